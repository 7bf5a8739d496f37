"""vdn_rope, vdn_qk_norm_rope and its gradients (CUDA, through the binding)
against the float64 oracle.

Tolerances count roundings.  An output is rounded once to its type (half a
step, eps/2 of its value).  Before that, in fp32 (u = 2^-24): the angle is off
by at most 2^-26 of a turn (the phase's conversion to float: 2 pi 2^-26 =
1.6 u) and sincospi by 2 ulp, the norm's factor by half of its sum's (at most
256 additions in a chain of 16 and 5, 21 u) and 2 ulp of rsqrt (4 u); four
products and a sum follow.  That is below 32 u of the pair's length, which the
head's largest value bounds up to sqrt 2: 48 u.
"""

import numpy as np
import pytest
import torch

from oracle import qk_prep
from tests.parity_util import ensure_built

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def vdn():
    ensure_built()
    from video_diffusion_hybrid_vda_b200 import vdn as _vdn
    return _vdn


def _half_step(dtype):
    return torch.finfo(dtype).eps / 2


def _f64(t):
    return t.detach().cpu().double().numpy()


def _wide(rows, cols, dtype, gen, pad=0, scale=1.0):
    """[rows, cols] view of a matrix with `pad` further columns."""
    full = (torch.randn(rows, cols + pad, generator=gen, device="cuda") * scale).to(dtype)
    return full[:, :cols]


def _check(got, ref, dtype, extra=48 * U):
    """got [rows, heads*d] against ref [rows, heads, d]; fp16 also rounds what
    is below its smallest normal number to steps of 2^-24."""
    got = _f64(got).reshape(ref.shape)
    big = np.abs(ref).max(-1, keepdims=True)
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0
    tol = _half_step(dtype) * np.abs(ref) * (1 + 2.0 ** -10) + extra * big + tiny
    assert np.isfinite(got).all()
    worst = float((np.abs(got - ref) - tol).max()) if ref.size else 0.0
    assert worst <= 0, worst


def _rotation(plan, positions, rows):
    axis = np.repeat(np.arange(plan.n_axes), plan.sections)
    pos = np.tile(np.arange(rows), (plan.n_axes, 1)) if positions is None else \
        positions.cpu().numpy().reshape(plan.n_axes, rows)
    # the factor as the kernel has it, in fp32
    return dict(positions=pos, frequencies=np.array(plan.frequencies), axis=axis,
                layout=plan.layout, scale=float(np.float32(plan.scale)))


ROPE = [  # rows, heads, d, rot, layout, dtype, sections, scaling, pad
    (1, 1, 8, 8, "half", "bf16", None, None, 0),
    (1, 3, 128, 128, "interleaved", "bf16", None, "yarn", 0),
    (257, 5, 128, 64, "half", "bf16", None, None, 24),
    (33, 2, 64, 64, "interleaved", "fp16", [10, 11, 11], None, 8),
    (19, 7, 96, 24, "half", "fp32", None, "ntk", 16),
    (700, 24, 128, 128, "half", "bf16", [22, 21, 21], None, 0),
    (40, 3, 256, 256, "interleaved", "fp32", [60, 60, 4, 4], "linear", 8),
    (64, 2, 40, 16, "interleaved", "fp16", [0, 8], None, 0),
    (5, 2, 16, 0, "half", "bf16", None, None, 0),
    (5000, 3, 64, 64, "half", "bf16", None, None, 0),
]


@pytest.mark.parametrize("rows,heads,d,rot,layout,dtype,sections,scaling,pad", ROPE)
@pytest.mark.parametrize("inverse", [False, True])
def test_rope(vdn, rows, heads, d, rot, layout, dtype, sections, scaling, pad, inverse):
    gen = torch.Generator("cuda").manual_seed(rows + d)
    plan = vdn.RopePlan(d, rot=rot, layout=layout, sections=sections, scaling=scaling, factor=4.0)
    x = _wide(rows, heads * d, DT[dtype], gen, pad)
    pos = torch.randint(-3, 4000000, (plan.n_axes, rows), generator=gen, device="cuda",
                        dtype=torch.int32)
    out = vdn.rope(x, heads, plan, positions=pos, inverse=inverse)
    ref = qk_prep.rotate(_f64(x).reshape(rows, heads, d), inverse=inverse,
                         **_rotation(plan, pos, rows))
    _check(out, ref, DT[dtype])
    if rot == 0:
        assert torch.equal(out, x)


@pytest.mark.parametrize("at", [0, (1 << 31) - 5, -(1 << 31), 123456789])
def test_rope_at_the_ends_of_the_positions(vdn, at):
    """Whole turns are dropped exactly: any 32-bit position keeps its angle.
    The oracle's own angle is a float64 product of up to 2^31 radians, off by
    2^-53 of it, so the sines are off by 2^-22 at most; the rest as above."""
    plan = vdn.RopePlan(64)
    gen = torch.Generator("cuda").manual_seed(3)
    x = _wide(4, 128, torch.float32, gen)
    pos = (at + torch.arange(4, device="cuda", dtype=torch.int64)).to(torch.int32)
    out = vdn.rope(x, 2, plan, positions=pos)
    ref = qk_prep.rotate(_f64(x).reshape(4, 2, 64), **_rotation(plan, pos, 4))
    _check(out, ref, torch.float32, 48 * U + 2 * 2.0 ** -22)


def test_rope_default_positions_in_place_and_empty(vdn):
    plan = vdn.RopePlan(64, rot=32, layout="interleaved", sections=[9, 7])
    gen = torch.Generator("cuda").manual_seed(4)
    x = _wide(77, 128, torch.bfloat16, gen, pad=8)
    out = vdn.rope(x, 2, plan)
    _check(out, qk_prep.rotate(_f64(x).reshape(77, 2, 64), **_rotation(plan, None, 77)),
           torch.bfloat16)
    whole = x._base.clone()
    view = whole[:, :128]
    assert vdn.rope(view, 2, plan, out=view) is view
    assert torch.equal(view, out)
    assert torch.equal(whole[:, 128:], x._base[:, 128:])  # columns past the heads untouched
    assert vdn.rope(x[:0], 2, plan).shape == (0, 128)


QK = [  # rows, H, Hkv, d, rot, layout, dtype, q_norm, k_norm, sections, pad
    (1, 1, 1, 16, 16, "half", "bf16", "rms", "l2", None, 0),
    (300, 6, 2, 64, 64, "half", "bf16", "rms", "rms", None, 0),
    (129, 4, 4, 128, 128, "interleaved", "bf16", "rms", "l2", [24, 20, 20], 16),
    (65, 3, 1, 96, 40, "half", "fp32", "l2", "rms", None, 8),
    (50, 8, 1, 256, 128, "interleaved", "fp16", "rms", "none", None, 0),
    (2500, 5, 1, 32, 32, "half", "fp16", "none", "l2", None, 0),
    (9, 1, 3, 24, 0, "half", "fp32", "rms", "l2", None, 0),   # norm alone, more key heads
    (1300, 24, 24, 128, 128, "half", "bf16", "rms", "l2", None, 0),
]


def _qk_case(vdn, rows, H, Hkv, d, rot, layout, dtype, sections, pad, seed=0):
    gen = torch.Generator("cuda").manual_seed(seed + rows)
    plan = vdn.RopePlan(d, rot=rot, layout=layout, sections=sections)
    dt = DT[dtype]
    q, k = _wide(rows, H * d, dt, gen, pad), _wide(rows, Hkv * d, dt, gen, pad, 3.0)
    w = [1 + 0.3 * torch.randn(d, generator=gen, device="cuda") for _ in range(2)]
    dy = [_wide(rows, H * d, dt, gen, pad), _wide(rows, Hkv * d, dt, gen, 0)]
    pos = torch.randint(0, 100000, (plan.n_axes, rows), generator=gen, device="cuda",
                        dtype=torch.int32)
    return plan, q, k, w, dy, pos


@pytest.mark.parametrize("rows,H,Hkv,d,rot,layout,dtype,q_norm,k_norm,sections,pad", QK)
def test_qk_norm_rope_and_gradients(vdn, rows, H, Hkv, d, rot, layout, dtype, q_norm, k_norm,
                                    sections, pad):
    plan, q, k, w, dy, pos = _qk_case(vdn, rows, H, Hkv, d, rot, layout, dtype, sections, pad)
    kw = dict(wq=w[0] if q_norm != "none" else None, wk=w[1] if k_norm != "none" else None,
              q_norm=q_norm, k_norm=k_norm, eps=1e-5, positions=pos)
    q0, k0 = q.clone(), k.clone()
    outs = vdn.qk_norm_rope(q, k, H, Hkv, plan, **kw)
    dq, dk, dwq, dwk, ws = vdn.qk_norm_rope_backward(q, k, dy[0], dy[1], H, Hkv, plan, **kw)
    assert torch.equal(q, q0) and torch.equal(k, k0)
    rt = _rotation(plan, pos, rows)
    for x, y, g, dx, dw, wt, kind, h in ((q, outs[0], dy[0], dq, dwq, kw["wq"], q_norm, H),
                                         (k, outs[1], dy[1], dk, dwk, kw["wk"], k_norm, Hkv)):
        xs = _f64(x).reshape(rows, h, d)
        ww = np.ones(d) if wt is None else _f64(wt)
        gs = _f64(g).reshape(rows, h, d)
        eps = float(np.float32(1e-5))
        _check(y, qk_prep.qk_norm_rope(xs, ww, kind, eps, rt), x.dtype)
        rx, rw = qk_prep.qk_norm_rope_backward(xs, ww, gs, kind, eps, rt)
        # dx: the rotated gradient's 48 u of its head's largest value, times r w; and the
        # second term's sum of d products (21 roundings in its chain, 48 u of each g)
        r = qk_prep.norm_factor(xs, kind, eps)
        c = 0.0 if kind == "none" else 1.0 / d if kind == "rms" else 1.0
        top = np.abs(gs).max(-1, keepdims=True) * 2 ** 0.5
        second = np.abs(xs) * r ** 3 * c * (top * np.abs(ww * xs).sum(-1, keepdims=True))
        off = 80 * U * (r * np.abs(ww) * top + second)
        tiny = 2.0 ** -25 if x.dtype == torch.float16 else 0.0
        tol = _half_step(x.dtype) * np.abs(rx) * (1 + 2.0 ** -10) + off + tiny
        assert (np.abs(_f64(dx).reshape(rx.shape) - rx) <= tol).all()
        if kind == "none":
            assert dw is None
            continue
        # dw: at most rows * h additions in a chain and the product's 80 u
        terms = (top * np.abs(xs) * r).sum((0, 1))
        assert (np.abs(_f64(dw) - rw) <= (80 + rows * h) * U * terms).all()
        # and what a sum of random signs is off by in practice
        assert np.linalg.norm(_f64(dw) - rw) <= 1e-5 * np.linalg.norm(terms)


def test_gradients_are_the_forwards_differences(vdn):
    """<dy, y(x + h e) - y(x - h e)> / 2h against dx and dw, in fp32: the
    difference quotient of values up to 4 with u roundings is off by 48 u 4 d /
    h from rounding and h^2 / 6 times a third derivative below 64 (h = 2^-7)."""
    plan, q, k, w, dy, pos = _qk_case(vdn, 3, 2, 1, 32, 16, "half", "fp32", None, 0)
    kw = dict(k_norm="l2", positions=pos)
    dq, dk, dwq, dwk, _ = vdn.qk_norm_rope_backward(q, k, dy[0], dy[1], 2, 1, plan, wq=w[0],
                                                    wk=w[1], **kw)

    def loss(q_, k_, wq, wk):
        a, b = vdn.qk_norm_rope(q_, k_, 2, 1, plan, wq=wq, wk=wk, **kw)
        return (a.double() * dy[0]).sum().item() + (b.double() * dy[1]).sum().item()

    h = 2.0 ** -7
    tol = 48 * U * 4 * 32 * 3 / h + h * h / 6 * 64
    for which, grad in ((0, dq), (1, dk), (2, dwq), (3, dwk)):
        for at in (0, 5, 17, 31):
            args = [[q.clone(), k.clone(), w[0].clone(), w[1].clone()] for _ in range(2)]
            args[0][which].view(-1)[at] += h
            args[1][which].view(-1)[at] -= h
            diff = (loss(*args[0]) - loss(*args[1])) / (2 * h)
            assert abs(diff - grad.reshape(-1)[at].item()) <= tol


def test_same_call_same_bits_in_place_and_captured(vdn):
    plan, q, k, w, dy, pos = _qk_case(vdn, 4001, 8, 2, 64, 64, "half", "bf16", None, 0)
    kw = dict(wq=w[0], wk=w[1], positions=pos)
    ref = vdn.qk_norm_rope(q, k, 8, 2, plan, **kw)
    a = vdn.qk_norm_rope_backward(q, k, dy[0], dy[1], 8, 2, plan, **kw)
    b = vdn.qk_norm_rope_backward(q, k, dy[0], dy[1], 8, 2, plan, **kw)
    for x, y in zip(a[:4], b[:4]):
        assert torch.equal(x, y)
    # in place: forward over its inputs, gradients over the outputs' gradients
    qi, ki = q.clone(), k.clone()
    vdn.qk_norm_rope(qi, ki, 8, 2, plan, q_out=qi, k_out=ki, **kw)
    assert torch.equal(qi, ref[0]) and torch.equal(ki, ref[1])
    g = [t.clone() for t in dy]
    vdn.qk_norm_rope_backward(q, k, g[0], g[1], 8, 2, plan, dq=g[0], dk=g[1], **kw)
    assert torch.equal(g[0], a[0]) and torch.equal(g[1], a[1])
    # captured on a stream of its own and replayed on new inputs
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    sq, sk = torch.zeros_like(q), torch.zeros_like(k)
    outs = [torch.empty_like(q), torch.empty_like(k), torch.empty_like(q), torch.empty_like(k),
            torch.empty_like(w[0]), torch.empty_like(w[0])]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        graph.capture_begin()
        vdn.qk_norm_rope(sq, sk, 8, 2, plan, q_out=outs[0], k_out=outs[1], **kw)
        vdn.qk_norm_rope_backward(sq, sk, dy[0], dy[1], 8, 2, plan, dq=outs[2], dk=outs[3],
                                  dwq=outs[4], dwk=outs[5], ws=a[4], **kw)
        graph.capture_end()
    torch.cuda.current_stream().wait_stream(st)
    sq.copy_(q)
    sk.copy_(k)
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(outs, (*ref, *a[:4])):
        assert torch.equal(x, y)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype,rot", [("bf16", 48), ("bf16", 40), ("fp32", 16)])
def test_columns_past_the_rotated_ones_are_copied(vdn, layout, dtype, rot):
    """Infinities and NaN there stay where they are, beside rotated columns too."""
    plan = vdn.RopePlan(64, rot=rot, layout=layout)
    gen = torch.Generator("cuda").manual_seed(1)
    x = _wide(50, 128, DT[dtype], gen).view(50, 2, 64)
    x[..., rot::3] = float("inf")
    x[3, 1, rot + 1] = float("nan")
    x = x.reshape(50, 128)
    for inverse in (False, True):
        y = vdn.rope(x, 2, plan, inverse=inverse).view(50, 2, 64)
        assert torch.isfinite(y[..., :rot]).all()
        same = torch.equal(y[..., rot:].nan_to_num(5.0, posinf=9.0),
                           x.view(50, 2, 64)[..., rot:].nan_to_num(5.0, posinf=9.0))
        assert same
    g = torch.ones_like(x)
    dq, _, _, _, _ = vdn.qk_norm_rope_backward(x, x, g, g, 2, 2, plan, q_norm="none",
                                               k_norm="none")
    assert torch.isfinite(dq).all()          # a rotation's gradient needs nothing of x


def test_positions_shared_by_the_axes(vdn):
    plan = vdn.RopePlan(64, sections=[8, 8, 16])
    x = torch.randn(37, 128, device="cuda").bfloat16()
    one = torch.randint(0, 9000, (37,), device="cuda", dtype=torch.int32)
    ref = vdn.rope(x, 2, plan, one.repeat(3, 1))
    assert torch.equal(vdn.rope(x, 2, plan, one.expand(3, 37)), ref)
    assert torch.equal(vdn.rope(x[:1], 2, plan, one[:1].expand(3, 1)), ref[:1])
    with pytest.raises(vdn.VdnError):                   # axes that overlap
        vdn.rope(x, 2, plan, torch.as_strided(one.repeat(3), (3, 37), (5, 1)))


def test_no_rows(vdn):
    plan = vdn.RopePlan(64)
    e = torch.empty((0, 128), dtype=torch.bfloat16, device="cuda")
    a, b = vdn.qk_norm_rope(e, e[:, :64], 2, 1, plan)
    assert a.shape == (0, 128) and b.shape == (0, 64)
    dq, dk, dwq, dwk, _ = vdn.qk_norm_rope_backward(e, e[:, :64], e, e[:, :64], 2, 1, plan)
    assert not dwq.any() and not dwk.any()


def test_offsets_past_32_bits(vdn):
    """Rows more than 2^31 elements into the tensor."""
    plan = vdn.RopePlan(64)
    ld = 1 << 20
    rows = (1 << 11) + 3
    big = torch.zeros((rows, ld), dtype=torch.bfloat16, device="cuda")
    view = big[:, ld - 64:]
    gen = torch.Generator("cuda").manual_seed(8)
    x = torch.randn(rows, 64, generator=gen, device="cuda").bfloat16()
    view.copy_(x)
    vdn.rope(view, 1, plan, out=view)
    assert torch.equal(view, vdn.rope(x, 1, plan))
    assert not big[:, :ld - 64].any()
