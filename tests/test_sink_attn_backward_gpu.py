"""vdn_sink_attn_backward (CUDA, through the binding) against the float64 oracle.

Tolerances count roundings (half a step of bf16: h = 2^-8), with P and dS the
oracle's.  dv_j = sum_i P dO: its own rounding h |dv| and P's, h sum P |dO|.
dq_i = scale sum_j dS k_j: h |dq|, dS's rounding h scale sum |dS| |k|, and the
error of D_i = dO_i . o_i, whose o is the forward's, rounded once and from a
rounded P: at most dD_i = h sum_c |dO| (|o| + P |v|), which enters dS as P dD.
P itself is off by 2^-12 of itself (see test_sink_attn_gpu.py), the products
by less; 2^-11 of every sum covers both.  dk like dq.  The whole result is held
tighter: the errors are independent and their vectors nearly orthogonal, so
the 2-norms add as squares, with 1.3 for what is not.
"""

import numpy as np
import pytest
import torch

from oracle.sink_attn import attend, visible
from tests.parity_util import ensure_built
from tests.test_sink_attn_gpu import CASES, _f64, make

pytestmark = pytest.mark.gpu

H_ = 2.0 ** -8
REST = 2.0 ** -11


@pytest.fixture(scope="module")
def vdn():
    ensure_built()
    from video_diffusion_hybrid_vda_b200 import vdn as _vdn
    return _vdn


def check(grads, q, k, v, g, H, Hkv, d, window, sinks, ahead, lens_q, lens_k):
    q, k, v, g = _f64(q), _f64(k), _f64(v), _f64(g)
    got = [_f64(x) for x in grads]
    assert all(np.isfinite(x).all() for x in got)
    scale = d ** -0.5
    refs = [np.zeros_like(x) for x in (q, k, v)]
    tols = [np.zeros_like(x) for x in (q, k, v)]
    norms = [np.zeros(len(x)) for x in (q, k, v)]      # squared, of each row's independent errors
    a = b = 0
    for nq, nk in zip(lens_q, lens_k):
        see = visible(nq, nk, window, sinks, ahead)
        rq, rk = slice(a, a + nq), slice(b, b + nk)
        for h in range(H):
            e = h // (H // Hkv)
            cq, ck = slice(h * d, (h + 1) * d), slice(e * d, (e + 1) * d)
            qs, gs, ks, vs = q[rq, cq], g[rq, cq], k[rk, ck], v[rk, ck]
            o, _, p = attend(qs, ks, vs, see, scale)
            ds = p * (gs @ vs.T - (gs * o).sum(1, keepdims=True))
            dD = H_ * (np.abs(gs) * (np.abs(o) + p @ np.abs(vs))).sum(1, keepdims=True)
            sD = H_ * np.sqrt((gs * gs * (o * o + (p * p) @ (vs * vs))).sum(1, keepdims=True))
            ads = np.abs(ds)
            refs[0][rq, cq] = scale * ds @ ks
            refs[1][rk, ck] += scale * ds.T @ qs
            refs[2][rk, ck] += p.T @ gs
            off = (H_ + REST) * ads + p * (dD * (1 + REST) + REST * np.abs(gs) @ np.abs(vs).T)
            tols[0][rq, cq] = scale * off @ np.abs(ks)
            tols[1][rk, ck] += scale * off.T @ np.abs(qs)
            tols[2][rk, ck] += (H_ + REST) * p.T @ np.abs(gs)
            k2, q2, g2 = ((x * x).sum(1) for x in (ks, qs, gs))
            norms[0][rq] += scale ** 2 * (H_ ** 2 * (ds * ds) @ k2 +
                                          sD[:, 0] ** 2 * ((p @ ks) ** 2).sum(1))
            norms[1][rk] += scale ** 2 * (H_ ** 2 * (ds * ds).T @ q2 + (p * p).T @ (sD[:, 0] ** 2 * q2))
            norms[2][rk] += H_ ** 2 * (p * p).T @ g2
        a, b = a + nq, b + nk
    for x, ref, tol, norm in zip(got, refs, tols, norms):
        err = np.abs(x - ref)
        assert (err <= H_ * np.abs(ref) * (1 + REST) + tol + 1e-30).all()
        assert np.linalg.norm(err) <= (H_ * np.linalg.norm(ref) + 1.3 * np.sqrt(norm.sum()) +
                                       REST * np.sqrt((tol * tol).sum()) + 1e-30)


def step(vdn, q, k, v, g, H, Hkv, d, window, sinks, ahead, cq, ck, **kw):
    lse = torch.empty((H, q.shape[0]), device="cuda")
    mask = dict(window=window, sinks=sinks, ahead=ahead, cu_q=cq, cu_k=ck)
    o, ws = vdn.sink_attn(q, k, v, H, Hkv, d, lse=lse, **mask)
    assert vdn.get_device_status(ws) == 0
    out = vdn.sink_attn_backward(q, k, v, o, lse, g, H, Hkv, d, **mask, **kw)
    assert vdn.get_device_status(out[3]) == 0
    return out


FAR = [  # long behind a short window: the tiles with sinks are split over far parts
    ([3000], [3000], 2, 1, 128, 100, 4, 0, 0),
    ([2500, 40, 1300], [2500, 40, 1300], 4, 2, 64, 200, 130, 0, 0),
    ([1800], [2100], 2, 2, 64, 1, 1, 5, 8),
]


@pytest.mark.parametrize("lens_q,lens_k,H,Hkv,d,window,sinks,ahead,pad", CASES + FAR)
def test_parity(vdn, lens_q, lens_k, H, Hkv, d, window, sinks, ahead, pad):
    q, k, v, cq, ck = make(lens_q, lens_k, H, Hkv, d, seed=sum(lens_q) + d, pad=pad)
    g = make(lens_q, [0], H, 1, d, seed=3, pad=pad)[0]
    wide = [torch.full((n, w + pad), 7.0, dtype=torch.bfloat16, device="cuda")
            for n, w in ((len(q), H * d), (len(k), Hkv * d), (len(k), Hkv * d))]
    views = [t[:, :t.shape[1] - pad] for t in wide]
    a = step(vdn, q, k, v, g, H, Hkv, d, window, sinks, ahead, cq, ck, dq=views[0], dk=views[1],
             dv=views[2])
    check(a[:3], q, k, v, g, H, Hkv, d, window, sinks, ahead, lens_q, lens_k)
    for t, w in zip(wide, views):
        assert (t[:, w.shape[1]:] == 7).all()
    b = step(vdn, q, k, v, g, H, Hkv, d, window, sinks, ahead, cq, ck)
    for x, y in zip(a[:3], b[:3]):
        assert torch.equal(x, y)                        # the same bits again


@pytest.mark.parametrize("lens,d,window,sinks,ahead", [
    ([700], 128, 2, 0, 0), ([700], 64, 3, 1, 0), ([900, 300], 128, 8, 2, 4), ([600], 64, 33, 4, 0),
    ([16] * 40, 128, 1 << 30, 0, 0), ([50, 61, 3, 64] * 5, 64, 1 << 30, 0, 7),
    ([500], 128, 20, 0, 100)])
def test_few_keys_lose_nothing(vdn, lens, d, window, sinks, ahead):
    """dq and dk of queries that see few keys are off by two roundings only,
    dS's and their own: D_i = dO_i . o_i with the rounded o would be off by as
    much again for all of a query's keys together.  A rounding's error is
    uniform over a step, at most 2^-8 / sqrt(3) of its value in the mean square
    (mantissa 1; less for others), and the errors add as squares, with 5 % for
    the finite number of them.  The last case sees few keys in its first rows'
    looks back and many ahead: its last rows alone see few."""
    H = 2
    q, k, v, cq, ck = make(lens, lens, H, H, d, seed=41)
    g = make(lens, [0], H, 1, d, seed=42)[0]
    out = step(vdn, q, k, v, g, H, H, d, window, sinks, ahead, cq, ck)
    q, k, v, g, dq, dk = (_f64(x) for x in (q, k, v, g, out[0], out[1]))
    err, ref, rounding, a = np.zeros(2), np.zeros(2), np.zeros(2), 0
    for n in lens:
        see, rows = visible(n, n, window, sinks, ahead), slice(a, a + n)
        few = see.sum(1) <= 64
        for h in range(H):
            c = slice(h * d, (h + 1) * d)
            qs, ks, vs, gs = (x[rows, c] for x in (q, k, v, g))
            o, _, p = attend(qs, ks, vs, see, d ** -0.5)
            ds = p * (gs @ vs.T - (gs * o).sum(1, keepdims=True)) * d ** -0.5
            sides = [(dq[rows, c][few], (ds @ ks)[few], (ds * ds)[few] @ (ks * ks).sum(1))]
            if few.all():
                sides.append((dk[rows, c], ds.T @ qs, (ds * ds).T @ (qs * qs).sum(1)))
            for i, (got, want, square) in enumerate(sides):
                err[i] += ((got - want) ** 2).sum()
                ref[i] += (want ** 2).sum()
                rounding[i] += square.sum()
        a += n
    assert ref[0] > 0
    assert (np.sqrt(err) <= 1.05 * H_ / 3 ** 0.5 * np.sqrt(ref + rounding)).all()


def test_random_shapes(vdn):
    rng = np.random.default_rng(23)
    for _ in range(25):
        n = int(rng.integers(1, 4))
        lens_k = [int(x) for x in rng.integers(0, 600, n)]
        lens_q = [int(rng.integers(0, x + 20)) for x in lens_k]
        if sum(lens_q) == 0:
            lens_q[0] = 3
        Hkv = int(rng.integers(1, 3))
        H, d = Hkv * int(rng.integers(1, 4)), int(rng.choice([64, 128]))
        window, ahead = int(rng.integers(1, 300)), int(rng.choice([0, 0, 1, 50, 300]))
        sinks = int(rng.choice([0, 1, 4, 127, 128, 129, 300]))
        q, k, v, cq, ck = make(lens_q, lens_k, H, Hkv, d, seed=n)
        g = make(lens_q, [0], H, 1, d, seed=4)[0]
        out = step(vdn, q, k, v, g, H, Hkv, d, window, sinks, ahead, cq, ck)
        check(out[:3], q, k, v, g, H, Hkv, d, window, sinks, ahead, lens_q, lens_k)


def test_against_differences_of_the_forward(vdn):
    """d/dh of <g, o(x + h e)> along random directions.  The forward's bf16
    output and P leave noise of at most 2^-8 |g| sum P |v| a query on each side
    (random signs: its 2-norm over the queries), so h is large, 1/2 on a
    direction of unit norm times the gradient's norm; the third-order term of a
    direction of unit length is below a percent of the first."""
    H, Hkv, d, lens = 2, 1, 64, [150, 90]
    q, k, v, cq, ck = make(lens, lens, H, Hkv, d, seed=31)
    g = make(lens, [0], H, 1, d, seed=32)[0]
    kw = dict(window=40, sinks=3, cu_q=cq, cu_k=ck)
    grads = step(vdn, q, k, v, g, H, Hkv, d, 40, 3, 0, cq, ck)

    def loss(*x):
        return (vdn.sink_attn(*x, H, Hkv, d, **kw)[0].double() * g.double()).sum().item()

    o = vdn.sink_attn(q, k, v, H, Hkv, d, **kw)[0].double()
    noise = H_ * 2 * (g.double() * (o.abs() + 0.3)).norm().item()
    for n in range(3):
        gen = torch.Generator("cuda").manual_seed(n)
        x = [q, k, v]
        e = grads[n].double()
        e = e / e.norm() + 0.01 * torch.randn(e.shape, generator=gen, device="cuda").double() / \
            e.numel() ** 0.5
        h = 4.0
        up, down = list(x), list(x)
        up[n], down[n] = (x[n].double() + h * e).bfloat16(), (x[n].double() - h * e).bfloat16()
        along = (up[n].double() - down[n].double())     # what rounding left of the step
        want = (grads[n].double() * along).sum().item()
        diff = loss(*up) - loss(*down)
        assert abs(diff - want) <= noise + 0.03 * abs(want), (n, diff, want, noise)


def test_other_sequences_and_rows_of_none_do_not_reach_in(vdn):
    H, d = 2, 128
    q, k, v, _, _ = make([400], [400], H, H, d)
    g = make([400], [0], H, 1, d, seed=6)[0]
    clean = [step(vdn, x[0], x[1], x[2], x[3], H, H, d, 50, 4, 0, None, None)[:3] for x in
             ([t[20:120] for t in (q, k, v, g)], [t[250:320] for t in (q, k, v, g)])]
    bad = torch.ones(400, dtype=torch.bool, device="cuda")
    bad[20:120] = bad[250:320] = False
    for value in (float("nan"), float("inf")):
        for t in (q, k, v, g):
            t[bad] = value
        cu = torch.tensor([20, 120, 250, 320], dtype=torch.int32, device="cuda")
        mask = dict(window=50, sinks=4, cu_q=cu, cu_k=cu)
        lse = torch.full((H, 400), float("nan"), device="cuda")
        o = torch.full_like(q, float("nan"))
        vdn.sink_attn(q, k, v, H, H, d, out=o, lse=lse, **mask)
        out = [torch.full_like(q, 9.0) for _ in range(3)]
        vdn.sink_attn_backward(q, k, v, o, lse, g, H, H, d, dq=out[0], dk=out[1], dv=out[2],
                               **mask)
        for n in range(3):
            assert torch.equal(out[n][20:120], clean[0][n])
            assert torch.equal(out[n][250:320], clean[1][n])
            assert (out[n][:20] == 9).all() and (out[n][320:] == 9).all()
        fresh = vdn.sink_attn_backward(q, k, v, o, lse, g, H, H, d, **mask)
        for n in range(3):                              # zeros in a new output
            assert torch.equal(fresh[n][20:120], clean[0][n])
            assert not fresh[n][:20].any() and not fresh[n][320:].any()


@pytest.mark.parametrize("lead", [127, 128, 300])
def test_rows_before_the_first_sequence(vdn, lead):
    H, d, lens = 2, 64, [300, 77]
    q, k, v, cq, ck = make(lens, lens, H, H, d, seed=lead)
    g = make(lens, [0], H, 1, d, seed=1)[0]
    qs, ks, vs, gs = (torch.cat([torch.full((lead, H * d), 5.0, device="cuda").bfloat16(), t])
                      for t in (q, k, v, g))
    mask = dict(window=90, sinks=4, ahead=400, cu_q=cq + lead, cu_k=ck + lead)
    lse = torch.zeros((H, lead + sum(lens)), device="cuda")
    o = torch.ones_like(qs)
    vdn.sink_attn(qs, ks, vs, H, H, d, out=o, lse=lse, **mask)
    out = [torch.full_like(qs, 9.0) for _ in range(3)]
    vdn.sink_attn_backward(qs, ks, vs, o, lse, gs, H, H, d, dq=out[0], dk=out[1], dv=out[2], **mask)
    fresh = vdn.sink_attn_backward(qs, ks, vs, o, lse, gs, H, H, d, **mask)
    check([x[lead:] for x in out], q, k, v, g, H, H, d, 90, 4, 400, lens, lens)
    for n in range(3):
        assert (out[n][:lead] == 9).all()
        assert torch.equal(fresh[n][lead:], out[n][lead:]) and not fresh[n][:lead].any()


def test_keys_no_query_sees_and_no_queries_at_all(vdn):
    q, k, v, _, _ = make([20], [300], 2, 1, 64)
    g = make([20], [0], 2, 1, 64, seed=1)[0]
    _, dk, dv, _ = step(vdn, q, k, v, g, 2, 1, 64, 30, 0, 0, None, None)
    assert not dk[:251].any() and not dv[:251].any()    # 300 - 20 - 30 + 1
    assert dk[251:].any()
    e = q[:0]
    lse = torch.empty((2, 0), device="cuda")
    dq, dk, dv, _ = vdn.sink_attn_backward(e, k, v, e, lse, e, 2, 1, 64, 30)
    assert dq.shape == (0, 128) and not dk.any() and not dv.any()


def test_captured_and_replayed(vdn):
    lens = [900, 77]
    q, k, v, cq, ck = make(lens, lens, 4, 2, 128, seed=2)
    g = make(lens, [0], 4, 1, 128, seed=1)[0]
    mask = dict(window=60, sinks=4, cu_q=cq, cu_k=ck)
    ref = step(vdn, q, k, v, g, 4, 2, 128, 60, 4, 0, cq, ck)
    sq, o = torch.zeros_like(q), torch.empty_like(q)
    lse = torch.empty((4, 977), device="cuda")
    outs = [torch.empty_like(t) for t in ref[:3]]
    ws = vdn.alloc_workspace(vdn.sink_attn_workspace(977, 977, 2, 4, 2, 128, 60, 4))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        graph.capture_begin()
        vdn.sink_attn(sq, k, v, 4, 2, 128, out=o, lse=lse, ws=ws, **mask)
        vdn.sink_attn_backward(sq, k, v, o, lse, g, 4, 2, 128, dq=outs[0], dk=outs[1], dv=outs[2],
                               ws=ref[3], **mask)
        graph.capture_end()
    torch.cuda.current_stream().wait_stream(st)
    sq.copy_(q)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(outs, ref):
        assert torch.equal(x, y)


def test_refusals(vdn):
    q, k, v, _, _ = make([8], [8], 2, 1, 64)
    lse = torch.empty((2, 8), device="cuda")
    o = torch.empty_like(q)
    for bad in (dict(lse=lse[:1]), dict(lse=lse.double()), dict(o=o.float()), dict(d_o=o[:4]),
                dict(o=o[:, :64])):
        args = dict(o=o, lse=lse, d_o=o)
        args.update(bad)
        with pytest.raises(ValueError):
            vdn.sink_attn_backward(q, k, v, args["o"], args["lse"], args["d_o"], 2, 1, 64, 4)
    with pytest.raises(vdn.VdnError):
        vdn.sink_attn_backward(q, k, v, o, lse, o, 2, 1, 64, 0)
    with pytest.raises(vdn.VdnError):                   # workspace too small
        vdn.sink_attn_backward(q, k, v, o, lse, o, 2, 1, 64, 4, ws=vdn.alloc_workspace(256))
