"""vdn_sink_attn_step (CUDA, through the binding) against the float64 oracle, and
the run of operators around it: normed and rotated queries and keys, a
prefill, then token by token, against one pass over the whole sequence.

Tolerances as for the forward pass (see test_sink_attn_gpu.py): half a step of
bf16, 2^-8, for the output and for each probability.
"""

import numpy as np
import pytest
import torch

from oracle.sink_attn import attend
from tests.parity_util import ensure_built

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8


@pytest.fixture(scope="module")
def vdn():
    ensure_built()
    from video_diffusion_hybrid_vda_b200 import vdn as _vdn
    return _vdn


def _f64(t):
    return t.detach().cpu().double().numpy()


def slot_of(p, window, sinks):
    return p if p < sinks + window else sinks + (p - sinks) % window


def check_rows(o, q, k, v, H, Hkv, d):
    """o, q [H*d] of one token; k, v [live, Hkv*d]."""
    see = np.ones((1, len(k)), bool)
    for h in range(H):
        e = h // (H // Hkv)
        c, ck = slice(h * d, (h + 1) * d), slice(e * d, (e + 1) * d)
        ro, _, p = attend(q[None, c], k[:, ck], v[:, ck], see, d ** -0.5)
        err = np.abs(o[None, c] - ro)
        assert (err <= HALF * np.abs(ro) + (HALF + 2.0 ** -12) * (p @ np.abs(v[:, ck]))).all()
        norm = np.sqrt((p * p) @ (v[:, ck] ** 2).sum(1))
        assert np.linalg.norm(err) <= HALF * (np.linalg.norm(ro) + 1.3 * norm[0])


CASES = [  # positions, H, Hkv, d, window, sinks, pad
    ([0], 1, 1, 64, 1, 0, 0),
    ([0, 1, 7], 2, 1, 128, 1, 0, 8),
    ([5, 6, 300], 4, 2, 64, 3, 4, 0),
    ([15, 16, 17, 31, 32, 33], 3, 3, 128, 40, 2, 0),
    ([1000, 99, 64], 16, 1, 128, 100, 0, 8),
    ([70, 5000], 34, 2, 64, 60, 5, 0),          # more than 16 query heads a key head
    ([4095, 4096, 100000], 8, 8, 128, 4092, 4, 0),   # over clusters of CTAs
    ([(1 << 31) - 1, 2000], 8, 1, 128, 1500, 7, 16),
    ([30000], 1, 1, 128, 20000, 0, 0),
]


@pytest.mark.parametrize("positions,H,Hkv,d,window,sinks,pad", CASES)
def test_parity(vdn, positions, H, Hkv, d, window, sinks, pad):
    gen = torch.Generator("cuda").manual_seed(len(positions) + H)
    B, slots = len(positions), window + sinks

    def normal(*shape):
        full = torch.randn(*shape[:-1], shape[-1] + pad, generator=gen, device="cuda").bfloat16()
        return full[..., :shape[-1]]

    q, kn, vn = normal(B, H * d), normal(B, Hkv * d), normal(B, Hkv * d)
    kc, vc = normal(B, slots, Hkv * d), normal(B, slots, Hkv * d)
    live = [min(p + 1, slots) for p in positions]
    for b in range(B):                         # slots that hold nothing are not read
        for c in (kc, vc):
            c[b, live[b]:] = float("nan")
            c[b, slot_of(positions[b], window, sinks)] = float("nan")
    k0, v0 = kc.clone(), vc.clone()
    pos = torch.tensor(positions, dtype=torch.int32, device="cuda")
    o = vdn.sink_attn_step(q, kn, vn, kc, vc, pos, H, Hkv, d, window, sinks)
    for b in range(B):
        at = slot_of(positions[b], window, sinks)
        for c, c0, new in ((kc, k0, kn), (vc, v0, vn)):
            want = c0[b].clone()
            want[at] = new[b]
            assert torch.equal(c[b].nan_to_num(7.0), want.nan_to_num(7.0))
        check_rows(_f64(o[b]), _f64(q[b]), _f64(kc[b, :live[b]]), _f64(vc[b, :live[b]]), H, Hkv, d)
    again = vdn.sink_attn_step(q, kn, vn, kc, vc, pos, H, Hkv, d, window, sinks)
    assert torch.equal(again, o)               # repeated: the same slot, the same bits


def test_inactive_sequences_are_left_alone(vdn):
    B, H, Hkv, d, window = 4, 4, 2, 64, 50
    gen = torch.Generator("cuda").manual_seed(0)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda").bfloat16()

    q, kn, vn = normal(B, H * d), normal(B, Hkv * d), normal(B, Hkv * d)
    kc, vc = normal(B, window, Hkv * d), normal(B, window, Hkv * d)
    k0, v0 = kc.clone(), vc.clone()
    pos = torch.tensor([3, -1, 60, -(1 << 31)], dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 5.0)
    vdn.sink_attn_step(q, kn, vn, kc, vc, pos, H, Hkv, d, window, out=out)
    for b in (1, 3):
        assert (out[b] == 5).all() and torch.equal(kc[b], k0[b]) and torch.equal(vc[b], v0[b])
    for b in (0, 2):
        assert not (out[b] == 5).all() and torch.equal(kc[b, slot_of(int(pos[b]), window, 0)], kn[b])
    none = torch.empty((0, H * d), dtype=torch.bfloat16, device="cuda")
    nk = torch.empty((0, Hkv * d), dtype=torch.bfloat16, device="cuda")
    assert vdn.sink_attn_step(none, nk, nk, kc[:0], vc[:0], pos[:0], H, Hkv, d,
                              window).shape == (0, H * d)


def test_offsets_past_32_bits(vdn):
    """A cache whose last sequence begins more than 2^31 elements in."""
    B, Hkv, d, window = 3, 1, 128, 100
    gen = torch.Generator("cuda").manual_seed(1)
    stride = 1 << 30
    flat = torch.zeros(2 * stride + 100 * 1024, dtype=torch.bfloat16, device="cuda")
    caches = [flat.as_strided((B, window, d), (stride, 1024, 1), off) for off in (0, 128)]
    q, kn, vn = (torch.randn(B, d, generator=gen, device="cuda").bfloat16() for _ in range(3))
    small = [torch.randn(B, window, d, generator=gen, device="cuda").bfloat16() for _ in range(2)]
    for c, x in zip(caches, small):
        c.copy_(x)
    pos = torch.tensor([150, 99, 3], dtype=torch.int32, device="cuda")
    a = vdn.sink_attn_step(q, kn, vn, *caches, pos, 1, Hkv, d, window)
    b = vdn.sink_attn_step(q, kn, vn, *small, pos, 1, Hkv, d, window)
    assert torch.equal(a, b)
    for c, x in zip(caches, small):
        assert torch.equal(c, x)


def test_stream_matches_one_pass(vdn):
    """Norm and rotation, prefill, then 40 tokens one at a time through a captured
    graph, against the same operators over the whole sequences at once: the
    same roundings of the same numbers, in another order (twice the bound)."""
    H, Hkv, d, window, sinks, eps = 6, 2, 128, 70, 3, 1e-6
    lens, new = [50, 200, 1], 40
    plan = vdn.RopePlan(d, rot=64, layout="interleaved")
    gen = torch.Generator("cuda").manual_seed(12)
    total = [n + new for n in lens]
    rows = sum(total)
    q, k, v = (torch.randn(rows, w * d, generator=gen, device="cuda").bfloat16()
               for w in (H, Hkv, Hkv))
    w = 1 + 0.1 * torch.randn(d, generator=gen, device="cuda")
    pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in total]).cuda()
    cu = torch.tensor(np.concatenate([[0], np.cumsum(total)]), dtype=torch.int32, device="cuda")
    kw = dict(wq=w, wk=w, eps=eps)
    qn, kn = vdn.qk_norm_rope(q, k, H, Hkv, plan, positions=pos, **kw)
    whole, _ = vdn.sink_attn(qn, kn, v, H, Hkv, d, window, sinks, cu_q=cu, cu_k=cu)
    # prefill: the prompts into the cache, by slot
    B = len(lens)
    kc, vc = (torch.zeros((B, window + sinks, Hkv * d), dtype=torch.bfloat16, device="cuda")
              for _ in range(2))
    for b, n in enumerate(lens):
        for p in range(n):
            r = int(cu[b]) + p
            kc[b, slot_of(p, window, sinks)] = kn[r]
            vc[b, slot_of(p, window, sinks)] = v[r]
    sq, sk, sv = (torch.zeros((B, x * d), dtype=torch.bfloat16, device="cuda")
                  for x in (H, Hkv, Hkv))
    at = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = torch.empty_like(sq)

    def token():
        a, b_ = vdn.qk_norm_rope(sq, sk, H, Hkv, plan, positions=at, **kw)
        vdn.sink_attn_step(a, b_, sv, kc, vc, at, H, Hkv, d, window, sinks, out=out)
        at.add_(1)

    warm = [t.clone() for t in (kc, vc, at)]
    token()                                     # kernels loaded before the capture
    for t, x in zip((kc, vc, at), warm):
        t.copy_(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        token()
    for i in range(new):
        r = cu[:-1].long() + torch.tensor(lens, device="cuda") + i
        sq.copy_(q[r])
        sk.copy_(k[r])
        sv.copy_(v[r])
        graph.replay()
        ref = whole[r].double()
        # every |v| row is below 4 sqrt(d)... the probabilities' part is at most h max |v|
        tol = 2 * (HALF * ref.abs() + 2 * HALF * 4.5)
        assert ((out.double() - ref).abs() <= tol).all()
        assert (out.double() - ref).norm() <= 3 * HALF * ref.norm()


def test_refusals(vdn):
    B, H, Hkv, d, window = 2, 4, 2, 64, 8
    q, kn = (torch.zeros((B, n * d), dtype=torch.bfloat16, device="cuda") for n in (H, Hkv))
    kc = torch.zeros((B, window + 1, Hkv * d), dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(B, dtype=torch.int32, device="cuda")
    good = dict(q=q, k_new=kn, v_new=kn, k_cache=kc, v_cache=kc.clone(), positions=pos, H=H,
                H_kv=Hkv, d=d, window=window, sinks=1)
    vdn.sink_attn_step(**good)
    for bad in (dict(k_cache=kc[:, :8]), dict(k_cache=kc.float()), dict(positions=pos.long()),
                dict(positions=pos[:1]), dict(q=q[:1]), dict(v_new=kn[:, :64]),
                dict(k_cache=kc.cpu()), dict(out=q[:, :64])):
        with pytest.raises(ValueError):
            vdn.sink_attn_step(**{**good, **bad})
    for bad in (dict(window=0, sinks=9), dict(window=10, sinks=-1), dict(H=3, q=q[:, :192])):
        with pytest.raises(vdn.VdnError):
            vdn.sink_attn_step(**{**good, **bad})
    shared = kc[:1].expand(2, -1, -1)             # two sequences in one cache
    with pytest.raises(vdn.VdnError):
        vdn.sink_attn_step(**{**good, "k_cache": shared, "v_cache": shared})
