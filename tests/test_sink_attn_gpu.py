"""vdn_sink_attn (CUDA, through the binding) against the float64 oracle.

Tolerances count roundings (half a step of bf16: 2^-8).  o = sum_j p_j v_j is
rounded once (2^-8 |o|) and each p_j once before the product (2^-8 sum p|v|).
The scores are fp32 sums of at most 128 exact products, off by at most 128
2^-24 sum |q k| scale, which stays below 16 for the inputs here: p is off by
2^-13 of itself, ex2 and the argument's rounding included below 2^-12.  lse is
off by the same 2^-12.  Whole rows are held tighter: errors of different keys
are independent and their values nearly orthogonal, so a row's error has at
most the 2-norm 2^-8 (|o| + 1.3 sqrt(sum p_j^2 |v_j|^2)).
"""

import numpy as np
import pytest
import torch

from oracle.sink_attn import attend, visible
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


def make(lens_q, lens_k, H, Hkv, d, seed=0, pad=0):
    gen = torch.Generator("cuda").manual_seed(seed)

    def normal(rows, cols):
        return torch.randn(rows, cols + pad, generator=gen, device="cuda").bfloat16()[:, :cols]

    nq, nk = sum(lens_q), sum(lens_k)
    cu = [torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device="cuda")
          for n in (lens_q, lens_k)]
    return normal(nq, H * d), normal(nk, Hkv * d), normal(nk, Hkv * d), cu[0], cu[1]


def check(o, lse, q, k, v, H, Hkv, d, window, sinks, ahead, lens_q, lens_k, heads=None):
    q, k, v, o, lse = _f64(q), _f64(k), _f64(v), _f64(o), _f64(lse)
    a = b = 0
    for nq, nk in zip(lens_q, lens_k):
        see = visible(nq, nk, window, sinks, ahead)
        for h in heads or range(H):
            e = h // (H // Hkv)
            ks, vs = (x[b:b + nk, e * d:(e + 1) * d] for x in (k, v))
            ro, rl, p = attend(q[a:a + nq, h * d:(h + 1) * d], ks, vs, see, d ** -0.5)
            go, gl = o[a:a + nq, h * d:(h + 1) * d], lse[h, a:a + nq]
            err = np.abs(go - ro)
            assert np.isfinite(go).all()
            assert (err <= HALF * np.abs(ro) + (HALF + 2.0 ** -12) * (p @ np.abs(vs)) + 1e-30).all()
            norm = np.sqrt((p * p) @ (vs * vs).sum(1))
            row = np.linalg.norm(ro, axis=1)
            assert (np.linalg.norm(err, axis=1) <= HALF * (row + 1.3 * norm) + 1e-30).all()
            empty = ~see.any(1)
            assert (gl[empty] == -np.inf).all() and not go[empty].any()
            assert (np.abs(gl[~empty] - rl[~empty]) <= 2.0 ** -12).all()
        a, b = a + nq, b + nk


CASES = [  # lens_q, lens_k, H, Hkv, d, window, sinks, ahead, pad
    ([1], [1], 1, 1, 64, 1, 0, 0, 0),
    ([1], [1], 2, 1, 128, 5, 3, 2, 8),
    ([128], [128], 2, 2, 128, 1000, 0, 0, 0),
    ([127, 129], [127, 129], 2, 1, 64, 64, 4, 0, 0),
    ([300], [300], 3, 1, 128, 1, 0, 0, 24),            # each query sees itself
    ([300], [300], 1, 1, 64, 1, 7, 0, 0),
    ([515], [515], 2, 2, 128, 100, 130, 0, 0),          # sinks over more than a tile
    ([700, 1, 0, 323], [700, 1, 0, 323], 2, 1, 64, 129, 5, 128, 0),
    ([5, 64, 200], [900, 64, 333], 4, 2, 128, 200, 4, 0, 0),   # chunks behind a context
    ([40, 3], [10, 3], 2, 2, 64, 100, 0, 0, 0),         # more queries than keys: empty rows
    ([40, 200], [10, 0], 2, 1, 128, 4, 2, 3, 0),        # no keys at all
    ([257], [257], 2, 1, 128, 4096, 0, 4096, 0),        # everything sees everything
    ([1000], [1000], 1, 1, 128, 256, 1, 17, 0),
    ([33], [5000], 4, 1, 128, 1 << 30, 0, 0, 0),        # split over the keys and joined
    ([3, 2], [4100, 77], 2, 1, 64, 2000, 4, 0, 8),
    ([300], [4000], 1, 1, 64, 1 << 30, 0, 0, 0),
    ([2600], [2600], 8, 2, 128, 513, 4, 0, 0),
    ([9], [2000], 8, 1, 64, 700, 4, 0, 0),              # heads that share a unit's rows
    ([1], [300], 32, 1, 128, 1 << 30, 0, 0, 8),
    ([16, 3, 30], [16, 500, 200], 16, 2, 128, 40, 3, 2, 0),
    ([100, 20], [100, 300], 6, 3, 64, 50, 2, 0, 0),
    ([0, 64, 0], [5, 64, 0], 4, 1, 128, 64, 0, 10, 0),
    # several units a CTA, some of whose row tiles take no keys
    ([257, 130, 1, 64, 300, 513] * 7, [257, 130, 1, 64, 300, 513] * 7, 8, 4, 64, 100, 4, 0, 0),
    ([257, 20, 384] * 12, [0, 500, 384] * 12, 6, 6, 128, 70, 2, 0, 0),
]


@pytest.mark.parametrize("lens_q,lens_k,H,Hkv,d,window,sinks,ahead,pad", CASES)
def test_parity(vdn, lens_q, lens_k, H, Hkv, d, window, sinks, ahead, pad):
    q, k, v, cq, ck = make(lens_q, lens_k, H, Hkv, d, seed=sum(lens_q) + d, pad=pad)
    lse = torch.full((H, q.shape[0]), float("nan"), device="cuda")
    wide = torch.full((q.shape[0], H * d + pad), 7.0, dtype=torch.bfloat16, device="cuda")
    kw = dict(window=window, sinks=sinks, ahead=ahead, cu_q=cq, cu_k=ck)
    o, ws = vdn.sink_attn(q, k, v, H, Hkv, d, out=wide[:, :H * d], lse=lse, **kw)
    assert vdn.get_device_status(ws) == 0
    check(o, lse, q, k, v, H, Hkv, d, window, sinks, ahead, lens_q, lens_k)
    assert (wide[:, H * d:] == 7).all()
    again, _ = vdn.sink_attn(q, k, v, H, Hkv, d, ws=ws, **kw)
    assert torch.equal(again, o)                        # no lse asked for, the same bits
    if len(lens_q) == 1:
        kw.update(cu_q=None, cu_k=None)
        assert torch.equal(vdn.sink_attn(q, k, v, H, Hkv, d, **kw)[0], o)


def test_random_shapes(vdn):
    rng = np.random.default_rng(17)
    for _ in range(25):
        n = int(rng.integers(1, 4))
        lens_k = [int(x) for x in rng.integers(0, 700, n)]
        lens_q = [int(rng.integers(0, x + 20)) for x in lens_k]
        if sum(lens_q) == 0:
            lens_q[0] = 3
        Hkv = int(rng.integers(1, 3))
        H, d = Hkv * int(rng.integers(1, 3)), int(rng.choice([64, 128]))
        window, ahead = int(rng.integers(1, 400)), int(rng.choice([0, 0, 1, 50, 300]))
        sinks = int(rng.choice([0, 1, 4, 127, 128, 129, 300]))
        q, k, v, cq, ck = make(lens_q, lens_k, H, Hkv, d, seed=n)
        lse = torch.empty((H, q.shape[0]), device="cuda")
        o, ws = vdn.sink_attn(q, k, v, H, Hkv, d, window, sinks, ahead, cq, ck, lse=lse)
        assert vdn.get_device_status(ws) == 0
        check(o, lse, q, k, v, H, Hkv, d, window, sinks, ahead, lens_q, lens_k)


def test_other_sequences_and_rows_of_none_do_not_reach_in(vdn):
    """NaN and infinity in the rows between and behind the sequences: results
    stay what they are without them, and rows of no sequence are not written."""
    H, d, lens = 2, 128, [100, 70]
    q, k, v, _, _ = make([400], [400], H, H, d)
    clean = [vdn.sink_attn(x, y, z, H, H, d, 50, 4)[0] for x, y, z in
             ((q[20:120], k[20:120], v[20:120]), (q[250:320], k[250:320], v[250:320]))]
    bad = torch.ones(400, dtype=torch.bool, device="cuda")
    bad[20:120] = bad[250:320] = False
    for value in (float("nan"), float("inf")):
        for t in (q, k, v):
            t[bad] = value
        # three sequences, the middle one all bad; rows 0..19 and 320.. of none
        cu = torch.tensor([20, 120, 250, 320], dtype=torch.int32, device="cuda")
        out = torch.full_like(q, 9.0)
        lse = torch.full((H, 400), 9.0, device="cuda")
        vdn.sink_attn(q, k, v, H, H, d, 50, 4, cu_q=cu, cu_k=cu, out=out, lse=lse)
        assert torch.equal(out[20:120], clean[0]) and torch.equal(out[250:320], clean[1])
        for none in (slice(0, 20), slice(320, 400)):
            assert (out[none] == 9).all() and (lse[:, none] == 9).all()
        fresh = vdn.sink_attn(q, k, v, H, H, d, 50, 4, cu_q=cu, cu_k=cu)[0]
        assert torch.equal(fresh[20:120], clean[0]) and torch.equal(fresh[250:320], clean[1])
        assert not fresh[:20].any() and not fresh[320:].any()   # zeros in a new output
    few = torch.tensor([5, 9], dtype=torch.int32, device="cuda")    # split over the keys
    kv = torch.tensor([0, 4000], dtype=torch.int32, device="cuda")
    q, k, v, _, _ = make([12], [4000], H, H, d)
    fresh = vdn.sink_attn(q, k, v, H, H, d, None, cu_q=few, cu_k=kv)[0]
    assert torch.equal(fresh[5:9], vdn.sink_attn(q[5:9], k, v, H, H, d, None)[0])
    assert not fresh[:5].any() and not fresh[9:].any()


def test_queries_behind_a_sequence_do_not_reach_its_roundings(vdn):
    """Rows that share a tile with a sequence's last ones: their maxima grow
    from key tile to key tile, and the sequence's bits stay."""
    lens_q, lens_k, H, d = [100, 90], [900, 90], 2, 128
    q, k, v, cq, ck = make(lens_q, lens_k, H, H, d, seed=8)
    kw = dict(window=None, cu_q=cq, cu_k=ck)
    ref = vdn.sink_attn(q, k, v, H, H, d, **kw)[0]
    loud = q.clone()
    loud[100:] *= 200
    assert torch.equal(vdn.sink_attn(loud, k, v, H, H, d, **kw)[0][:100], ref[:100])


@pytest.mark.parametrize("lead", [127, 128, 255, 256, 700])
def test_rows_before_the_first_sequence(vdn, lead):
    """Whole tiles of them, in front of queries and keys that look ahead (the
    rows in all decide how keys are split, so the bits are not those of a call
    without them)."""
    H, d, lens = 2, 64, [300, 77]
    q, k, v, cq, ck = make(lens, lens, H, H, d, seed=lead)
    kw = dict(window=90, sinks=4, ahead=400)
    for lead_k in (0, lead):
        qs, ks, vs = (torch.cat([torch.full((n, H * d), 5.0, device="cuda").bfloat16(), t])
                      for n, t in ((lead, q), (lead_k, k), (lead_k, v)))
        out, got = torch.full_like(qs, 9.0), torch.full((H, lead + sum(lens)), 9.0, device="cuda")
        vdn.sink_attn(qs, ks, vs, H, H, d, cu_q=cq + lead, cu_k=ck + lead_k, out=out, lse=got, **kw)
        check(out[lead:], got[:, lead:], q, k, v, H, H, d, 90, 4, 400, lens, lens)
        assert (out[:lead] == 9).all() and (got[:, :lead] == 9).all()
        fresh = vdn.sink_attn(qs, ks, vs, H, H, d, cu_q=cq + lead, cu_k=ck + lead_k, **kw)[0]
        assert torch.equal(fresh[lead:], out[lead:]) and not fresh[:lead].any()


def test_boundaries_outside_the_rows_are_clamped(vdn):
    q, k, v, _, _ = make([90], [90], 1, 1, 64)
    ref = vdn.sink_attn(q, k, v, 1, 1, 64, 33, 2)[0]
    cu = torch.tensor([-7, 1 << 30], dtype=torch.int32, device="cuda")
    assert torch.equal(vdn.sink_attn(q, k, v, 1, 1, 64, 33, 2, cu_q=cu, cu_k=cu)[0], ref)


def test_large_scores_and_a_row_of_equal_ones(vdn):
    """Scores of +-4000 before the scale and rows that tie: the running maximum
    moves by far more than its threshold."""
    q, k, v, _, _ = make([400], [400], 1, 1, 128, seed=5)
    q, k = q * 16, k * 16
    q[7] = 0
    lse = torch.empty((1, 400), device="cuda")
    o, _ = vdn.sink_attn(q, k, v, 1, 1, 128, 150, 4, lse=lse)
    qs, ks, vs = _f64(q), _f64(k), _f64(v)
    ro, rl, p = attend(qs, ks, vs, visible(400, 400, 150, 4, 0), 128 ** -0.5)
    # the scores' own rounding: 128 additions of up to sum |q k| scale (and as
    # much again in the exponent's argument) weigh here
    off = 130 * 2.0 ** -24 * (np.abs(qs) @ np.abs(ks).T).max() * 128 ** -0.5
    grow = np.expm1(2 * off) + 2.0 ** -12
    assert (np.abs(_f64(o) - ro) <= HALF * np.abs(ro) + (HALF + grow) * (p @ np.abs(vs))).all()
    assert (np.abs(_f64(lse)[0] - rl) <= 2 * off + 2.0 ** -12 + 2.0 ** -23 * np.abs(rl)).all()


def test_captured_replayed_and_on_another_stream(vdn):
    for lens, window in (([900], 100), ([20, 11], 1 << 30)):
        lens_k = [n + 3000 for n in lens] if window > 1000 else lens
        q, k, v, cq, ck = make(lens, lens_k, 4, 2, 128, seed=2)
        kw = dict(window=window, sinks=4, cu_q=cq, cu_k=ck)
        ref, ws = vdn.sink_attn(q, k, v, 4, 2, 128, **kw)
        st = torch.cuda.Stream()
        sq, out = torch.zeros_like(q), torch.empty_like(q)
        st.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(st):
            graph.capture_begin()
            vdn.sink_attn(sq, k, v, 4, 2, 128, out=out, ws=ws, **kw)
            graph.capture_end()
        torch.cuda.current_stream().wait_stream(st)
        sq.copy_(q)
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
        st.wait_stream(torch.cuda.current_stream())
        vdn.sink_attn(q, k, v, 4, 2, 128, out=out.zero_(), ws=ws, stream=torch.cuda.current_stream(),
                      **kw)
        assert torch.equal(out, ref)


@pytest.mark.parametrize("nq,nk,H,Hkv,d,window", [
    (64, 9000, 8, 1, 64, 1 << 30), (16, 8192, 2, 2, 128, 1 << 30), (5, 33, 8, 1, 64, 1 << 30),
    (100, 6000, 2, 1, 128, 5000), (257, 700, 1, 1, 64, 300)])
def test_keys_in_many_parts(vdn, nq, nk, H, Hkv, d, window):
    """Up to 32 parts of a key tile or more each, some of which a query does
    not see."""
    q, k, v, _, _ = make([nq], [nk], H, Hkv, d, seed=nk)
    lse = torch.empty((H, nq), device="cuda")
    o, ws = vdn.sink_attn(q, k, v, H, Hkv, d, window, 3, lse=lse)
    assert vdn.get_device_status(ws) == 0
    check(o, lse, q, k, v, H, Hkv, d, window, 3, 0, [nq], [nk])


def test_no_keys_at_all(vdn):
    q, k, _, _, _ = make([300], [5], 4, 2, 64)
    lse = torch.empty((4, 300), device="cuda")
    o, ws = vdn.sink_attn(q, k[:0], k[:0], 4, 2, 64, 9, 2, 3, lse=lse)
    assert not o.any() and (lse == -np.inf).all()
    dq, dk, dv, ws2 = vdn.sink_attn_backward(q, k[:0], k[:0], o, lse, q, 4, 2, 64, 9, 2, 3)
    assert not dq.any() and dk.shape == dv.shape == (0, 128)
    assert vdn.get_device_status(ws) == vdn.get_device_status(ws2) == 0


def test_two_calls_at_once(vdn):
    """On two streams, with a workspace each (one call splits its keys)."""
    jobs = []
    for lens, lens_k, seed in (([2000], [2000], 1), ([30], [9000], 2)):
        q, k, v, _, _ = make(lens, lens_k, 8, 2, 128, seed=seed)
        ref, ws = vdn.sink_attn(q, k, v, 8, 2, 128, 5000, 4)
        jobs.append((q, k, v, ref, ws, torch.empty_like(ref), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for q, k, v, _, ws, out, st in jobs:
            vdn.sink_attn(q, k, v, 8, 2, 128, 5000, 4, out=out, ws=ws, stream=st)
    torch.cuda.synchronize()
    for _, _, _, ref, ws, out, _ in jobs:
        assert torch.equal(out, ref) and vdn.get_device_status(ws) == 0


def test_long_rows_against_sampled_queries(vdn):
    """20000 tokens, the oracle on a few queries of each kind."""
    n, H, Hkv, d, window, sinks = 20000, 8, 2, 128, 3000, 4
    q, k, v, _, _ = make([n], [n], H, Hkv, d, seed=9)
    lse = torch.empty((H, n), device="cuda")
    o, _ = vdn.sink_attn(q, k, v, H, Hkv, d, window, sinks, lse=lse)
    for i in (0, 3, 127, 128, 2999, 3000, 3003, 3004, 9999, 16383, 19999):
        see = visible(i + 1, i + 1, window, sinks, 0)[-1:]
        for h in (0, 5):
            e = h // 4
            ks, vs = _f64(k[:i + 1, e * d:(e + 1) * d]), _f64(v[:i + 1, e * d:(e + 1) * d])
            ro, rl, p = attend(_f64(q[i:i + 1, h * d:(h + 1) * d]), ks, vs, see, d ** -0.5)
            go = _f64(o[i:i + 1, h * d:(h + 1) * d])
            norm = np.sqrt((p * p) @ (vs * vs).sum(1))
            assert (np.linalg.norm(go - ro, axis=1) <=
                    HALF * (np.linalg.norm(ro, axis=1) + 1.3 * norm)).all()
            assert abs(lse[h, i].item() - rl[0]) <= 2.0 ** -12


def test_refusals(vdn):
    q, k, v, cq, ck = make([8], [8], 2, 1, 64)
    for bad in (dict(window=0), dict(window=4, sinks=-1), dict(window=4, ahead=-1)):
        with pytest.raises(vdn.VdnError):
            vdn.sink_attn(q, k, v, 2, 1, 64, **bad)
    for args in ((q.float(), k, v), (q, k.half(), v), (q, k, v[:4]), (q[:, :64], k, v),
                 (q.cpu(), k, v)):
        with pytest.raises(ValueError):
            vdn.sink_attn(*args, 2, 1, 64, 4)
    with pytest.raises(ValueError):
        vdn.sink_attn(q, k, v, 2, 1, 64, 4, cu_q=cq)
    with pytest.raises(ValueError):
        vdn.sink_attn(q, k, v, 2, 1, 64, 4, cu_q=cq.long(), cu_k=ck.long())
    with pytest.raises(ValueError):
        vdn.sink_attn(q, k, v, 2, 1, 64, 4, lse=torch.empty((2, 9), device="cuda"))
