"""Sink-window attention and its gradients at sizes of their own: more key
tiles than the plan takes in at a time, element offsets past 2^31, two gradient
calls at once, long rows of head dim 64, many short sequences that forget
nothing."""

import numpy as np
import pytest
import torch

from oracle.sink_attn import attend, visible
from tests.parity_util import ensure_built
from tests.test_sink_attn_backward_gpu import check as check_gradients
from tests.test_sink_attn_backward_gpu import step
from tests.test_sink_attn_gpu import HALF, _f64, check, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vdn():
    ensure_built()
    from video_diffusion_hybrid_vda_b200 import vdn as _vdn
    return _vdn


@pytest.mark.parametrize("lens_q,lens_k,H,Hkv,d,window,sinks,ahead", [
    ([n % 97 for n in range(300)], [n % 97 for n in range(300)], 2, 1, 64, 40, 3, 0),
    ([0] * 255 + [200, 5], [0] * 254 + [1, 300, 130], 2, 2, 128, 1 << 30, 0, 4),
    ([1] * 600 + [700], [130] * 600 + [700], 1, 1, 64, 300, 2, 0),
])
def test_gradients_of_many_key_tiles(vdn, lens_q, lens_k, H, Hkv, d, window, sinks, ahead):
    """The plan's prefix sums run over 256 slots at a time (a slot a key tile of
    128, and one more a sequence)."""
    assert sum(lens_k) // 128 + len(lens_k) > 256
    q, k, v, cq, ck = make(lens_q, lens_k, H, Hkv, d, seed=8)
    g = make(lens_q, [0], H, 1, d, seed=9)[0]
    a = step(vdn, q, k, v, g, H, Hkv, d, window, sinks, ahead, cq, ck)
    check_gradients(a[:3], q, k, v, g, H, Hkv, d, window, sinks, ahead, lens_q, lens_k)
    b = step(vdn, q, k, v, g, H, Hkv, d, window, sinks, ahead, cq, ck)
    assert all(torch.equal(x, y) for x, y in zip(a[:3], b[:3]))


def test_gradients_at_offsets_past_32_bits(vdn):
    """Rows 2^23 elements apart: the last ones begin past element 2^31."""
    n, H, Hkv, d, ld = 290, 2, 1, 64, 1 << 23
    small = dict(zip("qkv", make([n], [n], H, Hkv, d, seed=4)[:3]))
    small["g"] = make([n], [0], H, 1, d, seed=5)[0]
    flat = torch.empty((n - 1) * ld + 8 * H * d, dtype=torch.bfloat16, device="cuda")
    assert (n - 1) * ld > 1 << 31

    def far(place, cols):
        return flat.as_strided((n, cols), (ld, 1), place * H * d)

    wide = {name: far(i, t.shape[1]).copy_(t) for i, (name, t) in enumerate(small.items())}
    dq, dk, dv = far(4, H * d), far(5, Hkv * d), far(6, Hkv * d)
    mask = dict(window=150, sinks=2)
    lse, lse2 = (torch.empty((H, n), device="cuda") for _ in range(2))
    ref, _ = vdn.sink_attn(*(small[c] for c in "qkv"), H, Hkv, d, lse=lse, **mask)
    o, ws = vdn.sink_attn(*(wide[c] for c in "qkv"), H, Hkv, d, out=far(7, H * d), lse=lse2,
                          **mask)
    assert torch.equal(o, ref) and torch.equal(lse, lse2) and vdn.get_device_status(ws) == 0
    want = vdn.sink_attn_backward(*(small[c] for c in "qkv"), ref, lse, small["g"], H, Hkv, d,
                                  **mask)
    got = vdn.sink_attn_backward(*(wide[c] for c in "qkv"), o, lse2, wide["g"], H, Hkv, d, dq=dq,
                                 dk=dk, dv=dv, **mask)
    assert all(torch.equal(x, y) for x, y in zip(got[:3], want[:3]))
    assert all(torch.equal(wide[c], small[c]) for c in small)


def test_two_gradient_calls_at_once(vdn):
    jobs = []
    for lens, H, Hkv, d, seed in (([2000, 77], 8, 2, 128, 1), ([300, 5], 2, 2, 64, 2)):
        q, k, v, cq, ck = make(lens, lens, H, Hkv, d, seed=seed)
        kw = dict(window=200, sinks=4, cu_q=cq, cu_k=ck)
        lse = torch.empty((H, len(q)), device="cuda")
        o, _ = vdn.sink_attn(q, k, v, H, Hkv, d, lse=lse, **kw)

        def call(q=q, k=k, v=v, o=o, lse=lse, H=H, Hkv=Hkv, d=d, kw=kw, **more):
            return vdn.sink_attn_backward(q, k, v, o, lse, q, H, Hkv, d, **kw, **more)

        jobs.append((call, call(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    results = [[call(stream=st) for call, _, st in jobs] for _ in range(5)]
    torch.cuda.synchronize()
    for row in results:
        for got, (_, ref, _) in zip(row, jobs):
            assert all(torch.equal(x, y) for x, y in zip(got[:3], ref[:3]))
            assert vdn.get_device_status(got[3]) == 0


def test_long_rows_of_head_dim_64(vdn):
    """20000 tokens, the oracle on a few queries of each kind."""
    n, H, Hkv, d, window, sinks = 20000, 6, 3, 64, 3000, 5
    q, k, v, _, _ = make([n], [n], H, Hkv, d, seed=9)
    lse = torch.empty((H, n), device="cuda")
    o, ws = vdn.sink_attn(q, k, v, H, Hkv, d, window, sinks, lse=lse)
    assert vdn.get_device_status(ws) == 0
    for i in (0, 4, 127, 128, 255, 256, 2999, 3000, 3004, 3005, 9999, 16383, 19999):
        see = visible(i + 1, i + 1, window, sinks, 0)[-1:]
        for h in (0, 5):
            e = h // 2
            ks, vs = _f64(k[:i + 1, e * d:(e + 1) * d]), _f64(v[:i + 1, e * d:(e + 1) * d])
            ro, rl, p = attend(_f64(q[i:i + 1, h * d:(h + 1) * d]), ks, vs, see, d ** -0.5)
            go = _f64(o[i:i + 1, h * d:(h + 1) * d])
            norm = np.sqrt((p * p) @ (vs * vs).sum(1))
            assert (np.linalg.norm(go - ro, axis=1) <=
                    HALF * (np.linalg.norm(ro, axis=1) + 1.3 * norm)).all()
            assert abs(lse[h, i].item() - rl[0]) <= 2.0 ** -12


@pytest.mark.parametrize("lens,H,Hkv,d", [([100] * 16, 2, 1, 128), ([64] * 32, 2, 2, 64),
                                          ([250] * 8, 2, 1, 128), ([1] * 40 + [900], 4, 1, 64)])
def test_many_short_sequences_that_forget_nothing(vdn, lens, H, Hkv, d):
    q, k, v, cq, ck = make(lens, lens, H, Hkv, d, seed=len(lens))
    lse = torch.empty((H, len(q)), device="cuda")
    o, ws = vdn.sink_attn(q, k, v, H, Hkv, d, None, cu_q=cq, cu_k=ck, lse=lse)
    assert vdn.get_device_status(ws) == 0
    check(o, lse, q, k, v, H, Hkv, d, 1 << 30, 0, 0, lens, lens)
