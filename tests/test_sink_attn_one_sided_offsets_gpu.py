"""The C entry points of the sink-window attention with row offsets for the
queries alone, or for the keys alone (the other side is one sequence of all
its rows): results against the float64 oracle, and the rows of no sequence
zeroed where the call asks for it and left alone where it does not."""

import ctypes

import numpy as np
import pytest
import torch

from tests.parity_util import ensure_built
from tests.test_sink_attn_backward_gpu import check as check_gradients
from tests.test_sink_attn_gpu import check, make

pytestmark = pytest.mark.gpu

H, HKV, WINDOW, SINKS, AHEAD = 4, 2, 90, 3, 2


@pytest.fixture(scope="module")
def vdn():
    ensure_built()
    from video_diffusion_hybrid_vda_b200 import vdn as _vdn
    return _vdn


@pytest.mark.parametrize("zero", range(8))
@pytest.mark.parametrize("given", ["keys", "queries", "both", "neither"])
@pytest.mark.parametrize("d,Lq,Lk", [(64, 200, 300), (128, 17, 900)])
def test_gradients_and_forward(vdn, d, Lq, Lk, given, zero):
    q, k, v, _, _ = make([Lq], [Lk], H, HKV, d, seed=Lq)
    g = make([Lq], [0], H, 1, d, seed=3)[0]
    has = (given in ("queries", "both"), given in ("keys", "both"))
    rows = [(5, n - 3) if on else (0, n) for on, n in zip(has, (Lq, Lk))]
    cu = [torch.tensor(r, dtype=torch.int32, device="cuda") if on else None
          for r, on in zip(rows, has)]
    shape = ctypes.byref(vdn.SinkShape(Lq, Lk, 1, H, HKV, d, WINDOW, AHEAD, SINKS))
    at = [None if c is None else c.data_ptr() for c in cu]
    stream = torch.cuda.current_stream().cuda_stream
    lib = vdn.lib()

    def workspace(call):
        return vdn.alloc_workspace(int(call(shape)))

    o, dq = (torch.full((Lq, H * d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dk, dv = (torch.full((Lk, HKV * d), 7.0, dtype=torch.bfloat16, device="cuda")
              for _ in range(2))
    lse = torch.full((H, Lq), 7.0, device="cuda")
    first = (shape, q.data_ptr(), H * d, k.data_ptr(), v.data_ptr(), HKV * d, *at, 0.0)
    ws = workspace(lib.vdn_sink_attn_workspace)
    assert lib.vdn_sink_attn(*first, o.data_ptr(), H * d, zero & 1, lse.data_ptr(), ws.data_ptr(),
                             ws.numel(), stream) == vdn.VDN_OK
    assert vdn.get_device_status(ws) == 0
    ws = workspace(lib.vdn_sink_attn_backward_workspace)
    assert lib.vdn_sink_attn_backward(
        *first, o.data_ptr(), H * d, lse.data_ptr(), g.data_ptr(), H * d, dq.data_ptr(), H * d,
        dk.data_ptr(), dv.data_ptr(), HKV * d, zero, ws.data_ptr(), ws.numel(),
        stream) == vdn.VDN_OK
    assert vdn.get_device_status(ws) == 0
    rq, rk = slice(*rows[0]), slice(*rows[1])
    lens = [rows[0][1] - rows[0][0]], [rows[1][1] - rows[1][0]]
    check(o[rq], lse[:, rq], q[rq], k[rk], v[rk], H, HKV, d, WINDOW, SINKS, AHEAD, *lens)
    check_gradients([dq[rq], dk[rk], dv[rk]], q[rq], k[rk], v[rk], g[rq], H, HKV, d, WINDOW,
                    SINKS, AHEAD, *lens)
    for x, keep, bit in ((o, rq, 1), (dq, rq, 1), (dk, rk, 2), (dv, rk, 4)):
        rest = np.ones(len(x), dtype=bool)
        rest[keep] = False
        rest = x[torch.from_numpy(rest).cuda()]
        assert (rest == (0.0 if zero & bit else 7.0)).all()
