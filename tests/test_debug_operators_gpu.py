"""The bounds-checking debug build on the query/key preparation and the
sink-window attention: a clean status word and the release library's bits (the
checks change no arithmetic).  Each library runs in a child process, since one
process loads one libvdn."""

import os
import subprocess
import sys

import numpy as np
import pytest

from tests.parity_util import ensure_built

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu

_CHILD = r"""
import sys, numpy as np, torch
sys.path.insert(0, {root!r})
from video_diffusion_hybrid_vda_b200 import vdn
vdn.LIB_PATH = {lib!r}
g = torch.Generator("cuda").manual_seed(7)
def normal(*s):
    return torch.randn(*s, generator=g, device="cuda").bfloat16()
H, Hkv, d = 6, 2, 64
lens = [300, 1, 150]
L = sum(lens)
cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
q, k, v, d_o = normal(L, H * d), normal(L, Hkv * d), normal(L, Hkv * d), normal(L, H * d)
out, st = [], []
plan = vdn.RopePlan(d, rot=48, layout="interleaved")
out.append(vdn.rope(q, H, plan))
qn, kn = vdn.qk_norm_rope(q, k, H, Hkv, plan)
out += [qn, kn]
*grads, ws = vdn.qk_norm_rope_backward(q, k, d_o, d_o[:, :Hkv * d], H, Hkv, plan)
out += grads; st.append(vdn.get_device_status(ws))
for kw in (dict(window=70, sinks=4, cu_q=cu, cu_k=cu), dict(window=400, sinks=200),
           dict(window=20, sinks=2, ahead=30)):
    lse = torch.empty((H, L), device="cuda")
    o, ws = vdn.sink_attn(qn, kn, v, H, Hkv, d, lse=lse, **kw)
    out += [o, lse]; st.append(vdn.get_device_status(ws))
    *grads, ws = vdn.sink_attn_backward(qn, kn, v, o, lse, d_o, H, Hkv, d, **kw)
    out += grads; st.append(vdn.get_device_status(ws))
long_k, long_v = normal(5000, Hkv * d), normal(5000, Hkv * d)
o, ws = vdn.sink_attn(q[:40], long_k, long_v, H, Hkv, d, None)   # split over the keys
out.append(o); st.append(vdn.get_device_status(ws))
*grads, ws = vdn.sink_attn_backward(long_k, long_k, long_v, long_v,
                                    torch.zeros((Hkv, 5000), device="cuda") + 9, long_v, Hkv, Hkv,
                                    d, 100, 4)
out += grads; st.append(vdn.get_device_status(ws))
caches = [normal(3, 104, Hkv * d) for _ in range(2)]
pos = torch.tensor([5, 103, 900], dtype=torch.int32, device="cuda")
out += [vdn.sink_attn_step(q[:3], k[:3], v[:3], *caches, pos, H, Hkv, d, 100, 4), *caches]
torch.cuda.synchronize()
np.savez({path!r}, *[t.float().cpu().numpy() for t in out], status=np.array(st),
         enabled=np.array(int(vdn.debug_bounds_enabled())))
"""


def _run(lib, path):
    code = _CHILD.format(root=ROOT, lib=lib, path=path)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stderr[-3000:]
    return np.load(path)


def test_debug_build_matches_release_with_clean_status(tmp_path):
    ensure_built()
    from video_diffusion_hybrid_vda_b200 import build
    rel = _run(build.LIB, str(tmp_path / "rel.npz"))
    dbg = _run(build.build(debug_bounds=True), str(tmp_path / "dbg.npz"))
    assert int(rel["enabled"]) == 0 and int(dbg["enabled"]) == 1
    assert not rel["status"].any() and not dbg["status"].any()
    for name in rel.files:
        if name not in ("status", "enabled"):
            assert np.array_equal(rel[name], dbg[name], equal_nan=True), name
