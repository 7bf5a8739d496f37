"""HybridLayer with qk_prep: the norm and rotation in the layer's own paths
(forward, head groups and staged videos of forward_many) against the operator
and the layer called one after the other: the same kernels on the same
numbers, so the same bits."""

import pytest
import torch

from tests.parity_util import ensure_built
from video_diffusion_hybrid_vda_b200 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vdn():
    ensure_built()
    from video_diffusion_hybrid_vda_b200 import vdn as _vdn
    return _vdn


def _layer(vdn, s, x, **kw):
    return vdn.HybridLayer(s.T, s.N, s.H, s.d, x["W_gs"], x["W_gl"], x["W_os"], x["W_ol"],
                           x["gamma"], **kw)


@pytest.mark.parametrize("T,rows,cols,H,d", [(7, 8, 12, 4, 64), (6, 6, 16, 2, 128)])
def test_layer_with_prep_is_the_operator_then_the_layer(vdn, T, rows, cols, H, d):
    s = synth.Shape(T, rows * cols, H, d)
    x = synth.make_inputs(s, seed=3, device="cuda", with_fuse=True)
    k = x["k"] * 5                              # not of unit length: the prep sees to it
    pos = vdn.video_positions(T, rows, cols)
    assert pos.shape == (3, s.L) and pos[:, rows * cols + cols + 2].tolist() == [1, 1, 2]
    third = d // 6
    plan = vdn.RopePlan(d, sections=[d // 2 - 2 * third, third, third])
    w = 1 + 0.1 * torch.randn(d, device="cuda")
    prep = vdn.QKPrep(plan, wq=w, positions=pos)
    plain, prepped = _layer(vdn, s, x), _layer(vdn, s, x, qk_prep=prep)
    assert prepped.kernels_per_forward == plain.kernels_per_forward + 1
    q0, k0 = x["q"].clone(), k.clone()
    y = prepped.forward(x["q"], k, x["v"], x["beta"], x["alpha"], x["x"]).clone()
    assert torch.equal(x["q"], q0) and torch.equal(k, k0)
    qn, kn = vdn.qk_norm_rope(x["q"], k, H, H, plan, wq=w, k_norm="l2", positions=pos)
    assert (kn.float().view(s.L, H, d).norm(dim=-1) - 1).abs().max() < 2 ** -7
    ref = plain.forward(qn, kn, x["v"], x["beta"], x["alpha"], x["x"])
    assert torch.equal(y, ref) and prepped.status() == 0
    # several videos from pinned host memory: head groups, then staged videos
    host = [t.cpu().pin_memory() for t in (x["q"], k, x["v"], x["beta"], x["alpha"], x["x"])]
    outs = [torch.empty((s.L, s.D), dtype=torch.bfloat16).pin_memory() for _ in range(3)]
    for _ in range(2):
        prepped.forward_many([host] * 3, outs)
        torch.cuda.synchronize()
        for o in outs:
            assert torch.equal(o, y.cpu())


def test_prep_of_another_head_dim_is_refused(vdn):
    s = synth.Shape(2, 16, 2, 64)
    x = synth.make_inputs(s, seed=1, device="cuda", with_fuse=True)
    with pytest.raises(ValueError):
        _layer(vdn, s, x, qk_prep=vdn.QKPrep(vdn.RopePlan(128)))
