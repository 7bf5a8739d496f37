"""The layer's calls on a stream of the caller's that is not torch's current
one, with outputs and workspaces of their own (the tests of the rotation and
sink-window calls), and the layer itself with host inputs."""

import pytest
import torch

from tests.parity_util import ensure_built
from tests.test_given_stream_gpu import (  # noqa: F401  (collected with the cases here)
    DELAY, _same, test_a_dropped_result_waits_for_the_current_stream,
    test_a_dropped_workspace_stays_with_the_call,
    test_new_outputs_do_not_take_memory_that_the_current_stream_still_writes)
from video_diffusion_hybrid_vda_b200 import synth

pytestmark = pytest.mark.gpu

S = synth.Shape(6, 96, 4, 128)
DIMS = (S.T, S.N, S.H, S.d)


@pytest.fixture(scope="module")
def vdn():
    ensure_built()
    from video_diffusion_hybrid_vda_b200 import vdn as _vdn
    return _vdn


@pytest.fixture(scope="module")
def inputs():
    x = synth.make_inputs(S, seed=5, device="cuda", with_fuse=True)
    x["weights"] = (x["W_gs"], x["W_gl"], x["gamma"], x["W_os"], x["W_ol"])
    return x


def _fuse_mxfp8(vdn, x, **kw):
    wg, wo = x["mx"]
    return [vdn.hybrid_fuse_mxfp8(x["x"], x["q"], x["v"], wg, x["gamma"], wo, S.H, **kw)[0]]


def _shard_rs(vdn, x, stream=None):
    with torch.cuda.stream(stream):
        owner = torch.zeros((S.L, S.D), device="cuda")
    owner.record_stream(torch.cuda.current_stream())
    vdn.hybrid_fuse_shard_rs(x["x"], x["q"], x["v"], *x["weights"], S.d, 0, [owner], stream=stream)
    return [owner]


CALLS = {
    "vda_scan": lambda vdn, x, **kw: [vdn.vda_scan(*x["scan"], *DIMS, **kw)[0]],
    "vda_scan_static": lambda vdn, x, **kw: list(vdn.vda_scan_static(*x["scan"], *DIMS, **kw)),
    "vda_backward": lambda vdn, x, **kw: list(
        vdn.vda_backward(*x["scan"], x["x"], *DIMS, **kw)[:5]),
    "mxfp8_quantize": lambda vdn, x, **kw: list(vdn.mxfp8_quantize(x["q"], **kw)),
    "gemm_mxfp8": lambda vdn, x, **kw: [vdn.gemm_mxfp8(x["mx"][0], x["mx"][1], **kw)[0]],
    "window_attn": lambda vdn, x, **kw: [
        vdn.window_attn(x["q"], x["k"], x["v"], *DIMS, **kw)[0]],
    "window_attn_mxfp8": lambda vdn, x, **kw: [
        vdn.window_attn_mxfp8(x["q"], x["k"], x["v"], *DIMS, **kw)[0]],
    "hybrid_fuse": lambda vdn, x, **kw: [
        vdn.hybrid_fuse(x["x"], x["q"], x["v"], *x["weights"], S.H, **kw)[0]],
    "hybrid_fuse_mxfp8": _fuse_mxfp8,
    "hybrid_fuse_shard": lambda vdn, x, **kw: [
        vdn.hybrid_fuse_shard(x["x"], x["q"], x["v"], *x["weights"], S.d, 0, **kw)[0]],
    "hybrid_fuse_shard_rs": _shard_rs,
    "selftest_exp2": lambda vdn, x, **kw: list(vdn.selftest_exp2(x["beta"], **kw)),
}


@pytest.fixture(params=list(CALLS))
def case(request, vdn, inputs):
    """(the call, its results on the current stream, another stream)"""
    inputs["scan"] = tuple(inputs[n] for n in ("q", "k", "v", "beta", "alpha"))
    wg, wo = vdn.mxfp8_fuse_weights(*(inputs[n] for n in ("W_gs", "W_gl", "W_os", "W_ol")))
    # as operands of a product: [2 D, D] and [D, D]
    inputs["mx"] = (wg, vdn.mxfp8_quantize(inputs["W_os"])) if request.param == "gemm_mxfp8" \
        else (wg, wo)

    def call(**kw):
        return CALLS[request.param](vdn, inputs, **kw)

    ref, st = call(), torch.cuda.Stream()
    torch.cuda._sleep(1)  # a kernel's first launch may wait for the whole device
    for t in (*ref, torch.empty(9, dtype=torch.uint8, device="cuda")):
        torch.empty_like(t).fill_(7)
        t.clone()
    torch.cuda.synchronize()
    return call, ref, st


def test_fuse_weights_that_arrive_late_on_the_stream(vdn, inputs):
    late = [inputs[n] for n in ("W_gs", "W_gl", "W_os", "W_ol")]
    ref = [t for pair in vdn.mxfp8_fuse_weights(*late) for t in pair]
    here, st = [torch.zeros_like(t) for t in late], torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        torch.cuda._sleep(DELAY)
        for t, x in zip(here, late):
            t.copy_(x)
    got = [t for pair in vdn.mxfp8_fuse_weights(*here, stream=st) for t in pair]
    [torch.empty((2 * S.D, S.D), dtype=torch.bfloat16, device="cuda").fill_(7) for _ in range(4)]
    torch.cuda.synchronize()
    assert _same(got, ref)


@pytest.mark.parametrize("many", [False, True])
def test_the_layers_buffers_for_host_inputs(vdn, inputs, many):
    """What the current stream has yet to read is not written."""
    names = ("q", "k", "v", "beta", "alpha", "x")
    host = [inputs[n].cpu().pin_memory() for n in names]
    layer = vdn.HybridLayer(*DIMS, *(inputs[n] for n in ("W_gs", "W_gl", "W_os", "W_ol", "gamma")))
    ref = layer.forward(*(inputs[n] for n in names)).cpu()
    outs = [torch.empty((S.L, S.D), dtype=torch.bfloat16).pin_memory() for _ in range(3)]
    st = torch.cuda.Stream()
    old = [torch.empty_like(inputs[n]).fill_(7) for n in names for _ in range(6)]
    [t.clone() for t in old]
    torch.cuda.synchronize()
    torch.cuda._sleep(DELAY)
    read = [t.clone() for t in old]
    del old
    if many:
        layer.forward_many([host] * 3, outs, stream=st)
    else:
        outs = outs[:1]
        layer.forward(*host, out=outs[0], stream=st)
    torch.cuda.synchronize()
    assert all((t == 7).all() for t in read)
    assert all(torch.equal(o, ref) for o in outs) and layer.status() == 0
