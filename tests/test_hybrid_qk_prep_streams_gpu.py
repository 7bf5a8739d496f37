"""HybridLayer with qk_prep on values that are views of a fused projection, and
on a stream of the caller's: the same kernels on the same numbers as the
contiguous call on the current stream, so the same bits."""

import pytest
import torch

from tests.parity_util import ensure_built
from video_diffusion_hybrid_vda_b200 import synth

pytestmark = pytest.mark.gpu

S_T = 6              # frames
DELAY = 100_000_000  # cycles, some 50 ms: what a stream does behind it comes last


@pytest.fixture(scope="module")
def vdn():
    ensure_built()
    from video_diffusion_hybrid_vda_b200 import vdn as _vdn
    return _vdn


def _case(vdn, d=64, **kw):
    s = synth.Shape(S_T, 96, 4, d)
    x = synth.make_inputs(s, seed=5, device="cuda", with_fuse=True)
    x["k"] = x["k"] * 5
    layer = vdn.HybridLayer(s.T, s.N, s.H, s.d, x["W_gs"], x["W_gl"], x["W_os"], x["W_ol"],
                            x["gamma"], qk_prep=vdn.QKPrep(vdn.RopePlan(d)), **kw)
    ref = layer.forward(x["q"], x["k"], x["v"], x["beta"], x["alpha"], x["x"]).clone()
    torch.cuda.synchronize()
    return s, x, layer, ref


# row strides of v: a fused q, k, v projection; v beside a little; two tensors in one
@pytest.mark.parametrize("wide", [0, 8, 256, 512])
def test_values_of_a_wider_row_are_read_in_place(vdn, wide, monkeypatch):
    s, x, layer, ref = _case(vdn)
    buf = torch.full((s.L, s.D + wide), float("nan"), dtype=torch.bfloat16, device="cuda")
    v = buf[:, wide:]
    v.copy_(x["v"])
    seen = []
    window_attn = vdn.window_attn
    monkeypatch.setattr(vdn, "window_attn", lambda q, k, v, *a, **kw: (
        seen.append((q.stride(0), k.stride(0), v.data_ptr())), window_attn(q, k, v, *a, **kw))[1])
    for _ in range(2):
        y = layer.forward(x["q"], x["k"], v, x["beta"], x["alpha"], x["x"])
        assert torch.equal(y, ref) and layer.status() == 0
        # a different video's contiguous v in between
        layer.forward(x["q"], x["k"], x["v"] * 2, x["beta"], x["alpha"], x["x"])
    assert seen[0] == seen[2] == (s.D + wide, s.D + wide, v.data_ptr())


@pytest.mark.parametrize("d,softmax", [(64, "bf16"), (128, "bf16"), (128, "mxfp8")])
def test_fused_projection_on_a_stream_that_is_behind(vdn, d, softmax):
    """q, k and v arrive late on the caller's stream: all that reads them comes
    after them."""
    s, x, layer, ref = _case(vdn, d, softmax=softmax)
    late = torch.cat([x["q"], x["k"], x["v"]], 1)
    qkv = torch.zeros_like(late)
    q, k, v = qkv[:, :s.D], qkv[:, s.D:2 * s.D], qkv[:, 2 * s.D:]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for _ in range(2):
        with torch.cuda.stream(st):
            torch.cuda._sleep(DELAY)
            qkv.copy_(late)
        y = layer.forward(q, k, v, x["beta"], x["alpha"], x["x"], stream=st)
        torch.empty_like(x["v"]).fill_(7)  # what the call dropped may not be in use
        torch.cuda.current_stream().wait_stream(st)
        assert torch.equal(y, ref) and layer.status() == 0
        qkv.zero_()
        st.wait_stream(torch.cuda.current_stream())


@pytest.mark.parametrize("kind", ["odd stride", "odd address", "columns apart", "one row"])
def test_values_that_the_branches_cannot_read_are_copied(vdn, kind):
    s, x, layer, ref = _case(vdn)
    late = x["v"]
    if kind == "odd stride":
        v = torch.zeros((s.L, s.D + 1), dtype=torch.bfloat16, device="cuda")[:, :s.D]
    elif kind == "odd address":
        v = torch.zeros((s.L, s.D + 8), dtype=torch.bfloat16, device="cuda")[:, 1:1 + s.D]
    elif kind == "columns apart":
        v = torch.zeros((s.D, s.L), dtype=torch.bfloat16, device="cuda").T
    else:  # expanded: every token has the first one's value
        v = torch.zeros((1, s.D), dtype=torch.bfloat16, device="cuda").expand(s.L, s.D)
        late = x["v"][:1]
        ref = layer.forward(x["q"], x["k"], late.expand(s.L, s.D).contiguous(), x["beta"],
                            x["alpha"], x["x"]).clone()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        torch.cuda._sleep(DELAY)
        (v[:1] if kind == "one row" else v).copy_(late)
    y = layer.forward(x["q"], x["k"], v, x["beta"], x["alpha"], x["x"], stream=st)
    torch.empty_like(x["v"]).fill_(7)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(y, ref) and layer.status() == 0


@pytest.mark.parametrize("bad", [lambda v: v.float(), lambda v: v.half(), lambda v: v[:-1]])
def test_values_of_another_type_or_size_are_refused(vdn, bad):
    s, x, layer, ref = _case(vdn)
    with pytest.raises(ValueError):
        layer.forward(x["q"], x["k"], bad(x["v"]), x["beta"], x["alpha"], x["x"])


@pytest.mark.parametrize("other", [
    lambda v: torch.cat([v, v[:5]]), lambda v: v.view(S_T, -1, v.shape[1]),
    lambda v: v.view(len(v), 4, -1),
    lambda v: torch.stack([v, v, v], 1)[:, 1].unflatten(1, (4, -1))])
def test_values_of_another_shape_or_with_more_rows(vdn, other):
    s, x, layer, ref = _case(vdn)
    y = layer.forward(x["q"], x["k"], other(x["v"]), x["beta"], x["alpha"], x["x"])
    assert torch.equal(y, ref) and layer.status() == 0


def test_captured_with_a_fused_projection_beside_contiguous_calls(vdn):
    """The buffers of a captured call stay, whatever strides later calls bring."""
    s, x, layer, ref = _case(vdn)
    qkv = torch.cat([x["q"], x["k"], x["v"]], 1)
    fused = [qkv[:, i * s.D:(i + 1) * s.D] for i in range(3)]
    rest = (x["beta"], x["alpha"], x["x"])
    layer.forward(*fused, *rest)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer.forward(*fused, *rest)
    for wide in (8, 256):
        v = torch.cat([x["v"], torch.zeros((s.L, wide), dtype=torch.bfloat16, device="cuda")], 1)
        layer.forward(x["q"], x["k"], v[:, :s.D] * 3, *rest)
        assert torch.equal(layer.forward(x["q"], x["k"], v[:, :s.D], *rest), ref)
    junk = [torch.full((s.L, 3 * s.D), float("nan"), device="cuda") for _ in range(4)]
    y.zero_()
    graph.replay()
    assert torch.equal(y, ref)
    del junk
