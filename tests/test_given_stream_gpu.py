"""The rotation and sink-window calls on a stream of the caller's that is not
torch's current one, with outputs and workspaces of their own: memory that the
current stream still uses is not written, and memory that the call uses is not
given away."""

import pytest
import torch

from tests.parity_util import ensure_built

pytestmark = pytest.mark.gpu

DELAY = 100_000_000  # cycles, some 50 ms: what a stream does behind it comes last


@pytest.fixture(scope="module")
def vdn():
    ensure_built()
    from video_diffusion_hybrid_vda_b200 import vdn as _vdn
    return _vdn


def _normal(rows, cols, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(rows, cols, generator=gen, device="cuda").bfloat16()


def _rope(vdn):
    x, plan = _normal(300, 256, 1), vdn.RopePlan(128)
    return lambda **kw: [vdn.rope(x, 2, plan, **kw)]


def _qk(vdn):
    q, k, plan = _normal(300, 256, 1), _normal(300, 128, 2), vdn.RopePlan(128)
    return lambda **kw: list(vdn.qk_norm_rope(q, k, 2, 1, plan, **kw))


def _qk_backward(vdn):
    q, k, plan = _normal(300, 256, 1), _normal(300, 128, 2), vdn.RopePlan(128)
    return lambda **kw: list(vdn.qk_norm_rope_backward(q, k, q, k, 2, 1, plan, **kw)[:4])


def _sink(nq, nk):
    def call(vdn):
        q, k, v = _normal(nq, 512, 1), _normal(nk, 256, 2), _normal(nk, 256, 3)
        return lambda **kw: [vdn.sink_attn(q, k, v, 4, 2, 128, 4000, 4, **kw)[0]]
    return call


def _sink_backward(nq, nk):
    def call(vdn):
        q, k, v = _normal(nq, 512, 1), _normal(nk, 256, 2), _normal(nk, 256, 3)
        lse = torch.empty((4, nq), device="cuda")
        o, _ = vdn.sink_attn(q, k, v, 4, 2, 128, 900, 4, lse=lse)
        return lambda **kw: list(vdn.sink_attn_backward(q, k, v, o, lse, q, 4, 2, 128, 900, 4,
                                                        **kw)[:3])
    return call


def _step(vdn):
    q, kn, vn = _normal(3, 512, 1), _normal(3, 256, 2), _normal(3, 256, 3)
    kc, vc = _normal(3 * 50, 256, 4).view(3, 50, 256), _normal(3 * 50, 256, 5).view(3, 50, 256)
    pos = torch.tensor([7, 100, 49], dtype=torch.int32, device="cuda")
    return lambda **kw: [vdn.sink_attn_step(q, kn, vn, kc, vc, pos, 4, 2, 128, 48, 2, **kw)]


CALLS = {"rope": _rope, "qk_norm_rope": _qk, "qk_norm_rope_backward": _qk_backward,
         "sink_attn": _sink(700, 700), "sink_attn in parts": _sink(40, 3000),
         "sink_attn_backward": _sink_backward(700, 700),
         "sink_attn_backward in parts": _sink_backward(1500, 2000), "sink_attn_step": _step}


@pytest.fixture(params=list(CALLS))
def case(request, vdn):
    """(the call, its results on the current stream, another stream)"""
    call = CALLS[request.param](vdn)
    ref = call()
    st = torch.cuda.Stream()
    torch.cuda._sleep(1)  # a kernel's first launch may wait for the whole device
    for t in (*ref, torch.empty(9, dtype=torch.uint8, device="cuda")):
        torch.empty_like(t).fill_(7)
        t.clone()
    torch.cuda.synchronize()
    return call, ref, st


def _same(got, ref):
    return all(torch.equal(a, b) for a, b in zip(got, ref))


def test_new_outputs_do_not_take_memory_that_the_current_stream_still_writes(case):
    call, ref, st = case
    first = call(stream=st)  # the stream's own first allocations
    torch.cuda.synchronize()
    old = [torch.empty_like(r) for r in ref for _ in range(8)]
    torch.cuda._sleep(DELAY)
    for t in old:
        t.fill_(7)
    del old, t
    got = call(stream=st)
    torch.cuda.synchronize()
    assert _same(got, ref) and _same(first, ref)


def test_a_dropped_workspace_stays_with_the_call(case, vdn, monkeypatch):
    call, ref, st = case
    sizes, alloc = [], vdn.alloc_workspace
    monkeypatch.setattr(vdn, "alloc_workspace",
                        lambda n, *a, **kw: (sizes.append(max(int(n), 256)), alloc(n, *a, **kw))[1])
    with torch.cuda.stream(st):
        torch.cuda._sleep(DELAY)
    got = call(stream=st)  # its workspace is dropped here, long before it runs
    junk = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(12)]
    torch.cuda.synchronize()
    assert all((j == 7).all() for j in junk)
    assert _same(got, ref)


def test_a_dropped_result_waits_for_the_current_stream(case):
    call, ref, st = case
    got = call(stream=st)
    torch.cuda.current_stream().wait_stream(st)
    torch.cuda._sleep(DELAY)
    read = [t.clone() for t in got]
    shapes = [(t.shape, t.dtype) for t in got]
    del got
    with torch.cuda.stream(st):
        for shape, dtype in shapes:
            torch.full(shape, 9, dtype=dtype, device="cuda")
    torch.cuda.synchronize()
    assert _same(read, ref)


def test_inputs_that_arrive_late_on_the_stream(vdn):
    """The call runs on the stream it is given, behind what is there."""
    late = [_normal(n, 256, n) for n in (40, 3000, 3000)]
    ref, _ = vdn.sink_attn(*late, 2, 2, 128, 4000, 4)
    q, k, v = (torch.zeros_like(t) for t in late)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        torch.cuda._sleep(DELAY)
        for t, x in zip((q, k, v), late):
            t.copy_(x)
    out, ws = vdn.sink_attn(q, k, v, 2, 2, 128, 4000, 4, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(out, ref)
    q.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        torch.cuda._sleep(DELAY)
        q.copy_(late[0])
    vdn.sink_attn(q, k, v, 2, 2, 128, 4000, 4, out=out, ws=ws, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(out, ref) and vdn.get_device_status(ws) == 0


def test_captured_on_a_stream_that_is_given(vdn):
    call = _sink(40, 3000)(vdn)
    ref, st, graph = call(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=st):
        got = call(stream=st)
    for _ in range(2):
        got[0].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert _same(got, ref)


def test_captured_on_a_forked_stream(vdn):
    """Two calls side by side in one graph, each with memory of its own."""
    calls = [_sink(40, 3000)(vdn), _sink(700, 700)(vdn)]
    refs, st, graph = [c() for c in calls], torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        st.wait_stream(here)
        got = [calls[0](stream=st), calls[1]()]
        here.wait_stream(st)
    for _ in range(2):
        for g in got:
            g[0].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(_same(g, r) for g, r in zip(got, refs))
