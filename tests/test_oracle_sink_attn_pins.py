"""The sink-window attention oracle against a loop over its definition, central
differences, and the library's refusals on the host."""

import ctypes
import math

import numpy as np
import pytest

import oracle
from oracle.sink_attn import sink_attn, visible
from tests.parity_util import ensure_built

RNG = np.random.default_rng(11)


def _plain(q, k, v, H, H_kv, window, sinks, ahead):
    d = q.shape[1] // H
    o, lse = np.zeros_like(q), np.full((H, len(q)), -np.inf)
    for h in range(H):
        e = h // (H // H_kv)
        for i in range(len(q)):
            p = i + len(k) - len(q)
            js = [j for j in range(len(k)) if j <= p + ahead and (p - j < window or j < sinks)]
            if not js:
                continue
            s = [float(q[i, h * d:(h + 1) * d] @ k[j, e * d:(e + 1) * d]) / math.sqrt(d)
                 for j in js]
            w = np.exp(s)
            lse[h, i] = math.log(w.sum())
            o[i, h * d:(h + 1) * d] = (w / w.sum()) @ v[js, e * d:(e + 1) * d]
    return o, lse


@pytest.mark.parametrize("nq,nk,window,sinks,ahead", [
    (9, 9, 3, 1, 0), (9, 9, 100, 0, 0), (4, 11, 2, 2, 0), (7, 3, 2, 0, 0), (6, 6, 2, 1, 2),
    (1, 5, 1, 0, 0), (3, 0, 4, 1, 0), (5, 2, 1, 5, 1)])
def test_against_the_definition(nq, nk, window, sinks, ahead):
    q, k, v = (RNG.standard_normal((n, w)) for n, w in ((nq, 32), (nk, 16), (nk, 16)))
    o, lse = sink_attn(q, k, v, 4, 2, window, sinks, ahead)
    ro, rl = _plain(q, k, v, 4, 2, window, sinks, ahead)
    np.testing.assert_allclose(o, ro, atol=1e-13)
    np.testing.assert_allclose(lse, rl, atol=1e-13)


def test_a_window_over_everything_is_the_window_softmax_of_one_frame():
    q, k, v = (RNG.standard_normal((12, 32)) for _ in range(3))
    o, lse = sink_attn(q, k, v, 2, 2, 100, 0, 100)
    ro, rl = oracle.window_attn(q, k, v, 1, 12, 2, 16)
    np.testing.assert_allclose(o, ro, atol=1e-12)
    np.testing.assert_allclose(lse, rl, atol=1e-12)


def test_gradients_against_central_differences():
    args = dict(H=4, H_kv=2, window=3, sinks=1, ahead=1, lens_q=[5, 0, 4], lens_k=[5, 2, 3])
    x = [RNG.standard_normal((9, 32)), RNG.standard_normal((10, 16)), RNG.standard_normal((10, 16))]
    g = RNG.standard_normal((9, 32))
    grads = sink_attn(*x, d_o=g, **args)[2:]
    h = 1e-5
    for n in range(3):
        for _ in range(25):
            at = tuple(RNG.integers(0, m) for m in x[n].shape)
            pair = []
            for sign in (1, -1):
                y = [t.copy() for t in x]
                y[n][at] += sign * h
                pair.append((sink_attn(*y, **args)[0] * g).sum())
            assert abs((pair[0] - pair[1]) / (2 * h) - grads[n][at]) < 1e-7


def test_what_a_query_before_the_first_key_sees():
    see = visible(4, 2, 3, 1, 0)
    assert not see[0].any() and not see[1].any()
    assert see[2].tolist() == [True, False] and see[3].tolist() == [True, True]


@pytest.fixture(scope="module")
def L():
    ensure_built()
    from video_diffusion_hybrid_vda_b200 import vdn
    return vdn


A = 4096  # an aligned stand-in address; nothing reads it


def _shape(L, **kw):
    base = dict(Lq=100, Lk=200, B=1, H=4, H_kv=2, d=128, window=64, ahead=0, sinks=4)
    base.update(kw)
    return L.SinkShape(*[base[n] for n, _ in L.SinkShape._fields_])


BAD_SHAPES = [(dict(Lq=-1), 1), (dict(Lk=-1), 1), (dict(B=0), 1), (dict(H=0), 1),
              (dict(H_kv=0), 1), (dict(H_kv=3), 1), (dict(d=0), 1), (dict(d=32), 2),
              (dict(d=96), 2), (dict(window=0), 1), (dict(ahead=-1), 1), (dict(sinks=-1), 1),
              (dict(Lq=1 << 30), 1), (dict(Lk=(1 << 31) - 1), 1), (dict(B=2), 1)]


@pytest.mark.parametrize("change,code", BAD_SHAPES)
def test_bad_shapes_are_refused_on_the_host(L, change, code):
    lib, P = L.lib(), ctypes.c_void_p
    s = _shape(L, **change)
    assert lib.vdn_sink_attn(ctypes.byref(s), P(A), 512, P(A), P(A), 256, None, None, 0.0, P(A),
                             512, 0, None, P(A), 1 << 40, None) == code
    if change != dict(B=2):
        assert lib.vdn_sink_attn_workspace(ctypes.byref(s)) == 0


@pytest.mark.parametrize("change", [
    dict(q=0), dict(k=0), dict(v=0), dict(o=0), dict(q=A + 8), dict(k=A + 2), dict(o=A + 4),
    dict(ld_q=504), dict(ld_q=516), dict(ld_kv=128), dict(ld_o=256), dict(lse=A + 2),
    dict(cu_q=A + 1)])
def test_bad_arguments_are_refused_on_the_host(L, change):
    lib, P = L.lib(), ctypes.c_void_p
    a = dict(q=A, ld_q=512, k=A, v=A, ld_kv=256, cu_q=0, o=A, ld_o=512, lse=0)
    a.update(change)
    s = _shape(L)
    assert lib.vdn_sink_attn(ctypes.byref(s), P(a["q"]), a["ld_q"], P(a["k"]), P(a["v"]),
                             a["ld_kv"], P(a["cu_q"]), None, 0.0, P(a["o"]), a["ld_o"],
                             0, P(a["lse"]), P(A), 1 << 40, None) == 1


def test_workspaces(L):
    lib, P = L.lib(), ctypes.c_void_p
    assert lib.vdn_sink_attn_workspace(None) == 0
    assert lib.vdn_sink_attn_workspace(ctypes.byref(_shape(L, Lq=100000, Lk=100000))) == 256
    few = _shape(L, Lq=16, Lk=8192, window=1 << 30)   # split over the keys: parts in fp32
    n = lib.vdn_sink_attn_workspace(ctypes.byref(few))
    assert n > 256 + 2 * 16 * 4 * 128 * 4
    for ws, size in ((0, 1 << 40), (A + 128, 1 << 40), (A, n - 1)):
        assert lib.vdn_sink_attn(ctypes.byref(few), P(A), 512, P(A), P(A), 256, None, None, 0.0,
                                 P(A), 512, 0, None, P(ws), size, None) == 3
    # no queries: nothing to do, nothing enqueued
    none = _shape(L, Lq=0)
    assert lib.vdn_sink_attn(ctypes.byref(none), None, 512, P(A), P(A), 256, None, None, 0.0,
                             None, 512, 0, None, P(A), 256, None) == 0


@pytest.mark.parametrize("change,code", [
    (dict(q=0), 1), (dict(o=0), 1), (dict(lse=0), 1), (dict(d_o=A + 8), 1), (dict(dq=0), 1),
    (dict(dk=A + 4), 1), (dict(dv=0), 1), (dict(ld_dq=500), 1), (dict(ld_dkv=128), 1),
    (dict(lse=A + 1), 1), (dict(ws=0), 3), (dict(ws=A + 16), 3), (dict(ws_bytes=256), 3)])
def test_bad_gradient_arguments_are_refused_on_the_host(L, change, code):
    lib, P = L.lib(), ctypes.c_void_p
    a = dict(q=A, o=A, lse=A, d_o=A, dq=A, dk=A, dv=A, ld_dq=512, ld_dkv=256, ws=A,
             ws_bytes=1 << 40)
    a.update(change)
    s = _shape(L)
    assert lib.vdn_sink_attn_backward(
        ctypes.byref(s), P(a["q"]), 512, P(A), P(A), 256, None, None, 0.0, P(a["o"]), 512,
        P(a["lse"]), P(a["d_o"]), 512, P(a["dq"]), a["ld_dq"], P(a["dk"]), P(a["dv"]),
        a["ld_dkv"], 0, P(a["ws"]), a["ws_bytes"], None) == code


@pytest.mark.parametrize("change,code", BAD_SHAPES)
def test_bad_gradient_shapes_are_refused_on_the_host(L, change, code):
    lib, P = L.lib(), ctypes.c_void_p
    s = _shape(L, **change)
    assert lib.vdn_sink_attn_backward(
        ctypes.byref(s), P(A), 512, P(A), P(A), 256, None, None, 0.0, P(A), 512, P(A), P(A), 512,
        P(A), 512, P(A), P(A), 256, 0, P(A), 1 << 40, None) == code


@pytest.mark.parametrize("change,code", [
    (dict(B=-1), 1), (dict(H=0), 1), (dict(H=3), 1), (dict(H_kv=0), 1), (dict(d=32), 2),
    (dict(window=0), 1), (dict(sinks=-1), 1), (dict(window=1 << 30), 1), (dict(B=70000), 2),
    (dict(q=0), 1), (dict(k_new=A + 8), 1), (dict(k_cache=0), 1), (dict(positions=0), 1),
    (dict(positions=A + 2), 1), (dict(o=0), 1), (dict(ld_q=500), 1), (dict(ld_new=128), 1),
    (dict(ld_cache=252), 1), (dict(ld_cache=128), 1), (dict(batch_stride=68 * 256 - 8), 1),
    (dict(batch_stride=68 * 256 + 4), 1), (dict(B=0, q=0), 0)])
def test_bad_step_arguments_are_refused_on_the_host(L, change, code):
    lib, P = L.lib(), ctypes.c_void_p
    a = dict(B=2, H=4, H_kv=2, d=128, window=64, sinks=4, q=A, ld_q=512, k_new=A, ld_new=256,
             k_cache=A, ld_cache=256, batch_stride=68 * 256, positions=A, o=A)
    a.update(change)
    assert lib.vdn_sink_attn_step(
        a["B"], a["H"], a["H_kv"], a["d"], a["window"], a["sinks"], P(a["q"]), a["ld_q"],
        P(a["k_new"]), P(A), a["ld_new"], P(a["k_cache"]), P(A), a["ld_cache"],
        a["batch_stride"], P(a["positions"]), 0.0, P(a["o"]), 512, None) == code
