"""The query/key preparation oracle against central differences and what fixes
a rotation: lengths kept, relative positions, the two layouts the same up to a
permutation; and the plan's frequencies and fixed-point phases."""

import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import qk_prep
from tests.parity_util import ensure_built
from video_diffusion_hybrid_vda_b200 import vdn

RNG = np.random.default_rng(5)


def _rotation(rot, layout, rows, axes=1, scale=1.0):
    n = rot // 2
    axis = np.arange(n) * axes // n
    return dict(positions=RNG.integers(-50, 50, (axes, rows)),
                frequencies=np.array(vdn.rope_frequencies(rot)[0]), axis=axis, layout=layout,
                scale=scale)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_a_rotation_keeps_lengths_and_its_inverse_undoes_it(layout):
    x = RNG.standard_normal((7, 3, 24))
    rt = _rotation(16, layout, 7, axes=2)
    y = qk_prep.rotate(x, **rt)
    np.testing.assert_allclose((y * y).sum(-1), (x * x).sum(-1), rtol=1e-13)
    np.testing.assert_allclose(qk_prep.rotate(y, inverse=True, **rt), x, atol=1e-13)
    np.testing.assert_array_equal(y[..., 16:], x[..., 16:])


def test_scores_depend_on_the_distance_of_two_positions():
    q, k = RNG.standard_normal((1, 1, 16)), RNG.standard_normal((1, 1, 16))
    f = np.array(vdn.rope_frequencies(16)[0])

    def score(p, j):
        kw = dict(frequencies=f, axis=np.zeros(8, int), layout="half")
        return (qk_prep.rotate(q, np.array([[p]]), **kw) *
                qk_prep.rotate(k, np.array([[j]]), **kw)).sum()

    assert abs(score(19, 4) - score(1019, 1004)) < 1e-11
    assert abs(score(19, 4) - score(19, 5)) > 1e-3


def test_layouts_are_a_permutation_of_each_other():
    x = RNG.standard_normal((4, 2, 16))
    a = _rotation(16, "half", 4)
    perm = np.stack(qk_prep.pair_columns(16, "half"), -1).ravel()  # half column of each slot
    y = qk_prep.rotate(x, **a)
    z = qk_prep.rotate(x[..., perm], **{**a, "layout": "interleaved"})
    np.testing.assert_allclose(z, y[..., perm], atol=1e-14)


@pytest.mark.parametrize("kind", ["rms", "l2", "none"])
def test_gradients_against_central_differences(kind):
    x, w = RNG.standard_normal((3, 2, 16)), 1 + 0.2 * RNG.standard_normal(16)
    dy = RNG.standard_normal(x.shape)
    rt = _rotation(8, "half", 3, scale=1.3)
    dx, dw = qk_prep.qk_norm_rope_backward(x, w, dy, kind, 1e-3, rt)

    def loss(x_, w_):
        return (qk_prep.qk_norm_rope(x_, w_, kind, 1e-3, rt) * dy).sum()

    h = 1e-5
    for _ in range(20):
        at = tuple(RNG.integers(0, n) for n in x.shape)
        e = np.zeros_like(x)
        e[at] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[at]) < 1e-7
    for i in range(16):
        e = np.zeros_like(w)
        e[i] = h
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[i]) < 1e-7


def test_frequencies_by_hand():
    f, s = vdn.rope_frequencies(8, base=10000.0)
    np.testing.assert_allclose(f, [1, 0.1, 0.01, 0.001], rtol=1e-14)
    assert s == 1.0
    np.testing.assert_allclose(vdn.rope_frequencies(8, scaling="linear", factor=4)[0],
                               [0.25, 0.025, 0.0025, 0.00025], rtol=1e-14)
    ntk = vdn.rope_frequencies(8, scaling="ntk", factor=4)[0]
    assert ntk[0] == 1.0 and abs(ntk[3] - 0.001 / 4) < 1e-17  # the slowest is interpolated
    y, s = vdn.rope_frequencies(64, scaling="yarn", factor=8, original=4096)
    plain = vdn.rope_frequencies(64)[0]
    assert y[0] == plain[0] and abs(y[-1] - plain[-1] / 8) < 1e-18
    assert abs(s - (0.1 * math.log(8) + 1)) < 1e-15
    assert all(b <= a for a, b in zip(plain, y))
    two = vdn.rope_frequencies(16, sections=[5, 3])[0]
    np.testing.assert_allclose(two[5:], [1, 10000 ** (-1 / 3), 10000 ** (-2 / 3)], rtol=1e-14)


def test_phase_words_are_turns_modulo_one():
    rng = np.random.default_rng(1)
    for f in [1.0, 0.1, 1e-4, 7.5, -0.3, 0.0, *rng.uniform(-10, 10, 20)]:
        w = vdn.RopePlan.phase_word(f)
        assert 0 <= w < 1 << 64
        for p in (0, 1, -1, 12345, -(1 << 31), (1 << 31) - 1):
            got = (p * w % (1 << 64)) / 2.0 ** 64
            want = (p * f / (2 * math.pi)) % 1.0
            off = abs(got - want)
            # float64 p * f / 2 pi: three roundings of a product up to |p f / 2 pi|
            assert min(off, 1 - off) <= 4 * 2.0 ** -53 * (abs(p * f / (2 * math.pi)) + 1)


def test_bad_plans_are_refused():
    for kw in (dict(layout="other"), dict(rot=7), dict(rot=24), dict(sections=[4, 3]),
               dict(sections=[2, 2, 2, 1, 1]), dict(sections=[9, -1]), dict(scaling="other"),
               dict(factor=0.0), dict(base=1.0), dict(frequencies=[1.0, 2.0]),
               dict(frequencies=[float("nan")] * 8)):
        with pytest.raises(ValueError):
            vdn.RopePlan(16, device="cpu", **kw)


# ---------------------------------------------------------------- refusals on the host

A = 4096  # an aligned stand-in address; nothing reads it


@pytest.fixture(scope="module")
def L():
    ensure_built()
    return vdn


def _plan(**kw):
    base = dict(head_dim=64, rot_dim=32, layout=0, n_axes=1, section_pairs=(16, 0, 0, 0), scale=1.0,
                phase=A)
    base.update(kw)
    pairs = (ctypes.c_int * 4)(*base["section_pairs"])
    return vdn.RopePlanC(base["head_dim"], base["rot_dim"], base["layout"], base["n_axes"], pairs,
                         base["scale"], base["phase"])


BAD_PLANS = [
    (dict(head_dim=0), 1), (dict(head_dim=60), 2), (dict(head_dim=264, rot_dim=0), 2),
    (dict(rot_dim=-8), 1), (dict(rot_dim=72), 1), (dict(rot_dim=12), 2), (dict(layout=2), 1),
    (dict(n_axes=0), 1), (dict(n_axes=5), 1), (dict(section_pairs=(15, 0, 0, 0)), 1),
    (dict(n_axes=2, section_pairs=(17, -1, 0, 0)), 1), (dict(phase=0), 1), (dict(phase=A + 4), 1)]
BAD_ARGS = [
    (dict(dtype=3), 1), (dict(dtype=-1), 1), (dict(rows=-1), 1), (dict(rows=1 << 31), 1),
    (dict(H=0), 1), (dict(x=0), 1), (dict(x=A + 8), 1), (dict(ld=120), 1), (dict(ld=132), 1),
    (dict(out=0), 1), (dict(ld_out=64), 1), (dict(positions=A + 2), 1), (dict(rows=0, x=0), 0)]


@pytest.mark.parametrize("plan,args,code", [(p, {}, c) for p, c in BAD_PLANS] +
                         [({}, a, c) for a, c in BAD_ARGS])
def test_rope_refuses_bad_arguments_on_the_host(L, plan, args, code):
    lib, P = L.lib(), ctypes.c_void_p
    a = dict(dtype=0, rows=10, H=2, x=A, ld=128, out=A, ld_out=128, positions=A)
    a.update(args)
    p = _plan(**plan)
    assert lib.vdn_rope(ctypes.byref(p), a["dtype"], a["rows"], a["H"], P(a["x"]), a["ld"],
                        P(a["positions"]), 10, 0, P(a["out"]), a["ld_out"], None) == code
    assert lib.vdn_rope(None, 0, 10, 2, P(A), 128, None, 0, 0, P(A), 128, None) == 1


def test_axes_need_a_stride_of_all_rows(L):
    lib, P = L.lib(), ctypes.c_void_p
    p = _plan(n_axes=2, section_pairs=(10, 6, 0, 0))
    assert lib.vdn_rope(ctypes.byref(p), 0, 10, 2, P(A), 128, P(A), 9, 0, P(A), 128, None) == 1


def test_stride_of_the_position_axes_is_the_tensors(L):
    """Positions shared by the axes (stride 0) and columns of wider ones."""
    plan = type("Plan", (), {"n_axes": 3})
    pos = torch.arange(50, dtype=torch.int32)
    for t, stride in ((pos.expand(3, 50), 0), (pos[:1].expand(3, 1), 0),
                      (pos[:30].view(3, 10)[:, 4:9], 10), (pos[:30].view(3, 10)[:, 4:5], 10),
                      (pos[:3].view(3, 1), 1)):
        assert L._rope_positions(t, plan, t.shape[1]) == (t.data_ptr(), stride)
    with pytest.raises(ValueError):
        L._rope_positions(pos[:30].view(10, 3).t(), plan, 10)


QK = dict(H=2, H_kv=1, q=A, ld_q=128, k=A, ld_k=64, q_norm=1, k_norm=2, wq=A, wk=0, eps=1e-6,
          g=A, dq=A, dk=A, dwq=A, dwk=A, ws=A, ws_bytes=1 << 30)


@pytest.mark.parametrize("change,code,forward", [
    (dict(H_kv=0), 1, True), (dict(q=A + 8), 1, True), (dict(k=0), 1, True),
    (dict(ld_k=60), 1, True), (dict(q_norm=3), 1, True), (dict(k_norm=-1), 1, True),
    (dict(wq=A + 4), 1, True), (dict(q_norm=0), 1, True),      # a weight without a norm
    (dict(eps=-1.0), 1, True), (dict(eps=float("nan")), 1, True), (dict(g=0), 1, False),
    (dict(dq=0), 1, False), (dict(dk=A + 2), 1, False), (dict(dwq=A + 2), 1, False),
    (dict(q_norm=0, wq=0), 1, False), (dict(ws=0), 3, False), (dict(ws=A + 16), 3, False),
    (dict(ws_bytes=1000), 3, False)])
def test_qk_norm_rope_refuses_bad_arguments_on_the_host(L, change, code, forward):
    lib, P = L.lib(), ctypes.c_void_p
    a = {**QK, **change}
    p = _plan()
    head = (ctypes.byref(p), 0, 10, a["H"], a["H_kv"], P(a["q"]), a["ld_q"], P(a["k"]), a["ld_k"],
            a["q_norm"], a["k_norm"], P(a["wq"]), P(a["wk"]), a["eps"], None, 0)
    if forward:
        assert lib.vdn_qk_norm_rope(*head, P(A), 128, P(A), 64, None) == code
    assert lib.vdn_qk_norm_rope_backward(
        *head, P(a["g"]), 128, P(A), 64, P(a["dq"]), 128, P(a["dk"]), 64, P(a["dwq"]), P(a["dwk"]),
        P(a["ws"]), a["ws_bytes"], None) == code
