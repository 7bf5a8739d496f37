"""The query/key preparation oracle against central differences and what fixes
a rotation: lengths kept, relative positions, the two layouts the same up to a
permutation; and the plan's frequencies and fixed-point phases."""

import math

import numpy as np
import pytest

from oracle import qk_prep
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
