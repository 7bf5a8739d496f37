"""Query/key preparation (per-head norm and rotary positions) and its
gradients, float64.  TEST INFRASTRUCTURE ONLY.

    r_i = (c sum x^2 + eps)^-1/2   (c = 1/d for "rms", 1 for "l2"; r = 1 for "none")
    n   = x r w
    y   = R(p) n: pair j turns by the angle p[axis_j] f_j, times `scale`

Angles are products of float64 frequencies and integer positions; the gradient
functions are the formulas, and tests/test_oracle_qk_prep_pins.py holds them
to central differences.
"""

import numpy as np


def pair_columns(rot, layout):
    """Columns (a, b) of every rotated pair."""
    j = np.arange(rot // 2)
    return (j, j + rot // 2) if layout == "half" else (2 * j, 2 * j + 1)


def rotate(x, positions, frequencies, axis, layout, scale=1.0, inverse=False):
    """x [rows, heads, d]; positions int [axes, rows]; frequencies, axis [rot/2]."""
    rot = 2 * len(frequencies)
    a, b = pair_columns(rot, layout)
    angle = positions[axis].astype(np.float64).T * np.asarray(frequencies, dtype=np.float64)
    cos = np.cos(angle)[:, None] * scale
    sin = np.sin(angle)[:, None] * (-scale if inverse else scale)
    y = np.array(x, dtype=np.float64)
    xa, xb = y[..., a].copy(), y[..., b].copy()
    y[..., a] = xa * cos - xb * sin
    y[..., b] = xb * cos + xa * sin
    return y


def norm_factor(x, kind, eps):
    if kind == "none":
        return np.ones(x.shape[:-1] + (1,))
    c = 1.0 / x.shape[-1] if kind == "rms" else 1.0
    return 1.0 / np.sqrt((x * x).sum(-1, keepdims=True) * c + eps)


def qk_norm_rope(x, w, kind, eps, rotation):
    """One side; rotation: keyword arguments of rotate()."""
    x = np.asarray(x, dtype=np.float64)
    return rotate(x * norm_factor(x, kind, eps) * w, **rotation)


def qk_norm_rope_backward(x, w, dy, kind, eps, rotation):
    """(dx, dw) of one side."""
    x = np.asarray(x, dtype=np.float64)
    g = rotate(np.asarray(dy, dtype=np.float64), inverse=True, **rotation)
    r = norm_factor(x, kind, eps)
    dw = (g * x * r).sum((0, 1))
    gw = g * w
    if kind == "none":
        return gw, dw
    c = 1.0 / x.shape[-1] if kind == "rms" else 1.0
    return r * gw - x * (r ** 3 * c * (gw * x).sum(-1, keepdims=True)), dw
