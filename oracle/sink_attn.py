"""Attention with a sliding window and sinks, and its gradients, float64.
TEST INFRASTRUCTURE ONLY.

Query i of a sequence with n_q queries and n_k keys has the position
p = i + n_k - n_q and sees key j iff
    j <= p + ahead and (p - j < window or j < sinks).
o_i = sum_j P_ij v_j with P the softmax of scale q_i . k_j over the visible
keys; a query that sees nothing has o = 0 and lse = -inf and no gradient.
"""

import numpy as np


def visible(n_q, n_k, window, sinks, ahead):
    p = np.arange(n_q)[:, None] + n_k - n_q
    j = np.arange(n_k)[None]
    return (j <= p + ahead) & ((p - j < window) | (j < sinks))


def attend(q, k, v, see, scale):
    """One head of one sequence: (o, lse, P)."""
    s = np.where(see, q @ k.T * scale, -np.inf)
    top = s.max(1, initial=-np.inf, keepdims=True)
    top = np.where(np.isfinite(top), top, 0.0)
    e = np.where(see, np.exp(s - top), 0.0)
    total = e.sum(1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = (np.log(total) + top)[:, 0]
    p = e / np.where(total == 0, 1.0, total)
    return p @ v, lse, p


def sink_attn(q, k, v, H, H_kv, window, sinks=0, ahead=0, lens_q=None, lens_k=None, scale=None,
              d_o=None):
    """q [Lq, H*d], k, v [Lk, H_kv*d] -> (o, lse [H, Lq]) and, with d_o, (dq, dk, dv)."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    d = q.shape[1] // H
    scale = d ** -0.5 if scale is None else scale
    lens_q = [q.shape[0]] if lens_q is None else lens_q
    lens_k = [k.shape[0]] if lens_k is None else lens_k
    o, lse = np.zeros_like(q), np.full((H, q.shape[0]), -np.inf)
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    a = b = 0
    for n_q, n_k in zip(lens_q, lens_k):
        see = visible(n_q, n_k, window, sinks, ahead)
        rq, rk = slice(a, a + n_q), slice(b, b + n_k)
        for h in range(H):
            c = slice(h * d, (h + 1) * d)
            e = h // (H // H_kv)
            ck = slice(e * d, (e + 1) * d)
            o[rq, c], lse[h, rq], p = attend(q[rq, c], k[rk, ck], v[rk, ck], see, scale)
            if d_o is None:
                continue
            g = np.asarray(d_o[rq, c], dtype=np.float64)
            ds = p * (g @ v[rk, ck].T - (g * o[rq, c]).sum(1, keepdims=True)) * scale
            dv[rk, ck] += p.T @ g
            dq[rq, c] = ds @ k[rk, ck]
            dk[rk, ck] += ds.T @ q[rq, c]
        a, b = a + n_q, b + n_k
    return (o, lse) if d_o is None else (o, lse, dq, dk, dv)
