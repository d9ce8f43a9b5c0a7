"""Rotary positions and drafted trees in numpy, written from their definitions (test infrastructure)."""
from __future__ import annotations

import numpy as np


def angles(positions, inv_freq):
    """position * frequency in extended precision, reduced to (-pi, pi], as fp64 [T, n]."""
    a = np.asarray(positions, np.longdouble)[:, None] * np.asarray(inv_freq, np.longdouble)[None, :]
    two_pi = np.longdouble("6.283185307179586476925286766559005768")
    return (a - two_pi * np.rint(a / two_pi)).astype(np.float64)


def pairs(n, first, interleaved):
    f = np.arange(n)
    return (first + 2 * f, first + 2 * f + 1) if interleaved else (first + f, first + n + f)


def rotate(x, c, s, first=0, interleaved=False):
    """x [T, H, d], c and s [T, n]: the rotated x, in x's precision."""
    i1, i2 = pairs(c.shape[1], first, interleaved)
    y = x.copy()
    c, s = c[:, None, :], s[:, None, :]
    y[..., i1] = x[..., i1] * c - x[..., i2] * s
    y[..., i2] = x[..., i2] * c + x[..., i1] * s
    return y


def path(parents, i):
    """Node i and its ancestors, upwards."""
    out = [i]
    while True:
        p = i - 1 if parents is None else int(parents[i])
        if p < 0 or p >= i:
            return out
        i = p
        out.append(i)


def attention(q, k, v, L, parents, *, scale=None, window=-1, sink=None):
    """Attention of one sequence's nodes q [n, H_q, d] over its tokens k, v [tokens, H_kv, d] (fp64, as
    held; L before the tree, the nodes' behind them as far as they exist).  Returns o [n, H_q, d], lse
    [H_q, n], and per output element sum_j P_j |v_j| and per row max_j scale sum_x |q_x k_jx|."""
    n, H, d = q.shape
    G = H // k.shape[1]
    scale = 1 / np.sqrt(d) if scale is None else scale
    o, a = np.zeros((n, H, d)), np.zeros((n, H, d))
    lse, mag = np.full((H, n), -np.inf), np.zeros((H, n))
    for i in range(n):
        up = path(parents, i)
        depth = len(up) - 1
        js = list(range(max(0, L + depth - window) if window >= 0 else 0, min(L, k.shape[0])))
        js += [L + a_ for a_ in (up if window < 0 else up[:window + 1]) if L + a_ < k.shape[0]]
        for h in range(H):
            kk, vv = k[js, h // G], v[js, h // G]
            t = kk @ q[i, h] * scale
            m = np.max(t, initial=-np.inf)
            if sink is not None:
                m = max(m, sink[h])
            if np.isinf(m) and m < 0:
                continue
            e = np.exp(t - m)
            z = e.sum() + (np.exp(sink[h] - m) if sink is not None else 0.0)
            o[i, h], a[i, h] = (e / z) @ vv, (e / z) @ np.abs(vv)
            lse[h, i] = m + np.log(z)
            mag[h, i] = np.max(np.abs(kk) @ np.abs(q[i, h]) * scale, initial=0.0)
    return o, lse, a, mag


def keep(tokens, L, kept):
    """tokens: a list of one sequence's tokens; the moves in order."""
    for i, a in enumerate(kept):
        if a < 0:
            break
        tokens[L + i] = tokens[L + a]
