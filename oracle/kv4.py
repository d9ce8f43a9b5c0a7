"""The 4-bit paged key/value cache in numpy, written from the format's definition (test
infrastructure): which values a token is held as, where its bytes lie in a page, and
attention of the newest tokens over a cache, in fp64.

Format: 16 consecutive dims share an unsigned 8-bit float scale (5 exponent bits, bias 15,
3 mantissa bits, gradual underflow), a value is (c - 8) * scale for a code c in 0..15.
"""
from __future__ import annotations

import numpy as np

# every finite scale, byte 0x00 .. 0xF7: e = byte >> 3, m = byte & 7
SCALES = np.array([(1 + (b & 7) / 8) * 2.0 ** ((b >> 3) - 15) if b >> 3 else (b & 7) / 8 * 2.0 ** -14
                   for b in range(0xF8)])


def scale_bytes(r):
    """Nearest scale to each r >= 0, the even byte where two are as near, the largest above them all."""
    r = np.minimum(np.asarray(r, np.float64), SCALES[-1])
    hi = np.clip(np.searchsorted(SCALES, r), 0, len(SCALES) - 1)
    lo = np.maximum(hi - 1, 0)
    dh, dl = np.abs(SCALES[hi] - r), np.abs(r - SCALES[lo])
    return np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)


def quantise(x):
    """x [..., d] fp64 -> codes [..., d] (0..15), scale bytes [..., d/16]; 0xFF where 16 values are not all finite."""
    x = np.asarray(x, np.float64)
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    ok = np.isfinite(g).all(-1)
    z = np.where(ok[..., None], g, 0.0)
    b = scale_bytes(np.abs(z).max(-1) / 7)
    s = SCALES[b][..., None]
    c = np.where(s > 0, np.clip(np.rint(z / np.where(s > 0, s, 1)), -8, 7), 0) + 8
    return c.astype(np.int64).reshape(x.shape), np.where(ok, b, 0xFF)


def values(codes, byts):
    """What codes and scale bytes stand for, in fp64."""
    s = np.where(byts < 0xF8, SCALES[np.minimum(byts, 0xF7)], np.nan)
    g = codes.reshape(*codes.shape[:-1], -1, 16) - 8.0
    return (g * s[..., None]).reshape(codes.shape)


def held(x):
    """The values that x [..., d] is held as."""
    return values(*quantise(x))


def block_bytes(P, d):
    return P * d * 9 // 8


def k_code_at(w, x, P, d):
    """(byte, shift) of dim x of token w's key inside a block."""
    return w * (d // 2) + x // 2, 4 * (x % 2)


def v_code_at(w, x, P, d):
    u, g = w // 2, x // (d // 8)
    slot = g ^ (2 * (u % 4) if d == 128 else 4 * ((u // 2) % 2))
    return P * d // 2 + u * d + slot * (d // 8) + (w % 2) * (d // 16) + (x % (d // 8)) // 2, 4 * (x % 2)


def k_scale_at(w, g, P, d):
    return P * d + w * (d // 16) + g


def v_scale_at(w, g, P, d):
    return P * d + P * d // 16 + (w // 2) * (d // 8) + 2 * g + w % 2


def write_token(block, w, k, v, P):
    """Token w's key and value [d] into one page's block of one head (uint8 [block_bytes])."""
    d = len(k)
    for x_, code_at, scale_at in ((k, k_code_at, k_scale_at), (v, v_code_at, v_scale_at)):
        c, b = quantise(x_)
        for x in range(d):
            at, sh = code_at(w, x, P, d)
            block[at] = (int(block[at]) & ~(15 << sh) & 0xFF) | (int(c[x]) << sh)
        for g in range(d // 16):
            block[scale_at(w, g, P, d)] = int(b[g])


def decode(q, k, v, seq_len, *, scale=None, window=-1, sink=None):
    """Attention of the last S_q tokens of one sequence: q [S_q, H_q, d] over k, v [seq_len, H_kv, d]
    (fp64, as held), sink [H_q] logits or None.  Returns o [S_q, H_q, d], lse [H_q, S_q], and per
    output element sum_j P_j |v_j| and per row max_j scale sum_x |q_x k_jx|, for error bounds."""
    S, H, d = q.shape
    G = H // k.shape[1]
    scale = 1 / np.sqrt(d) if scale is None else scale
    o, a = np.zeros((S, H, d)), np.zeros((S, H, d))
    lse, mag = np.full((H, S), -np.inf), np.zeros((H, S))
    for h in range(H):
        for s in range(S):
            pos = seq_len - S + s
            lo = max(0, pos - window) if window >= 0 else 0
            kk, vv = k[lo:pos + 1, h // G], v[lo:pos + 1, h // G]
            if pos < 0:
                kk, vv = k[:0, h // G], v[:0, h // G]
            t = kk @ q[s, h] * scale
            m = np.max(t, initial=-np.inf)
            if sink is not None:
                m = max(m, sink[h])
            if np.isinf(m) and m < 0:
                continue
            e = np.exp(t - m)
            z = e.sum() + (np.exp(sink[h] - m) if sink is not None else 0.0)
            o[s, h], a[s, h] = (e / z) @ vv, (e / z) @ np.abs(vv)
            lse[h, s] = m + np.log(z)
            mag[h, s] = np.max(np.abs(kk) @ np.abs(q[s, h]) * scale, initial=0.0)
    return o, lse, a, mag
