"""Float64 definitions of the decode-side operators, one row at a time."""
from __future__ import annotations

import numpy as np


def visible_keys(k_prefix, k_own, own_len: int, q_len: int, i: int):
    """Keys that token i of q_len sees: the prefix, then own keys j <= own_len - q_len + i."""
    n = max(0, own_len - q_len + 1 + i)
    return np.concatenate([k_prefix, k_own[:n]], axis=0)


def prefix_attention(q, prefixes, owns, groups, scale=0.125):
    """q [n, t, H, 64]; prefixes[g] = (k, v) [Lp, Hkv, 64]; owns[s] = (k, v) [Ls, Hkv, 64]; groups[s] = g.

    Returns (out, absv, amax): the output, sum_j p_j |v_j| of every element, and the largest
    sum_i |q_i k_i| of every row (what the rounding bounds need)."""
    n, t, H, hd = q.shape
    out, absv, amax = np.zeros((n, t, H, hd)), np.zeros((n, t, H, hd)), np.zeros((n, t, H))
    for s in range(n):
        kp, vp = prefixes[groups[s]]
        ko, vo = owns[s]
        r = H // kp.shape[1]
        for i in range(t):
            K = visible_keys(kp, ko, ko.shape[0], t, i)
            V = visible_keys(vp, vo, vo.shape[0], t, i)
            if K.shape[0] == 0:
                continue
            for h in range(H):
                kh, vh = K[:, h // r], V[:, h // r]
                z = kh @ q[s, i, h] * scale
                p = np.exp(z - z.max())
                p /= p.sum()
                out[s, i, h] = p @ vh
                absv[s, i, h] = p @ np.abs(vh)
                amax[s, i, h] = (np.abs(kh) @ np.abs(q[s, i, h])).max()
    return out, absv, amax


def rotate(x, pos, inv_freq, interleaved):
    """x [tokens, heads, 64] turned by pos [tokens] * inv_freq; also sum of the magnitudes of each
    element's two products."""
    y, mag = x.copy(), np.abs(x)
    half = len(inv_freq)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        w = (pos.astype(np.float64) * float(inv_freq[i]))[:, None]
        c, s = np.cos(w), np.sin(w)
        y[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
        y[:, :, b] = x[:, :, b] * c + x[:, :, a] * s
        mag[:, :, a] = mag[:, :, b] = np.abs(x[:, :, a]) + np.abs(x[:, :, b])
    return y, mag


def quantize_rows(x):
    """(integers, scales): scale = fp32(max|row| * fp32(1 / 127)), integers = nearest of x / scale (ties to even);
    zero rows have scale 0, rows with a non-finite element scale NaN, both integers 0."""
    x = np.asarray(x, np.float32)
    with np.errstate(all="ignore"):
        amax = np.abs(x).max(axis=1)
        scale = amax * (np.float32(1) / np.float32(127))
        bad = ~np.isfinite(x).all(axis=1)
        q = np.rint(x.astype(np.float64) / scale.astype(np.float64)[:, None])
    q = np.clip(q, -127, 127)
    q[bad | (scale == 0)] = 0
    scale[bad] = np.nan
    return q.astype(np.int8), scale


def linear_i8(a, a_scale, w, w_scale, bias):
    """(pre-activation, sum of the magnitudes of its products) in float64."""
    acc = a.astype(np.float64) @ w.astype(np.float64).T
    mag = np.abs(a.astype(np.float64)) @ np.abs(w.astype(np.float64)).T
    ss = a_scale.astype(np.float64)[:, None] * w_scale.astype(np.float64)[None]
    return acc * ss + bias.astype(np.float64), mag * ss
