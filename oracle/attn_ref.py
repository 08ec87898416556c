"""CPU fp64 reference of the paged-cache operators: the rotation and append, and causal
attention over the cache with a window, first tokens that stay visible and shared prefixes.
Loops over sequences and heads; numpy only."""
from __future__ import annotations

import numpy as np


def positions(q_off, kv_len):
    """(row, sequence, position) of every new token."""
    out = []
    for s in range(len(kv_len)):
        n = int(q_off[s + 1] - q_off[s])
        for i in range(n):
            out.append((int(q_off[s]) + i, s, int(kv_len[s]) - n + i))
    return out


def rotate(x, cs, pos_of_pair, interleaved):
    """One head x [D] rotated: pair i by table row pos_of_pair[i] of cs [n_pos, rot]; a
    position outside the table leaves its pair as it is."""
    x = np.array(x, np.float64)
    y = x.copy()
    half = cs.shape[1] // 2
    for i in range(half):
        p = pos_of_pair[i]
        if not 0 <= p < cs.shape[0]:
            continue
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, half + i)
        c, s = float(cs[p, i]), float(cs[p, half + i])
        y[a] = x[a] * c - x[b] * s
        y[b] = x[b] * c + x[a] * s
    return y


def attention(q, rows_k, rows_v, q_off, kv_len, scale, window=0, n_sink=0):
    """q [T, Hq, D]; rows_k[s], rows_v[s] [kv_len[s], Hkv, D] of each sequence.  Returns out
    [T, Hq, D] and weight_v [T, Hq, D] = sum_j w_j |v_j| (for error bounds); rows of no
    sequence are NaN in out."""
    T, hq, d = q.shape
    out = np.full((T, hq, d), np.nan)
    bound = np.zeros((T, hq, d))
    for t, s, p in positions(q_off, kv_len):
        hkv = rows_k[s].shape[1] if len(rows_k[s]) else 1
        seen = [j for j in range(p + 1) if window == 0 or j > p - window or j < n_sink]
        if not seen:
            out[t] = 0
            continue
        for h in range(hq):
            k = rows_k[s][seen, h // (hq // hkv)]
            v = rows_v[s][seen, h // (hq // hkv)]
            x = scale * (k @ q[t, h])
            w = np.exp(x - x.max())
            w /= w.sum()
            out[t, h] = w @ v
            bound[t, h] = w @ np.abs(v)
    return out, bound
