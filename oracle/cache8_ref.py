"""CPU reference of the 8-bit paged cache: e4m3 codes and block scales, the append with its
growing scales, and a batch's plan from the lengths of its requests.  Loops; numpy only."""
from __future__ import annotations

import numpy as np

BLOCK = 16


def _values():
    out = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[c] = np.nan if c & 127 == 127 else -x if c & 128 else x
    return out


VALUES = _values()   # of the 256 codes


def encode(x):
    """The codes nearest to x, ties to the even code, magnitudes above 448 to 448, NaN to 127."""
    x = np.asarray(x, np.float64)
    pos = VALUES[:127]
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(pos, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up = pos[hi] - a
    down = a - pos[lo]
    code = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.isnan(x), 127, code)
    return (code + 128 * np.signbit(x)).astype(np.uint8)


def scale_byte(top):
    """The byte of the least power of two 2^(b - 127), b >= 1, with top <= 448 * 2^(b - 127)."""
    b = 1
    while top > 448 * 2.0 ** (b - 127):
        b += 1
    return b


def scale_read(byte):
    return np.clip(np.asarray(byte, np.int64), 1, 253)


def dequantize(codes, scale):
    """codes [..., page, d] and scale bytes [..., page / B] to values."""
    n = codes.shape[-2] // scale.shape[-1]
    return VALUES[codes] * np.repeat(2.0 ** (scale_read(scale) - 127.0), n, -1)[..., None]


def append(codes, scale, rows, places):
    """Appends rows [n, heads, d] (fp64) of one sequence to consecutive positions, places
    [(page, row)], in place.  codes [pages, heads, page, d], scale [pages, heads, blocks]."""
    page = codes.shape[2]
    block = min(BLOCK, page)
    i = 0
    while i < len(places):
        at, first = places[i]
        n = 1
        while i + n < len(places) and (first + n) % block:
            n += 1
        held = first % block
        for h in range(codes.shape[1]):
            x = rows[i:i + n, h]
            b = scale_byte(np.max(np.abs(x)))
            if held:
                old = int(scale_read(scale[at, h, first // block]))
                b = max(b, old)
                before = codes[at, h, first - held:first]
                if b > old:
                    before[:] = encode(VALUES[before] * 2.0 ** (old - b))
            scale[at, h, first // block] = b
            codes[at, h, first:first + n] = encode(x * 2.0 ** (127 - b))
        i += n


def plan(table, n_cached, n_new, n_shared, free, n_free, page, n_pages, T):
    """The plan of a batch; changes table and free.  Returns q_off, kv_len, slots, pos, n_free."""
    n, max_pages = table.shape
    stack = [int(x) for x in free[:n_free]]
    for s in range(n):
        if n_new[s] < 0:
            for c in range(n_shared[s], min(-(-int(n_cached[s]) // page), max_pages)):
                if 0 <= table[s, c] < n_pages:
                    stack.append(int(table[s, c]))
    stack = stack[:len(free)]
    free[:len(stack)] = stack
    q_off, kv_len, slots, pos = [0], [], [], []
    for s in range(n):
        rows = min(max(int(n_new[s]), 0), T - q_off[-1])
        cached = int(n_cached[s])
        q_off.append(q_off[-1] + rows)
        kv_len.append(0 if n_new[s] < 0 else cached + rows)
        for c in range(-(-cached // page), min(-(-(cached + rows) // page), max_pages)):
            table[s, c] = stack.pop() if stack else -1
        for p in range(cached, cached + rows):
            ok = p // page < max_pages and 0 <= table[s, p // page] < n_pages
            slots.append(int(table[s, p // page]) * page + p % page if ok else -1)
            pos.append(p)
    pad = [-1] * (T - len(slots))
    return np.array(q_off), np.array(kv_len), np.array(slots + pad), np.array(pos + pad), len(stack)
