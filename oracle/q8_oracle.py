"""Oracle of the 8-bit paged KV cache: plain loops in fp64 and Python integers
(test infrastructure only; shares no code with the CUDA library).

The cache has no counterpart on the pages; the definitions are those of the C
header: a stored byte stands for its e4m3 or int8 value times its block's
scale, K and V pages are [num_pages, Hkv, P, d], scales [num_pages, Hkv, P/S, 2].
"""
from __future__ import annotations

import math

import numpy as np

__all__ = ["e4m3_values", "decode_bytes", "nearest", "scale_for", "page_tables", "append", "rows_of", "attend"]


def e4m3_values() -> np.ndarray:
    """The 256 values of e4m3 by byte: sign, 4 exponent bits (bias 7), 3
    fraction bits; exponent 0 is subnormal, 0x7f and 0xff are NaN."""
    out = np.zeros(256)
    for b in range(256):
        e, f = (b >> 3) & 15, b & 7
        v = math.ldexp(f / 8.0, -6) if e == 0 else math.ldexp(1.0 + f / 8.0, e - 7)
        if e == 15 and f == 7:
            v = math.nan
        out[b] = -v if b & 0x80 else v
    return out


def decode_bytes(raw: np.ndarray, kind: str) -> np.ndarray:
    """Bytes (uint8) to the values they hold."""
    if kind == "int8":
        return raw.view(np.int8).astype(np.float64)
    return e4m3_values()[raw]


def nearest(y: np.ndarray, kind: str) -> np.ndarray:
    """Values to the nearest of the type, ties to the even one, saturated;
    NaN stays (e4m3) or becomes 0 (int8).  By search in the list of values."""
    y = np.asarray(y, dtype=np.float64)
    if kind == "int8":
        grid = np.arange(0.0, 128.0)
    else:
        grid = e4m3_values()[:127]          # 0 .. 448 ascending; even bytes have an even fraction
    mag = np.minimum(np.abs(np.where(np.isnan(y), 0.0, y)), grid[-1])
    hi = np.clip(np.searchsorted(grid, mag, side="left"), 1, len(grid) - 1)
    lo = hi - 1
    down, up = mag - grid[lo], grid[hi] - mag
    pick = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    out = np.copysign(grid[pick], y)
    return np.where(np.isnan(y), math.nan if kind == "e4m3" else 0.0, out)


def scale_for(amax: float, kind: str) -> float:
    """The smallest power of two s, exponent in [-100, 122], with amax <= top s."""
    top = 448.0 if kind == "e4m3" else 127.0
    e = -100
    while e < 122 and amax > math.ldexp(top, e):
        e += 1
    return math.ldexp(1.0, e)


def page_tables(page, kv_lens, new_lens, free, table, capacity):
    """(table, lens, offsets, slots, info) after adding new_lens tokens."""
    table = [list(r) for r in table]
    width, n = len(table[0]), len(kv_lens)
    need = [-(-(a + b) // page) - -(-a // page) for a, b in zip(kv_lens, new_lens)]
    total = sum(new_lens)
    if (min(kv_lens) < 0 or min(new_lens) < 0 or any(a + b > min(width * page, 1 << 20) for a, b in zip(kv_lens, new_lens))
            or total > capacity or sum(need) > len(free)):
        return table, list(kv_lens), [0] * (n + 1), [-1] * capacity, [-1, 0]
    at, slots, offsets = 0, [], [0]
    for b in range(n):
        first = -(-kv_lens[b] // page)
        for i in range(need[b]):
            table[b][first + i] = free[at]
            at += 1
        for pos in range(kv_lens[b], kv_lens[b] + new_lens[b]):
            slots.append(table[b][pos // page] * page + pos % page)
        offsets.append(len(slots))
    lens = [a + b for a, b in zip(kv_lens, new_lens)]
    return table, lens, offsets, slots + [-1] * (capacity - total), [at, total]


def append(values, scales, x, slots, which, block, kind):
    """One tensor's append, in place: values [num_pages, Hkv, P, d] (what the
    bytes hold), scales [num_pages, Hkv, P/S, 2], x [T, Hkv, d].  Tokens with
    a slot outside the pool count for nothing (fewer than 32 in a row)."""
    page = values.shape[2]
    keep = [t for t, sl in enumerate(slots) if 0 <= sl < values.shape[0] * page]
    x, slots = x[keep], [slots[t] for t in keep]
    i = 0
    while i < len(slots):
        j = i + 1
        while j < len(slots) and slots[j] // block == slots[i] // block:
            j += 1
        pg, row = divmod(slots[i], page)
        cell, before = divmod(row, block)
        for h in range(values.shape[1]):
            new = x[i:j, h].astype(np.float64)
            fin = np.abs(new[np.isfinite(new)])
            s = scale_for(float(fin.max()) if fin.size else 0.0, kind)
            old = float(scales[pg, h, cell, which])
            if before and old >= s:
                s = old
            elif before:
                rows = slice(cell * block, cell * block + before)
                values[pg, h, rows] = nearest(values[pg, h, rows] * (old / s), kind)
            scales[pg, h, cell, which] = s
            for t in range(i, j):
                values[pg, h, slots[t] % page] = nearest(x[t, h].astype(np.float64) / s, kind)
        i = j


def rows_of(values, scales, which, table_row, h, n):
    """Head h's first n rows of the request with page list table_row."""
    page, block = values.shape[2], values.shape[2] // scales.shape[2]
    out = np.zeros((n, values.shape[3]))
    for j in range(n):
        pg, r = table_row[j // page], j % page
        out[j] = values[pg, h, r] * float(scales[pg, h, r // block, which])
    return out


def attend(q, k, v):
    """Softmax attention of rows q [G, d] over k, v [n, d]: (o, lse, the sum of
    p |v| per output, the largest sum of |q k| / sqrt(d))."""
    if len(k) == 0:
        z = np.zeros((len(q), q.shape[1]))
        return z, np.full(len(q), -math.inf), z, 0.0
    s = q @ k.T / math.sqrt(q.shape[1])
    m = s.max(1, keepdims=True)
    p = np.exp(s - m)
    l = p.sum(1, keepdims=True)
    mass = float((np.abs(q) @ np.abs(k).T).max() / math.sqrt(q.shape[1]))
    return p @ v / l, (m + np.log(l))[:, 0], p @ np.abs(v) / l, mass
