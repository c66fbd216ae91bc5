"""Oracle for the 4-bit KV cache, the accumulated attention weights and the eviction by them: plain,
slow fp64 / integer numpy restatements of what include/oda.h defines.

TEST INFRASTRUCTURE ONLY, as oda_oracle: it shares no code with the CUDA library. Every function is
pinned by tests/test_kv4_oracle_pins.py.
"""
from __future__ import annotations

import numpy as np

from oracle import oda_oracle as O

PAGE_BYTES = 2304
GROUP = 64


def bf16_up(x: float) -> float:
    """The least bf16 value that is not below x >= 0, by trying the bit patterns around it."""
    bits = int(np.float32(x).view(np.uint32)) >> 16
    best = None
    for c in range(max(0, bits - 1), bits + 3):
        v = float(np.uint32(c << 16).view(np.float32))
        if v >= x and (best is None or v < best):
            best = v
    return best


def quantise_group(x):
    """(codes, scale, minimum) of one group of fp64 values that are bf16 values: minimum = the
    least, scale = the bf16 at or above span / 15, codes = the nearest whole number of scales."""
    x = np.asarray(x, dtype=np.float64)
    span = x.max() - x.min() if np.all(np.isfinite(x)) else np.inf
    if not np.isfinite(np.float32(span)):
        return np.zeros(len(x), dtype=np.int64), np.nan, np.nan
    scale = bf16_up(span / 15.0)
    if scale == 0.0:
        return np.zeros(len(x), dtype=np.int64), 0.0, x.min()
    return np.minimum(np.rint((x - x.min()) / scale).astype(np.int64), 15), scale, x.min()


def round_trip(rows):
    """What bf16 rows [..., 128] (as fp64) read back as."""
    rows = np.asarray(rows, dtype=np.float64)
    flat = rows.reshape(-1, GROUP)
    out = np.empty_like(flat)
    for i, x in enumerate(flat):
        c, s, m = quantise_group(x)
        out[i] = m + c * s
    return out.reshape(rows.shape)


def unpack_pages(pages):
    """Pages uint8 [..., 2304] -> K, V fp64 [..., 16, 128], byte by byte from the layout."""
    pages = np.asarray(pages, dtype=np.uint8)
    lead = pages.shape[:-1]
    p = pages.reshape(-1, PAGE_BYTES)
    meta = O.widen_bf16(p[:, 2048:].copy().view(np.uint16).reshape(-1, 16, 4, 2))
    out = []
    for part in (0, 1):
        codes = p[:, 1024 * part:1024 * (part + 1)].reshape(-1, 16, 64)
        x = np.empty(codes.shape[:2] + (128,))
        for dim in range(128):
            g, i, k = dim // 64, (dim % 64) // 8, dim % 8
            c = (codes[:, :, 4 * (2 * i + g) + k // 2] >> (4 * (k % 2))) & 15
            with np.errstate(invalid="ignore"):
                x[:, :, dim] = meta[:, :, 2 * part + g, 1] + c * meta[:, :, 2 * part + g, 0]
        out.append(x.reshape(lead + (16, 128)))
    return out


def attention_mass(q, k_rows, scale, group):
    """Softmax weights of positions, summed over the query heads of each KV head: q [Hq][128],
    k_rows a list of [n][128] per KV head -> [Hkv][n]."""
    out = np.zeros((len(k_rows), k_rows[0].shape[0]))
    for g, k in enumerate(k_rows):
        for h in range(g * group, (g + 1) * group):
            z = k @ np.asarray(q[h], dtype=np.float64) * scale
            if z.size:
                w = np.exp(z - z.max())
                out[g] += w / w.sum()
    return out


def kept_slots(mass, n, sink, recent, budget):
    """The slots of one (sequence, KV head) of n tokens that stay, ascending."""
    if n <= budget:
        return np.arange(n)
    free = list(range(sink, n - recent))
    free.sort(key=lambda p: (-(float(mass[p]) + 0.0), p))
    best = sorted(free[:budget - sink - recent])
    return np.array(list(range(sink)) + best + list(range(n - recent, n)), dtype=np.int64)
