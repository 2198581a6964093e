"""Seeded inputs of the paged 8-bit key/value cache: a pool with random codes
and scales, table rows of given lengths, rotary frequencies and positions.
Holds no arithmetic of the method."""
from __future__ import annotations

import numpy as np


def make_kv_pool(rng, layers, pages, heads, dim, fmt):
    """Codes near normal, scales that differ from block to block."""
    shape = (layers, pages, heads, 64 * dim)
    cache = {"format": fmt}
    for w in ("k", "v"):
        x = rng.standard_normal(shape).astype(np.float32)
        if fmt == "int8":
            cache[w] = (np.clip(np.rint(x * 36), -127, 127) + 128).astype(np.uint8)
        else:
            # every finite e4m3 byte
            cache[w] = (rng.integers(0, 127, shape) + 128 * rng.integers(0, 2, shape)).astype(np.uint8)
        top = 3.5 / 127 if fmt == "int8" else 3.5 / 448
        cache[w + "s"] = (top * 2.0 ** rng.uniform(-2, 1, (layers, pages, heads, 4))).astype(np.float32)
    return cache


def make_kv_table(rng, lens, spare=2, extra=1):
    """(table [rows][max_pages], pages): the rows' pages in random order."""
    need = [-(-n // 64) for n in lens]
    pages = sum(need) + spare
    order = rng.permutation(pages).tolist()
    width = max(max(need), 1) + extra
    table = np.full((len(lens), width), -1, np.int32)
    for i, n in enumerate(need):
        table[i, :n] = [order.pop() for _ in range(n)]
    return table, max(pages, 1)


def rope_freqs(rot, theta=1e6):
    return (theta ** (-2 * np.arange(rot // 2) / max(rot, 1))).astype(np.float32)
