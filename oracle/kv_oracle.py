"""Plain fp64 forms of the rotary positions, the paged 8-bit key/value cache,
its attention and its page operations, from their definitions.

A cache is a dict of NumPy arrays: k, v uint8 [layers][pages][heads][64*D],
ks, vs [layers][pages][heads][4], and "format" ("int8" or "e4m3")."""
from __future__ import annotations

import numpy as np

PAGE, BLOCK = 64, 16
QMAX = {"int8": 127.0, "e4m3": 448.0}


def kv_place_k(token: int, dim: int, D: int) -> int:
    """Byte of (token, dim) in a K page: [token/16][dim/64][dim/16%4][token%16][dim%16]."""
    return (token // 16) * 16 * D + (dim // 64) * 1024 + (dim // 16 % 4) * 256 + (token % 16) * 16 + dim % 16


def kv_place_v(token: int, dim: int, D: int) -> int:
    """Byte of (token, dim) in a V page: [dim/16][token/4%4][dim%16][token/16][token%4]."""
    return (dim // 16) * 1024 + (token // 4 % 4) * 256 + (dim % 16) * 16 + (token // 16) * 4 + token % 4


def kv_places(which: str, D: int) -> np.ndarray:
    place = kv_place_k if which == "k" else kv_place_v
    return np.array([[place(t, d, D) for d in range(D)] for t in range(PAGE)])


def kv_table(fmt: str) -> np.ndarray:
    """Value of each byte."""
    b = np.arange(256)
    if fmt == "int8":
        return b - 128.0
    sign = np.where(b & 128, -1.0, 1.0)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    return np.where((b & 127) == 127, np.nan, sign * v)


def kv_encode(x: np.ndarray, fmt: str) -> np.ndarray:
    """Bytes of the codes nearest to x (in units of the scale), ties to even;
    past the largest code: that code; NaN: 0."""
    x = np.asarray(x, dtype=np.float64)
    zero = 128 if fmt == "int8" else 0
    if fmt == "int8":
        return np.where(np.isnan(x), zero, np.clip(np.rint(np.nan_to_num(x, nan=0.0)), -127, 127) + 128).astype(np.uint8)
    a = np.minimum(np.abs(np.nan_to_num(x, nan=0.0)), 448.0)
    top = kv_table(fmt)[:127]                       # rising, bytes 0..126
    hi = np.clip(np.searchsorted(top, a), 1, 126)
    lo = hi - 1
    dl, dh = a - top[lo], top[hi] - a
    byte = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    byte = np.where(a == 0, 0, byte)
    return np.where(np.isnan(x), zero, byte + np.where(np.signbit(np.nan_to_num(x, nan=0.0)), 128, 0)).astype(np.uint8)


def rope_f64(x, pos, inv_freq, axis=None, adjacent=False):
    """x [tokens][heads][D] fp64; pos [axes][tokens]."""
    x = np.asarray(x, dtype=np.float64)
    y, rot = x.copy(), 2 * len(inv_freq)
    for r in range(rot // 2):
        ax = 0 if axis is None else int(axis[r])
        a = (np.asarray(pos[ax], dtype=np.float64) * float(inv_freq[r]))[:, None]
        i, j = (2 * r, 2 * r + 1) if adjacent else (r, r + rot // 2)
        y[..., i] = x[..., i] * np.cos(a) - x[..., j] * np.sin(a)
        y[..., j] = x[..., j] * np.cos(a) + x[..., i] * np.sin(a)
    return y


def kv_sequence(cache, layer, row, n, which):
    """Held values [n][heads][D] of a table row's first n tokens, fp64."""
    D = cache["k"].shape[3] // PAGE
    ids = np.asarray(row[:-(-n // PAGE)], dtype=np.int64)
    held = (ids >= 0) & (ids < cache["k"].shape[1])
    ids = np.where(held, ids, 0)
    codes = kv_table(cache["format"])[cache[which][layer][ids]][:, :, kv_places(which, D).ravel()]
    codes = codes.reshape(codes.shape[0], codes.shape[1], PAGE, D)
    values = codes * np.repeat(cache[which + "s"][layer][ids].astype(np.float64), BLOCK, axis=-1)[..., None]
    # [pages][heads][64][D] to tokens; a page that is none holds nothing
    return np.where(held[:, None, None, None], values, 0.0).swapaxes(1, 2).reshape(-1, values.shape[1], D)[:n]


def kv_append_f64(cache, layer, row, start, k, v):
    """Writes rows k, v [n][heads][D] (already turned) of one sequence as its tokens from start on."""
    n, heads, D = k.shape
    top, zero = QMAX[cache["format"]], (128 if cache["format"] == "int8" else 0)
    for which, new in (("k", k), ("v", v)):
        place = kv_places(which, D)
        for block in range(start // BLOCK, (start + n - 1) // BLOCK + 1):
            page, b = int(row[block * BLOCK // PAGE]), block % (PAGE // BLOCK)
            for h in range(heads):
                codes, scales = cache[which][layer, page, h], cache[which + "s"][layer, page, h]
                tokens = np.arange(block * BLOCK, (block + 1) * BLOCK)
                fresh = new[[t - start for t in tokens if start <= t < start + n], h]
                finite = np.abs(fresh[np.isfinite(fresh)])
                scale = (finite.max() if finite.size else 0.0) / top
                held = float(scales[b]) if tokens[0] < start else 0.0
                scale = max(scale, held)
                for t in tokens:
                    at = place[t % PAGE]
                    if t < start:
                        x = kv_table(cache["format"])[codes[at]] * (held / scale if scale > 0 else 0.0)
                    elif t < start + n:
                        with np.errstate(invalid="ignore"):
                            x = new[t - start, h] / scale if scale > 0 else np.where(np.isinf(new[t - start, h]), np.nan, 0.0)
                    else:
                        codes[at] = zero
                        continue
                    codes[at] = kv_encode(x, cache["format"])
                scales[b] = scale


def kv_attn_f64(cache, layer, row, n, q, scale, causal=True, window=0):
    """(out [rows][q_heads][D], mass of the same shape) of one sequence that
    holds n tokens: mass = sum p|v| / sum p."""
    k, v = (kv_sequence(cache, layer, row, n, w) for w in ("k", "v"))
    rows, heads, D = q.shape
    group = heads // k.shape[1]
    out, mass = np.zeros((rows, heads, D)), np.zeros((rows, heads, D))
    held = np.array([0 <= int(row[t // PAGE]) < cache["k"].shape[1] for t in range(n)], dtype=bool)
    for i in range(rows):
        pos = n - rows + i
        j = np.arange(n)
        seen = held & (j <= pos if causal else np.ones(n, bool))
        if causal and window > 0:
            seen &= j > pos - window
        if not seen.any():
            continue
        for h in range(heads):
            s = k[seen, h // group] @ q[i, h].astype(np.float64) * scale
            p = np.exp(s - s.max())
            out[i, h] = p @ v[seen, h // group] / p.sum()
            mass[i, h] = p @ np.abs(v[seen, h // group]) / p.sum()
    return out, mass


class PagesOracle:
    """Tables, lengths, reference counts and page contents (one hashable value
    per page) as plain lists, changed a page at a time."""

    def __init__(self, table, lens, refs, contents):
        self.table, self.lens = [list(r) for r in table], list(lens)
        self.refs, self.contents = list(refs), list(contents)

    def _pages(self, n):
        return -(-n // PAGE)

    def _take(self):
        return self.refs.index(0)

    def _free(self):
        return self.refs.count(0)

    def fork(self, src, dst):
        """(told, copies)"""
        rows = len(self.lens)
        if len(set(dst)) < len(dst) or any(not (0 <= s < rows and 0 <= d < rows) or s == d for s, d in zip(src, dst)):
            return -1, 0
        if any(self.lens[d] != 0 for d in dst):
            return -1, 0
        need = sum(self.lens[s] % PAGE != 0 for s in src)
        if need > self._free():
            return need - self._free(), 0
        lens = [self.lens[s] for s in src]
        for s, d, n in zip(src, dst, lens):
            full = n // PAGE
            row = [-1] * len(self.table[d])
            for c in range(full):
                row[c] = self.table[s][c]
                self.refs[row[c]] += 1
            if n % PAGE:
                row[full] = self._take()
                self.refs[row[full]] = 1
                self.contents[row[full]] = self.contents[self.table[s][full]]
            self.table[d], self.lens[d] = row, n
        return 0, need

    def resize(self, want):
        if any(not -1 <= w <= len(self.table[0]) * PAGE for w in want):
            return -1, 0
        want = [n if w < 0 else w for n, w in zip(self.lens, want)]
        refs = list(self.refs)
        for row, n, w in zip(self.table, self.lens, want):
            for c in range(self._pages(w), self._pages(n)):
                refs[row[c]] -= 1
        split = [w < n and w % PAGE != 0 and refs[row[self._pages(w) - 1]] > 1
                 for row, n, w in zip(self.table, self.lens, want)]
        need = sum(max(self._pages(w) - self._pages(n), 0) + s for n, w, s in zip(self.lens, want, split))
        if need > refs.count(0):
            return need - refs.count(0), 0
        self.refs = refs
        let_go = []
        for i, (n, w) in enumerate(zip(self.lens, want)):
            row = self.table[i]
            for c in range(self._pages(w), self._pages(n)):
                row[c] = -1
            if split[i]:
                old, new = row[self._pages(w) - 1], self._take()
                self.refs[new], row[self._pages(w) - 1] = 1, new
                self.contents[new] = self.contents[old]
                let_go.append(old)
            for c in range(self._pages(n), self._pages(w)):
                row[c] = self._take()
                self.refs[row[c]] = 1
            self.lens[i] = w
        for p in let_go:
            self.refs[p] -= 1
        return 0, len(let_go)

    def compact(self):
        live = sum(r > 0 for r in self.refs)
        src = [p for p in range(live, len(self.refs)) if self.refs[p] > 0]
        dst = [p for p in range(live) if self.refs[p] <= 0]
        for s, d in zip(src, dst):
            self.contents[d], self.refs[d], self.refs[s] = self.contents[s], self.refs[s], 0
        to = dict(zip(src, dst))
        self.table = [[to.get(p, p) for p in row] for row in self.table]
        return 0, len(src)
