"""Plain fp64 forms of a decoding step with a tree of drafted tokens: per-head
norms, trees, attention by an explicit matrix of who sees whom, accepting a
path and moving its tokens, and log probabilities, from their definitions."""
from __future__ import annotations

import math

import numpy as np

from .kv_oracle import BLOCK, PAGE, kv_encode, kv_places, kv_sequence, kv_table


def norm_f64(x, weight, eps):
    """x [..., D] normed over its last axis."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(all="ignore"):
        return x / np.sqrt((x * x).sum(-1, keepdims=True) / x.shape[-1] + eps) * np.asarray(weight, dtype=np.float64)


def tree_above(parent):
    """Of each row the rows from itself up, itself first."""
    out = []
    for i, p in enumerate(parent):
        out.append([i] + (out[p] if 0 <= p < i else []))
    return out


def tree_seen(parent, window=0):
    """bool [n][n]: row i sees row j."""
    n = len(parent)
    seen = np.zeros((n, n), bool)
    for i, rows in enumerate(tree_above(parent)):
        seen[i, rows[:window] if window else rows] = True
    return seen


def tree_words(seen, words):
    """uint64 [n][words] of a bool [n][n]; rows past 64 * words are left out."""
    out = np.zeros((len(seen), words), np.uint64)
    for i, row in enumerate(seen):
        for j in np.nonzero(row)[0]:
            if j < 64 * words:
                out[i, j // 64] |= np.uint64(1) << np.uint64(j % 64)
    return out


def tree_context(n, base, seen, window=0, sinks=0):
    """bool [n][base + n] of what a tree's rows see of a sequence of base + n tokens."""
    out = np.zeros((n, base + n), bool)
    for i in range(n):
        count = int(seen[i].sum())
        for j in range(base):
            out[i, j] = not window or j >= base - max(window - count, 0) or j < sinks
        out[i, base:] = seen[i]
    return out


def causal_context(n, base, window=0, sinks=0):
    """bool [n][base + n] of what the last n rows see; base may be negative."""
    out = np.zeros((n, max(base + n, 0)), bool)
    for i in range(n):
        for j in range(max(base + i + 1, 0)):
            out[i, j] = not window or j > base + i - window or j < sinks
    return out


def kv_attn_seen_f64(cache, layer, row, n, q, scale, seen):
    """As kv_attn_f64 with seen bool [rows][n]."""
    k, v = (kv_sequence(cache, layer, row, n, w) for w in ("k", "v"))
    rows, heads, D = q.shape
    group = heads // k.shape[1]
    out, mass = np.zeros((rows, heads, D)), np.zeros((rows, heads, D))
    held = np.array([0 <= int(row[t // PAGE]) < cache["k"].shape[1] for t in range(n)], dtype=bool)
    for i in range(rows):
        at = np.nonzero(seen[i] & held)[0]
        if not at.size:
            continue
        for h in range(heads):
            s = k[at, h // group] @ q[i, h].astype(np.float64) * scale
            p = np.exp(s - s.max())
            out[i, h] = p @ v[at, h // group] / p.sum()
            mass[i, h] = p @ np.abs(v[at, h // group]) / p.sum()
    return out, mass


def tree_accept(target, token, parent, max_path):
    """(rows taken, the token behind them) of one sequence."""
    if not len(target):
        return [], -1
    path = [0]
    while len(path) < max_path:
        at = path[-1]
        nxt = [i for i in range(at + 1, len(parent)) if parent[i] == at and token[i] == target[at]]
        if not nxt:
            break
        path.append(nxt[0])
    return path, int(target[path[-1]])


def kv_keep_f64(cache, row, base, path):
    """Moves tokens base + path[i] of one sequence to base + i in all layers, in
    place; the ratio of two scales and its product with a code are fp32."""
    D = cache["k"].shape[3] // PAGE
    fmt, table = cache["format"], kv_table(cache["format"])
    pages = cache["k"].shape[1]
    held = lambda t: 0 <= int(row[t // PAGE]) < pages
    moves = {base + i: base + p for i, p in enumerate(path) if p != i and held(base + i) and held(base + p)}
    for which in ("k", "v"):
        place = kv_places(which, D)
        for layer in range(cache["k"].shape[0]):
            for block in sorted({t // BLOCK for t in moves}):
                page, b = int(row[block * BLOCK // PAGE]), block % (PAGE // BLOCK)
                for h in range(cache["k"].shape[2]):
                    codes, scales = cache[which][layer, page, h], cache[which + "s"][layer, page, h]
                    made = []
                    own = scales[b]
                    for t in range(block * BLOCK, (block + 1) * BLOCK):
                        src = moves.get(t, t)
                        p = int(row[src // PAGE]) if t in moves else page
                        made.append((cache[which][layer, p, h][place[src % PAGE]].copy(),
                                     cache[which + "s"][layer, p, h, src % PAGE // BLOCK] if t in moves else own))
                    top = max(s for _, s in made + [(None, own)])
                    for t, (c, s) in zip(range(block * BLOCK, (block + 1) * BLOCK), made):
                        codes[place[t % PAGE]] = c if s == top else kv_encode(table[c].astype(np.float32) * (np.float32(s) / np.float32(top)), fmt)
                    scales[b] = top


def logprobs_f64(x, tokens, top):
    """(logprob [count], entropy, top_tokens, top_logprobs) of one row, by value with ties to the lowest token, NaN first."""
    x = np.asarray(x, dtype=np.float64)
    order = sorted(range(len(x)), key=lambda v: (not math.isnan(x[v]), -x[v] if not math.isnan(x[v]) else 0.0, v))[:top]
    with np.errstate(all="ignore"):
        m = x.max()
        if not np.isfinite(m):
            lp, entropy = np.full(len(x), np.nan), np.nan
        else:
            e = np.exp(x - m)
            lp = (x - m) - np.log(e.sum())
            p = e / e.sum()
            entropy = -float(np.sum(np.where(p > 0, p * np.where(p > 0, lp, 0), 0)))
    fine = np.isfinite(m)
    given = np.array([(lp[t] if 0 <= t < len(x) else -np.inf) if fine else np.nan for t in tokens])
    tt = np.array(order + [-1] * (top - len(order)))
    tl = np.array([lp[t] if fine else np.nan for t in order] + [-np.inf] * (top - len(order)))
    return given, entropy, tt, tl
