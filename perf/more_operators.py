"""What is measured of a decoding step with a tree of drafted tokens, over the paged key/value cache in 8 bits: norms of
queries and keys with the rotation on their way into the cache, attention with a window and sinks, attention of the tree,
log probabilities with entropy and top alternatives, and accepting a path of the tree.

The cache: pages of 64 tokens, one scale for each block of 16 tokens and head.  A page's codes are held in the order
in which the matrix instructions of the attention take them (`_k_at`, `_v_at`); a value is scale * code, the code
an int8 held as byte code + 128, or an e4m3 number.
"""
import math
import random

import torch

own = False

PAGE, BLOCK = 64, 16
QMAX = {"int8": 127.0, "e4m3": 448.0}
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    wide = {"heads": 48, "kv_heads": 8, "dim": 128}  # q 6144, k/v 1024 columns: the repository's projection shapes
    attn = {"window": 0, "sinks": 0, "words": 0, "format": "int8"}
    return [
        # one decode step of 32 sequences: q and k are normed, turned, and k and v join partly filled blocks
        {"name": "norm_step", "op": "norm", **wide, "batch": 32, "new": 1, "ctx": 4001, "axes": 1, "format": "int8"},
        # a prompt's chunk behind an odd number of held tokens
        {"name": "norm_prompt", "op": "norm", **wide, "batch": 1, "new": 4093, "ctx": 5120, "axes": 1, "format": "int8"},
        # one token each of eight long sequences in a layer that sees a window and the first tokens
        {"name": "sink_token", "op": "attn", **wide, **attn, "batch": 8, "new": 1, "ctx": 131001, "window": 4096, "sinks": 4},
        # a prompt's chunk in such a layer
        {"name": "sink_prompt", "op": "attn", **wide, **attn, "batch": 1, "new": 2047, "ctx": 10240, "window": 1024, "sinks": 4},
        # a small tree behind a short context: a latency-bound call
        {"name": "tree_one", "op": "attn", **wide, **attn, "batch": 1, "new": 13, "ctx": 1003, "words": 1},
        # trees of 61 rows of sequences of very different lengths
        {"name": "tree_batch", "op": "attn", **wide, **attn, "batch": 16, "new": 61, "ctx": 16384, "words": 1, "format": "e4m3"},
        # a tree over a long context: bound by the matrix cores
        {"name": "tree_long", "op": "attn", **wide, **attn, "batch": 1, "new": 64, "ctx": 131001, "words": 1},
        # the rows of a short draft: the token's probability and the alternatives that a server answers with
        {"name": "logprob_step", "op": "logprobs", "rows": 5, "vocab": 151936, "half": True, "count": 1, "top": 20, "entropy": False},
        # a drafting model's next level for a batch: alternatives for the tree, fp32 logits
        {"name": "logprob_draft", "op": "logprobs", "rows": 301, "vocab": 32000, "half": False, "count": 0, "top": 10, "entropy": True},
        # scoring a long text
        {"name": "logprob_score", "op": "logprobs", "rows": 2047, "vocab": 151936, "half": True, "count": 1, "top": 5, "entropy": True},
        # a tree's masks, its accepted path, and that path's keys and values moved behind the context: one sequence
        {"name": "accept_one", "op": "accept", "kv_heads": 8, "dim": 128, "layers": 2, "batch": 1, "new": 13, "ctx": 1003, "levels": 4, "format": "int8"},
        # and a batch of larger trees
        {"name": "accept_batch", "op": "accept", "kv_heads": 8, "dim": 128, "layers": 4, "batch": 32, "new": 61, "ctx": 4001, "levels": 8, "format": "int8"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rows", "norm", "attn", "attn", "attn", "logprobs", "logprobs", "accept"])
    dim = rng.choice([64, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 6, 8])
    form = rng.choice(["int8", "e4m3"])
    if op == "rows":  # norm and rotation of rows that go to no cache
        return {"op": op, "tokens": _log(rng, 1, 8000), "heads": kv_heads * group, "dim": dim,
                "rot": rng.choice([dim, dim // 2, 0]), "axes": rng.choice([1, 2, 3]), "adjacent": rng.random() < 0.3}
    if op == "norm":
        new = _log(rng, 1, 4000)
        batch = max(1, min(64, _log(rng, 1, 64), 4000 // new))
        return {"op": op, "heads": kv_heads * group, "kv_heads": kv_heads, "dim": dim, "batch": batch, "new": new,
                "ctx": new + _log(rng, 1, 4000), "axes": rng.choice([1, 3]), "format": form}
    if op == "logprobs":
        vocab, count = _log(rng, 100, 160000), rng.choice([0, 1, 1, 7])
        return {"op": op, "rows": _log(rng, 1, max(1, min(2000, 100_000_000 // vocab))), "vocab": vocab, "half": rng.random() < 0.6,
                "count": count, "top": rng.choice([0, 1, 5, 20, 64] if count else [1, 5, 20, 64]), "entropy": rng.random() < 0.5}
    if op == "accept":
        new = _log(rng, 2, 250)
        return {"op": op, "kv_heads": kv_heads, "dim": dim, "layers": rng.choice([1, 2, 3]), "batch": min(_log(rng, 1, 64), max(1, 4000 // new)),
                "new": new, "ctx": new + _log(rng, 1, 4000), "levels": rng.randint(1, 8), "format": form}
    tree = rng.random() < 0.6
    window = _log(rng, 16, 8192) if not tree or rng.random() < 0.3 else 0
    new = _log(rng, 2, 250) if tree else rng.choice([1, 1, 2, 5, _log(rng, 6, 2000)])
    batch = _log(rng, 1, max(1, min(64, 2000 // new)))
    ctx = new + _log(rng, 1, max(16, min(262144, 8_000_000 // new) // batch))
    return {"op": op, "heads": kv_heads * group, "kv_heads": kv_heads, "dim": dim, "batch": batch, "new": new, "ctx": ctx,
            "window": window, "sinks": rng.choice([0, 1, 4, 4, 70]) if window else 0, "words": -(-new // 64) if tree else 0, "format": form}


def _lens(case):
    """Tokens held for each sequence: from ctx down to ctx / 16, spread over the logarithm."""
    b = case["batch"]
    return [max(case["new"], int(case["ctx"] * 16.0 ** (-i / max(1, b - 1)))) for i in range(b)]


def _tree(rng, n, levels):
    """parent of each of n rows, level by level behind row 0, the last token."""
    size = [1] + [1] * min(levels, n - 1)
    for _ in range(n - len(size) if len(size) > 1 else 0):
        size[rng.randint(1, len(size) - 1)] += 1
    parent, at = [-1], 0
    for k in size[1:]:
        before = len(parent)
        parent += sorted(rng.randint(at, before - 1) for _ in range(k))
        at = before
    return parent


def _path(rng, parent):
    """Rows of a path from row 0: it can be moved to the front again and again (no row that it comes from is one that it goes to)."""
    node, path = len(parent) - 1 - rng.randint(0, len(parent) // 3), []
    while node >= 0:
        path.append(node)
        node = parent[node]
    path.reverse()
    k = len(path)
    while any(p != i and p < k for i, p in enumerate(path[:k])):
        k -= 1
    return path[:k]


def _trees(case):
    """(parents, accepted paths) of the sequences of a case: the same for every seed."""
    rng = random.Random(11)
    parents = [_tree(rng, case["new"], case.get("levels", 8)) for _ in range(case["batch"])]
    return parents, [_path(rng, p) for p in parents]


def work(case):
    op = case["op"]
    if op == "rows":
        n = case["tokens"] * case["heads"] * case["dim"]
        return {"bytes": 4 * n + 4 * case["tokens"] * case["axes"], "flops": 7 * n}
    if op == "logprobs":
        n, r = case["rows"] * case["vocab"], case["rows"]
        return {"bytes": n * (2 if case["half"] else 4) + r * (8 * case["count"] + 8 * case["top"] + 4 * case["entropy"]), "flops": 4 * n}
    kh, d, new, b = case["kv_heads"], case["dim"], case["new"], case["batch"]
    t = b * new
    if op == "norm":
        # q read and written, k and v read, codes written; then the codes read back and given as fp16
        h = case["heads"]
        return {"bytes": 4 * t * h * d + 4 * t * kh * d + 2 * t * kh * d + 6 * t * kh * d, "flops": t * (h + 3 * kh) * d * 7}
    if op == "accept":
        kept = sum(map(len, _trees(case)[1]))
        # parents, tokens, targets; masks and positions; the kept rows' codes; all rows read back as fp16
        return {"bytes": 12 * t + t * (8 * -(-new // 64) + 4) + 4 * kept + case["layers"] * kh * d * (4 * kept + 6 * t), "flops": 0}
    pairs = held = 0
    w, sinks, h = case["window"], case["sinks"], case["heads"]
    parents = _trees(case)[0] if case["words"] else []
    for i, n in enumerate(_lens(case)):
        first = n - new
        if case["words"]:
            depth = []
            for p in parents[i]:
                depth.append(1 if p < 0 else depth[p] + 1)  # rows that a row sees of the tree
            low = [max(first - max(w - k, 0), 0) if w else 0 for k in depth]
            pairs += sum(k + first - lo + min(sinks, lo) for k, lo in zip(depth, low))
            held += new + first - min(low) + min(sinks, min(low))
        else:
            low = [max(p - w + 1, 0) if w else 0 for p in range(first, n)]
            pairs += sum(p + 1 - lo + min(sinks, lo) for p, lo in zip(range(first, n), low))
            held += n - low[0] + min(sinks, low[0])
    return {"bytes": held * kh * (2 * d + 8 / BLOCK) + 4 * t * h * d + 8 * t * case["words"], "flops": 4 * pairs * h * d}


# ------------------------------------------------------------------ inputs
def _codes(gen, n, form):
    """n random codes as a trained model's keys and values give them: near normal, the largest of a block at the range's end."""
    out = torch.empty(n, dtype=torch.uint8, device="cuda")
    step = 1 << 27
    for at in range(0, n, step):
        x = torch.randn(min(step, n - at), generator=gen, device="cuda")
        if form == "int8":
            out[at:at + step] = ((x * 36).round().clamp(-127, 127) + 128).to(torch.uint8)
        else:
            out[at:at + step] = (x * 120).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return out


def _pool(gen, layers, pages, case):
    kh, d, form = case["kv_heads"], case["dim"], case["format"]
    n = layers * pages * kh * PAGE * d
    s = {"k": _codes(gen, n, form), "v": _codes(gen, n, form)}
    top = 3.5 / QMAX[form]
    for x in ("k", "v"):
        s[x] = s[x].view(layers, pages, kh, PAGE * d)
        s[x + "_scales"] = (torch.rand(layers, pages, kh, PAGE // BLOCK, generator=gen, device="cuda") * 0.5 + 0.75) * top
    s["format"] = form
    return s


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _positions(gen, axes, tokens):
    """[axes][tokens]: text runs up on every axis, every second stretch of 256 tokens is a picture of 16 x 16."""
    t = torch.arange(tokens, device="cuda") + int(torch.randint(0, 30000, (1,), generator=gen, device="cuda"))
    pos = t.repeat(axes, 1)
    if axes > 1:
        at = torch.arange(tokens, device="cuda")
        picture = (at // 256) % 2 == 1
        for a in range(1, axes):
            inside = (at % 256) // 16 if a == 1 else at % 16
            pos[a] = torch.where(picture, pos[a] - at % 256 + inside, pos[a])
    return pos.to(torch.int32).contiguous()


def _angles(axes, rot):
    """(inv_freq [rot/2], axis of each pair): theta 1e6, the axes share the pairs in turn."""
    r = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    inv = (1e6 ** (-2 * r / max(rot, 1))).to(torch.float32)
    return inv, (torch.arange(rot // 2, device="cuda") % axes).to(torch.int32)


def _weight(gen, d):
    """A norm's weights as training leaves them: near 1, some dimensions several times that."""
    return torch.exp(0.4 * torch.randn(d, generator=gen, device="cuda"))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    s = {"op": op, "case": dict(case)}
    if op == "rows":
        s["x"] = (torch.randn(case["tokens"], case["heads"], case["dim"], generator=gen, device="cuda") * 3).half()
        s["pos"] = _positions(gen, case["axes"], case["tokens"])
        s["inv_freq"], s["axis"] = _angles(case["axes"], case["rot"])
        s["weight"] = _weight(gen, case["dim"])
        return s
    if op == "logprobs":
        r, v = case["rows"], case["vocab"]
        x = torch.empty(r, v, dtype=torch.float16 if case["half"] else torch.float32, device="cuda")
        for at in range(0, r, 512):
            x[at:at + 512] = torch.randn(min(512, r - at), v, generator=gen, device="cuda") * 2.5
        # each row has a few likely tokens, and the vocabulary is padded with columns that no token has
        likely = torch.randint(0, v // 6, (r, 6), generator=gen, device="cuda") + torch.arange(6, device="cuda") * (v // 6)
        x.scatter_add_(1, likely, (torch.rand(r, 6, generator=gen, device="cuda") * 16).to(x.dtype))
        pad = v // 570
        if pad:
            x[:, v - pad:] = -math.inf
        s["logits"] = x
        s["tokens"] = torch.where(torch.rand(r, case["count"], generator=gen, device="cuda") < 0.7, likely[:, :1],
                                  torch.randint(0, v - pad, (r, case["count"]), generator=gen, device="cuda")).int() if case["count"] else None
        s["workspace"] = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
        return s
    lens, new, b = _lens(case), case["new"], case["batch"]
    need = [-(-n // PAGE) for n in lens]
    pages, width = sum(need) + 3, max(need) + 1
    order = torch.randperm(pages, generator=gen, device="cuda").tolist()
    table, at = [], 0
    for n in need:
        table.append(order[at:at + n] + [-1] * (width - n))
        at += n
    s |= _pool(gen, case.get("layers", 1), pages, case)
    s |= {"table": _ints(table), "lens": _ints(lens), "cu": _ints([new * i for i in range(b + 1)]), "max_len": max(lens)}
    kh, d = case["kv_heads"], case["dim"]
    if op == "accept" or op == "attn" and case["words"]:
        parents, paths = _trees(case)
        s["parent"] = _ints([p for row in parents for p in row])
        s["max_path"] = case.get("levels", 8) + 1
    if op == "accept":
        # siblings have tokens of their own; the target model takes the path's, and tokens that no row has where it ends
        s["token"] = torch.randperm(b * new, generator=gen, device="cuda").int()
        target = torch.randint(100000, 150000, (b * new,), generator=gen, device="cuda").int()
        last = [(i * new + p, i * new + q) for i, path in enumerate(paths) for p, q in zip(path, path[1:])]
        if last:
            f, t = torch.tensor(last, device="cuda").t()
            target[f] = s["token"][t]
        s["target"] = target
        s["total"] = b * new
        return s
    h = case["heads"]
    if op == "attn":
        s["q"] = (2 * torch.randn(b * new, h, d, generator=gen, device="cuda")).half()
        s["workspace"] = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
        if case["words"]:
            s["mask"] = _plain_plan(s)[0]
        return s
    # the rows of a fused q, k, v product
    qkv = torch.randn(b * new, (h + 2 * kh) * d, generator=gen, device="cuda").half()
    for name, lo, n in (("q", 0, h), ("k_new", h, kh), ("v_new", h + kh, kh)):
        s[name] = qkv[:, lo * d:(lo + n) * d].unflatten(1, (n, d))
    s["pos"] = _positions(gen, case["axes"], b * new)
    s["inv_freq"], s["axis"] = _angles(case["axes"], d // 2 if d == 256 else d)
    s["q_weight"], s["k_weight"] = _weight(gen, d), _weight(gen, d)
    # read back: the new tokens and the older ones of the block that the first of them went to
    back = [new + (n - new) % BLOCK for n in lens]
    s["cu_read"] = _ints([sum(back[:i]) for i in range(b + 1)])
    s["read"] = sum(back)
    return s


# ------------------------------------------------------------------ plain forms
def _value(codes, form):
    return codes.float() - 128 if form == "int8" else codes.view(torch.float8_e4m3fn).float()


def _code(x, form):
    if form == "int8":
        return (x.round().clamp(-127, 127) + 128).to(torch.uint8)
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _unpack_k(page, d):
    """[..., 64 * d] in held order -> [..., 64, d]"""
    x = page.unflatten(-1, (4, d // 64, 4, 16, 16))  # i c g t j: token 16i + t, dim 64c + 16g + j
    n = x.dim() - 5
    return x.permute(*range(n), n, n + 3, n + 1, n + 2, n + 4).flatten(n + 2).flatten(n, n + 1)


def _unpack_v(page, d):
    """[..., 64 * d] in held order -> [..., 64, d]"""
    x = page.unflatten(-1, (d // 16, 4, 16, 4, 4))  # n g d i j: token 16i + 4g + j, dim 16n + d
    n = x.dim() - 5
    return x.permute(*range(n), n + 3, n + 1, n + 4, n, n + 2).flatten(n + 3).flatten(n, n + 2)


def _k_at(token, dim, d):
    """Place of (token, dim) in a page."""
    return (((token // 16 * (d // 64) + dim // 64) * 4 + dim % 64 // 16) * 16 + token % 16) * 16 + dim % 16


def _v_at(token, dim, d):
    return (((dim // 16 * 4 + token % 16 // 4) * 16 + dim % 16) * 4 + token // 16) * 4 + token % 4


def _plain_norm(x, weight):
    x = x.float()
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight


def _plain_rope(x, pos, inv_freq, axis, adjacent):
    rot = 2 * inv_freq.numel()
    angle = (pos.double()[axis.long()].t() * inv_freq.double())  # [tokens][rot / 2], in 64 bits: far positions
    c, s = angle.cos().float()[:, None], angle.sin().float()[:, None]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if adjacent else (x[..., :rot // 2], x[..., rot // 2:rot])
    y1, y2 = a * c - b * s, b * c + a * s
    y = torch.stack((y1, y2), -1).flatten(-2) if adjacent else torch.cat((y1, y2), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _tokens(cu, lens, total):
    """(sequence, position in its cache) of each of the `total` last tokens."""
    at = torch.arange(total, device=cu.device)
    b = torch.searchsorted(cu[1:].long(), at, right=True)
    return b, lens[b].long() - cu[b + 1] + at


def _plain_read(s, layer, cu, total):
    d, form = s["case"]["dim"], s["format"]
    b, n = _tokens(cu, s["lens"], total)
    page, inside = s["table"][b, n // PAGE].long(), n % PAGE
    dims = torch.arange(d, device="cuda")
    out = []
    for x, place in (("k", _k_at), ("v", _v_at)):
        codes = s[x][layer][page].gather(-1, place(inside[:, None], dims, d)[:, None].expand(-1, s[x].shape[2], -1))
        scale = s[x + "_scales"][layer][page].gather(-1, (inside // BLOCK)[:, None, None].expand(-1, s[x].shape[2], 1))
        out.append((_value(codes, form) * scale).half())
    return out


def _plain_append(s):
    case, form = s["case"], s["format"]
    d, kh, top = case["dim"], case["kv_heads"], QMAX[form]
    q = _plain_rope(_plain_norm(s["q"], s["q_weight"]), s["pos"], s["inv_freq"], s["axis"], False).half()
    k = _plain_rope(_plain_norm(s["k_new"], s["k_weight"]), s["pos"], s["inv_freq"], s["axis"], False)
    total = k.shape[0]
    b, n = _tokens(s["cu"], s["lens"], total)
    page, inside = s["table"][b, n // PAGE].long(), n % PAGE
    block = page * (PAGE // BLOCK) + inside // BLOCK  # of each new token
    first = (s["lens"] - (s["cu"][1:] - s["cu"][:-1])).long()
    seqs = torch.arange(first.numel(), device="cuda")
    # older tokens of the blocks that the first new tokens go to, and what is left of the last ones
    lane = torch.arange(BLOCK, device="cuda")
    old_n = first[:, None] // BLOCK * BLOCK + lane
    old = old_n < first[:, None]
    old_b, old_n = seqs[:, None].expand_as(old)[old], old_n[old]
    end_n = (s["lens"].long()[:, None] - 1) // BLOCK * BLOCK + lane
    end = end_n >= s["lens"][:, None]
    end_b, end_n = seqs[:, None].expand_as(end)[end], end_n[end]
    old_page, end_page = (s["table"][x, y // PAGE].long() for x, y in ((old_b, old_n), (end_b, end_n)))
    old_block = old_page * (PAGE // BLOCK) + old_n % PAGE // BLOCK
    dims = torch.arange(d, device="cuda")
    heads = torch.arange(kh, device="cuda")[None, :, None]
    for x, new, place in (("k", k, _k_at), ("v", s["v_new"].float(), _v_at)):
        codes, scales = s[x][0], s[x + "_scales"][0].transpose(1, 2).reshape(-1, kh)  # scales: [block][head]
        held = torch.zeros_like(scales)
        held[old_block] = scales[old_block]
        most = torch.zeros_like(scales).scatter_reduce_(0, block[:, None].expand(-1, kh), new.abs().amax(-1), "amax")
        now = torch.maximum(most / top, held)
        where = (old_page[:, None, None], heads, place((old_n % PAGE)[:, None], dims, d)[:, None])
        ratio = (scales[old_block] / now[old_block]).nan_to_num(0.0)
        codes[where] = _code(_value(codes[where], form) * ratio[..., None], form)
        inv = torch.where(now > 0, 1 / now, torch.zeros_like(now))
        codes[page[:, None, None], heads, place(inside[:, None], dims, d)[:, None]] = _code(new * inv[block][..., None], form)
        codes[end_page[:, None, None], heads, place((end_n % PAGE)[:, None], dims, d)[:, None]] = 128 if form == "int8" else 0
        touched = torch.cat((block, old_block))
        scales[touched] = now[touched]
        s[x + "_scales"][0] = scales.view(-1, PAGE // BLOCK, kh).transpose(1, 2)
    return q


def _plain_plan(s):
    """(masks int64 [total][words], positions [total], depths and which rows each sees) of the trees that `parent` gives."""
    case = s["case"]
    b, new = case["batch"], case["new"]
    words = -(-new // 64)
    parent = s["parent"].view(b, new).long()
    rows = torch.arange(new, device="cuda")
    up = (parent[..., None] == rows) | torch.eye(new, dtype=torch.bool, device="cuda")  # a row and its parent
    up = up.float()
    for _ in range(max(1, math.ceil(math.log2(new)))):  # twice as many generations each time
        up = (up @ up > 0).float()
    depth = up.sum(-1)
    w = case.get("window", 0)
    if w:
        up = up * ((depth[:, :, None] - depth[:, None, :]) < w)  # of a row's own, the last w
    bit = torch.ones((), dtype=torch.int64, device="cuda") << (rows % 64)
    mask = torch.stack([(up.long() * bit * (rows // 64 == i)).sum(-1) for i in range(words)], -1)
    pos = (s["lens"][:, None] - new + depth - 1).int()
    return mask.view(b * new, words), pos.flatten(), depth.view(b, new), up.view(b, new, new)


def _plain_attn(s):
    case, form = s["case"], s["format"]
    h, kh, d, new, b = case["heads"], case["kv_heads"], case["dim"], case["new"], case["batch"]
    w, sinks = case["window"], case["sinks"]
    width = s["table"].shape[1]
    lens = s["lens"].long()[:, None]
    if w and w + new + PAGE * 2 < s["max_len"]:
        # the pages that some row may see: those of the sinks, and those from the first row's window on
        front = torch.arange(-(-sinks // PAGE), device="cuda")
        back = (lens - new - w).clamp(min=0) // PAGE + torch.arange((w + new) // PAGE + 2, device="cuda")
        back = torch.where(back < front.numel(), width, back)  # (not twice)
        col = torch.cat((front.expand(b, -1), back), 1)
    else:
        col = torch.arange(width, device="cuda").expand(b, -1)
    page = s["table"].gather(1, col.clamp(max=width - 1)).clamp(min=0).long()
    at = (col[..., None] * PAGE + torch.arange(PAGE, device="cuda")).flatten(1)  # [b][n] positions
    n = at.shape[1]

    def held(x, unpack):  # [b][kh][n][d]
        codes = _value(unpack(s[x][0][page], d), form)  # [b][pages][kh][64][d]
        codes = codes.unflatten(3, (PAGE // BLOCK, BLOCK)) * s[x + "_scales"][0][page][..., None, None]
        return codes.flatten(3, 4).transpose(1, 2).reshape(b, kh, n, d)

    base = lens - new
    i = torch.arange(new, device="cuda")
    if case["words"]:
        mask = s["mask"].view(b, new, -1)
        off = (at - base).clamp(0, 64 * case["words"] - 1)[:, None].expand(b, new, n)
        tree = (mask.gather(2, off // 64) >> (off % 64)) & 1
        at3 = at[:, None]
        inside = (at3 >= base[..., None]) & (at3 < lens[..., None])
        low = torch.zeros_like(base)[..., None]
        if w:
            bits = (mask[..., None] >> torch.arange(64, device="cuda")) & 1
            low = base[..., None] - (w - bits.sum((-1, -2))[..., None]).clamp(min=0)
        seen = (inside & (tree > 0)) | ((at3 < base[..., None]) & ((at3 >= low) | (at3 < sinks)))
    else:
        pos = (base + i)[..., None]
        at3 = at[:, None]
        seen = at3 <= pos
        if w:
            seen = seen & ((at3 > pos - w) | (at3 < sinks))
    q = s["q"].float().view(b, new, kh, h // kh, d).permute(0, 2, 3, 1, 4).reshape(b, kh, h // kh * new, d)
    x = (q @ held("k", _unpack_k).transpose(2, 3)).view(b, kh, h // kh, new, n) * d ** -0.5
    x = x.masked_fill(~seen[:, None, None], -torch.inf)
    x = (x - x.amax(-1, keepdim=True).clamp(min=-1e30)).exp()
    total = x.sum(-1, keepdim=True)
    v = torch.where((at < lens)[:, None, :, None], held("v", _unpack_v), 0)
    o = x.view(b, kh, h // kh * new, n) @ v
    o = o.view(b, kh, h // kh, new, d) / total.clamp(min=1e-30)
    return o.permute(0, 3, 1, 2, 4).reshape(b * new, h, d).half()


def _order(x):
    """Whole numbers in the order of the values x; -0 as 0."""
    bits = (x.float() + 0.0).view(torch.int32).long()
    return torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)


def _plain_logprobs(s):
    case, x = s["case"], s["logits"].float()
    m = x.amax(-1, keepdim=True)
    y = x - m
    e = y.exp()
    total = e.sum(-1, keepdim=True)
    log = total.log()
    out = {}
    if case["count"]:
        out["logprob"] = y.gather(1, s["tokens"].long()) - log
    if case["entropy"]:
        out["entropy"] = (log - torch.where(e > 0, e * y, 0).sum(-1, keepdim=True) / total)[:, 0]
    if case["top"]:
        del e
        v = x.shape[1]
        key = (_order(x) << 18) + (v - 1 - torch.arange(v, device="cuda"))  # a larger value first, then a lower token
        token = v - 1 - (key.topk(case["top"], -1).values & ((1 << 18) - 1))
        out |= {"top_tokens": token.int(), "top_logprobs": y.gather(1, token) - log}
    return out


def _plain_accept(s):
    """The rows that the target tokens take, from row 0 on: path [batch][max_path] (-1 behind it), their number, the
    token after them, the length that is left of the sequence."""
    case, most = s["case"], s["max_path"]
    b, new = case["batch"], case["new"]
    mask, pos, depth, up = _plain_plan(s)
    parent, token, target = (s[x].view(b, new).long() for x in ("parent", "token", "target"))
    rows = torch.arange(new, device="cuda")
    fits = target.gather(1, parent.clamp(min=0)) == token
    # of siblings with the same token only the first is one
    twin = (parent[:, :, None] == parent[:, None]) & (token[:, :, None] == token[:, None]) & (rows[None, :] < rows[:, None])
    fits = fits & ~twin.any(-1)
    fits[:, 0] = True
    taken = ((up > 0) <= fits[:, None]).all(-1) & (depth <= most)
    kept = taken.sum(-1).int()
    order = torch.where(taken, rows, new).sort(-1).values
    order = torch.nn.functional.pad(order, (0, max(0, most - new)), value=new)[:, :most]
    path = torch.where(order < new, order, -1).int()
    last = path.gather(1, (kept.long() - 1)[:, None])
    return mask, pos, path, kept, target.gather(1, last.long())[:, 0].int(), s["lens"] - new + kept


def _plain_keep(s, path, kept):
    case, form = s["case"], s["format"]
    d, kh, b, new = case["dim"], case["kv_heads"], case["batch"], case["new"]
    base = (s["lens"] - new).long()[:, None]
    i = torch.arange(path.shape[1], device="cuda")
    live = (i < kept[:, None]) & (path != i)
    seq = torch.arange(b, device="cuda")[:, None].expand_as(live)[live]
    src, dst = (base + path)[live], (base + i)[live]
    sp, dp = s["table"][seq, src // PAGE].long(), s["table"][seq, dst // PAGE].long()
    sb, db = sp * (PAGE // BLOCK) + src % PAGE // BLOCK, dp * (PAGE // BLOCK) + dst % PAGE // BLOCK
    dims, lane = torch.arange(d, device="cuda"), torch.arange(BLOCK, device="cuda")
    block = db.unique()  # what a block holds beside comes to its new scale
    layers, heads = torch.arange(s["k"].shape[0], device="cuda")[:, None, None, None], torch.arange(kh, device="cuda")[None, None, :, None]
    for x, place in (("k", _k_at), ("v", _v_at)):
        codes, scales = s[x], s[x + "_scales"].transpose(2, 3).flatten(1, 2)  # scales: [layer][block][head]
        now = scales.scatter_reduce(1, db[None, :, None].expand(scales.shape[0], -1, kh), scales[:, sb], "amax")
        moved = codes[layers, sp[None, :, None, None], heads, place((src % PAGE)[:, None], dims, d)[None, :, None]]
        moved = _code(_value(moved, form) * (scales[:, sb] / now[:, db]).nan_to_num(0.0)[..., None], form)
        t = (block[:, None] % (PAGE // BLOCK) * BLOCK + lane).flatten()
        at = (layers, (block // (PAGE // BLOCK)).repeat_interleave(BLOCK)[None, :, None, None], heads, place(t[:, None], dims, d)[None, :, None])
        ratio = (scales[:, block] / now[:, block]).nan_to_num(0.0).repeat_interleave(BLOCK, 1)
        codes[at] = _code(_value(codes[at], form) * ratio[..., None], form)
        codes[layers, dp[None, :, None, None], heads, place((dst % PAGE)[:, None], dims, d)[None, :, None]] = moved
        s[x + "_scales"].copy_(now.unflatten(1, (-1, PAGE // BLOCK)).transpose(2, 3))


# ------------------------------------------------------------------ one pass
def run(s):
    op, case = s["op"], s["case"]
    if own:
        import bit_quantized_decode_qmv_amd as bq
        if op == "rows":
            return bq.norm_rope(s["x"], s["weight"], EPS, s["pos"], s["inv_freq"], axis=s["axis"], adjacent=case["adjacent"])
        if op == "logprobs":
            got = bq.logprobs(s["logits"], s["tokens"], top=case["top"], entropy=case["entropy"], workspace=s["workspace"])
            return {k: x for k, x in zip(("logprob", "entropy", "top_tokens", "top_logprobs"), got) if x is not None}
        cache = bq.KVCache(s["k"], s["v"], s["k_scales"], s["v_scales"], s["format"])
        if op == "attn" and case["words"]:
            return bq.kv_attn_tree(cache, 0, s["q"], s["cu"], s["lens"], s["table"], s["mask"], window=case["window"],
                                   sinks=case["sinks"], workspace=s["workspace"])
        if op == "attn":
            return bq.kv_attn(cache, 0, s["q"], s["cu"], s["lens"], s["table"], window=case["window"], sinks=case["sinks"],
                              workspace=s["workspace"])
        if op == "norm":
            q = bq.kv_append_norm(cache, 0, s["k_new"], s["v_new"], s["cu"], s["lens"], s["table"], q=s["q"], q_weight=s["q_weight"],
                                  k_weight=s["k_weight"], eps=EPS, pos=s["pos"], inv_freq=s["inv_freq"], axis=s["axis"])
            k, v = bq.kv_read(cache, 0, s["cu_read"], s["lens"], s["table"], s["read"])
            return {"q": q, "k": k, "v": v}
        mask, pos = bq.tree_plan(s["parent"], s["cu"], s["lens"], words=-(-case["new"] // 64))
        path, kept, token, want = bq.tree_accept(s["target"], s["token"], s["parent"], s["cu"], s["lens"], s["max_path"])
        bq.kv_keep(cache, s["cu"], s["lens"], s["table"], path, kept)
        read = [bq.kv_read(cache, i, s["cu"], s["lens"], s["table"], s["total"]) for i in range(cache.layers)]
    else:
        if op == "rows":
            return _plain_rope(_plain_norm(s["x"], s["weight"]), s["pos"], s["inv_freq"], s["axis"], case["adjacent"]).half()
        if op == "logprobs":
            return _plain_logprobs(s)
        if op == "attn":
            return _plain_attn(s)
        if op == "norm":
            q = _plain_append(s)
            k, v = _plain_read(s, 0, s["cu_read"], s["read"])
            return {"q": q, "k": k, "v": v}
        mask, pos, path, kept, token, want = _plain_accept(s)
        _plain_keep(s, path, kept)
        read = [_plain_read(s, i, s["cu"], s["total"]) for i in range(s["k"].shape[0])]
    return {"mask": mask, "pos": pos, "path": path, "kept": kept, "next": token, "want": want, "k": [x[0] for x in read], "v": [x[1] for x in read]}


# ------------------------------------------------------------------ 64 bits
def _exact_norm_rope(x, weight, s, adjacent):
    """The norm from its definition, the rotation as a product of complex numbers."""
    x = x.double()
    x = x / ((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * weight.double()
    inv = s["inv_freq"].double()
    r = inv.numel()
    if r == 0:
        return x
    angle = torch.stack([s["pos"][int(a)].double() * f for a, f in zip(s["axis"].tolist(), inv)], 1)[:, None]
    turn = torch.polar(torch.ones_like(angle), angle)
    y = x.clone()
    if adjacent:
        z = torch.complex(x[..., 0:2 * r:2], x[..., 1:2 * r:2]) * turn
        y[..., 0:2 * r:2], y[..., 1:2 * r:2] = z.real, z.imag
    else:
        z = torch.complex(x[..., :r], x[..., r:2 * r]) * turn
        y[..., :r], y[..., r:2 * r] = z.real, z.imag
    return y


def _sequence(s, x, b, n, layer=0):
    """(values [kv_heads][n][dim] of the first n tokens of sequence b in 64 bits, byte by byte from their places in a page;
    scales [kv_heads][n])."""
    d = s["case"]["dim"]
    page = s["table"][b, :-(-n // PAGE)].long()
    t, c = torch.arange(PAGE, device="cuda")[:, None], torch.arange(d, device="cuda")[None]
    if x == "k":
        place = t // 16 * 16 * d + c // 64 * 1024 + c % 64 // 16 * 256 + t % 16 * 16 + c % 16
    else:
        place = c // 16 * 1024 + t % 16 // 4 * 256 + c % 16 * 16 + t // 16 * 4 + t % 4
    raw = s[x][layer][page][:, :, place.flatten()].view(page.numel(), -1, PAGE, d)
    value = raw.double() - 128 if s["format"] == "int8" else raw.view(torch.float8_e4m3fn).double()
    scale = s[x + "_scales"][layer][page].double().repeat_interleave(BLOCK, -1)
    return (value * scale[..., None]).transpose(0, 1).flatten(1, 2)[:, :n], scale.transpose(0, 1).flatten(1)[:, :n]


def _nearest(code, form):
    """The code nearest to it: whole, or one of e4m3's by its exponent."""
    unit = torch.ones_like(code) if form == "int8" else torch.exp2(code.abs().clamp(min=2.0 ** -6).log2().floor() - 3)
    return (code / unit).round() * unit


def _exact_append(s, case):
    lens, new, d = _lens(case), case["new"], case["dim"]
    q, k, v = _exact_norm_rope(s["q"], s["q_weight"], s, False), _exact_norm_rope(s["k_new"], s["k_weight"], s, False), s["v_new"].double()
    got = {"q": q, "k": [], "v": []}
    top = QMAX[s["format"]]
    for b, n in enumerate(lens):
        for x, made in (("k", k), ("v", v)):
            first = n - new
            at = first // BLOCK * BLOCK
            old, held = _sequence(s, x, b, first) if first else (made.new_zeros(case["kv_heads"], 0, d), None)
            both = torch.cat((old[:, at:], made[b * new:(b + 1) * new].transpose(0, 1)), 1)
            for j in range(0, both.shape[1], BLOCK):
                part = both[:, j:j + BLOCK]
                since = first - at if j == 0 else 0
                scale = part[:, since:].abs().amax((1, 2)) / top
                if since:
                    scale = torch.maximum(scale, held[:, at])
                scale = scale[:, None, None]
                both[:, j:j + BLOCK] = _nearest(part / scale.clamp(min=1e-300), s["format"]) * scale
            got[x].append(both.transpose(0, 1))
    return {"q": q, "k": torch.cat(got["k"]), "v": torch.cat(got["v"])}


def _exact_accept(s, case):
    """The tokens at the tree's places after the path has moved, a token at a time."""
    parents, paths = _trees(case)
    lens, new = _lens(case), case["new"]
    out = {"mask": None, "pos": None, "path": None, "kept": None, "next": None, "want": None, "k": [], "v": []}
    for layer in range(case["layers"]):
        for x in ("k", "v"):
            rows = []
            for b, n in enumerate(lens):
                value, scale = _sequence(s, x, b, n, layer)
                top = scale.clone()  # of the block that a token lies in
                first, path = n - new, paths[b]
                moves = [(first + p, first + i) for i, p in enumerate(path) if p != i]
                for f, t in moves:
                    lo = t // BLOCK * BLOCK
                    most = torch.maximum(top[:, lo:lo + 1], scale[:, f:f + 1])
                    top[:, lo:lo + BLOCK] = most
                for f, t in moves:
                    value[:, t] = value[:, f]
                rows.append((_nearest(value / top[..., None], s["format"]) * top[..., None])[:, first:].transpose(0, 1))
            out[x].append(torch.cat(rows))
    return out


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op == "rows":
        return _exact_norm_rope(s["x"], s["weight"], s, case["adjacent"])
    if op == "norm":
        return _exact_append(s, case)
    if op == "accept":
        return _exact_accept(s, case)
    if op == "logprobs":
        out = {k: [] for k, on in (("logprob", case["count"]), ("entropy", case["entropy"]), ("top_logprobs", case["top"])) if on}
        if case["top"]:
            out["top_tokens"] = None
        for at in range(0, case["rows"], 256):
            x = s["logits"][at:at + 256].double()
            lse = x.logsumexp(-1, keepdim=True)
            if case["count"]:
                out["logprob"].append(x.gather(1, s["tokens"][at:at + 256].long()) - lse)
            if case["entropy"]:
                p = (x - lse).exp()
                out["entropy"].append(-torch.special.xlogy(p, p).sum(-1))
            if case["top"]:
                out["top_logprobs"].append(x.topk(case["top"], -1).values - lse)
        return {k: torch.cat(v) if isinstance(v, list) else v for k, v in out.items()}
    lens, new, d = _lens(case), case["new"], case["dim"]
    out = torch.zeros(case["batch"] * new, case["heads"], d, dtype=torch.float64, device="cuda")
    group = case["heads"] // case["kv_heads"]
    parents = _trees(case)[0] if case["words"] else []
    for b, n in enumerate(lens):
        k, v = _sequence(s, "k", b, n)[0], _sequence(s, "v", b, n)[0]
        j, first = torch.arange(n, device="cuda"), n - new
        if case["words"]:
            sees = []  # rows of the tree that a row sees, itself among them
            for i, p in enumerate(parents[b]):
                sees.append((sees[p] if p >= 0 else []) + [i])
            w = case["window"] or n + new
            hide = torch.ones(new, n, dtype=torch.bool, device="cuda")
            for i, rows in enumerate(sees):
                rows = rows[-w:]
                hide[i, max(first - (w - len(rows)), 0):first] = False
                hide[i, :min(case["sinks"], first)] = False
                hide[i, torch.tensor(rows, device="cuda") + first] = False
        else:
            dist = (first + torch.arange(new, device="cuda"))[:, None] - j
            hide = dist < 0
            if case["window"]:
                hide = hide | ((dist >= case["window"]) & (j >= case["sinks"]))
        for h in range(case["heads"]):
            x = s["q"][b * new:(b + 1) * new, h].double() @ k[h // group].T / math.sqrt(d)
            out[b * new:(b + 1) * new, h] = torch.softmax(x.masked_fill(hide, -math.inf), -1) @ v[h // group]
    return out
