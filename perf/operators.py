"""What is measured of the paged key/value cache in 8 bits and of the operators around it: rotary positions with
several axes, writing new tokens into the cache, attention over the cache, and the pages' fork, resize and compaction.

The cache: pages of 64 tokens, one scale for each block of 16 tokens and head.  A page's codes are held in the order
in which the matrix instructions of the attention take them (`unpack_k`, `unpack_v`); a value is scale * code, the code
an int8 held as byte code + 128, or an e4m3 number.
"""
import math
import random

import torch

own = False

PAGE, BLOCK = 64, 16
QMAX = {"int8": 127.0, "e4m3": 448.0}


# ------------------------------------------------------------------ cases
def listed():
    wide = {"heads": 48, "kv_heads": 8, "dim": 128}  # q 6144, k/v 1024 columns: the repository's projection shapes
    return [
        # the five rows of a draft verification, one axis: a latency-bound call
        {"name": "rope_draft", "op": "rope", "tokens": 5, "heads": 48, "dim": 128, "rot": 128, "axes": 1, "adjacent": False},
        # a prompt of images or video: time, height and width positions
        {"name": "rope_image", "op": "rope", "tokens": 8191, "heads": 48, "dim": 128, "rot": 128, "axes": 3, "adjacent": False},
        # one decode step of 32 sequences: each adds one token to a block that is partly filled
        {"name": "append_step", "op": "append", **wide, "batch": 32, "new": 1, "ctx": 4001, "axes": 1, "format": "int8"},
        # a prompt's chunk behind an odd number of held tokens
        {"name": "append_prompt", "op": "append", **wide, "batch": 1, "new": 4093, "ctx": 5120, "axes": 3, "format": "int8"},
        # several short prompts with half of the dimensions rotated, wide heads, codes in e4m3
        {"name": "append_batch", "op": "append", "heads": 24, "kv_heads": 4, "dim": 256, "batch": 8, "new": 301, "ctx": 777, "axes": 3, "format": "e4m3"},
        # one token of one sequence, short context: the smallest step
        {"name": "attn_token", "op": "attn", **wide, "batch": 1, "new": 1, "ctx": 1003, "causal": True, "window": 0, "format": "int8"},
        # one token of one sequence over a long context: the cache's bytes
        {"name": "attn_token_long", "op": "attn", **wide, "batch": 1, "new": 1, "ctx": 131001, "causal": True, "window": 0, "format": "int8"},
        # the five rows of a draft for 32 sequences of very different lengths
        {"name": "attn_draft", "op": "attn", **wide, "batch": 32, "new": 5, "ctx": 16384, "causal": True, "window": 0, "format": "e4m3"},
        # a prompt's chunk over what the cache already holds: bound by the matrix cores
        {"name": "attn_prompt", "op": "attn", **wide, "batch": 1, "new": 2047, "ctx": 10240, "causal": True, "window": 0, "format": "int8"},
        # queries of a decoder over an encoder's states: no causal mask, no shared heads
        {"name": "attn_encoder", "op": "attn", "heads": 16, "kv_heads": 16, "dim": 64, "batch": 6, "new": 77, "ctx": 1500, "causal": False, "window": 0, "format": "int8"},
        # a prompt's sequence forked into eight samples; others are cut, grown and freed
        {"name": "pages_fork", "op": "fork", "kv_heads": 8, "dim": 128, "layers": 16, "pages": 600, "ctx": 5000, "forks": 8},
        # a pool with holes is compacted before its upper part is given back
        {"name": "pages_compact", "op": "compact", "kv_heads": 8, "dim": 128, "layers": 16, "pages": 600, "ctx": 4700, "forks": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attn", "attn", "fork", "compact"])
    dim = rng.choice([64, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 6, 8])
    if op == "rope":
        return {"op": op, "tokens": _log(rng, 1, 8000), "heads": kv_heads * group, "dim": dim,
                "rot": rng.choice([dim, dim // 2]), "axes": rng.choice([1, 2, 3]), "adjacent": rng.random() < 0.3}
    if op in ("fork", "compact"):
        return {"op": op, "kv_heads": kv_heads, "dim": min(dim, 128), "layers": rng.choice([1, 2, 4, 8, 16]),
                "pages": rng.randint(300, 600), "ctx": _log(rng, 700, 4600), "forks": rng.randint(1, 8) if op == "fork" else 0}
    form = rng.choice(["int8", "e4m3"])
    if op == "append":
        new = _log(rng, 1, 4000)
        batch = max(1, min(64, _log(rng, 1, 64), 4000 // new))
        return {"op": op, "heads": kv_heads * group, "kv_heads": kv_heads, "dim": dim, "batch": batch, "new": new,
                "ctx": new + _log(rng, 1, 4000), "axes": rng.choice([1, 3]), "format": form}
    causal = rng.random() < 0.8
    new = rng.choice([1, 1, 2, 3, 4, 5, 5, _log(rng, 6, 2000)])
    if new > 5:
        batch, ctx = rng.randint(1, max(1, min(8, 2000 // new))), new + _log(rng, 1, 8000)
    else:
        batch = _log(rng, 1, 64)
        ctx = _log(rng, 16, 262144 // batch)
    return {"op": op, "heads": kv_heads * group, "kv_heads": kv_heads, "dim": dim, "batch": batch, "new": new,
            "ctx": max(ctx, new), "causal": causal, "window": _log(rng, 16, 4096) if causal and rng.random() < 0.25 else 0,
            "format": form}


def _lens(case):
    """Tokens held for each sequence: from ctx down to ctx / 16, spread over the logarithm."""
    b = case["batch"]
    return [max(case["new"], int(case["ctx"] * 16.0 ** (-i / max(1, b - 1)))) for i in range(b)]


def work(case):
    op = case["op"]
    if op == "rope":
        n = case["tokens"] * case["heads"]
        return {"bytes": 4 * n * case["dim"] + 4 * case["tokens"] * case["axes"], "flops": 3 * n * case["rot"]}
    if op in ("fork", "compact"):
        page = case["layers"] * case["kv_heads"] * (2 * PAGE * case["dim"] + 32)
        seqs, held = _pool_of(case)
        if op == "fork":
            _, _, copies = _fork_plan(case, seqs)
            ints = 4 * (case["pages"] * 2 + sum(seqs) // PAGE)
        else:
            live = set(p for row in held for p in row)
            copies = sum(p >= len(live) for p in live)
            ints = 4 * (case["pages"] * 2 + 2 * len(live))
        return {"bytes": 2 * copies * page + ints, "flops": 0}
    h, kh, d, new, b = case["heads"], case["kv_heads"], case["dim"], case["new"], case["batch"]
    if op == "append":
        # q read and written, k and v read, codes written; then the codes read back and given as fp16
        t = b * new
        return {"bytes": 4 * t * h * d + 4 * t * kh * d + 2 * t * kh * d + 6 * t * kh * d, "flops": t * (h + 3 * kh) * d * 3}
    pairs = held = 0
    for n in _lens(case):
        first = n - new  # position of the first query
        if not case["causal"]:
            pairs, held = pairs + new * n, held + n
        else:
            w = case["window"] or n
            pairs += sum(min(p + 1, w) for p in range(first, n)) if w < n else new * first + new * (new + 1) // 2
            held += min(n, w + new - 1)
    return {"bytes": held * kh * (2 * d + 8 / BLOCK) + 4 * b * new * h * d, "flops": 4 * pairs * h * d}


# ------------------------------------------------------------------ inputs
def _rows(case):
    """The sequences' lengths of a pool and which pages hold them."""
    r = random.Random(7)
    n, left, lens = 0, case["pages"] * (PAGE - 8) // 2, []
    while left > 0 and n < 24:
        lens.append(min(case["ctx"] - 37 * n if n == 0 else r.randint(1, case["ctx"]), left))
        left -= lens[-1] + PAGE
        n += 1
    return lens, r


def _pool_of(case):
    lens, r = _rows(case)
    free = list(range(case["pages"]))
    r.shuffle(free)
    held = [[free.pop() for _ in range(-(-n // PAGE))] for n in lens]
    return lens, held


def _fork_plan(case, lens):
    """(source of each fork, wanted lengths after it, pages that fork and resize copy): fork i goes to row len(lens) + i.
    The first samples are cut inside a shared page, as after a rejected draft, one sequence of its own is freed, one grows."""
    n, f = len(lens), case["forks"]
    src = [0] * f
    want = [-1] * (n + f)
    copies = f if lens[0] % PAGE else 0
    for i in range(0, f, 3):
        cut = max(1, lens[0] - PAGE - 2 * i - 1)
        want[n + i] = cut
        if cut < lens[0] // PAGE * PAGE and cut % PAGE:
            copies += 1
    if n > 1:
        want[1] = 0
    if n > 2:
        want[2] = lens[2] + 100
    return src, want, copies


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


def _pool(gen, layers, pages, case, form):
    kh, d = case["kv_heads"], case["dim"]
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
    inv = (1e6 ** (-2 * r / rot)).to(torch.float32)
    return inv, (torch.arange(rot // 2, device="cuda") % axes).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    s = {"op": op, "case": dict(case)}
    if op == "rope":
        s["x"] = torch.randn(case["tokens"], case["heads"], case["dim"], generator=gen, device="cuda").half()
        s["pos"] = _positions(gen, case["axes"], case["tokens"])
        s["inv_freq"], s["axis"] = _angles(case["axes"], case["rot"])
        return s
    if op in ("fork", "compact"):
        lens, held = _pool_of(case)
        rows, width = len(lens) + case["forks"], max(-(-case["ctx"] // PAGE), max(map(len, held))) + 3
        s |= _pool(gen, case["layers"], case["pages"], case, "int8")
        table = [row + [-1] * (width - len(row)) for row in held] + [[-1] * width] * (rows - len(held))
        refs = [0] * case["pages"]
        for row in held:
            for p in row:
                refs[p] += 1
        s |= {"table": _ints(table), "lens": _ints(lens + [0] * (rows - len(lens))), "refs": _ints(refs)}
        src, want, _ = _fork_plan(case, lens)
        s |= {"src": _ints(src), "dst": _ints([len(lens) + i for i in range(case["forks"])]), "want": _ints(want)}
        return s
    lens, new, b = _lens(case), case["new"], case["batch"]
    need = [-(-n // PAGE) for n in lens]
    pages, width = sum(need) + 3, max(need) + 1
    order = torch.randperm(pages, generator=gen, device="cuda").tolist()
    table, at = [], 0
    for n in need:
        table.append(order[at:at + n] + [-1] * (width - n))
        at += n
    s |= _pool(gen, 1, pages, case, case["format"])
    s |= {"table": _ints(table), "lens": _ints(lens), "cu": _ints([new * i for i in range(b + 1)]), "max_len": max(lens)}
    h, kh, d = case["heads"], case["kv_heads"], case["dim"]
    if op == "attn":
        s["q"] = 2 * torch.randn(b * new, h, d, generator=gen, device="cuda")
        s["q"] = s["q"].half()
        s["workspace"] = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
        return s
    # the rows of a fused q, k, v product
    qkv = torch.randn(b * new, (h + 2 * kh) * d, generator=gen, device="cuda").half()
    for name, lo, n in (("q", 0, h), ("k_new", h, kh), ("v_new", h + kh, kh)):
        s[name] = qkv[:, lo * d:(lo + n) * d].unflatten(1, (n, d))
    s["pos"] = _positions(gen, case["axes"], b * new)
    s["inv_freq"], s["axis"] = _angles(case["axes"], d // 2 if d == 256 else d)
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


def unpack_k(page, d):
    """[..., 64 * d] in held order -> [..., 64, d]"""
    x = page.unflatten(-1, (4, d // 64, 4, 16, 16))  # i c g t j: token 16i + t, dim 64c + 16g + j
    n = x.dim() - 5
    return x.permute(*range(n), n, n + 3, n + 1, n + 2, n + 4).flatten(n + 2).flatten(n, n + 1)


def unpack_v(page, d):
    """[..., 64 * d] in held order -> [..., 64, d]"""
    x = page.unflatten(-1, (d // 16, 4, 16, 4, 4))  # n g d i j: token 16i + 4g + j, dim 16n + d
    n = x.dim() - 5
    return x.permute(*range(n), n + 3, n + 1, n + 4, n, n + 2).flatten(n + 3).flatten(n, n + 2)


def _k_at(token, dim, d):
    """Place of (token, dim) in a page."""
    return (((token // 16 * (d // 64) + dim // 64) * 4 + dim % 64 // 16) * 16 + token % 16) * 16 + dim % 16


def _v_at(token, dim, d):
    return (((dim // 16 * 4 + token % 16 // 4) * 16 + dim % 16) * 4 + token // 16) * 4 + token % 4


def _plain_rope(x, pos, inv_freq, axis, adjacent):
    rot = 2 * inv_freq.numel()
    angle = pos.float()[axis.long()].t() * inv_freq  # [tokens][rot / 2]
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    x = x.float()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if adjacent else (x[..., :rot // 2], x[..., rot // 2:rot])
    y1, y2 = a * c - b * s, b * c + a * s
    y = torch.stack((y1, y2), -1).flatten(-2) if adjacent else torch.cat((y1, y2), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _tokens(cu, lens, total):
    """(sequence, position in its cache) of each of the `total` last tokens."""
    at = torch.arange(total, device=cu.device)
    b = torch.searchsorted(cu[1:].long(), at, right=True)
    return b, lens[b].long() - cu[b + 1] + at


def _plain_read(s, cu, total):
    d, form = s["case"]["dim"], s["format"]
    b, n = _tokens(cu, s["lens"], total)
    page, inside = s["table"][b, n // PAGE].long(), n % PAGE
    dims = torch.arange(d, device="cuda")
    out = []
    for x, place in (("k", _k_at), ("v", _v_at)):
        codes = s[x][0][page].gather(-1, place(inside[:, None], dims, d)[:, None].expand(-1, s[x].shape[2], -1))
        scale = s[x + "_scales"][0][page].gather(-1, (inside // BLOCK)[:, None, None].expand(-1, s[x].shape[2], 1))
        out.append((_value(codes, form) * scale).half())
    return out


def _plain_append(s):
    case, form = s["case"], s["format"]
    d, kh, top = case["dim"], case["kv_heads"], QMAX[form]
    q = _plain_rope(s["q"], s["pos"], s["inv_freq"], s["axis"], False).half()
    k = _plain_rope(s["k_new"], s["pos"], s["inv_freq"], s["axis"], False)
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


def _plain_attn(s):
    case, form = s["case"], s["format"]
    h, kh, d, new, b = case["heads"], case["kv_heads"], case["dim"], case["new"], case["batch"]
    page = s["table"].clamp(min=0).long()
    n = page.shape[1] * PAGE

    def held(x, unpack):  # [b][kh][n][d]
        codes = _value(unpack(s[x][0][page], d), form)  # [b][pages][kh][64][d]
        codes = codes.unflatten(3, (PAGE // BLOCK, BLOCK)) * s[x + "_scales"][0][page][..., None, None]
        return codes.flatten(3, 4).transpose(1, 2).reshape(b, kh, n, d)

    at = torch.arange(n, device="cuda")
    lens = s["lens"][:, None, None]
    seen = (at < lens).expand(b, new, n)
    if case["causal"]:
        pos = lens - new + torch.arange(new, device="cuda")[None, :, None]
        seen = seen & (at <= pos)
        if case["window"]:
            seen = seen & (at > pos - case["window"])
    q = s["q"].float().view(b, new, kh, h // kh, d).permute(0, 2, 3, 1, 4).reshape(b, kh, h // kh * new, d)
    x = (q @ held("k", unpack_k).transpose(2, 3)).view(b, kh, h // kh, new, n) * d ** -0.5
    x = x.masked_fill(~seen[:, None, None], -torch.inf)
    x = (x - x.amax(-1, keepdim=True).clamp(min=-1e30)).exp()
    total = x.sum(-1, keepdim=True)
    v = torch.where((at < lens[..., 0])[:, None, :, None], held("v", unpack_v), 0)
    o = x.view(b, kh, h // kh * new, n) @ v
    o = o.view(b, kh, h // kh, new, d) / total.clamp(min=1e-30)
    return o.permute(0, 3, 1, 2, 4).reshape(b * new, h, d).half()


def _lowest_free(refs):
    return torch.argsort((refs != 0).int(), stable=True)


def _copy(s, src, dst):
    for x in ("k", "v", "k_scales", "v_scales"):
        s[x][:, dst] = s[x][:, src]


def _plain_fork(s, table, lens, refs):
    rows, n = table[s["src"].long()], lens[s["src"].long()]
    full, tail = n // PAGE, n % PAGE > 0
    col = torch.arange(table.shape[1], device="cuda")
    keep = col < full[:, None]
    last = rows.gather(1, full.long()[:, None])[:, 0]
    new = torch.where(tail, _lowest_free(refs)[tail.cumsum(0) - tail.long()].int(), last)
    refs.scatter_add_(0, rows.clamp(min=0).flatten().long(), keep.flatten().int())
    refs.scatter_add_(0, new.clamp(min=0).long(), tail.int())
    made = torch.where(keep, rows, torch.where((col == full[:, None]) & tail[:, None], new[:, None], -1))
    table[s["dst"].long()] = made
    lens[s["dst"].long()] = n
    _copy(s, last[tail].long(), new[tail].long())
    return torch.stack((torch.zeros_like(full[0]), tail.sum().int()))


def _plain_resize(s, table, lens, refs):
    want = torch.where(s["want"] < 0, lens, s["want"])
    have, need = (lens + PAGE - 1) // PAGE, (want + PAGE - 1) // PAGE
    col = torch.arange(table.shape[1], device="cuda")
    drop = (col >= need[:, None]) & (col < have[:, None])
    refs.scatter_add_(0, table.clamp(min=0).flatten().long(), -drop.flatten().int())
    last = table.gather(1, (need.long() - 1).clamp(min=0)[:, None])[:, 0]
    split = (want < lens) & (want % PAGE != 0) & (refs[last.clamp(min=0).long()] > 1)
    count = (need - have).clamp(min=0) + split.int()
    first, free = count.cumsum(0) - count, _lowest_free(refs).int()
    grow = (col >= have[:, None]) & (col < need[:, None])
    change = split[:, None] & (col == need[:, None] - 1)
    at = first[:, None] + torch.where(grow, col - have[:, None], 0)
    taken = free[at.clamp(max=free.numel() - 1)]
    refs.scatter_add_(0, last.clamp(min=0).long(), -split.int())
    refs.scatter_add_(0, taken.flatten().long(), (grow | change).flatten().int())
    table.copy_(torch.where(grow | change, taken, torch.where(drop, -1, table)))
    lens.copy_(want)
    _copy(s, last[split].long(), taken[change].long())
    return torch.stack((torch.zeros_like(lens[0]), split.sum().int()))


def _plain_compact(s, table, refs):
    live = refs > 0
    at = torch.arange(refs.numel(), device="cuda")
    low = at < live.sum()
    src, dst = (live & ~low).nonzero()[:, 0], (~live & low).nonzero()[:, 0]
    _copy(s, src, dst)
    to = at.int()
    to[src] = dst.int()
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()], -1))
    refs[dst] = refs[src]
    refs[src] = 0
    return torch.stack((torch.zeros_like(to[0]), torch.full_like(to[0], src.numel())))


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["op"]
    if own:
        import bit_quantized_decode_qmv_amd as bq
        if op == "rope":
            return bq.rope(s["x"], s["pos"], s["inv_freq"], axis=s["axis"], adjacent=s["case"]["adjacent"])
        cache = bq.KVCache(s["k"], s["v"], s["k_scales"], s["v_scales"], s["format"])
        if op == "attn":
            return bq.kv_attn(cache, 0, s["q"], s["cu"], s["lens"], s["table"], causal=s["case"]["causal"],
                              window=s["case"]["window"], workspace=s["workspace"])
        if op == "append":
            q = bq.kv_append(cache, 0, s["k_new"], s["v_new"], s["cu"], s["lens"], s["table"], q=s["q"], pos=s["pos"],
                             inv_freq=s["inv_freq"], axis=s["axis"])
            k, v = bq.kv_read(cache, 0, s["cu_read"], s["lens"], s["table"], s["read"])
            return {"q": q, "k": k, "v": v}
        table, lens, refs = s["table"].clone(), s["lens"].clone(), s["refs"].clone()
        if op == "fork":
            told = [bq.kv_fork(cache, table, lens, refs, s["src"], s["dst"]), bq.kv_resize(cache, table, lens, refs, s["want"])]
        else:
            told = [bq.kv_compact(cache, table, refs)]
    else:
        if op == "rope":
            return _plain_rope(s["x"], s["pos"], s["inv_freq"], s["axis"], s["case"]["adjacent"]).half()
        if op == "attn":
            return _plain_attn(s)
        if op == "append":
            q = _plain_append(s)
            k, v = _plain_read(s, s["cu_read"], s["read"])
            return {"q": q, "k": k, "v": v}
        table, lens, refs = s["table"].clone(), s["lens"].clone(), s["refs"].clone()
        if op == "fork":
            told = [_plain_fork(s, table, lens, refs), _plain_resize(s, table, lens, refs)]
        else:
            told = [_plain_compact(s, table, refs)]
    return {"table": table, "lens": lens, "refs": refs, "told": told, "k": s["k"], "v": s["v"],
            "k_scales": s["k_scales"].view(torch.int32), "v_scales": s["v_scales"].view(torch.int32)}


# ------------------------------------------------------------------ 64 bits
def _exact_rope(x, s, adjacent):
    """The rotation as a product of complex numbers."""
    inv, x = s["inv_freq"].double(), x.double()
    r = inv.numel()
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


def _sequence(s, x, b, n):
    """The first n held values of sequence b: [kv_heads][n][dim] in 64 bits, byte by byte from their places in a page."""
    d = s["case"]["dim"]
    page = s["table"][b, :-(-n // PAGE)].long()
    t, c = torch.arange(PAGE, device="cuda")[:, None], torch.arange(d, device="cuda")[None]
    if x == "k":
        place = t // 16 * 16 * d + c // 64 * 1024 + c % 64 // 16 * 256 + t % 16 * 16 + c % 16
    else:
        place = c // 16 * 1024 + t % 16 // 4 * 256 + c % 16 * 16 + t // 16 * 4 + t % 4
    raw = s[x][0][page][:, :, place.flatten()].view(page.numel(), -1, PAGE, d)
    value = raw.double() - 128 if s["format"] == "int8" else raw.view(torch.float8_e4m3fn).double()
    value = value * s[x + "_scales"][0][page].double().repeat_interleave(BLOCK, -1)[..., None]
    return value.transpose(0, 1).flatten(1, 2)[:, :n]


def exact(case, seed):
    op = case["op"]
    if op in ("fork", "compact"):
        return None
    s = prepare(case, seed)
    if op == "rope":
        return _exact_rope(s["x"], s, case["adjacent"])
    lens, new, d = _lens(case), case["new"], case["dim"]
    if op == "append":
        q, k, v = _exact_rope(s["q"], s, False), _exact_rope(s["k_new"], s, False), s["v_new"].double()
        got = {"q": q, "k": [], "v": []}
        top = QMAX[s["format"]]
        for b, n in enumerate(lens):
            for x, made in (("k", k), ("v", v)):
                first = n - new
                at = first // BLOCK * BLOCK
                old = _sequence(s, x, b, first)[:, at:] if first > at else made.new_zeros(case["kv_heads"], 0, d)
                both = torch.cat((old, made[b * new:(b + 1) * new].transpose(0, 1)), 1)
                held = s[x + "_scales"][0][s["table"][b].long()].double()  # [pages][heads][4]
                for j in range(0, both.shape[1], BLOCK):
                    part = both[:, j:j + BLOCK]
                    since = first - at if j == 0 else 0
                    scale = part[:, since:].abs().amax((1, 2)) / top
                    if since:
                        scale = torch.maximum(scale, held[at // PAGE, :, at % PAGE // BLOCK])
                    scale = scale[:, None, None]
                    code = part / scale.clamp(min=1e-300)
                    # the code nearest to it: whole, or one of e4m3's by its exponent
                    unit = torch.ones_like(code) if s["format"] == "int8" else torch.exp2(code.abs().clamp(min=2.0 ** -6).log2().floor() - 3)
                    both[:, j:j + BLOCK] = (code / unit).round() * unit * scale
                got[x].append(both.transpose(0, 1))
        return {"q": q, "k": torch.cat(got["k"]), "v": torch.cat(got["v"])}
    out = torch.zeros(case["batch"] * new, case["heads"], d, dtype=torch.float64, device="cuda")
    group = case["heads"] // case["kv_heads"]
    for b, n in enumerate(lens):
        k, v = _sequence(s, "k", b, n), _sequence(s, "v", b, n)
        dist = (n - new + torch.arange(new, device="cuda"))[:, None] - torch.arange(n, device="cuda")
        hide = (dist < 0) if case["causal"] else torch.zeros_like(dist, dtype=torch.bool)
        if case["window"]:
            hide = hide | (dist >= case["window"])
        for h in range(case["heads"]):
            x = s["q"][b * new:(b + 1) * new, h].double() @ k[h // group].T / math.sqrt(d)
            out[b * new:(b + 1) * new, h] = torch.softmax(x.masked_fill(hide, -math.inf), -1) @ v[h // group]
    return out
