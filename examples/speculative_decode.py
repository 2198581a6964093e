#!/usr/bin/env python3
"""A small decoder with 2-bit weights and a paged key/value cache in 8 bits.

One prompt is read, forked into several samples, and every sample is decoded
with drafts: a step takes the last token and L draft tokens of each sample
(their L + 1 rows share one read of the weights), the target tokens verify the
draft, and what was rejected is cut from the cache again.  Finished samples
are freed and the pool is compacted.

    python examples/speculative_decode.py            # needs an MI355X

Products go through bq.linear, positions and cache through bq.kv_append, the
attention through bq.kv_attn, verification through bq.spec_decode_verify, the
pages through bq.kv_resize, bq.kv_fork and bq.kv_compact.  Weights are random
(nothing is downloaded): the tokens mean nothing, the calls are those of a
real decoder.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import bit_quantized_decode_qmv_amd as bq


def ints(values, device="cuda"):
    return torch.tensor(values, dtype=torch.int32, device=device)


class Decoder:
    """`layers` blocks of attention and one output product, hidden size heads * dim."""

    def __init__(self, layers=2, heads=8, kv_heads=2, dim=64, vocab=1024, group_size=64, seed=0):
        self.layers, self.heads, self.kv_heads, self.dim, self.vocab = layers, heads, kv_heads, dim, vocab
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        hidden = heads * dim

        def weight(n, k):
            # 2-bit codes, symmetric: values -1.5, -0.5, 0.5, 1.5 times the scale
            w = torch.randint(-2 ** 31, 2 ** 31 - 1, (n, k // 16), dtype=torch.int64, generator=gen, device="cuda").int()
            s = ((torch.rand(n, k // group_size, generator=gen, device="cuda") + 0.5) / k ** 0.5).half()
            s = (s.view(torch.int16) & ~3).view(torch.float16)  # two low bits clear: -1.5 s is exact
            return bq.QuantizedWeight(w, s, -1.5 * s, 2, group_size)

        self.qkv = [weight((heads + 2 * kv_heads) * dim, hidden) for _ in range(layers)]
        self.o = [weight(hidden, hidden) for _ in range(layers)]
        self.head = weight(vocab, hidden)
        self.embed = torch.randn(vocab, hidden, generator=gen, device="cuda").half()
        # three axes in turn (time, height, width); text has the same position on all
        self.inv_freq = (1e4 ** (-torch.arange(dim // 2, device="cuda", dtype=torch.float64) * 2 / dim)).float()
        self.axis = (torch.arange(dim // 2, device="cuda") % 3).int()

    def forward(self, tokens, cache, cu, lens, table, workspace):
        """Logits [rows][vocab] of the packed rows `tokens`; the rows join the cache."""
        count = cu[1:] - cu[:-1]
        at = torch.arange(tokens.numel(), device="cuda", dtype=torch.int32)
        row = torch.searchsorted(cu[1:], at, right=True, out_int32=True)
        pos = (lens[row] - count[row] + at - cu[row]).int().repeat(3, 1).contiguous()
        x = self.embed[tokens.long()]
        h, k, d = self.heads, self.kv_heads, self.dim
        for layer in range(self.layers):
            y = bq.linear(normed(x), self.qkv[layer], workspace="auto")
            q, new_k, new_v = (y[:, a * d:b * d].unflatten(1, (b - a, d)) for a, b in ((0, h), (h, h + k), (h + k, h + 2 * k)))
            q = bq.kv_append(cache, layer, new_k, new_v, cu, lens, table, q=q, pos=pos, inv_freq=self.inv_freq, axis=self.axis)
            y = bq.kv_attn(cache, layer, q, cu, lens, table, workspace=workspace)
            x = x + bq.linear(y.flatten(1), self.o[layer], workspace="auto")
        return bq.linear(normed(x), self.head, workspace="auto")


def normed(x):
    y = x.float()
    return (y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)).half()


class Session:
    """The cache, its pages and the sequences (rows of the table) of one decoder."""

    def __init__(self, model, rows=8, pages=64, max_pages=16, format="int8"):
        self.model, self.rows = model, rows
        self.cache = bq.KVCache.empty(model.layers, pages, model.kv_heads, model.dim, format)
        self.table = torch.full((rows, max_pages), -1, dtype=torch.int32, device="cuda")
        self.lens, self.refs = ints([0] * rows), ints([0] * pages)
        # zero once; every attention call leaves it so
        self.workspace = torch.zeros(16 << 20, dtype=torch.uint8, device="cuda")

    def resize(self, want):
        status = bq.kv_resize(self.cache, self.table, self.lens, self.refs, want)
        if int(status[0]):
            raise RuntimeError(f"the pool cannot hold the sequences: {status.tolist()}")

    def feed(self, tokens, counts):
        """Logits of `tokens`, counts[i] of them the next of row i."""
        self.resize(self.lens + counts)
        cu = torch.zeros(self.rows + 1, dtype=torch.int32, device="cuda")
        cu[1:] = counts.cumsum(0)
        return self.model.forward(tokens, self.cache, cu, self.lens, self.table, self.workspace)

    def fork(self, src, dst):
        status = bq.kv_fork(self.cache, self.table, self.lens, self.refs, ints(src), ints(dst))
        if int(status[0]):
            raise RuntimeError(f"cannot fork: {status.tolist()}")

    def compact(self):
        return int(bq.kv_compact(self.cache, self.table, self.refs)[1])


def decode(session, prompt, samples, steps, draft_len, seed=0, compact=True):
    """`samples` continuations of the prompt (token ids), as lists of tokens."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rows, vocab = session.rows, session.model.vocab
    counts = ints([prompt.numel()] + [0] * (rows - 1))
    logits = session.feed(prompt, counts)
    first = int(logits[-1].float().argmax())
    if samples > 1:
        session.fork([0] * (samples - 1), list(range(1, samples)))
    counts = ints([draft_len + 1] * samples + [0] * (rows - samples))
    # each sample goes on from a token of its own
    last = (torch.arange(samples, device="cuda", dtype=torch.int32) + first) % vocab
    out = [[int(t)] for t in last]
    for _ in range(steps):
        draft = torch.randint(0, vocab, (samples, draft_len), dtype=torch.int32, generator=gen, device="cuda")
        held = session.lens.clone()
        logits = session.feed(torch.cat((last[:, None], draft), 1).flatten(), counts)
        accepted, last, _ = bq.spec_decode_verify(logits.view(samples, draft_len + 1, vocab), draft)
        want = held
        want[:samples] += accepted + 1  # the rejected rows leave the cache
        session.resize(want)
        for i, (n, t) in enumerate(zip(accepted.tolist(), last.tolist())):
            out[i] += draft[i, :n].tolist() + [t]
    # the first half of the samples is done: their pages are given back
    half = samples // 2
    want = session.lens.clone()
    want[:half] = 0
    session.resize(want)
    moved = session.compact() if compact else 0
    # the others go on from pages that have moved into the gaps
    counts = ints([0] * half + [1] * (samples - half) + [0] * (rows - samples))
    logits = session.feed(last[half:].contiguous(), counts)
    return out, logits, moved


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--format", choices=sorted(bq.KV_FORMATS), default="int8")
    ap.add_argument("--samples", type=int, default=4)
    ap.add_argument("--steps", type=int, default=6)
    a = ap.parse_args()
    model = Decoder()
    session = Session(model, rows=max(a.samples, 2), format=a.format)
    prompt = torch.randint(0, model.vocab, (150,), dtype=torch.int32, device="cuda")
    out, logits, moved = decode(session, prompt, a.samples, a.steps, draft_len=4)
    for i, tokens in enumerate(out):
        print(f"sample {i}: {tokens}")
    print(f"{moved} pages moved by the compaction, {int((session.refs > 0).sum())} of {session.refs.numel()} in use")


if __name__ == "__main__":
    main()
