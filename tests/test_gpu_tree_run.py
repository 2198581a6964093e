"""The tree operators together, as a decoding step uses them: a tree is planned,
its rows are normed, turned and appended, attend, the target's tokens choose a
path, the path stays; step after step, over pages that are forked, moved and cut.

What each call makes is compared with the oracle on what the cache held before
it; tolerances are those of the tests of the single calls."""
import os
import sys

import numpy as np
import pytest

import oracle
import synth
from gpu_helpers import torch_mod
from kv_helpers import cu_of, download_cache, up
from test_gpu_kv_attn_tree import check as check_attention

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def ex():
    torch = torch_mod()
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import speculative_decode
    return speculative_decode


@pytest.mark.parametrize("fmt,window,sinks", [("int8", 0, 0), ("e4m3", 0, 0), ("int8", 40, 5)])
def test_steps_against_the_oracle(ex, fmt, window, sinks):
    import bit_quantized_decode_qmv_amd as bq
    torch = torch_mod()
    rng = np.random.default_rng(window + len(fmt))
    heads, group, D, rows, vocab, steps = 2, 3, 64, 3, 6, 5
    cache = bq.KVCache.empty(2, 40, heads, D, fmt)
    for t in (cache.k, cache.v, cache.k_scales, cache.v_scales):
        t.zero_()
    table = torch.full((rows, 8), -1, dtype=torch.int32, device="cuda:0")
    lens, refs = ex.ints([0] * rows), ex.ints([0] * 40)
    ws = torch.zeros(16 << 20, dtype=torch.uint8, device="cuda:0")
    w = [np.exp(rng.uniform(-1, 1, D)).astype(np.float32) for _ in range(2)]
    inv = synth.rope_freqs(D)

    def resize(want):
        status = bq.kv_resize(cache, table, lens, refs, want)
        assert int(status[0]) == 0

    def feed(news, pos, mask):
        """Rows of new tokens on both layers; the attention's result is checked."""
        total = sum(news)
        cu = up(cu_of(news))
        for layer in range(2):
            q, k, v = (rng.standard_normal((total, h, D)).astype(np.float16) for h in (heads * group, heads, heads))
            turned = bq.kv_append_norm(cache, layer, up(k), up(v), cu, lens, table, q=up(q), k_weight=up(w[0]), q_weight=up(w[1]),
                                       pos=pos, inv_freq=up(inv))
            args = dict(window=window, sinks=sinks, workspace=ws)
            if mask is None:
                out = bq.kv_attn(cache, layer, turned, cu, lens, table, **args)
                seen = [oracle.causal_context(n, m - n, window, sinks) for n, m in zip(news, lens.tolist())]
            else:
                out = bq.kv_attn_tree(cache, layer, turned, cu, lens, table, mask[0], **args)
                seen = [oracle.tree_context(n, m - n, oracle.tree_seen(p, window), window, sinks)
                        for n, m, p in zip(news, lens.tolist(), mask[1])]
            c = download_cache(cache)
            check_attention(out.cpu().numpy(), c, layer, table.cpu().numpy(), lens.tolist(), cu_of(news), turned.cpu().numpy(), D ** -0.5, seen)

    # a prompt on row 0, and two samples of it
    resize(ex.ints([77, 0, 0]))
    feed([77, 0, 0], up(np.arange(77)[None], np.int32), None)
    status = bq.kv_fork(cache, table, lens, refs, ex.ints([0, 0]), ex.ints([1, 2]))
    assert int(status[0]) == 0
    for step in range(steps):
        news = [int(n) for n in rng.integers(1, 30, rows)]
        if step == 2:
            news[1] = 0                                         # a sample that waits
        parents = [synth.make_tree(rng, n, 5) for n in news]
        flat = up(np.concatenate(parents), np.int32)
        cu = up(cu_of(news))
        before = lens.tolist()
        resize(lens + (cu[1:] - cu[:-1]))
        mask, pos = bq.tree_plan(flat, cu, lens, window=window)
        feed(news, pos[None].contiguous(), (mask, parents))
        # targets that some rows of the tree have
        logits = rng.standard_normal((sum(news), vocab)).astype(np.float16)
        token = rng.integers(0, vocab, sum(news))
        target = bq.logprobs(up(logits), top=1, workspace=ws)[2].flatten()
        path, kept, nxt, want = bq.tree_accept(target, up(token, np.int32), flat, cu, lens, 4)
        held, tables, at = download_cache(cache), table.cpu().numpy(), cu_of(news)
        bq.kv_keep(cache, cu, lens, table, path, kept)
        now = download_cache(cache)
        for b, n in enumerate(news):
            s = slice(at[b], at[b + 1])
            rows_kept, after = oracle.tree_accept(logits[s].argmax(1), token[s], parents[b], 4)
            assert path[b].tolist()[:len(rows_kept)] == rows_kept and int(kept[b]) == len(rows_kept) and int(nxt[b]) == after
            assert int(want[b]) == before[b] + len(rows_kept)
            if n:
                oracle.kv_keep_f64(held, tables[b], before[b], rows_kept)
        for x in ("k", "v", "ks", "vs"):
            assert np.array_equal(now[x], held[x]), (step, x)
        resize(want)
        assert lens.tolist() == want.tolist()
        if step == 3:
            bq.kv_compact(cache, table, refs)
    assert int(ws[:bq.KV_ATTN_COUNTER_BYTES].max()) == 0


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_example(ex, fmt):
    model = ex.Decoder(norms=True, window=64, sinks=4)
    torch = torch_mod()
    prompt = torch.from_numpy(np.random.default_rng(1).integers(0, 1024, 150).astype(np.int32)).to("cuda:0")
    runs = []
    for _ in range(2):
        s = ex.Session(model, rows=4, format=fmt)
        runs.append(ex.decode_tree(s, prompt, 3, 5))
        # a step adds the row that it began with, those that were taken and the token behind them
        assert all(1 + 5 <= len(t) <= 1 + 5 * 4 for t in runs[-1])
        assert s.lens.tolist()[:3] == [150 + len(t) - 1 for t in runs[-1]] and s.lens.tolist()[3] == 0
        refs, table = s.refs.cpu().numpy(), s.table.cpu().numpy()
        assert np.array_equal(np.bincount(table[table >= 0], minlength=refs.size), refs)
    assert runs[0] == runs[1]


def test_a_step_that_takes_nothing_is_a_decoding_step(ex):
    """A tree of the last token alone: the token behind it is what a plain step gives."""
    torch = torch_mod()
    model = ex.Decoder(norms=True, window=32, sinks=2)
    prompt = torch.from_numpy(np.random.default_rng(2).integers(0, 1024, 90).astype(np.int32)).to("cuda:0")
    last = ex.ints([7, 9])
    counts = ex.ints([1, 1])
    a, b = ex.Session(model, rows=2), ex.Session(model, rows=2)
    for s in (a, b):
        s.feed(prompt, ex.ints([60, 30]))
    path, kept, after, _ = a.feed_tree(last, ex.ints([-1, -1]), counts, 4)
    logits = b.feed(last, counts)
    assert path.tolist() == [[0, -1, -1, -1]] * 2 and kept.tolist() == [1, 1] and a.lens.tolist() == b.lens.tolist() == [61, 31]
    # either kernel's attention is within some 2^-11 of the exact one, so the logits differ by about 2^-9 of their spread
    # through two layers: two tokens may change places only if they are closer than 0.05 of it, 25 times that
    for i in range(2):
        row = logits[i].float()
        assert float(row.max() - row[int(after[i])]) <= 0.05 * float(row.std())
