"""bq_kv_attn over batches, lengths and head counts whose work is laid out in
several steps: more sequences than a wave has lanes, more pages than a wave
holds table entries, more tiles than one launch, parts of every kind; whole
decode steps in a graph.  Oracle and tolerances are those of the other
attention tests."""
import numpy as np
import pytest

import oracle
import synth
from gpu_helpers import torch_mod
from kv_helpers import cu_of, download_cache, up, upload_cache
from test_gpu_kv_attn import check, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = torch_mod()
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import bit_quantized_decode_qmv_amd as bq
    bq.load_library()


@pytest.mark.parametrize("workspace", ["auto", "none"])
@pytest.mark.parametrize("fmt,D,heads,group", [("int8", 64, 3, 1), ("e4m3", 128, 1, 4)])
def test_more_sequences_than_lanes(fmt, D, heads, group, workspace):
    """150 sequences, some without rows, some without tokens, a few long enough for several parts."""
    rng = np.random.default_rng(31)
    lens = rng.integers(0, 200, 150).tolist()
    news = rng.integers(0, 4, 150).tolist()
    for b in (0, 63, 64, 100, 128, 149):
        lens[b], news[b] = 2300 + b, 1
    run(rng, fmt, D, heads, group, lens, news, workspace=workspace)


@pytest.mark.parametrize("workspace", ["auto", "none"])
def test_more_prompts_than_lanes(workspace):
    rng = np.random.default_rng(32)
    lens = rng.integers(40, 90, 70).tolist()
    news = [min(n, 40) for n in lens]
    lens[3], lens[66], news[66] = 1500, 1900, 300
    lens[10], news[20] = 0, 0
    run(rng, "int8", 64, 1, 1, lens, news, workspace=workspace)


@pytest.mark.parametrize("group,new", [(4, 6), (6, 5), (32, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_two_row_groups_in_parts(D, group, new):
    """17 to 32 rows of a sequence, its tokens in several parts, heads that do not divide the chip."""
    run(np.random.default_rng(33), "e4m3", D, 3, group, [2600, 1900], [new, new])


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("news,workspace", [([1], "none"), ([2], "auto"), ([70], "none"), ([70], "auto")])
def test_long_contexts(fmt, news, workspace):
    """More pages than the 64 whose table entries the lanes hold at a time: 8 waves in turn, and one after the other."""
    run(np.random.default_rng(34), fmt, 64, 1, 1, [40000 if news[0] < 3 else 9000], news, workspace=workspace)


@pytest.mark.parametrize("D", [192, 256])
@pytest.mark.parametrize("new", [1, 40])
def test_wide_heads_in_parts(D, new):
    run(np.random.default_rng(35), "int8", D, 2, 2, [4500, 300], [new, new])


@pytest.mark.parametrize("window", [100, 2000])
@pytest.mark.parametrize("new", [2, 64])
def test_windows_in_parts(window, new):
    """The pages ahead of the window are no part of the work, the tile's first rows see further back than its last."""
    run(np.random.default_rng(36), "int8", 64, 1, 2, [6000, 90], [new, new], window=window)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("new", [1, 5, 60])
def test_scores_that_leap_over_blocks_without_values(fmt, new):
    """A page whose V is zero (scale 0) has scores 200 above the page before, and the page after it 300 more: sums that
    followed V's units only would pass the range of fp32.  A page's keys are equal, so its scores are."""
    import bit_quantized_decode_qmv_amd as bq
    rng = np.random.default_rng(43)
    D, lens = 64, [256, 200]
    table, pages = synth.make_kv_table(rng, lens)
    c = synth.make_kv_pool(rng, 1, pages, 1, D, fmt)
    c["k"][:] = 128 + 127 if fmt == "int8" else 0x7E          # the largest code
    for row in table:
        for at, score in enumerate((0, 200, 500, 0)):
            if row[at] >= 0:
                # q = 1 in every dimension, scale 1/8: 8 scale code = score
                c["ks"][0, row[at]] = score / 8 / (127 if fmt == "int8" else 448)
                if at == 1:
                    c["vs"][0, row[at]] = 0
    q = np.ones((2 * new, 2, D), np.float16)
    cu = cu_of([new] * 2)
    for causal in (True, False):
        for workspace in (None, torch_mod().zeros(0, dtype=torch_mod().uint8, device="cuda:0")):
            out = bq.kv_attn(upload_cache(c), 0, up(q), up(cu), up(lens, np.int32), up(table), causal=causal,
                             workspace=workspace)
            check(out.cpu().numpy(), c, 0, table, lens, cu, q, 0.125, causal, 0)


@pytest.mark.parametrize("news", [[3, 2], [60, 40]])
def test_windows_longer_than_any_sequence(news):
    """The largest window is no window, also where rows are more than tokens."""
    lens = [20, 70]
    out = [run(np.random.default_rng(44), "int8", 64, 1, 2, lens, news, window=w)[0] for w in (0, 1 << 30, 2 ** 31 - 1)]
    assert np.array_equal(out[0], out[1]) and np.array_equal(out[0], out[2])


def test_same_bits_on_every_call():
    import bit_quantized_decode_qmv_amd as bq
    torch = torch_mod()
    for news in ([1, 1], [20, 1], [200, 64]):
        rng = np.random.default_rng(37)
        out, cache, table, q, cu = run(rng, "int8", 128, 2, 4, [3000, 700], news)
        side = torch.cuda.Stream()
        for i in range(4):
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side if i % 2 else torch.cuda.current_stream()):
                again = bq.kv_attn(cache, 1, up(q), up(cu), up([3000, 700], np.int32), up(table))
            torch.cuda.synchronize()
            assert np.array_equal(out, again.cpu().numpy())


def test_more_tiles_than_one_launch():
    """70000 sequences of one token: each output is its token's value, whatever the query."""
    import bit_quantized_decode_qmv_amd as bq
    rng = np.random.default_rng(38)
    n, pages = 70000, 50
    c = synth.make_kv_pool(rng, 1, pages, 1, 64, "int8")
    table = rng.integers(0, pages, (n, 1)).astype(np.int32)
    q = rng.standard_normal((n, 1, 64)).astype(np.float16)
    out = bq.kv_attn(upload_cache(c), 0, up(q), up(np.arange(n + 1), np.int32), up(np.ones(n), np.int32), up(table))
    first = np.stack([oracle.kv_sequence(c, 0, [p], 1, "v")[0, 0] for p in range(pages)])
    np.testing.assert_allclose(out.cpu().numpy()[:, 0], first[table[:, 0]], rtol=2.0 ** -10, atol=2.0 ** -24)


def test_many_prompts_tiles():
    """40000 sequences of three rows of 16 heads: tiles of 128 rows in two launches.  Every row sees the values of
    identical tokens, so each output is that value."""
    import bit_quantized_decode_qmv_amd as bq
    rng = np.random.default_rng(39)
    n, pages, group = 40000, 20, 16
    c = synth.make_kv_pool(rng, 1, pages, 1, 64, "int8")
    c["v"][:] = 128 + 90
    c["vs"][:] = 0.01 * (1 + np.arange(pages))[None, :, None, None]
    table = rng.integers(0, pages, (n, 1)).astype(np.int32)
    q = rng.standard_normal((3 * n, group, 64)).astype(np.float16)
    out = bq.kv_attn(upload_cache(c), 0, up(q), up(3 * np.arange(n + 1), np.int32), up(np.full(n, 50), np.int32), up(table))
    want = np.repeat(c["vs"][0, table[:, 0], 0, 0].astype(np.float64) * 90, 3)
    got = out.cpu().numpy().astype(np.float64)
    assert np.max(np.abs(got / want[:, None, None] - 1)) <= 2.0 ** -9


def test_falling_offsets_give_no_work():
    """Offsets that fall: nothing is written, and the workspace serves the next call."""
    import bit_quantized_decode_qmv_amd as bq
    torch = torch_mod()
    rng = np.random.default_rng(40)
    ws = torch.zeros(16 << 20, dtype=torch.uint8, device="cuda:0")
    for new in (1, 40):
        lens = [3000, 2000, 900]
        out, cache, table, q, cu = run(rng, "int8", 64, 2, 2, lens, [new] * 3, workspace=ws)
        dst = torch.full((3 * new, 4, 64), 7.0, dtype=torch.float16, device="cuda:0")
        bq.kv_attn(cache, 1, up(q), up([0, 3 * new, 0, 3 * new], np.int32), up(lens, np.int32), up(table), out=dst, workspace=ws)
        assert bool((dst == 7.0).all()) and int(ws[:bq.KV_ATTN_COUNTER_BYTES].max()) == 0
        again = bq.kv_attn(cache, 1, up(q), up(cu), up(lens, np.int32), up(table), workspace=ws)
        assert np.array_equal(out, again.cpu().numpy())


@pytest.mark.parametrize("new", [1, 4, 70])
def test_steps_in_a_graph(new):
    """Resize, append with rotation and attention captured once and replayed: every replay is the next step of the
    sequences, and equals the same calls made one by one on a second cache."""
    import bit_quantized_decode_qmv_amd as bq
    torch = torch_mod()
    rng = np.random.default_rng(41)
    heads, group, D, rows = 2, 2, 64, 2
    steps = 5
    # outputs of a step, of two separate states
    def make():
        cache = bq.KVCache.empty(1, 40, heads, D)
        for t in (cache.k, cache.v, cache.k_scales, cache.v_scales):
            t.zero_()                                # bytes never written are compared too
        table = torch.full((rows, 16), -1, dtype=torch.int32, device="cuda:0")
        return cache, table, up([0] * rows, np.int32), up([0] * 40, np.int32)

    k, v = (up(rng.standard_normal((steps, rows * new, heads, D)).astype(np.float16)) for _ in range(2))
    q = up(rng.standard_normal((steps, rows * new, heads * group, D)).astype(np.float16))
    cu, inv = up([0, new, 2 * new], np.int32), up(synth.rope_freqs(D))
    ws = [torch.zeros(16 << 20, dtype=torch.uint8, device="cuda:0") for _ in range(2)]

    def step(state, kk, vv, qq, pos, workspace):
        cache, table, lens, refs = state
        bq.kv_resize(cache, table, lens, refs, lens + new)
        turned = bq.kv_append(cache, 0, kk, vv, cu, lens, table, q=qq, pos=pos, inv_freq=inv)
        return bq.kv_attn(cache, 0, turned, cu, lens, table, workspace=workspace)

    a, b = make(), make()
    at = [t[0].clone() for t in (k, v, q)]
    pos = up(np.tile(np.arange(new), rows)[None], np.int32)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = step(a, *at, pos, ws[0])
    for i in range(steps):
        for t, src in zip(at, (k, v, q)):
            t.copy_(src[i])
        if i:
            pos += new
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = step(b, k[i], v[i], q[i], pos, ws[1])
        assert torch.equal(out, want) and bool(out.abs().max() > 0)
        for x, y in zip(a[1:], b[1:]):
            assert torch.equal(x, y)
        assert torch.equal(a[0].k, b[0].k) and torch.equal(a[0].k_scales, b[0].k_scales)
    c = download_cache(b[0])
    n = steps * new
    turned = bq.rope(q[-1], pos, inv).cpu().numpy()
    check(want.cpu().numpy(), c, 0, b[1].cpu().numpy(), [n] * rows, cu_of([new] * rows), turned, D ** -0.5, True, 0)


def test_pages_in_a_graph():
    """Fork, resize and compact captured; replays follow the arrays and equal the calls made one by one."""
    import bit_quantized_decode_qmv_amd as bq
    torch = torch_mod()
    rng = np.random.default_rng(42)
    codes = [up(rng.integers(0, 256, (2, 30, 2, 64 * 64)).astype(np.uint8)) for _ in range(2)]
    scales = [up(rng.random((2, 30, 2, 4)).astype(np.float32)) for _ in range(2)]

    def make():
        cache = bq.KVCache(*(t.clone() for t in codes + scales))
        table = up([[5, 9, 2, -1, -1], [7, -1, -1, -1, -1]] + [[-1] * 5] * 4, np.int32)
        refs = np.zeros(30, np.int32)
        refs[[5, 9, 2, 7]] = 1
        return cache, table, up([170, 30, 0, 0, 0, 0], np.int32), up(refs)

    def step(s, src, dst, want):
        cache, table, lens, refs = s
        return bq.kv_fork(cache, table, lens, refs, src, dst), bq.kv_resize(cache, table, lens, refs, want), bq.kv_compact(cache, table, refs)

    a, b = make(), make()
    args = [up(x, np.int32) for x in ([0, 1], [2, 3], [0, -1, 100, 64, -1, -1])]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        told = step(a, *args)
    for src, dst, want in (([0, 1], [2, 3], [0, -1, 100, 64, -1, -1]), ([2, 2], [0, 4], [-1, 0, 90, 200, 10, -1]),
                           ([0, 0], [1, 5], [-1, 300, -1, 0, -1, 40]), ([9, 0], [1, 5], [-1, -1, -1, -1, 0, 0])):
        for t, x in zip(args, (src, dst, want)):
            t.copy_(up(x, np.int32))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        eager = step(b, *args)
        for x, y in zip(told + a[1:], eager + b[1:]):
            assert torch.equal(x, y)
        live = b[3] > 0
        for x, y in zip(download_cache(a[0]).values(), download_cache(b[0]).values()):
            if not isinstance(x, str):
                assert np.array_equal(x[:, live.cpu().numpy()], y[:, live.cpu().numpy()])


def test_helpers_refuse():
    import bit_quantized_decode_qmv_amd as bq
    torch = torch_mod()
    cache = bq.KVCache.empty(1, 4, 2, 64)
    h = lambda *shape: torch.zeros(shape, dtype=torch.float16, device="cuda:0")
    cu, lens, table = up([0, 2], np.int32), up([2], np.int32), up([[0]], np.int32)
    ok = dict(q=h(2, 4, 64), cu=cu, lens=lens, table=table)
    bq.kv_attn(cache, 0, **ok)
    for change in (dict(q=h(2, 3, 64)), dict(q=h(2, 4, 128)), dict(q=h(2, 4, 64).float()), dict(q=h(2, 4, 64).cpu()),
                   dict(q=h(2, 64, 4).transpose(1, 2)), dict(lens=up([2, 2], np.int32)), dict(cu=cu.long()),
                   dict(table=table[0]), dict(out=h(3, 4, 64)), dict(causal=False, window=3), dict(window=-1),
                   dict(scale=float("nan")), dict(workspace=h(100))):
        with pytest.raises((ValueError, TypeError, bq.BQError)):
            bq.kv_attn(cache, 0, **{**ok, **change})
    for layer in (-1, 1):
        with pytest.raises((ValueError, TypeError, bq.BQError)):
            bq.kv_attn(cache, layer, **ok)
    with pytest.raises((ValueError, TypeError, bq.BQError)):
        bq.kv_append(cache, 0, h(2, 2, 64), h(3, 2, 64), cu, lens, table)
    with pytest.raises((ValueError, TypeError, bq.BQError)):
        bq.kv_append(cache, 0, h(2, 2, 64), h(2, 2, 64), cu, lens, table, q=h(1, 4, 64))
    with pytest.raises((ValueError, TypeError, bq.BQError)):
        bq.rope(h(2, 2, 64), up([[0, 1]], np.int32), up(np.ones(33), np.float32))
    refs = up([1, 0, 0, 0], np.int32)
    with pytest.raises((ValueError, TypeError, bq.BQError)):
        bq.kv_resize(cache, table, lens, refs[:3], up([5], np.int32))
    with pytest.raises((ValueError, TypeError, bq.BQError)):
        bq.kv_fork(cache, table, lens, refs, up([0, 0], np.int32), up([0], np.int32))
