"""GPU parity of bq_kv_attn_sinks and bq_kv_attn_tree against the fp64 oracle,
which takes who sees whom as an explicit matrix.  Tolerance: that of the tests
of bq_kv_attn."""
import numpy as np
import pytest

import oracle
import synth
from gpu_helpers import torch_mod
from kv_helpers import cu_of, up, upload_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = torch_mod()
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import bit_quantized_decode_qmv_amd as bq
    bq.load_library()


def check(out, cache, layer, table, lens, cu, q, scale, seen):
    for b, n in enumerate(lens):
        if cu[b] == cu[b + 1]:
            continue
        rows = slice(cu[b], cu[b + 1])
        ref, mass = oracle.kv_attn_seen_f64(cache, layer, table[b], n, q[rows], scale, seen[b])
        top = float(np.abs(oracle.kv_sequence(cache, layer, table[b], n, "v")).max()) if n else 0.0
        tol = 2.0 ** -11 * np.abs(ref) + 2.0 ** -10 * mass + 2.0 ** -25 * (1 + top * 256)
        worst = np.max(np.abs(out[rows].astype(np.float64) - ref) / tol)
        assert worst <= 1.0, (b, n, worst)


def make(rng, fmt, D, heads, group, lens, news, spoil=None):
    table, pages = synth.make_kv_table(rng, lens)
    c = synth.make_kv_pool(rng, 2, pages, heads, D, fmt)
    if spoil:
        spoil(c, table)
    q = (rng.standard_normal((sum(news), heads * group, D)) * 2).astype(np.float16)
    return c, table, q, cu_of(news)


def workspaces():
    torch = torch_mod()
    return None, torch.zeros(0, dtype=torch.uint8, device="cuda:0")


def sinks_case(rng, fmt, D, heads, group, lens, news, window, sinks, spoil=None):
    import bit_quantized_decode_qmv_amd as bq
    c, table, q, cu = make(rng, fmt, D, heads, group, lens, news, spoil)
    seen = [oracle.causal_context(n, m - n, window, sinks) for n, m in zip(news, lens)]
    for workspace in workspaces():
        out = bq.kv_attn(upload_cache(c), 1, up(q), up(cu), up(lens, np.int32), up(table), window=window, sinks=sinks,
                         workspace=workspace).cpu().numpy()
        check(out, c, 1, table, lens, cu, q, D ** -0.5, seen)
    return out, c, table, q, cu


SINKS = [  # D, heads, group, lens, news, window, sinks
    (128, 2, 6, [1003], [1], 100, 4),
    (128, 2, 6, [64, 65, 63, 1, 130, 700], [1] * 6, 16, 4),
    (64, 2, 1, [500, 77], [5, 5], 33, 70),                  # more than a page of sinks
    (128, 1, 8, [700, 9, 333], [5, 2, 4], 64, 64),          # whole pages of both
    (192, 1, 3, [400], [7], 1, 1),
    (256, 1, 4, [600, 40], [5, 1], 50, 200),
    (64, 1, 2, [560], [90], 70, 3),                         # a prompt's chunk
    (128, 1, 3, [450], [450], 40, 130),                     # a whole prompt
    (128, 1, 5, [633, 20], [100, 20], 200, 1),
    (256, 1, 2, [340], [70], 30, 65),
    (192, 1, 2, [300], [67], 128, 5),
    (64, 1, 2, [300], [90], 128, 1000),                     # all are sinks
    (128, 1, 2, [300, 10], [1, 10], 5, 2 ** 31 - 1),
    (64, 1, 16, [200], [9], 0, 4),                          # no window
    (64, 2, 2, [20, 70], [60, 40], 8, 3),                   # rows ahead of the first token
]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("D,heads,group,lens,news,window,sinks", SINKS)
def test_sinks(fmt, D, heads, group, lens, news, window, sinks):
    sinks_case(np.random.default_rng(D + sum(lens) + window), fmt, D, heads, group, lens, news, window, sinks)


@pytest.mark.parametrize("new", [1, 5, 60])
def test_long_contexts_split(new):
    sinks_case(np.random.default_rng(new), "int8", 64, 2, 4, [9000, 5000], [new] * 2, 4000, 150)


@pytest.mark.parametrize("new", [1, 60])
def test_pages_that_no_row_sees_are_not_read(new):
    """Between the sinks and the window: no page at all, or codes and scales that are no numbers."""
    import bit_quantized_decode_qmv_amd as bq
    rng = np.random.default_rng(5)
    lens = [1500]
    c, table, q, cu = make(rng, "e4m3", 64, 2, 2, lens, [new])
    args = dict(window=200, sinks=70)
    out = bq.kv_attn(upload_cache(c), 1, up(q), up(cu), up(lens, np.int32), up(table), **args)
    first = (1500 - new - 200 + 1) // 64
    for w in "kv":
        c[w][:, table[0, 2:first]] = 0x7F
        c[w + "s"][:, table[0, 2:first]] = np.nan
    assert torch_mod().equal(out, bq.kv_attn(upload_cache(c), 1, up(q), up(cu), up(lens, np.int32), up(table), **args))
    table[0, 2:first] = -1
    assert torch_mod().equal(out, bq.kv_attn(upload_cache(c), 1, up(q), up(cu), up(lens, np.int32), up(table), **args))


def tree_case(rng, fmt, D, heads, group, lens, news, window=0, sinks=0, words=None, masks=None, spoil=None, scale=None):
    """masks: "tree" (of bq.tree_plan), or bool [n][n] of each sequence."""
    import bit_quantized_decode_qmv_amd as bq
    torch = torch_mod()
    c, table, q, cu = make(rng, fmt, D, heads, group, lens, news, spoil)
    words = words or max(1, -(-max(news) // 64))
    if masks is None:
        parents = [synth.make_tree(rng, n, 7) for n in news]
        rows = [oracle.tree_seen(p, window) for p in parents]
        mask, _ = bq.tree_plan(up(np.concatenate(parents), np.int32), up(cu), up(lens, np.int32), words, window)
        want = np.concatenate([oracle.tree_words(r, words) for r in rows])
        assert np.array_equal(mask.cpu().numpy().view(np.uint64), want)
    else:
        rows = masks
        mask = up(np.concatenate([oracle.tree_words(r, words) for r in rows]).view(np.int64))
    for r in rows:
        r[:, 64 * words:] = False
    seen = [oracle.tree_context(n, max(m - n, 0), r, window, sinks) for n, m, r in zip(news, lens, rows)]
    # rows that no token holds (fewer tokens than rows): the last ones remain
    seen = [x[:, n - m:] if m < n else x for x, n, m in zip(seen, news, lens)]
    for workspace in workspaces():
        out = bq.kv_attn_tree(upload_cache(c), 1, up(q), up(cu), up(lens, np.int32), up(table), mask, window=window,
                              sinks=sinks, workspace=workspace, scale=scale).cpu().numpy()
        check(out, c, 1, table, lens, cu, q, D ** -0.5 if scale is None else scale, seen)
    return out, c, table, q, cu, mask


TREES = [  # D, heads, group, lens, news, window, sinks
    (128, 2, 6, [1], [1], 0, 0),                            # a root alone
    (128, 2, 6, [1003], [13], 0, 0),
    (128, 1, 2, [64, 65, 63, 7, 130], [5, 2, 8, 7, 1], 0, 0),
    (64, 2, 1, [200, 77, 50], [16, 9, 0], 0, 0),
    (128, 1, 4, [130, 90], [8, 4], 0, 0),                   # 32 rows a tile
    (64, 1, 8, [300], [61], 0, 0),
    (128, 1, 6, [500, 64, 61], [61, 64, 61], 0, 0),         # trees without a context, and across a page's end
    (192, 1, 3, [129], [7], 0, 0),
    (192, 1, 2, [260], [61], 0, 0),
    (256, 1, 4, [300, 40], [5, 3], 0, 0),
    (256, 1, 2, [240], [70], 0, 0),                         # more than 64 rows
    (64, 1, 2, [560], [250], 0, 0),
    (128, 1, 6, [700, 300], [13, 61], 100, 4),              # a window and sinks
    (128, 2, 1, [700, 90], [5, 9], 3, 1),                   # shallower than the tree
    (64, 1, 4, [600], [130], 90, 70),
    (64, 1, 3, [800], [61], 200, 0),
    (256, 1, 2, [500], [61], 64, 64),
    (64, 1, 1, [20, 30], [30, 30], 0, 0),                   # rows that no token holds
]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("D,heads,group,lens,news,window,sinks", TREES)
def test_trees(fmt, D, heads, group, lens, news, window, sinks):
    tree_case(np.random.default_rng(D + sum(lens) + sum(news)), fmt, D, heads, group, lens, news, window, sinks)


@pytest.mark.parametrize("D,news", [(64, [3, 20]), (128, [70, 130]), (256, [9, 40])])
@pytest.mark.parametrize("window", [0, 9])
def test_masks_of_any_kind(D, news, window):
    """Rows that see later rows, not themselves, nothing at all; sequences with and without a context."""
    rng = np.random.default_rng(D + window)
    masks = [rng.random((n, n)) < 0.3 for n in news]
    for m in masks:
        m[1] = False
        m[2] = True
    tree_case(rng, "int8", D, 2, 2, [news[0], news[1] + 100], news, window, 2, masks=masks)
    out = tree_case(rng, "e4m3", D, 1, 3, news, news, window, masks=masks)[0]
    assert not out[1].any() and not out[news[0] + 1].any()  # neither a context nor a row


def test_rows_past_the_words_are_seen_by_none():
    rng = np.random.default_rng(8)
    masks = [np.ones((100, 100), bool)]
    tree_case(rng, "int8", 64, 1, 2, [150], [100], words=1, masks=masks)


def test_bits_past_the_rows_do_not_count():
    import bit_quantized_decode_qmv_amd as bq
    rng = np.random.default_rng(9)
    for window in (0, 20):
        out, c, table, q, cu, mask = tree_case(rng, "int8", 64, 2, 2, [90, 200], [5, 13], window, 1, words=2)
        for b, n in enumerate((5, 13)):
            mask[int(cu[b]):int(cu[b + 1]), 0] |= -1 << n
        mask[:, 1] = -1
        again = bq.kv_attn_tree(upload_cache(c), 1, up(q), up(cu), up([90, 200], np.int32), up(table), mask, window=window, sinks=1,
                                workspace=workspaces()[1])
        assert np.array_equal(out, again.cpu().numpy())


@pytest.mark.parametrize("new", [1, 13, 61])
def test_long_trees_split(new):
    tree_case(np.random.default_rng(new), "int8", 64, 2, 4, [9000, 5000], [new] * 2)


@pytest.mark.parametrize("new", [4, 61])
def test_what_lies_behind_the_length_is_not_read(new):
    """NaN codes and scales behind the last row, in the tree's own page."""
    def spoil(c, table):
        places = [oracle.kv_places(w, 64) for w in "kv"]
        for w, p in zip("kv", places):
            c[w][1, table[0, 2]][:, p[150 % 64:].ravel()] = 0x7F
            c[w + "s"][1, table[0, 2], :, 2:] = np.nan
    tree_case(np.random.default_rng(new), "e4m3", 64, 2, 2, [150], [new], spoil=spoil)


def test_missing_pages():
    def spoil(c, table):
        table[0, 1] = -1
        table[1, 0] = 1 << 29
    rng = np.random.default_rng(11)
    tree_case(rng, "int8", 64, 1, 2, [200, 70], [9, 30], spoil=spoil)
    sinks_case(rng, "int8", 64, 1, 2, [200, 70], [9, 30], 100, 3, spoil=spoil)


def test_negative_and_zero_scale():
    for scale in (-0.2, 0.0):
        tree_case(np.random.default_rng(12), "int8", 64, 1, 4, [300], [40], scale=scale)
        tree_case(np.random.default_rng(12), "int8", 64, 1, 2, [300], [4], scale=scale)


def test_many_sequences():
    rng = np.random.default_rng(13)
    news = rng.integers(0, 6, 150).tolist()
    lens = [n + int(rng.integers(0, 90)) for n in news]
    tree_case(rng, "int8", 64, 1, 2, lens, news)
    sinks_case(rng, "int8", 64, 1, 2, lens, news, 20, 3)


def test_same_bits_on_every_call_and_stream():
    import bit_quantized_decode_qmv_amd as bq
    torch = torch_mod()
    for new in (2, 30):
        rng = np.random.default_rng(14)
        out, c, table, q, cu, mask = tree_case(rng, "int8", 128, 2, 4, [3000, 700], [new] * 2)
        cache, side = upload_cache(c), torch.cuda.Stream()
        got = []
        for i in range(4):
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side if i % 2 else torch.cuda.current_stream()):
                got.append(bq.kv_attn_tree(cache, 1, up(q), up(cu), up([3000, 700], np.int32), up(table), mask))
            torch.cuda.synchronize()
        assert all(torch.equal(got[0], g) for g in got)


def test_strided_rows_and_rows_behind_the_last_sequence():
    import bit_quantized_decode_qmv_amd as bq
    torch = torch_mod()
    out, c, table, q, cu, mask = tree_case(np.random.default_rng(15), "int8", 64, 2, 2, [90], [13])
    wide = torch.full((16, 4 * 64 + 24), 7.0, dtype=torch.float16, device="cuda:0")
    view = wide[:, 8:8 + 256].unflatten(1, (4, 64))
    rows = torch.zeros((16, 4, 64), dtype=torch.float16, device="cuda:0")
    rows[:13] = up(q)
    masks = torch.cat((mask, mask[:3]))
    bq.kv_attn_tree(upload_cache(c), 1, rows, up(cu), up([90], np.int32), up(table), masks, out=view, workspace=workspaces()[1])
    assert np.array_equal(view[:13].cpu().numpy(), out)
    assert bool((view[13:] == 7).all()) and bool((wide[:, :8] == 7).all()) and bool((wide[:, 264:] == 7).all())


@pytest.mark.parametrize("new", [3, 40])
def test_two_graphs_with_one_workspace(new):
    """Captured calls of both kinds that share a workspace, replayed in turn over changing lengths and masks, with eager
    calls between: every replay equals the eager call."""
    import bit_quantized_decode_qmv_amd as bq
    torch = torch_mod()
    rng = np.random.default_rng(16)
    c, table, q, cu = make(rng, "int8", 64, 2, 2, [3000, 900], [new] * 2)
    cache, dq, dcu, lens, dt = upload_cache(c), up(q), up(cu), up([3000, 900], np.int32), up(table)
    ws = torch.zeros(16 << 20, dtype=torch.uint8, device="cuda:0")
    parent = up(np.concatenate([synth.make_tree(rng, new, 4)] * 2), np.int32)

    def calls(workspace):
        mask, pos = bq.tree_plan(parent, dcu, lens)
        return [lambda: bq.kv_attn_tree(cache, 1, dq, dcu, lens, dt, mask, workspace=workspace),
                lambda: bq.kv_attn(cache, 1, dq, dcu, lens, dt, window=500, sinks=4, workspace=workspace)]

    graphs, outs = [], []
    torch.cuda.synchronize()
    for k in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(calls(ws)[k]())
        graphs.append(g)
    for i in range(4):
        lens.copy_(up([3000 - 317 * i, 900 - 100 * i], np.int32))
        parent.copy_(up(np.concatenate([synth.make_tree(rng, new, 4) for _ in range(2)]), np.int32))
        torch.cuda.synchronize()
        graphs[i % 2].replay()
        graphs[1 - i % 2].replay()
        torch.cuda.synchronize()
        for out, call in zip(outs, calls(torch.zeros(16 << 20, dtype=torch.uint8, device="cuda:0"))):
            assert torch.equal(out, call())
        assert int(ws[:bq.KV_ATTN_COUNTER_BYTES].max()) == 0


def test_helpers_refuse():
    import bit_quantized_decode_qmv_amd as bq
    torch = torch_mod()
    cache = bq.KVCache.empty(1, 4, 2, 64)
    cache.k_scales.zero_()
    cache.v_scales.zero_()
    h = lambda *shape: torch.zeros(shape, dtype=torch.float16, device="cuda:0")
    m = lambda *shape: torch.zeros(shape, dtype=torch.int64, device="cuda:0")
    ok = dict(q=h(2, 4, 64), cu=up([0, 2], np.int32), lens=up([2], np.int32), table=up([[0]], np.int32), mask=m(2, 1))
    bq.kv_attn_tree(cache, 0, **ok)
    for change in (dict(mask=m(3, 1)), dict(mask=m(2)), dict(mask=m(2, 1).int()), dict(mask=m(2, 1).cpu()), dict(mask=m(2, 17)),
                   dict(mask=m(2, 2)[:, :1]), dict(mask=m(2, 0)), dict(window=-1), dict(sinks=-1), dict(q=h(2, 3, 64)), dict(workspace=h(100))):
        with pytest.raises((ValueError, TypeError, bq.BQError)):
            bq.kv_attn_tree(cache, 0, **{**ok, **change})
    del ok["mask"]
    for change in (dict(sinks=-1, window=4), dict(sinks=4, causal=False), dict(sinks=2 ** 40 * -1)):
        with pytest.raises((ValueError, TypeError, bq.BQError)):
            bq.kv_attn(cache, 0, **{**ok, **change})
