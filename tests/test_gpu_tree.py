"""GPU parity of bq_tree_plan, bq_tree_accept and bq_kv_keep: whole numbers,
and codes and scales, equal to the oracle's."""
import numpy as np
import pytest

import oracle
import synth
from gpu_helpers import torch_mod
from kv_helpers import cu_of, download_cache, up, upload_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = torch_mod()
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import bit_quantized_decode_qmv_amd as bq
    bq.load_library()


def plan_of(parents, lens, words, window):
    """(masks, positions) of all sequences"""
    mask, pos = [], []
    for p, n in zip(parents, lens):
        rows = min(len(p), 64 * words)
        seen = np.zeros((len(p), len(p)), bool)
        seen[:rows, :rows] = oracle.tree_seen(p[:rows], window)
        mask.append(oracle.tree_words(seen, words))
        depth = [len(a) - 1 for a in oracle.tree_above(p[:rows])] + [0] * (len(p) - rows)
        pos += [max(n - len(p), 0) + d for d in depth]
    return np.concatenate(mask), np.array(pos)


@pytest.mark.parametrize("news,levels,words,window", [
    ([1], 1, 1, 0), ([13, 0, 61, 64], 6, 1, 0), ([61] * 3, 60, 1, 0), ([65, 130, 2], 9, 3, 0), ([1024, 300], 1023, 16, 0),
    ([61, 20], 30, 1, 4), ([200], 150, 4, 70), ([100, 10], 8, 1, 0), ([50], 5, 16, 0), ([40] * 200, 5, 1, 0),
])
def test_plan(news, levels, words, window):
    import bit_quantized_decode_qmv_amd as bq
    rng = np.random.default_rng(sum(news) + levels)
    parents = [synth.make_tree(rng, n, levels) for n in news]
    lens = [n + int(rng.integers(0, 500)) for n in news]
    mask, pos = bq.tree_plan(up(np.concatenate(parents), np.int32), up(cu_of(news)), up(lens, np.int32), words, window)
    want, want_pos = plan_of(parents, lens, words, window)
    assert np.array_equal(mask.cpu().numpy().view(np.uint64), want)
    assert np.array_equal(pos.cpu().numpy(), want_pos)


def test_parents_that_are_none_stand_behind_the_context():
    import bit_quantized_decode_qmv_amd as bq
    parent = [-1, 0, 2, 99, -7, 1, 2 ** 31 - 1, -2 ** 31]
    plain = [-1, 0, -1, -1, -1, 1, -1, -1]
    mask, pos = bq.tree_plan(up(parent, np.int32), up([0, 8], np.int32), up([20], np.int32))
    want, want_pos = plan_of([plain], [20], 1, 0)
    assert np.array_equal(mask.cpu().numpy().view(np.uint64), want) and np.array_equal(pos.cpu().numpy(), want_pos)


def test_rows_outside_any_sequence_and_offsets_past_the_end():
    import bit_quantized_decode_qmv_amd as bq
    torch = torch_mod()
    parent = up(np.full(10, -1), np.int32)
    lib_mask = torch.full((10, 1), -9, dtype=torch.int64, device="cuda:0")
    pos = torch.full((10,), -9, dtype=torch.int32, device="cuda:0")
    cu, lens = up([0, 3, 7], np.int32), up([3, 2], np.int32)
    bq.bq_tree_plan(parent.data_ptr(), cu.data_ptr(), lens.data_ptr(), 2, 10, 1, 0, lib_mask.data_ptr(), pos.data_ptr(), 0)
    torch.cuda.synchronize()
    assert (lib_mask[7:] == -9).all() and (pos[7:] == -9).all() and pos[:7].tolist() == [0] * 7
    cu = up([0, 3, 900], np.int32)
    bq.bq_tree_plan(parent.data_ptr(), cu.data_ptr(), lens.data_ptr(), 2, 10, 1, 0, None, pos.data_ptr(), 0)
    torch.cuda.synchronize()
    assert (pos >= 0).all()


def accept(targets, tokens, parents, lens, most):
    import bit_quantized_decode_qmv_amd as bq
    news = [len(p) for p in parents]
    flat = lambda xs: up(np.concatenate([np.asarray(x, np.int32) for x in xs]), np.int32)
    return [t.cpu().numpy() for t in bq.tree_accept(flat(targets), flat(tokens), flat(parents), up(cu_of(news)), up(lens, np.int32), most)]


@pytest.mark.parametrize("news,levels,most,vocab", [
    ([1], 1, 1, 5), ([13, 0, 61, 2], 6, 8, 3), ([61] * 40, 9, 10, 2), ([500, 1024], 300, 1024, 1), ([61] * 3, 20, 4, 1), ([7] * 5, 3, 20, 2),
])
def test_accept(news, levels, most, vocab):
    rng = np.random.default_rng(sum(news) + most)
    parents = [synth.make_tree(rng, n, levels) for n in news]
    targets, tokens = ([rng.integers(0, vocab, n) for n in news] for _ in range(2))
    lens = [n + int(rng.integers(0, 500)) for n in news]
    path, kept, nxt, want = accept(targets, tokens, parents, lens, most)
    for b, n in enumerate(news):
        rows, after = oracle.tree_accept(targets[b], tokens[b], parents[b], most)
        assert path[b].tolist() == rows + [-1] * (most - len(rows)) and kept[b] == len(rows) and nxt[b] == after
        assert want[b] == lens[b] - n + len(rows)


def test_accept_ignores_rows_past_the_limit_and_parents_that_are_none():
    n = 1030
    parent = np.zeros(n, np.int64)
    parent[0] = -1
    token = np.arange(n)
    target = np.zeros(n, np.int64)
    target[0] = 1025                                    # only a row past the limit has it
    path, kept, nxt, want = accept([target], [token], [parent], [2000], 3)
    assert kept[0] == 1 and nxt[0] == 1025 and want[0] == 2000 - n + 1
    # a row that names itself, a later row, and one that is negative
    path, kept, nxt, want = accept([[5, 5, 5, 5, 7]], [[0, 5, 5, 5, 5]], [[-1, 1, 3, -4, 0]], [50], 4)
    assert path[0].tolist() == [0, 4, -1, -1] and nxt[0] == 7


def test_no_rows_at_all():
    import bit_quantized_decode_qmv_amd as bq
    torch = torch_mod()
    none = torch.empty(0, dtype=torch.int32, device="cuda:0")
    cu, lens = up([0, 0, 0], np.int32), up([5, 0], np.int32)
    mask, pos = bq.tree_plan(none, cu, lens, words=2)
    assert mask.shape == (0, 2) and pos.shape == (0,)
    path, kept, nxt, want = bq.tree_accept(none, none, none, cu, lens, 3)
    assert path.tolist() == [[-1] * 3] * 2 and kept.tolist() == [0, 0] and nxt.tolist() == [-1, -1] and want.tolist() == [5, 0]


def keep(c, table, lens, news, paths, kept=None, most=None):
    import bit_quantized_decode_qmv_amd as bq
    most = most or max(max(map(len, paths)), 1)
    path = np.full((len(paths), most), -1, np.int32)
    for b, p in enumerate(paths):
        path[b, :len(p)] = p
    cache = upload_cache(c)
    bq.kv_keep(cache, up(cu_of(news)), up(lens, np.int32), up(table), up(path), up([len(p) for p in paths] if kept is None else kept, np.int32))
    return download_cache(cache)


def same(got, want):
    for x in ("k", "v", "ks", "vs"):
        assert np.array_equal(got[x], want[x]), x


KEEPS = [  # D, heads, lens, news, paths
    (128, 2, [1003], [13], [[0, 2, 7]]),
    (64, 1, [20], [20], [[0, 3, 4, 19]]),                       # no context, one block and the next
    (128, 2, [70, 64, 130, 61], [13, 5, 61, 61], [[0, 1, 2], [0, 4], [0, 5, 9, 30, 60], [0]]),
    (192, 1, [200], [100], [[0] + list(range(2, 100, 2))]),     # four blocks, rows read from the next ones
    (256, 2, [90, 5], [40, 0], [[0, 20, 21, 22, 39], []]),
    (64, 3, [500], [250], [list(range(100)) + list(range(150, 250))]),
    (64, 1, [300], [64], [[5, 9, 10]]),                         # not from row 0 on
]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("D,heads,lens,news,paths", KEEPS)
def test_keep(fmt, D, heads, lens, news, paths):
    rng = np.random.default_rng(D + sum(lens))
    table, pages = synth.make_kv_table(rng, lens)
    c = synth.make_kv_pool(rng, 2, pages, heads, D, fmt)
    c["ks"][0, :, 0] = 0                                        # a head whose scales are all 0
    want = {x: y.copy() if x != "format" else y for x, y in c.items()}
    for b, p in enumerate(paths):
        oracle.kv_keep_f64(want, table[b], lens[b] - news[b], p)
    same(keep(c, table, lens, news, paths), want)


def test_paths_that_do_not_rise_change_nothing():
    rng = np.random.default_rng(3)
    lens, news = [100] * 6, [20] * 6
    table, pages = synth.make_kv_table(rng, lens)
    c = synth.make_kv_pool(rng, 1, pages, 1, 64, "int8")
    same(keep(c, table, lens, news, [[0, 5, 5], [0, 7, 6], [0, 20], [-1, 3], [2 ** 31 - 1], [0, 1, 2]]), c)
    # numbers of rows that do not fit: none, or what the arrays hold
    same(keep(c, table, lens, news, [[0, 4]] * 6, kept=[0, -1, -2 ** 31, 1, 0, 0]), c)
    want = {x: y.copy() if x != "format" else y for x, y in c.items()}
    for b in range(6):
        oracle.kv_keep_f64(want, table[b], 80, [0, 4])
    same(keep(c, table, lens, news, [[0, 4]] * 6, kept=[2, 3, 2 ** 31 - 1, 2, 9, 2]), want)


def test_missing_pages_and_short_sequences():
    rng = np.random.default_rng(4)
    lens, news = [130, 130, 10, 130], [61, 61, 20, 61]
    table, pages = synth.make_kv_table(rng, lens)
    table[0, 2] = -1                                            # rows 128 - 69 and on have no page
    table[1, 1] = 1 << 20                                       # nor the places that are written
    c = synth.make_kv_pool(rng, 1, pages, 1, 64, "int8")
    paths = [[0, 30, 59, 60], [0, 30, 59, 60], [0, 15], [0, 30, 59, 60]]
    want = {x: y.copy() if x != "format" else y for x, y in c.items()}
    for b in (0, 1, 3):
        oracle.kv_keep_f64(want, table[b], lens[b] - news[b], paths[b])
    same(keep(c, table, lens, news, paths), want)


def test_layers_past_32_bits():
    """Two layers of 2.6 GB: the second one's offset does not fit 32 bits."""
    import bit_quantized_decode_qmv_amd as bq
    torch = torch_mod()
    cache = bq.KVCache.empty(2, 40000, 8, 128)
    assert cache.k.numel() > 2 ** 32
    rng = np.random.default_rng(5)
    pages = [39998, 39999]
    small = synth.make_kv_pool(rng, 2, 2, 8, 128, "int8")
    for x, t in (("k", cache.k), ("v", cache.v), ("ks", cache.k_scales), ("vs", cache.v_scales)):
        t[:, pages] = up(small[x])
    bq.kv_keep(cache, up([0, 61], np.int32), up([120], np.int32), up([pages], np.int32), up([[0, 8, 40, 60]], np.int32), up([4], np.int32))
    oracle.kv_keep_f64(small, [0, 1], 59, [0, 8, 40, 60])
    for x, t in (("k", cache.k), ("v", cache.v), ("ks", cache.k_scales), ("vs", cache.v_scales)):
        assert np.array_equal(t[:, pages].cpu().numpy(), small[x]), x


def test_a_step_in_a_graph():
    """Plan, accept and keep captured once: replays follow the arrays and equal the calls made one by one."""
    import bit_quantized_decode_qmv_amd as bq
    torch = torch_mod()
    rng = np.random.default_rng(6)
    news, lens0 = [13, 40], [100, 90]
    table, pages = synth.make_kv_table(rng, lens0)
    c = synth.make_kv_pool(rng, 2, pages, 2, 64, "int8")
    a, b = upload_cache(c), upload_cache(c)
    args = [up(np.zeros(53), np.int32) for _ in range(3)]
    lens, cu, dt = up(lens0, np.int32), up(cu_of(news)), up(table)

    def step(cache):
        target, token, parent = args
        mask, pos = bq.tree_plan(parent, cu, lens)
        path, kept, nxt, want = bq.tree_accept(target, token, parent, cu, lens, 6)
        bq.kv_keep(cache, cu, lens, dt, path, kept)
        return mask, pos, path, kept, nxt, want

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        told = step(a)
    for i in range(4):
        for t in args[:2]:
            t.copy_(up(rng.integers(0, 2, 53), np.int32))
        args[2].copy_(up(np.concatenate([synth.make_tree(rng, n, 5) for n in news]), np.int32))
        lens.copy_(up([100 - 9 * i, 90 - 7 * i], np.int32))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(told, step(b)):
            assert torch.equal(x, y)
        assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v) and torch.equal(a.k_scales, b.k_scales) and torch.equal(a.v_scales, b.v_scales)


def test_helpers_refuse():
    import bit_quantized_decode_qmv_amd as bq
    torch = torch_mod()
    i = lambda *v: up(list(v), np.int32)
    ok = (i(-1, 0), i(0, 2), i(5))
    bq.tree_plan(*ok)
    for bad in ((i(-1, 0).long(), *ok[1:]), (ok[0], i(0, 1, 2), ok[2]), (ok[0][None], *ok[1:]), (ok[0], ok[1], ok[2].cpu())):
        with pytest.raises((ValueError, TypeError)):
            bq.tree_plan(*bad)
        with pytest.raises((ValueError, TypeError)):
            bq.tree_accept(i(1, 2), i(1, 2), *bad, 4)
    for words in (0, 17):
        with pytest.raises(ValueError):
            bq.tree_plan(*ok, words=words)
    with pytest.raises(bq.BQError):
        bq.tree_plan(*ok, window=-1)
    for most in (0, 1025):
        with pytest.raises(ValueError):
            bq.tree_accept(i(1, 2), i(1, 2), *ok, most)
    with pytest.raises(ValueError):
        bq.tree_accept(i(1, 2, 3), i(1, 2), *ok, 4)
    cache = bq.KVCache.empty(1, 4, 2, 64)
    args = (cache, i(0, 2), i(2), up([[0]], np.int32))
    for path, kept in ((i(0, 1), i(1)), (up([[0], [1]], np.int32), i(1)), (up([[0]], np.int32), i(1, 1)), (up([[0]], np.int32).long(), i(1)),
                       (torch.zeros((1, 0), dtype=torch.int32, device="cuda:0"), i(0)),
                       (torch.zeros((1, 1025), dtype=torch.int32, device="cuda:0"), i(0))):
        with pytest.raises((ValueError, TypeError, bq.BQError)):
            bq.kv_keep(*args, path, kept)
