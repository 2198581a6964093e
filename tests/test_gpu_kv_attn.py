"""GPU parity of bq_kv_attn against the fp64 oracle.

Tolerance of an output o = sum p v / sum p, with mass = sum p |v| / sum p:
its own rounding to fp16, 2^-11 |o| + 2^-25; the rounding of each p to fp16,
2^-11 mass, and below the normal range 2^-25 of the largest |v|; scores in
fp32: sums of D products, D 2^-24 sum |q k| <= 2^-14 |score mass| for these
inputs, an exponent error of at most 2^-11 here, so 2^-11 mass once more."""
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


def check(out, cache, layer, table, lens, cu, q, scale, causal, window, heads_checked=None):
    for b, n in enumerate(lens):
        if cu[b] == cu[b + 1]:
            continue
        rows = slice(cu[b], cu[b + 1])
        ref, mass = oracle.kv_attn_f64(cache, layer, table[b], n, q[rows], scale, causal, window)
        top = max((float(np.abs(oracle.kv_sequence(cache, layer, table[b], n, "v")).max()) if n else 0.0), 0.0)
        got = out[rows].astype(np.float64)
        tol = 2.0 ** -11 * np.abs(ref) + 2.0 ** -10 * mass + 2.0 ** -25 * (1 + top * 256)
        worst = np.max(np.abs(got - ref) / tol)
        assert worst <= 1.0, (b, n, worst)


def run(rng, fmt, D, heads, group, lens, news, causal=True, window=0, layers=2, layer=1, q_scale=2.0, spoil=None,
        workspace="auto", scale=None):
    import bit_quantized_decode_qmv_amd as bq
    torch = torch_mod()
    table, pages = synth.make_kv_table(rng, lens)
    c = synth.make_kv_pool(rng, layers, pages, heads, D, fmt)
    if spoil:
        spoil(c, table)
    q = (rng.standard_normal((sum(news), heads * group, D)) * q_scale).astype(np.float16)
    cu = cu_of(news)
    cache = upload_cache(c)
    if workspace == "none":
        workspace = torch.zeros(0, dtype=torch.uint8, device="cuda:0")
    elif workspace == "auto":
        workspace = None
    out = bq.kv_attn(cache, layer, up(q), up(cu), up(lens, np.int32), up(table), scale=scale, causal=causal,
                     window=window, workspace=workspace).cpu().numpy()
    check(out, c, layer, table, lens, cu, q, D ** -0.5 if scale is None else scale, causal, window)
    return out, cache, table, q, cu


CASES = [  # D, heads, group, lens, news, causal, window
    (128, 2, 6, [1], [1], True, 0),                       # one token of context
    (128, 1, 6, [1003], [1], True, 0),
    (128, 2, 6, [64, 65, 63, 1, 130, 16], [1] * 6, True, 0),
    (64, 2, 1, [200, 77], [5, 5], True, 0),
    (128, 1, 8, [700, 9, 333], [5, 2, 4], True, 0),       # 40 rows, 16 and 32
    (192, 1, 3, [129], [7], True, 0),
    (256, 1, 4, [300, 40], [5, 1], True, 0),
    (64, 1, 2, [260], [90], True, 0),                     # a prompt's chunk
    (128, 1, 3, [150], [150], True, 0),                   # a whole prompt
    (128, 1, 5, [333, 20], [100, 20], True, 0),
    (256, 1, 2, [140], [70], True, 0),
    (192, 1, 2, [100], [67], True, 0),
    (64, 2, 1, [150, 31], [40, 9], False, 0),             # every row sees all of an encoder's states
    (128, 1, 6, [100], [70], False, 0),
    (128, 1, 6, [500, 64, 70], [1, 3, 5], True, 33),      # windows
    (64, 1, 4, [400], [100], True, 70),
    (128, 1, 2, [300], [90], True, 1),                    # a window of the row's own token
]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("D,heads,group,lens,news,causal,window", CASES)
def test_attn(fmt, D, heads, group, lens, news, causal, window):
    run(np.random.default_rng(D + sum(lens)), fmt, D, heads, group, lens, news, causal, window)


@pytest.mark.parametrize("news", [[1], [5], [30]])
def test_split_and_unsplit(news):
    """Without a workspace one workgroup takes all of a tile's tokens; with one several share them."""
    rng = lambda: np.random.default_rng(11)
    a = run(rng(), "int8", 128, 1, 6, [2500], news)[0]
    b = run(rng(), "int8", 128, 1, 6, [2500], news, workspace="none")[0]
    assert np.allclose(a, b, rtol=2.0 ** -9, atol=2.0 ** -9)


@pytest.mark.parametrize("new,group", [(1, 6), (5, 6), (64, 4)])
def test_workspace_is_left_ready(new, group):
    """Calls of several shapes on one workspace, each twice: the same bits, and the counters zero again."""
    import bit_quantized_decode_qmv_amd as bq
    torch = torch_mod()
    ws = torch.zeros(16 << 20, dtype=torch.uint8, device="cuda:0")
    rng = np.random.default_rng(12)
    for lens in ([3000, 100], [70], [1500, 1400, 64, 900]):
        lens = [max(n, new) for n in lens]
        out, cache, table, q, cu = run(rng, "int8", 128, 2, group, lens, [new] * len(lens), workspace=ws)
        again = bq.kv_attn(cache, 1, up(q), up(cu), up(lens, np.int32), up(table), workspace=ws)
        assert np.array_equal(out, again.cpu().numpy())
        assert int(ws[:bq.KV_ATTN_COUNTER_BYTES].max()) == 0


def test_small_workspaces():
    import bit_quantized_decode_qmv_amd as bq
    torch = torch_mod()
    need = bq.bq_kv_attn_workspace(upload_cache(synth.make_kv_pool(np.random.default_rng(0), 1, 2, 2, 128, "int8")).desc, 12, 1, 1)
    for size in (0, 100, bq.KV_ATTN_COUNTER_BYTES, bq.KV_ATTN_COUNTER_BYTES + 50000, need // 2):
        run(np.random.default_rng(13), "int8", 128, 2, 6, [1900], [1],
            workspace=torch.zeros(size, dtype=torch.uint8, device="cuda:0"))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("news", [[1, 3], [20, 40]])
def test_what_lies_past_the_length_is_not_used(fmt, news):
    """Scales that are NaN or infinite and e4m3 codes that are NaN behind the last token; pages in the table past it."""
    lens = [77, 64 + 33]

    def spoil(c, table):
        table[:, 2:] = 1 << 29
        for b, n in enumerate(lens):
            page = table[b, n // 64]
            first = (n % 64 + 15) // 16
            c["ks"][:, page, :, first:], c["vs"][:, page, :, first:] = np.nan, np.inf
            for w, byte in (("k", 0x7F), ("v", 0xFF)):
                at = oracle.kv_places(w, 128)[n % 64:].ravel()
                c[w][:, page, :, at] = byte
    run(np.random.default_rng(14), fmt, 128, 2, 3, lens, news, spoil=spoil)


@pytest.mark.parametrize("news", [[1, 2, 1, 3], [40, 33, 12, 50]])
def test_rows_that_see_nothing_are_zero(news):
    """No token held; more rows than tokens; a page that is none."""
    import bit_quantized_decode_qmv_amd as bq
    lens = [0, 1, 20, 64]

    def spoil(c, table):
        table[3, 0] = -1
    out, *_ = run(np.random.default_rng(15), "int8", 64, 2, 2, lens, news, spoil=spoil)
    assert not out[:news[0]].any() and not out[sum(news[:3]):].any()
    first = max(news[1] - 1, 0)
    assert not out[news[0]:news[0] + first].any()


def test_missing_page_in_the_middle():
    def spoil(c, table):
        table[0, 1] = c["k"].shape[1] + 3
    for news in ([1], [50]):
        run(np.random.default_rng(16), "int8", 128, 1, 2, [200], news, spoil=spoil)


@pytest.mark.parametrize("new", [1, 5, 60])
def test_extreme_scores_and_scales(new):
    """Scores of some hundreds (one token takes all), V scales that differ by 2^40 from block to block, zero scales."""
    def spoil(c, table):
        rng = np.random.default_rng(1)
        c["vs"][:] *= 2.0 ** rng.integers(-40, 1, c["vs"].shape)
        c["vs"][:, :, :, 1] = 0
        c["ks"][:, ::2, :, 2] = 0
    run(np.random.default_rng(17), "int8", 128, 1, 4, [700], [new], q_scale=16.0, spoil=spoil)


@pytest.mark.parametrize("scale", [0.0, -0.1, 1e-3])
def test_scales_of_the_scores(scale):
    run(np.random.default_rng(18), "int8", 64, 1, 2, [150], [3], scale=scale)
    run(np.random.default_rng(18), "int8", 64, 1, 2, [150], [70], scale=scale)


def test_one_hot_values_come_back_exactly():
    """A key that one row's query picks out by far: the output is that token's V, exactly rounded, at every place of a
    page, from workgroups all over the chip."""
    import bit_quantized_decode_qmv_amd as bq
    rng = np.random.default_rng(19)
    D, heads, n = 128, 4, 1024
    table, pages = synth.make_kv_table(rng, [n])
    c = synth.make_kv_pool(rng, 1, pages, heads, D, "int8")
    # K: token t has the signs of a random word; q asks for one token's signs
    signs = rng.integers(0, 2, (heads, n, D)) * 2 - 1
    place = oracle.kv_places("k", D)
    for t in range(n):
        c["k"][0, table[0, t // 64], :, place[t % 64]] = (128 + 100 * signs[:, t]).T.astype(np.uint8)
    c["ks"][:] = 1.0
    cache = upload_cache(c)
    v = oracle.kv_sequence(c, 0, table[0], n, "v")
    pick = rng.integers(0, n, (256, heads))
    q = np.stack([signs[np.arange(heads), pick[i]] for i in range(256)]).astype(np.float16)
    want = np.stack([v[pick[i], np.arange(heads)] for i in range(256)])
    for rows in (256, 32, 1):
        out = bq.kv_attn(cache, 0, up(q[:rows]), up([0, rows], np.int32), up([n], np.int32), up(table), causal=False)
        # p = 1 for the token, 0 for the others; v's scale has at most 24 bits: the product in fp16 units, one rounding
        np.testing.assert_allclose(out.cpu().numpy(), want[:rows], rtol=2.0 ** -10, atol=0)


def test_strides_streams_and_graph():
    import bit_quantized_decode_qmv_amd as bq
    torch = torch_mod()
    rng = np.random.default_rng(20)
    out, cache, table, q, cu = run(rng, "int8", 128, 2, 6, [900, 300], [2, 1])
    ws = torch.zeros(8 << 20, dtype=torch.uint8, device="cuda:0")
    dcu, dlens, dtable = up(cu), up([900, 300], np.int32), up(table)
    wide = torch.zeros((3, 12 * 128 * 3), dtype=torch.float16, device="cuda:0")
    wide[:, 1536:3072] = up(q).flatten(1)
    view = wide[:, 1536:3072].unflatten(1, (12, 128))
    into = torch.zeros((3, 12 * 128 * 2), dtype=torch.float16, device="cuda:0")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        bq.kv_attn(cache, 1, view, dcu, dlens, dtable, out=into[:, 1536:].unflatten(1, (12, 128)), workspace=ws)
    side.synchronize()
    assert np.array_equal(into[:, 1536:].unflatten(1, (12, 128)).cpu().numpy(), out) and not into[:, :1536].any()
    # a captured call follows the device arrays: the same graph over a shorter context
    dst = torch.zeros_like(view.contiguous())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bq.kv_attn(cache, 1, view, dcu, dlens, dtable, out=dst, workspace=ws)
    for lens in ([900, 300], [850, 1], [900, 300], [64, 256]):
        dlens.copy_(up(lens, np.int32))
        eager = bq.kv_attn(cache, 1, view, dcu, dlens, dtable, workspace=ws)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dst, eager)


def test_offsets_past_32_bits():
    """A pool of more than 4 GiB of codes: the sequence's pages lie at its end."""
    import bit_quantized_decode_qmv_amd as bq
    torch = torch_mod()
    rng = np.random.default_rng(21)
    D, heads = 128, 8
    lens, news = [150], [2]
    table, pages = synth.make_kv_table(rng, lens)
    c = synth.make_kv_pool(rng, 1, pages, heads, D, "int8")
    total = 70000                                     # 64 KiB of K a page: 4.3 GiB
    shift = total - pages
    big = {w: torch.empty((1, total, heads, 64 * D), dtype=torch.uint8, device="cuda:0") for w in ("k", "v")}
    scales = {w: torch.zeros((1, total, heads, 4), dtype=torch.float32, device="cuda:0") for w in ("k", "v")}
    for w in ("k", "v"):
        big[w][:, shift:] = up(c[w])
        scales[w][:, shift:] = up(c[w + "s"])
    cache = bq.KVCache(big["k"], big["v"], scales["k"], scales["v"], "int8")
    q = rng.standard_normal((2, heads * 2, D)).astype(np.float16)
    far = np.where(table >= 0, table + shift, -1).astype(np.int32)
    out = bq.kv_attn(cache, 0, up(q), up([0, 2], np.int32), up(lens, np.int32), up(far))
    check(out.cpu().numpy(), c, 0, table, lens, [0, 2], q, D ** -0.5, True, 0)
    k, v = bq.kv_read(cache, 0, up([0, 150], np.int32), up(lens, np.int32), up(far), 150)
    assert np.allclose(k.cpu().numpy(), oracle.kv_sequence(c, 0, table[0], 150, "k"), rtol=2.0 ** -10)
    bq.kv_append(cache, 0, k[:3].clone(), v[:3].clone(), up([0, 3], np.int32), up(lens, np.int32), up(far))
    k2, _ = bq.kv_read(cache, 0, up([0, 3], np.int32), up(lens, np.int32), up(far), 3)
    assert float((k2 - k[:3]).abs().max()) <= float(k[:3].abs().max()) / 100
