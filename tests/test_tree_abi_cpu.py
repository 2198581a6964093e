"""The entry points of norms, sinks, trees and log probabilities reject invalid
arguments with their documented status before they touch the GPU, and the
tensor helpers what is not theirs."""
import ctypes
import os

import pytest

import bit_quantized_decode_qmv_amd as bq

OK, NULL, BITS, SHAPE, ALIGN, FLAGS = 0, -1, -2, -4, -6, -8
P = 0x10000  # fake, aligned, never dereferenced addresses
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    # a call that got past validation would launch on the fake addresses
    if os.path.exists("/dev/kfd"):
        pytest.skip("fake-pointer validation tests run only on machines without a GPU")
    return bq.load_library()


def desc(**kw):
    d = dict(k=P, v=2 * P, k_scales=3 * P, v_scales=4 * P, layers=2, num_pages=10, kv_heads=2, head_dim=128, format=1)
    d.update(kw)
    return bq.KVCacheDesc(**d)


def norm(lib, x=P, y=P, xs=256, ys=256, tokens=4, heads=2, dim=128, w=P, eps=1e-6, pos=P, inv=P, axis=None, rot=128, axes=1, flags=0):
    return lib.bq_norm_rope(x, y, xs, ys, tokens, heads, dim, w, eps, pos, inv, axis, rot, axes, flags, None)


def append(lib, cache=None, layer=0, k=P, v=P, ks=256, vs=256, q=P, qo=P, qs=512, qos=512, heads=4, cu=P, lens=P,
           table=P, batch=1, pages=4, total=3, kw=P, qw=P, eps=1e-6, pos=P, inv=P, axis=None, rot=128, axes=1, flags=0):
    return lib.bq_kv_append_norm(desc() if cache is None else cache, layer, k, v, ks, vs, q, qo, qs, qos, heads, cu, lens,
                                 table, batch, pages, total, kw, qw, eps, pos, inv, axis, rot, axes, flags, None)


def sinks(lib, cache=None, layer=0, q=P, out=P, qs=512, os=512, heads=4, cu=P, lens=P, table=P, batch=1, pages=4,
          total=3, scale=1.0, window=0, sinks=4, ws=None, ws_bytes=0):
    return lib.bq_kv_attn_sinks(desc() if cache is None else cache, layer, q, out, qs, os, heads, cu, lens, table, batch,
                                pages, total, scale, window, sinks, ws, ws_bytes, None)


def tree(lib, cache=None, layer=0, q=P, out=P, qs=512, os=512, heads=4, cu=P, lens=P, table=P, batch=1, pages=4,
         total=3, mask=P, words=1, scale=1.0, window=0, sinks=4, ws=None, ws_bytes=0):
    return lib.bq_kv_attn_tree(desc() if cache is None else cache, layer, q, out, qs, os, heads, cu, lens, table, batch,
                               pages, total, mask, words, scale, window, sinks, ws, ws_bytes, None)


def keep(lib, cache=None, cu=P, lens=P, table=P, batch=1, pages=4, path=P, most=4, kept=P):
    return lib.bq_kv_keep(desc() if cache is None else cache, cu, lens, table, batch, pages, path, most, kept, None)


def plan(lib, parent=P, cu=P, lens=P, batch=1, total=3, words=1, window=0, mask=P, pos=P):
    return lib.bq_tree_plan(parent, cu, lens, batch, total, words, window, mask, pos, None)


def accept(lib, target=P, token=P, parent=P, cu=P, lens=P, batch=1, total=3, most=4, path=P, kept=P, nxt=P, want=P):
    return lib.bq_tree_accept(target, token, parent, cu, lens, batch, total, most, path, kept, nxt, want, None)


def logprobs(lib, x=P, dtype=1, stride=100, rows=2, V=100, tokens=P, count=1, lp=P, ent=P, top=5, tt=P, tl=P, ws=None, ws_bytes=0):
    return lib.bq_logprobs(x, dtype, stride, rows, V, tokens, count, lp, ent, top, tt, tl, ws, ws_bytes, None)


@pytest.mark.parametrize("call", [append, sinks, tree, keep])
def test_cache_description(lib, call):
    for field in ("k", "v", "k_scales", "v_scales"):
        assert call(lib, cache=desc(**{field: None})) == NULL
        assert call(lib, cache=desc(**{field: P + 8})) == ALIGN
    assert call(lib, cache=desc(format=3)) == BITS
    for bad in ({"head_dim": 96}, {"layers": 0}, {"num_pages": 0}, {"kv_heads": 0}):
        assert call(lib, cache=desc(**bad)) == SHAPE


@pytest.mark.parametrize("call", [append, sinks, tree, keep])
def test_batches(lib, call):
    for bad in ({"batch": 0}, {"batch": (1 << 20) + 1}, {"pages": 0}, {"pages": (1 << 24) + 1}):
        assert call(lib, **bad) == SHAPE, bad
    for x in ("cu", "lens", "table"):
        assert call(lib, **{x: None}) == NULL
        assert call(lib, **{x: P + 2}) == ALIGN
    if call is not keep:
        for bad in ({"layer": -1}, {"layer": 2}, {"total": -1}, {"total": (1 << 28) + 1}):
            assert call(lib, **bad) == SHAPE, bad
        assert call(lib, total=0) == OK


def test_norm(lib):
    assert norm(lib, x=None) == NULL and norm(lib, y=None) == NULL and norm(lib, w=None) == NULL
    assert norm(lib, pos=None) == NULL and norm(lib, inv=None) == NULL
    for x in ("x", "y"):
        assert norm(lib, **{x: P + 8}) == ALIGN
    assert norm(lib, w=P + 2) == ALIGN and norm(lib, xs=260) == ALIGN and norm(lib, ys=248) == ALIGN
    for bad in ({"dim": 8}, {"dim": 72}, {"dim": 1040}, {"heads": 0}, {"heads": 70000}, {"tokens": -1}, {"rot": 8},
                {"rot": 144}, {"axes": 0}, {"axes": 9}, {"eps": -1e-6}, {"eps": NAN}, {"eps": INF}):
        assert norm(lib, **bad) == SHAPE, bad
    assert norm(lib, flags=2) == FLAGS and norm(lib, tokens=0) == OK and norm(lib, tokens=0, x=None, y=None) == OK


def test_append(lib):
    assert append(lib, k=None) == NULL and append(lib, v=None) == NULL and append(lib, qo=None) == NULL
    assert append(lib, kw=P + 2) == ALIGN and append(lib, qw=P + 1) == ALIGN
    for eps in (-1.0, NAN, INF):
        assert append(lib, eps=eps) == SHAPE
    for x in ("k", "v", "q", "qo"):
        assert append(lib, **{x: P + 8}) == ALIGN
    assert append(lib, heads=0) == SHAPE and append(lib, rot=160) == SHAPE and append(lib, flags=4) == FLAGS


@pytest.mark.parametrize("call", [sinks, tree])
def test_attention(lib, call):
    assert call(lib, q=None) == NULL and call(lib, out=None) == NULL
    assert call(lib, heads=3) == SHAPE and call(lib, window=-1) == SHAPE and call(lib, sinks=-1) == SHAPE
    assert call(lib, scale=NAN) == SHAPE and call(lib, qs=504) == ALIGN and call(lib, os=516) == ALIGN
    assert call(lib, ws=P + 8, ws_bytes=1 << 20) == ALIGN
    for x in ("q", "out"):
        assert call(lib, **{x: P + 8}) == ALIGN


def test_masks(lib):
    assert tree(lib, mask=None) == NULL and tree(lib, mask=P + 4) == ALIGN
    assert tree(lib, words=0) == SHAPE and tree(lib, words=17) == SHAPE
    assert tree(lib, total=0, mask=None) == OK


def test_keep(lib):
    assert keep(lib, path=None) == NULL and keep(lib, kept=None) == NULL
    assert keep(lib, path=P + 2) == ALIGN and keep(lib, kept=P + 1) == ALIGN
    assert keep(lib, most=0) == SHAPE and keep(lib, most=1025) == SHAPE
    assert keep(lib, cache=desc(kv_heads=1024), batch=1 << 14) == SHAPE      # more workgroups than a launch holds


@pytest.mark.parametrize("call", [plan, accept])
def test_trees(lib, call):
    for x in ("parent", "cu", "lens"):
        assert call(lib, **{x: None}) == NULL and call(lib, **{x: P + 2}) == ALIGN
    for bad in ({"batch": 0}, {"batch": (1 << 20) + 1}, {"total": -1}, {"total": (1 << 28) + 1}):
        assert call(lib, **bad) == SHAPE


def test_plan(lib):
    assert plan(lib, mask=None, pos=None) == NULL and plan(lib, mask=P + 4) == ALIGN and plan(lib, pos=P + 2) == ALIGN
    assert plan(lib, words=0) == SHAPE and plan(lib, words=17) == SHAPE and plan(lib, window=-1) == SHAPE
    assert plan(lib, total=0, parent=None, mask=None, pos=None) == OK


def test_accept(lib):
    for x in ("target", "token", "path", "kept", "nxt", "want"):
        assert accept(lib, **{x: None}) == NULL, x
        assert accept(lib, **{x: P + 2}) == ALIGN, x
    assert accept(lib, most=0) == SHAPE and accept(lib, most=1025) == SHAPE


def test_logprobs(lib):
    for x in ("x", "tokens", "lp", "tt", "tl"):
        assert logprobs(lib, **{x: None}) == NULL, x
    assert logprobs(lib, x=P + 1) == ALIGN and logprobs(lib, x=P + 2, dtype=2) == ALIGN
    for x in ("tokens", "lp", "ent", "tt", "tl"):
        assert logprobs(lib, **{x: P + 2}) == ALIGN, x
    assert logprobs(lib, ws=P + 8, ws_bytes=1 << 20) == ALIGN
    for d in (0, 3):
        assert logprobs(lib, dtype=d) == BITS
    for bad in ({"rows": -1}, {"rows": 1 << 24}, {"V": 0}, {"V": 1 << 28, "stride": 1 << 28}, {"stride": 99}, {"top": -1}, {"top": 65},
                {"count": -1}, {"count": 1025}, {"count": 0, "ent": None, "top": 0}):
        assert logprobs(lib, **bad) == SHAPE, bad
    assert logprobs(lib, rows=0) == OK


def test_logprobs_workspace(lib):
    n = ctypes.c_size_t(7)
    ws = lambda rows=5, V=151936, dtype=1, top=20: (lib.bq_logprobs_workspace(rows, V, dtype, top, ctypes.byref(n)), n.value)[0]
    assert ws() == OK and bq.LOGPROBS_COUNTER_BYTES < n.value < 1 << 20
    assert ws(rows=5000) == OK and n.value == 0            # rows enough: none is shared
    assert ws(V=100) == OK and n.value == 0
    assert ws(rows=-1) == SHAPE and ws(V=0) == SHAPE and ws(top=65) == SHAPE and ws(dtype=3) == BITS
    assert lib.bq_logprobs_workspace(1, 1, 1, 1, None) == NULL
    # one of the attention serves too
    assert bq.LOGPROBS_COUNTER_BYTES == bq.KV_ATTN_COUNTER_BYTES


def test_helpers_refuse_cpu_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 2, 64, dtype=torch.float16)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        bq.norm_rope(x, torch.ones(64), 1e-6)
    with pytest.raises(ValueError, match="GPU"):
        bq.logprobs(torch.zeros(2, 9), top=1)
    with pytest.raises(TypeError):
        bq.logprobs(None, top=1)
    with pytest.raises(ValueError, match="GPU"):
        bq.tree_plan(i, i, i)
    with pytest.raises(ValueError, match="GPU"):
        bq.tree_accept(i, i, i, i, i, 4)
