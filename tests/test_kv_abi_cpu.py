"""Every cache entry point rejects invalid arguments with its documented
status before it touches the GPU, and the tensor helpers what is not theirs."""
import ctypes
import os

import pytest

import bit_quantized_decode_qmv_amd as bq

OK, NULL, BITS, SHAPE, ALIGN, HIP_ERR, FLAGS, WORKSPACE = 0, -1, -2, -4, -6, -7, -8, -9
P = 0x10000  # fake, aligned, never dereferenced addresses


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


def rope(lib, x=P, y=P, xs=256, ys=256, tokens=4, heads=2, dim=128, pos=P, inv=P, axis=None, rot=128, axes=1, flags=0):
    return lib.bq_rope(x, y, xs, ys, tokens, heads, dim, pos, inv, axis, rot, axes, flags, None)


def append(lib, cache=None, layer=0, k=P, v=P, ks=256, vs=256, q=P, qo=P, qs=512, qos=512, heads=4, cu=P, lens=P,
           table=P, batch=1, pages=4, total=3, pos=P, inv=P, axis=None, rot=128, axes=1, flags=0):
    return lib.bq_kv_append(desc() if cache is None else cache, layer, k, v, ks, vs, q, qo, qs, qos, heads, cu, lens,
                            table, batch, pages, total, pos, inv, axis, rot, axes, flags, None)


def read(lib, cache=None, layer=0, k=P, v=P, cu=P, lens=P, table=P, batch=1, pages=4, total=3):
    return lib.bq_kv_read(desc() if cache is None else cache, layer, k, v, cu, lens, table, batch, pages, total, None)


def attn(lib, cache=None, layer=0, q=P, out=P, qs=512, os=512, heads=4, cu=P, lens=P, table=P, batch=1, pages=4,
         total=3, scale=1.0, window=0, flags=1, ws=None, ws_bytes=0):
    return lib.bq_kv_attn(desc() if cache is None else cache, layer, q, out, qs, os, heads, cu, lens, table, batch,
                          pages, total, scale, window, flags, ws, ws_bytes, None)


def fork(lib, cache=None, table=P, lens=P, refs=P, rows=4, pages=4, src=P, dst=P, n=1, status=P, ws=P, ws_bytes=1 << 20):
    return lib.bq_kv_fork(desc() if cache is None else cache, table, lens, refs, rows, pages, src, dst, n, status, ws,
                          ws_bytes, None)


def resize(lib, cache=None, table=P, lens=P, refs=P, rows=4, pages=4, want=P, status=P, ws=P, ws_bytes=1 << 20):
    return lib.bq_kv_resize(desc() if cache is None else cache, table, lens, refs, rows, pages, want, status, ws,
                            ws_bytes, None)


def compact(lib, cache=None, table=P, refs=P, rows=4, pages=4, status=P, ws=P, ws_bytes=1 << 20):
    return lib.bq_kv_compact(desc() if cache is None else cache, table, refs, rows, pages, status, ws, ws_bytes, None)


def copy(lib, cache=None, src=P, dst=P, n=1):
    return lib.bq_kv_copy_pages(desc() if cache is None else cache, src, dst, n, None)


CACHE_CALLS = [append, read, attn, fork, resize, compact, copy]


@pytest.mark.parametrize("call", CACHE_CALLS)
def test_cache_description(lib, call):
    for field in ("k", "v", "k_scales", "v_scales"):
        assert call(lib, cache=desc(**{field: None})) == NULL
        assert call(lib, cache=desc(**{field: P + 8})) == ALIGN
    for fmt in (0, 3, -1):
        assert call(lib, cache=desc(format=fmt)) == BITS
    for dim in (0, 16, 32, 80, 96, 320, 512, -64):
        assert call(lib, cache=desc(head_dim=dim)) == SHAPE
    for bad in ({"layers": 0}, {"num_pages": 0}, {"num_pages": (1 << 24) + 1}, {"kv_heads": 0}, {"kv_heads": 1025}):
        assert call(lib, cache=desc(**bad)) == SHAPE


@pytest.mark.parametrize("call", [append, read, attn])
def test_layers_and_batches(lib, call):
    for bad in ({"layer": -1}, {"layer": 2}, {"batch": 0}, {"batch": (1 << 20) + 1}, {"pages": 0},
                {"pages": (1 << 24) + 1}, {"total": -1}, {"total": (1 << 28) + 1}):
        assert call(lib, **bad) == SHAPE, bad
    for x in ("cu", "lens", "table"):
        assert call(lib, **{x: None}) == NULL
        assert call(lib, **{x: P + 2}) == ALIGN
    assert call(lib, total=0) == OK


def test_rope(lib):
    assert rope(lib, x=None) == NULL and rope(lib, y=None) == NULL
    assert rope(lib, pos=None) == NULL and rope(lib, inv=None) == NULL
    assert rope(lib, x=P + 8) == ALIGN and rope(lib, y=P + 2) == ALIGN
    assert rope(lib, xs=260) == ALIGN and rope(lib, ys=248) == ALIGN      # not whole 16 bytes; rows overlap
    assert rope(lib, pos=P + 1) == ALIGN and rope(lib, inv=P + 2) == ALIGN and rope(lib, axis=P + 2) == ALIGN
    for bad in ({"dim": 8}, {"dim": 72}, {"dim": 1040}, {"heads": 0}, {"heads": 70000}, {"tokens": -1}, {"rot": 8},
                {"rot": 144}, {"rot": -16}, {"axes": 0}, {"axes": 9}):
        assert rope(lib, **bad) == SHAPE, bad
    assert rope(lib, flags=2) == FLAGS and rope(lib, flags=-1) == FLAGS
    assert rope(lib, tokens=0) == OK and rope(lib, tokens=0, x=None, y=None, pos=None) == OK


def test_append(lib):
    assert append(lib, k=None) == NULL and append(lib, v=None) == NULL and append(lib, qo=None) == NULL
    assert append(lib, pos=None) == NULL and append(lib, inv=None) == NULL
    for x in ("k", "v", "q", "qo"):
        assert append(lib, **{x: P + 8}) == ALIGN
    for x in ("ks", "vs"):
        assert append(lib, **{x: 252}) == ALIGN and append(lib, **{x: 248}) == ALIGN
    for x in ("qs", "qos"):
        assert append(lib, **{x: 504}) == ALIGN
    assert append(lib, heads=0) == SHAPE and append(lib, rot=136) == SHAPE and append(lib, rot=160) == SHAPE
    assert append(lib, flags=4) == FLAGS


def test_read(lib):
    assert read(lib, k=None) == NULL and read(lib, v=None) == NULL
    assert read(lib, k=P + 8) == ALIGN and read(lib, v=P + 4) == ALIGN


def test_attn(lib):
    assert attn(lib, q=None) == NULL and attn(lib, out=None) == NULL
    assert attn(lib, heads=3) == SHAPE and attn(lib, heads=0) == SHAPE and attn(lib, window=-1) == SHAPE
    assert attn(lib, scale=float("nan")) == SHAPE and attn(lib, scale=float("inf")) == SHAPE
    assert attn(lib, flags=2) == FLAGS and attn(lib, flags=0, window=5) == FLAGS
    for x in ("q", "out"):
        assert attn(lib, **{x: P + 8}) == ALIGN
    assert attn(lib, qs=504) == ALIGN and attn(lib, os=516) == ALIGN
    assert attn(lib, ws=P + 8, ws_bytes=1 << 20) == ALIGN


def test_attn_workspace(lib):
    n = ctypes.c_size_t(7)
    ws = lambda **kw: lib.bq_kv_attn_workspace(kw.get("cache", desc()), kw.get("heads", 4), kw.get("batch", 1),
                                               kw.get("total", 1), ctypes.byref(n))
    assert ws() == OK and n.value > bq.KV_ATTN_COUNTER_BYTES and n.value < 64 << 20
    assert ws(total=1 << 20) == OK and n.value == 0          # rows enough: nothing is split
    assert ws(heads=3) == SHAPE and ws(batch=0) == SHAPE and ws(cache=desc(format=9)) == BITS
    assert lib.bq_kv_attn_workspace(desc(), 4, 1, 1, None) == NULL
    assert bq.bq_kv_attn_workspace(desc(), 4, 1, 1) > 0
    with pytest.raises(bq.BQError):
        bq.bq_kv_attn_workspace(desc(), 3, 1, 1)


@pytest.mark.parametrize("call", [fork, resize, compact])
def test_pages(lib, call):
    for x in ("table", "refs", "status"):
        assert call(lib, **{x: None}) == NULL
        assert call(lib, **{x: P + 2}) == ALIGN
    for bad in ({"rows": 0}, {"rows": (1 << 20) + 1}, {"pages": 0}):
        assert call(lib, **bad) == SHAPE
    assert call(lib, ws=None) == WORKSPACE and call(lib, ws_bytes=64) == WORKSPACE
    assert call(lib, ws=P + 4) == ALIGN
    if call is not compact:
        assert call(lib, lens=None) == NULL and call(lib, lens=P + 1) == ALIGN


def test_fork_resize_copy(lib):
    assert fork(lib, src=None) == NULL and fork(lib, dst=None) == NULL and resize(lib, want=None) == NULL
    assert fork(lib, n=0) == SHAPE and fork(lib, n=5) == SHAPE
    assert fork(lib, src=P + 2) == ALIGN and fork(lib, dst=P + 2) == ALIGN and resize(lib, want=P + 2) == ALIGN
    assert copy(lib, src=None) == NULL and copy(lib, dst=None) == NULL and copy(lib, n=-1) == SHAPE
    assert copy(lib, src=P + 1) == ALIGN and copy(lib, n=0) == OK


def test_pages_workspace(lib):
    small = bq.bq_kv_pages_workspace(desc(num_pages=10), 4)
    assert 0 < small < bq.bq_kv_pages_workspace(desc(num_pages=1000), 4) and small % 4 == 0
    n = ctypes.c_size_t(0)
    assert lib.bq_kv_pages_workspace(desc(), 0, ctypes.byref(n)) == SHAPE
    assert lib.bq_kv_pages_workspace(desc(), 4, None) == NULL


def test_helpers_refuse_cpu_tensors_and_formats():
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 2, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="GPU"):
        bq.rope(x, torch.zeros(1, 2, dtype=torch.int32), torch.zeros(32))
    codes, scales = torch.zeros(1, 2, 1, 64 * 64, dtype=torch.uint8), torch.zeros(1, 2, 1, 4)
    with pytest.raises(ValueError, match="GPU"):
        bq.KVCache(codes, codes, scales, scales)
    with pytest.raises(ValueError, match="format"):
        bq.KVCache(codes, codes, scales, scales, format="int4")
