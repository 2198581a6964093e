"""Attention with a paged key/value cache in 8 bits: the binding of the
``bq_rope`` and ``bq_kv_*`` entry points of ``include/bq.h`` and their tensor
helpers (``rope``, ``kv_append``, ``kv_read``, ``kv_attn``, ``kv_fork``,
``kv_resize``, ``kv_compact``, ``kv_copy_pages``) over a :class:`KVCache`.

As in the rest of the package every step runs in the HIP kernels; a helper
checks its arguments, allocates what it returns and passes the current stream.
"""
from __future__ import annotations

import ctypes
import sys
from typing import Optional

KV_PAGE = 64
KV_BLOCK = 16
KV_I8 = 1
KV_E4M3 = 2
KV_FORMATS = {"int8": KV_I8, "e4m3": KV_E4M3}
KV_CAUSAL = 1
KV_ATTN_COUNTER_BYTES = 65536
ROPE_ADJACENT = 1
ROPE_MAX_AXES = 8

KV_POINTS = ("bq_rope", "bq_kv_append", "bq_kv_read", "bq_kv_attn_workspace", "bq_kv_attn", "bq_kv_pages_workspace",
             "bq_kv_fork", "bq_kv_resize", "bq_kv_compact", "bq_kv_copy_pages")


class KVCacheDesc(ctypes.Structure):
    """bq_kv_cache of include/bq.h."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("layers", ctypes.c_int), ("num_pages", ctypes.c_int),
                ("kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("format", ctypes.c_int)]


def declare(lib) -> None:
    """Argument types of the entry points."""
    vp, i, ll, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_size_t
    cache = ctypes.POINTER(KVCacheDesc)
    size = ctypes.POINTER(sz)
    types = {
        "bq_rope": [vp, vp, ll, ll, i, i, i, vp, vp, vp, i, i, i, vp],
        "bq_kv_append": [cache, i, vp, vp, ll, ll, vp, vp, ll, ll, i, vp, vp, vp, i, i, i, vp, vp, vp, i, i, i, vp],
        "bq_kv_read": [cache, i, vp, vp, vp, vp, vp, i, i, i, vp],
        "bq_kv_attn_workspace": [cache, i, i, i, size],
        "bq_kv_attn": [cache, i, vp, vp, ll, ll, i, vp, vp, vp, i, i, i, ctypes.c_float, i, i, vp, sz, vp],
        "bq_kv_pages_workspace": [cache, i, size],
        "bq_kv_fork": [cache, vp, vp, vp, i, i, vp, vp, i, vp, vp, sz, vp],
        "bq_kv_resize": [cache, vp, vp, vp, i, i, vp, vp, vp, sz, vp],
        "bq_kv_compact": [cache, vp, vp, i, i, vp, vp, sz, vp],
        "bq_kv_copy_pages": [cache, vp, vp, i, vp],
    }
    for name, args in types.items():
        fn = getattr(lib, name)
        fn.restype = ctypes.c_int
        fn.argtypes = args


# the package (its library, errors and checks) and torch, which is imported
# when the first tensor comes
_bq = sys.modules[__package__]
_torch = None
_raw_stream = None
_device_now = None


def _use_torch():
    global _torch, _raw_stream, _device_now
    import torch
    # the current stream's handle and device by themselves where torch offers
    # them: a call's host time is a few microseconds in all
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    _device_now = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    _torch = torch
    return torch


def _stream(device) -> int:
    if _raw_stream is not None and device.index is not None:
        return _raw_stream(device.index)
    return _bq._stream_handle(device)


def _need(t, name, dtype, device) -> None:
    """A contiguous tensor of dtype on device; what it is not is said by the package's check."""
    try:
        if t.dtype is dtype and t.device == device and t.is_contiguous():
            return
    except AttributeError:
        pass
    _bq._check(t, name, dtype, device)


def _call(name, *args):
    lib = _bq._lib or _bq.load_library()
    st = getattr(lib, name)(*args)
    if st < 0:
        raise _bq.BQError(st, lib.bq_strerror(st).decode(), name)
    return st


def _launch(device, name, *args):
    """The entry point on the current stream of the tensors' device, with that
    device current (as the package's _launch)."""
    if _device_now() == device.index:
        return _call(name, *args, _stream(device))
    with _torch.cuda.device(device):
        return _call(name, *args, _stream(device))


def _c_entry(name):
    def fn(*args):
        return _call(name, *args)
    fn.__name__ = name
    fn.__doc__ = f"C entry point {name} of include/bq.h (pointers and stream as integers, the cache as KVCache.desc)."
    return fn


bq_rope = _c_entry("bq_rope")
bq_kv_append = _c_entry("bq_kv_append")
bq_kv_read = _c_entry("bq_kv_read")
bq_kv_attn = _c_entry("bq_kv_attn")
bq_kv_fork = _c_entry("bq_kv_fork")
bq_kv_resize = _c_entry("bq_kv_resize")
bq_kv_compact = _c_entry("bq_kv_compact")
bq_kv_copy_pages = _c_entry("bq_kv_copy_pages")


def bq_kv_attn_workspace(desc, q_heads, batch, total):
    """Workspace bytes bq_kv_attn wants for its full split (host only)."""
    n = ctypes.c_size_t(0)
    _call("bq_kv_attn_workspace", desc, q_heads, batch, total, ctypes.byref(n))
    return n.value


def bq_kv_pages_workspace(desc, rows):
    """Workspace bytes the page calls need (host only)."""
    n = ctypes.c_size_t(0)
    _call("bq_kv_pages_workspace", desc, rows, ctypes.byref(n))
    return n.value


# bq_kv_pages_workspace by (pages, rows), of which alone it is a function
_pages_bytes = {}


class KVCache:
    """A paged key/value cache in 8 bits over the caller's tensors:
    k, v uint8 [layers][pages][kv_heads][64 * head_dim], k_scales, v_scales
    float32 [layers][pages][kv_heads][4] (``include/bq.h`` gives the order of
    a page's bytes).  format: "int8" or "e4m3"."""

    __slots__ = ("k", "v", "k_scales", "v_scales", "format", "device", "layers", "num_pages", "kv_heads", "head_dim",
                 "desc")

    def __init__(self, k, v, k_scales, v_scales, format: str = "int8"):
        torch = _torch or _use_torch()
        if format not in KV_FORMATS:
            raise ValueError(f"format must be one of {sorted(KV_FORMATS)}, got {format!r}")
        if not isinstance(k, torch.Tensor) or not k.is_cuda:
            _bq._check(k, "k", torch.uint8, None)
        dev = k.device
        _need(k, "k", torch.uint8, dev)
        _need(v, "v", torch.uint8, dev)
        _need(k_scales, "k_scales", torch.float32, dev)
        _need(v_scales, "v_scales", torch.float32, dev)
        shape = k.shape
        if len(shape) != 4 or shape[3] % KV_PAGE:
            raise ValueError(f"k has shape {tuple(shape)}, expected [layers][pages][kv_heads][{KV_PAGE} * head_dim]")
        if v.shape != shape:
            raise ValueError(f"v has shape {tuple(v.shape)}, k {tuple(shape)}")
        layers, pages, heads, row = shape
        scales = (layers, pages, heads, KV_PAGE // KV_BLOCK)
        if k_scales.shape != scales or v_scales.shape != scales:
            raise ValueError(f"scales have shapes {tuple(k_scales.shape)}, {tuple(v_scales.shape)}, expected {scales}")
        self.k, self.v, self.k_scales, self.v_scales, self.format = k, v, k_scales, v_scales, format
        self.device = dev
        self.layers, self.num_pages, self.kv_heads, self.head_dim = layers, pages, heads, row // KV_PAGE
        self.desc = KVCacheDesc(k.data_ptr(), v.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(), layers, pages,
                                heads, row // KV_PAGE, KV_FORMATS[format])

    @classmethod
    def empty(cls, layers: int, num_pages: int, kv_heads: int, head_dim: int, format: str = "int8", device="cuda"):
        """A cache of its own memory, uninitialised: tokens exist once they are appended."""
        torch = _torch or _use_torch()
        codes = (layers, num_pages, kv_heads, KV_PAGE * head_dim)
        scales = (layers, num_pages, kv_heads, KV_PAGE // KV_BLOCK)
        return cls(*(torch.empty(codes, dtype=torch.uint8, device=device) for _ in range(2)),
                   *(torch.empty(scales, dtype=torch.float32, device=device) for _ in range(2)), format=format)


def _int(value, name) -> int:
    """A number as the C entry points hold it; ctypes would drop the bits past the 32nd."""
    if not -1 << 31 <= value < 1 << 31:
        raise ValueError(f"{name} = {value} does not fit 32 bits")
    return value


def _rows(t, name, device, heads=None, head_dim=None):
    """Checks a row array [tokens][heads][head_dim], fp16, any row stride; returns its row stride."""
    torch = _torch or _use_torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU, got {t.device}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype is not torch.float16:
        raise TypeError(f"{name} must be torch.float16, got {t.dtype}")
    shape = t.shape
    if len(shape) != 3 or (heads is not None and shape[1] != heads) or (head_dim is not None and shape[2] != head_dim):
        raise ValueError(f"{name} has shape {tuple(shape)}, expected [tokens][{heads or 'heads'}][{head_dim or 'head_dim'}]")
    n, h, d = shape
    _int(n, f"the rows of {name}")
    s0, s1, s2 = t.stride()
    row = h * d
    if s2 != 1 or (s1 != d and h > 1):
        raise ValueError(f"{name} must hold each row [heads][head_dim] contiguously")
    if n <= 1:
        return row  # a single row has no stride
    if s0 < row:
        raise ValueError(f"{name} has overlapping rows (stride {s0}, row {row})")
    return s0


def _batch(cu, lens, table, device):
    i32 = _torch.int32
    _need(cu, "cu", i32, device)
    _need(lens, "lens", i32, device)
    _need(table, "table", i32, device)
    n = lens.shape[0]
    if lens.dim() != 1 or cu.dim() != 1 or cu.shape[0] != n + 1 or table.dim() != 2 or table.shape[0] != n:
        raise ValueError(f"expected lens [batch], cu [batch + 1], table [batch][max_pages]; got {tuple(lens.shape)}, "
                         f"{tuple(cu.shape)}, {tuple(table.shape)}")
    return n, table.shape[1]


def _angles(pos, inv_freq, axis, adjacent, tokens, device):
    """(pos, inv_freq, axis pointers, rot_dim, axes, flags)"""
    if inv_freq is None:
        if pos is not None or axis is not None:
            raise ValueError("pos and axis need inv_freq")
        return None, None, None, 0, 1, 0
    _need(inv_freq, "inv_freq", _torch.float32, device)
    _need(pos, "pos", _torch.int32, device)
    rot = 2 * inv_freq.numel()
    axes = 1 if pos.dim() == 1 else pos.shape[0]
    if pos.dim() not in (1, 2) or pos.shape[-1] != tokens:
        raise ValueError(f"pos has shape {tuple(pos.shape)}, expected [axes][{tokens}]")
    if axis is not None:
        _need(axis, "axis", _torch.int32, device)
        if axis.numel() * 2 != rot:
            raise ValueError(f"axis has {axis.numel()} values, inv_freq {inv_freq.numel()}")
    return (pos.data_ptr(), inv_freq.data_ptr(), axis.data_ptr() if axis is not None else None, rot, axes,
            ROPE_ADJACENT if adjacent else 0)


def _out(t, name, like, device):
    """(tensor, row stride): t checked against the rows of `like`, or new contiguous rows."""
    if t is None:
        shape = like.shape
        return like.new_empty(shape), shape[1] * shape[2]
    return t, _rows_like(t, name, like, device)


def _rows_like(t, name, like, device):
    stride = _rows(t, name, device, like.shape[1], like.shape[2])
    if t.shape[0] != like.shape[0]:
        raise ValueError(f"{name} has {t.shape[0]} rows, expected {like.shape[0]}")
    return stride


def rope(x, pos, inv_freq, axis=None, adjacent: bool = False, out=None):
    """x [tokens][heads][head_dim] with its first 2 * len(inv_freq) dimensions
    turned by pos[axis[r]][token] * inv_freq[r] (pair r: dimensions r and
    r + rot/2; adjacent: 2r and 2r + 1).  pos int32 [axes][tokens] (or
    [tokens]), inv_freq float32, axis int32 (None: the first axis for all).
    out may be x."""
    stride = _rows(x, "x", None)
    dev = x.device
    tokens, heads, dim = x.shape
    a = _angles(pos, inv_freq, axis, adjacent, tokens, dev)
    out, out_stride = _out(out, "out", x, dev)
    _launch(dev, "bq_rope", x.data_ptr(), out.data_ptr(), stride, out_stride, tokens, heads, dim, *a)
    return out


def kv_append(cache: KVCache, layer: int, k, v, cu, lens, table, q=None, pos=None, inv_freq=None, axis=None,
              adjacent: bool = False, q_out=None):
    """Writes the rows k, v [total][kv_heads][head_dim] to the cache as the
    last tokens of their sequences (lens counts them), k turned as rope()
    does; with q [total][q_heads][head_dim] also returns q turned (into q_out
    when given).  Without inv_freq nothing turns."""
    dev = cache.device
    k_stride = _rows(k, "k", dev, cache.kv_heads, cache.head_dim)
    v_stride = _rows_like(v, "v", k, dev)
    total = k.shape[0]
    batch, max_pages = _batch(cu, lens, table, dev)
    a = _angles(pos, inv_freq, axis, adjacent, total, dev)
    qp = op = None
    q_stride = out_stride = q_heads = 0
    if q is not None:
        q_stride = _rows(q, "q", dev, None, cache.head_dim)
        if q.shape[0] != total:
            raise ValueError(f"q has {q.shape[0]} rows, k {total}")
        q_out, out_stride = _out(q_out, "q_out", q, dev)
        qp, op, q_heads = q.data_ptr(), q_out.data_ptr(), q.shape[1]
    _launch(dev, "bq_kv_append", cache.desc, _int(layer, "layer"), k.data_ptr(), v.data_ptr(), k_stride, v_stride, qp, op,
            q_stride, out_stride, q_heads, cu.data_ptr(), lens.data_ptr(), table.data_ptr(), batch, max_pages, total, *a)
    return q_out if q is not None else None


def kv_read(cache: KVCache, layer: int, cu, lens, table, total: int):
    """(k, v) fp16 [total][kv_heads][head_dim]: the values held for the last
    cu[b+1] - cu[b] tokens of each sequence; total = cu[-1]."""
    dev = cache.device
    batch, max_pages = _batch(cu, lens, table, dev)
    _int(total, "total")
    k, v = (_torch.empty((total, cache.kv_heads, cache.head_dim), dtype=_torch.float16, device=dev) for _ in range(2))
    _launch(dev, "bq_kv_read", cache.desc, _int(layer, "layer"), k.data_ptr(), v.data_ptr(), cu.data_ptr(), lens.data_ptr(),
            table.data_ptr(), batch, max_pages, total)
    return k, v


def kv_attn(cache: KVCache, layer: int, q, cu, lens, table, scale: Optional[float] = None, causal: bool = True,
            window: int = 0, out=None, workspace=None):
    """Attention of the rows q [total][q_heads][head_dim] over the cache; scale
    defaults to head_dim ** -0.5.  causal: a row sees the tokens up to its own
    position (the rows are the last of their sequence), window > 0: only the
    last `window` of them; else every token held.  workspace: a uint8 tensor,
    zero before its first use and kept for later calls (see
    bq_kv_attn_workspace); allocated here when None."""
    dev = cache.device
    stride = _rows(q, "q", dev, None, cache.head_dim)
    total, heads, dim = q.shape
    batch, max_pages = _batch(cu, lens, table, dev)
    out, out_stride = _out(out, "out", q, dev)
    ws, ws_bytes = None, 0
    if workspace is None:
        ws_bytes = bq_kv_attn_workspace(cache.desc, heads, batch, total)
        workspace = _torch.zeros(ws_bytes, dtype=_torch.uint8, device=dev) if ws_bytes else None
    else:
        _need(workspace, "workspace", _torch.uint8, dev)
        ws_bytes = workspace.numel()
    if workspace is not None:
        ws = workspace.data_ptr()
    _launch(dev, "bq_kv_attn", cache.desc, _int(layer, "layer"), q.data_ptr(), out.data_ptr(), stride, out_stride, heads,
            cu.data_ptr(), lens.data_ptr(), table.data_ptr(), batch, max_pages, total, dim ** -0.5 if scale is None else scale,
            _int(min(window, (1 << 31) - 1), "window"), KV_CAUSAL if causal else 0, ws, ws_bytes)
    return out


def _ints(t, name, device, *shape):
    _need(t, name, _torch.int32, device)
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")


def _page_call(name, cache, table, refs, workspace, before, after):
    """before, after: the pointers and sizes ahead of refs and behind max_pages."""
    dev = cache.device
    _ints(refs, "refs", dev, cache.num_pages)
    rows, max_pages = table.shape
    status = _torch.empty(2, dtype=_torch.int32, device=dev)
    if workspace is None:
        size = _pages_bytes.get((cache.num_pages, rows))
        if size is None:
            size = _pages_bytes[cache.num_pages, rows] = bq_kv_pages_workspace(cache.desc, rows)
        workspace = _torch.empty(size, dtype=_torch.uint8, device=dev)
    else:
        _need(workspace, "workspace", _torch.uint8, dev)
        size = workspace.numel()
    _launch(dev, name, cache.desc, table.data_ptr(), *before, refs.data_ptr(), rows, max_pages, *after,
            status.data_ptr(), workspace.data_ptr(), size)
    return status


def _table(table, device):
    _need(table, "table", _torch.int32, device)
    if table.dim() != 2:
        raise ValueError(f"table has shape {tuple(table.shape)}, expected [rows][max_pages]")
    return table.shape[0]


def kv_fork(cache: KVCache, table, lens, refs, src, dst, workspace=None):
    """Row dst[i] becomes a copy of row src[i]: whole pages shared, a partly
    filled last page copied.  Updates table, lens, refs on the GPU and
    returns status int32 [2] (0 / -1 invalid / pages short; pages copied)."""
    dev = cache.device
    rows = _table(table, dev)
    _ints(lens, "lens", dev, rows)
    n = src.shape[0]
    _ints(src, "src", dev, n)
    _ints(dst, "dst", dev, n)
    return _page_call("bq_kv_fork", cache, table, refs, workspace, (lens.data_ptr(),),
                      (src.data_ptr(), dst.data_ptr(), n))


def kv_resize(cache: KVCache, table, lens, refs, want, workspace=None):
    """Row i gets the length want[i] (-1: as it is): pages are let go or
    taken, a shared page that becomes the partly filled last one is copied.
    Returns status as kv_fork."""
    dev = cache.device
    rows = _table(table, dev)
    _ints(lens, "lens", dev, rows)
    _ints(want, "want", dev, rows)
    return _page_call("bq_kv_resize", cache, table, refs, workspace, (lens.data_ptr(),), (want.data_ptr(),))


def kv_compact(cache: KVCache, table, refs, workspace=None):
    """Moves pages so that those in use have the lowest ids; table and refs
    follow.  Returns status as kv_fork (status[1]: pages moved)."""
    _table(table, cache.device)
    return _page_call("bq_kv_compact", cache, table, refs, workspace, (), ())


def kv_copy_pages(cache: KVCache, src, dst) -> None:
    """Copies pages src[i] to dst[i] over all layers."""
    dev = cache.device
    n = src.shape[0]
    _ints(src, "src", dev, n)
    _ints(dst, "dst", dev, n)
    _launch(dev, "bq_kv_copy_pages", cache.desc, src.data_ptr(), dst.data_ptr(), n)


__all__ = [
    "KV_ATTN_COUNTER_BYTES", "KV_BLOCK", "KV_CAUSAL", "KV_E4M3", "KV_FORMATS", "KV_I8", "KV_PAGE", "KV_POINTS",
    "KVCache", "KVCacheDesc", "ROPE_ADJACENT", "ROPE_MAX_AXES", "bq_kv_append", "bq_kv_attn", "bq_kv_attn_workspace",
    "bq_kv_compact", "bq_kv_copy_pages", "bq_kv_fork", "bq_kv_pages_workspace", "bq_kv_read", "bq_kv_resize",
    "bq_rope", "kv_append", "kv_attn", "kv_compact", "kv_copy_pages", "kv_fork", "kv_read", "kv_resize", "rope",
]
