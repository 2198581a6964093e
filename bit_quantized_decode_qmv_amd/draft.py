"""Drafted tokens and what a model says of them: the binding of the
``bq_logprobs`` and ``bq_tree_*`` entry points of ``include/bq.h`` and their
tensor helpers (``logprobs``, ``tree_plan``, ``tree_accept``).

A step of decoding with a tree: the drafting model's alternatives
(``logprobs``) make the tree, ``tree_plan`` its masks and positions; its rows
join the cache (``kv_append_norm``) and attend (``kv_attn_tree``); the target
model's most likely tokens (``logprobs`` again) choose a path (``tree_accept``),
whose keys and values stay (``kv_keep``, ``kv_resize``).
"""
from __future__ import annotations

import ctypes
import sys

from . import kv as _kv

LOGPROBS_MAX_TOP = 64
LOGPROBS_MAX_COUNT = 1024
LOGPROBS_COUNTER_BYTES = 65536

DRAFT_POINTS = ("bq_tree_plan", "bq_tree_accept", "bq_logprobs_workspace", "bq_logprobs")


def declare(lib) -> None:
    """Argument types of the entry points."""
    vp, i, ll, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_size_t
    types = {
        "bq_tree_plan": [vp, vp, vp, i, i, i, i, vp, vp, vp],
        "bq_tree_accept": [vp, vp, vp, vp, vp, i, i, i, vp, vp, vp, vp, vp],
        "bq_logprobs_workspace": [i, i, i, i, ctypes.POINTER(sz)],
        "bq_logprobs": [vp, i, ll, i, i, vp, i, vp, vp, i, vp, vp, vp, sz, vp],
    }
    for name, args in types.items():
        fn = getattr(lib, name)
        fn.restype = ctypes.c_int
        fn.argtypes = args


_bq = sys.modules[__package__]

bq_tree_plan = _kv._c_entry("bq_tree_plan")
bq_tree_accept = _kv._c_entry("bq_tree_accept")
bq_logprobs = _kv._c_entry("bq_logprobs")


def bq_logprobs_workspace(rows, V, logits_dtype, top):
    """Workspace bytes bq_logprobs wants to share rows among workgroups (host only)."""
    n = ctypes.c_size_t(0)
    _kv._call("bq_logprobs_workspace", rows, V, logits_dtype, top, ctypes.byref(n))
    return n.value


def _gpu(t, name):
    """The tensor's device, which has to be a GPU."""
    torch = _kv._torch or _kv._use_torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU, got {t.device}")
    return t.device


def _sequences(parent, cu, lens):
    """(device, batch, total)"""
    dev = _gpu(parent, "parent")
    _kv._need(lens, "lens", _kv._torch.int32, dev)
    if parent.dim() != 1 or lens.dim() != 1:
        raise ValueError(f"expected parent [total], lens [batch]; got {tuple(parent.shape)}, {tuple(lens.shape)}")
    total, batch = parent.shape[0], lens.shape[0]
    _kv._int(total, "total")
    _kv._ints(parent, "parent", dev, total)
    _kv._ints(cu, "cu", dev, batch + 1)
    return dev, batch, total


def tree_plan(parent, cu, lens, words: int = 1, window: int = 0):
    """(mask int64 [total][words], pos int32 [total]) of the trees that parent
    int32 [total] gives (a row's parent in its sequence, -1: the context; cu
    and lens as in kv_attn): the rows that each row sees, itself and those
    above it (window > 0: the nearest `window`), and its position."""
    dev, batch, total = _sequences(parent, cu, lens)
    torch = _kv._torch
    if not 1 <= words <= _kv.TREE_MAX_WORDS:
        raise ValueError(f"words = {words}, expected 1 .. {_kv.TREE_MAX_WORDS}")
    mask = torch.empty((total, words), dtype=torch.int64, device=dev)
    pos = torch.empty_like(parent)
    _kv._launch(dev, "bq_tree_plan", parent.data_ptr(), cu.data_ptr(), lens.data_ptr(), batch, total, words,
                _kv._window(window, "window"), mask.data_ptr(), pos.data_ptr())
    return mask, pos


def tree_accept(target, token, parent, cu, lens, max_path: int):
    """The path that the target tokens take through each tree from its row 0
    on: (path [batch][max_path], kept [batch], next_token [batch], want
    [batch]), int32: the rows taken (-1 behind them), their number, the token
    behind the last, and the sequence's length with these rows alone.
    target, token, parent: int32 [total], target[row] the token that the target
    model has after the row, token[row] the row's own."""
    dev, batch, total = _sequences(parent, cu, lens)
    _kv._ints(target, "target", dev, total)
    _kv._ints(token, "token", dev, total)
    if not 1 <= max_path <= _kv.TREE_MAX_ROWS:
        raise ValueError(f"max_path = {max_path}, expected 1 .. {_kv.TREE_MAX_ROWS}")
    path = parent.new_empty((batch, max_path))
    told = parent.new_empty((3, batch))
    at = told.data_ptr()
    _kv._launch(dev, "bq_tree_accept", target.data_ptr(), token.data_ptr(), parent.data_ptr(), cu.data_ptr(),
                lens.data_ptr(), batch, total, max_path, path.data_ptr(), at, at + 4 * batch, at + 8 * batch)
    return path, *told.unbind()


def logprobs(logits, tokens=None, top: int = 0, entropy: bool = False, workspace=None):
    """Log probabilities under softmax(logits), logits [rows][V] float16 or
    float32 with any row stride: (logprob float32 of the given tokens int32
    [rows] or [rows][count], in their shape; entropy float32 [rows]; top_tokens
    int32 [rows][top]; top_logprobs float32 [rows][top]), None for what is not
    asked for.  Equal values: the lowest token first.  workspace: a uint8
    tensor, zero before its first use and kept for later calls (see
    bq_logprobs_workspace; one of kv_attn will do); allocated here when None
    and wanted."""
    dev = _gpu(logits, "logits")
    torch = _kv._torch
    if logits.dtype not in (torch.float16, torch.float32):
        raise TypeError(f"logits must be float16 or float32, got {logits.dtype}")
    if logits.dim() != 2:
        raise ValueError(f"logits have shape {tuple(logits.shape)}, expected [rows][V]")
    rows, V = logits.shape
    _kv._int(rows, "rows")
    _kv._int(V, "V")
    stride = logits.stride(0) if rows > 1 else V
    if V > 1 and logits.stride(1) != 1 or stride < V:
        raise ValueError("logits must hold each row contiguously, rows that do not overlap")
    dtype = _bq.DTYPE_F16 if logits.dtype is torch.float16 else _bq.DTYPE_F32
    count, logprob, entropies, top_tokens, top_logprobs = 0, None, None, None, None
    if tokens is not None:
        _gpu(tokens, "tokens")
        if tokens.dim() not in (1, 2):
            raise ValueError(f"tokens have shape {tuple(tokens.shape)}, expected [{rows}] or [{rows}][count]")
        count = 1 if tokens.dim() == 1 else _kv._int(tokens.shape[1], "count")
        _kv._ints(tokens, "tokens", dev, *((rows,) if tokens.dim() == 1 else (rows, count)))
        logprob = torch.empty(tokens.shape, dtype=torch.float32, device=dev)
    if entropy:
        entropies = torch.empty(rows, dtype=torch.float32, device=dev)
    if not 0 <= top <= LOGPROBS_MAX_TOP:
        raise ValueError(f"top = {top}, expected 0 .. {LOGPROBS_MAX_TOP}")
    if top:
        top_tokens = torch.empty((rows, top), dtype=torch.int32, device=dev)
        top_logprobs = torch.empty((rows, top), dtype=torch.float32, device=dev)
    if not count and not entropy and not top:
        raise ValueError("nothing is asked for: give tokens, top or entropy")
    ws, ws_bytes = None, 0
    if workspace is None:
        ws_bytes = bq_logprobs_workspace(rows, V, dtype, top)
        if ws_bytes:
            workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
            workspace[:LOGPROBS_COUNTER_BYTES].zero_()
    else:
        _kv._need(workspace, "workspace", torch.uint8, dev)
        ws_bytes = workspace.numel()
    if workspace is not None:
        ws = workspace.data_ptr()
    _kv._launch(dev, "bq_logprobs", logits.data_ptr(), dtype, stride, rows, V, tokens.data_ptr() if count else None, count,
                logprob.data_ptr() if count else None, entropies.data_ptr() if entropy else None, top,
                top_tokens.data_ptr() if top else None, top_logprobs.data_ptr() if top else None, ws, ws_bytes)
    return logprob, entropies, top_tokens, top_logprobs


__all__ = [
    "DRAFT_POINTS", "LOGPROBS_COUNTER_BYTES", "LOGPROBS_MAX_COUNT", "LOGPROBS_MAX_TOP", "bq_logprobs",
    "bq_logprobs_workspace", "bq_tree_accept", "bq_tree_plan", "logprobs", "tree_accept", "tree_plan",
]
