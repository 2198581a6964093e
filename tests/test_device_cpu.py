"""The tensor helpers launch on their tensors' device, whichever is current: tensors that say they are on cuda:1 go
through every helper, and a library that only notes the current device stands in for the built one."""
import types

import pytest

import bit_quantized_decode_qmv_amd as bq

torch = pytest.importorskip("torch")


class Far(torch.Tensor):
    device = torch.device("cuda", 1)
    is_cuda = True


def far(*shape, dtype=torch.float16):
    return torch.zeros(shape, dtype=dtype).as_subclass(Far)


def ints(*shape):
    return far(*shape, dtype=torch.int32)


@pytest.fixture
def calls(monkeypatch):
    """(entry point, device that was current) of each launch; device 0 is current ahead of every call."""
    bq.kv._use_torch()
    state, noted = {"now": 0}, []

    class On:
        def __init__(self, device):
            self.to = torch.device(device).index

        def __enter__(self):
            self.was, state["now"] = state["now"], self.to

        def __exit__(self, *_):
            state["now"] = self.was

    class Library:
        def __getattr__(self, name):
            def entry(*args):
                if "workspace" not in name or args[-1] is None or isinstance(args[-1], int):
                    noted.append((name, state["now"]))
                return 0
            return entry

    empty, zeros = torch.empty, torch.zeros
    for name, make in (("empty", empty), ("zeros", zeros)):
        monkeypatch.setattr(torch, name, lambda *s, make=make, device=None, **kw: make(*s, **kw).as_subclass(Far))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: state["now"])
    monkeypatch.setattr(torch.cuda, "device", On)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: types.SimpleNamespace(cuda_stream=0))
    monkeypatch.setattr(bq.kv, "_device_now", lambda: state["now"], raising=False)
    monkeypatch.setattr(bq.kv, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(bq, "_lib", Library())
    return types.SimpleNamespace(state=state, noted=noted)


def run(calls, names, call):
    calls.noted.clear()
    call()
    assert [n for n, _ in calls.noted] == names
    assert all(d == 1 for _, d in calls.noted), calls.noted
    assert calls.state["now"] == 0


def test_products(calls):
    x, s, b = far(2, 128), far(8, 2), far(8, 2)
    w, t5 = ints(8, 8), far(8, 26, dtype=torch.uint8)
    run(calls, ["bq_qmv"], lambda: bq.qmv(x, w, s, b, 2, 64))
    run(calls, ["bq_qmv_wide"], lambda: bq.qmv_wide(x, w, s, b, 2, 64))
    run(calls, ["bq_qmv_sym"], lambda: bq.qmv_sym(x, w, s, 2, 64))
    run(calls, ["bq_t5_qmv"], lambda: bq.t5_qmv(x, t5, s, 64))
    run(calls, ["bq_t5_qmm"], lambda: bq.t5_qmm(x, t5, s, 64))
    run(calls, ["bq_qmm"], lambda: bq.qmm(x, w, s, 2, 64))
    run(calls, ["bq_t5_qmm_ws"], lambda: bq.t5_qmm_ws(x, t5, s, 64))
    run(calls, ["bq_qmm_ws"], lambda: bq.qmm_ws(x, w, s, 2, 64))
    run(calls, ["bq_dequant"], lambda: bq.dequant(w, s, b, 2, 64, 128))
    run(calls, ["bq_sym_check"], lambda: bq.sym_check(s, b, 2, 64))
    run(calls, ["bq_t5_repack"], lambda: bq.t5_repack(w, 2, 64, 128))
    qw = bq.QuantizedWeight(w, s, None, 2, 64)
    run(calls, ["bq_linear"], lambda: bq.linear(x, qw))
    run(calls, ["bq_linear_ws"], lambda: bq.linear(x, qw, workspace="auto"))
    run(calls, ["bq_spec_decode_verify"], lambda: bq.spec_decode_verify(far(2, 4, 50), ints(2, 3)))


def test_cache_calls(calls):
    codes = lambda: far(1, 3, 2, 64 * 64, dtype=torch.uint8)
    scales = lambda: far(1, 3, 2, 4, dtype=torch.float32)
    cache = bq.KVCache(codes(), codes(), scales(), scales())
    cu, lens, table = ints(3), ints(2), ints(2, 4)
    inv, pos = far(32, dtype=torch.float32), ints(1, 5)
    rows = lambda heads: far(5, heads, 64)
    run(calls, ["bq_rope"], lambda: bq.rope(rows(4), pos, inv, out=rows(4)))
    run(calls, ["bq_kv_append"], lambda: bq.kv_append(cache, 0, rows(2), rows(2), cu, lens, table, q=rows(4), pos=pos,
                                                       inv_freq=inv, q_out=rows(4)))
    run(calls, ["bq_kv_read"], lambda: bq.kv_read(cache, 0, cu, lens, table, 5))
    ws = far(1 << 16, dtype=torch.uint8)
    run(calls, ["bq_kv_attn"], lambda: bq.kv_attn(cache, 0, rows(4), cu, lens, table, out=rows(4), workspace=ws))
    run(calls, ["bq_kv_fork"], lambda: bq.kv_fork(cache, table, lens, ints(3), ints(1), ints(1), workspace=ws))
    run(calls, ["bq_kv_resize"], lambda: bq.kv_resize(cache, table, lens, ints(3), ints(2), workspace=ws))
    run(calls, ["bq_kv_compact"], lambda: bq.kv_compact(cache, table, ints(3), workspace=ws))
    run(calls, ["bq_kv_copy_pages"], lambda: bq.kv_copy_pages(cache, ints(2), ints(2)))


def test_the_device_is_put_back_after_an_error(calls, monkeypatch):
    class Broken:
        def bq_strerror(self, st):
            return b"as asked"

        def __getattr__(self, name):
            return lambda *args: -4
    monkeypatch.setattr(bq, "_lib", Broken())
    with pytest.raises(bq.BQError):
        bq.qmv(far(2, 128), ints(8, 8), far(8, 2), far(8, 2), 2, 64)
    with pytest.raises(bq.BQError):
        bq.rope(far(5, 4, 64), ints(1, 5), far(32, dtype=torch.float32), out=far(5, 4, 64))
    assert calls.state["now"] == 0
