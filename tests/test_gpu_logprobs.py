"""GPU parity of bq_logprobs against the fp64 oracle.

Tolerance.  A term 2^y, y = x log2(e) - B, carries 2^-24 |y| (rounding of y),
2^-26 |y| (of log2(e)) and 2^-23 (the hardware's exponential) of itself; under
p the mean |y| is at most log2(V) + 1.  A lane adds at most V / 1024 + 16
terms one after the other into one of four sums, each addition off by 2^-24 of
the sum, then some 16 partial sums.  So log s is within
2^-24 (V / 1024 + 96), and a log probability within that, 2^-23 of itself
and of log s <= 20, and 2^-24 of x - m.  The entropy's second sum is of terms
|y| times as large and its error goes by the mean |y|: the first bound times
2 + 2 log(V)."""
import numpy as np
import pytest

import oracle
import synth
from gpu_helpers import torch_mod
from kv_helpers import up

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = torch_mod()
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import bit_quantized_decode_qmv_amd as bq
    bq.load_library()


def close(got, want, tol):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)])
    if fine.any():
        worst = np.max(np.abs(got[fine] - want[fine]) / tol[fine])
        assert worst <= 1, worst


def check(x, tokens, top, got):
    lp, ent, tt, tl = (None if t is None else t.cpu().numpy() for t in got)
    V = x.shape[1]
    base = 2.0 ** -24 * (V / 1024 + 96)
    for r in range(x.shape[0]):
        given, entropy, order, values = oracle.logprobs_f64(x[r], tokens[r] if tokens is not None else [], top)
        bound = lambda v: base + 2.0 ** -23 * (2 * np.abs(np.nan_to_num(v, posinf=0, neginf=0)) + 20)
        if lp is not None:
            close(lp[r], given, bound(given))
        if ent is not None:
            close(ent[r:r + 1], [entropy], np.array([base * (2 + 2 * np.log(V))]))
        if top:
            assert tt[r].tolist() == order.tolist(), r
            close(tl[r], values, bound(values))


def run(x, tokens=None, top=0, entropy=True, workspace=None):
    import bit_quantized_decode_qmv_amd as bq
    got = bq.logprobs(up(x), None if tokens is None else up(tokens, np.int32), top, entropy, workspace)
    check(x, tokens, top, got)
    return got


@pytest.mark.parametrize("dtype", [np.float16, np.float32])
@pytest.mark.parametrize("rows,V,count,top", [
    (1, 1, 1, 1), (3, 2, 2, 5), (2, 7, 1, 7), (5, 63, 0, 64), (4, 64, 1, 64), (3, 65, 3, 10), (7, 1000, 1, 20), (2, 4097, 5, 64),
    (3, 8191, 1, 1), (2, 32000, 1, 20), (300, 1003, 1, 3), (1100, 77, 1, 2), (2, 151936, 1024, 5), (1, 300001, 1, 64),
])
def test_logprobs(dtype, rows, V, count, top):
    rng = np.random.default_rng(rows * 1000 + V)
    x = (rng.standard_normal((rows, V)) * 3).astype(dtype)
    x[rng.integers(0, rows, 3), rng.integers(0, V, 3)] += 9
    tokens = rng.integers(0, V, (rows, count)) if count else None
    a = run(x, tokens, top)
    b = run(x, tokens, top, entropy=False)
    for p, q in zip(a, b):
        if p is not None and q is not None:
            assert torch_mod().equal(p, q)
    if tokens is not None:
        run(x, tokens, 0, entropy=False)
    run(x, None, 0)


def test_equal_values_go_by_the_lowest_token():
    rng = np.random.default_rng(1)
    for dtype in (np.float16, np.float32):
        run(np.zeros((3, 9000), dtype), top=64)
        run(np.full((2, 40000), -7.5, dtype), [[0]] * 2, top=20)
        run(rng.integers(0, 3, (4, 30000)).astype(dtype), top=64)
        x = np.zeros((2, 5000), dtype)
        x[0, ::2] = -0.0                               # equal to 0
        x[1, 1::3] = -0.0
        run(x, top=10)


@pytest.mark.parametrize("dtype", [np.float16, np.float32])
def test_rising_and_falling_rows(dtype):
    """Rows in which every value, or none after the first ones, is among the largest so far."""
    up_ = np.linspace(-20, 20, 60000).astype(dtype)
    saw = np.tile(np.linspace(-5, 5, 700), 86)[:60000].astype(dtype)
    run(np.stack([up_, up_[::-1], saw, -saw]), [[0, 59999, 30000]] * 4, top=64)


@pytest.mark.parametrize("top", [1, 30, 64])
def test_floors_between_equal_values(top):
    """Few values over a long row, the largest of them rare, at its ends, in the middle: which of the equal ones are
    among the largest is decided by tokens that other waves and parts hold."""
    rng = np.random.default_rng(10)
    for n in (3, 40, 200):
        x = rng.integers(0, 2, (6, 90000)).astype(np.float16)
        x[0, -n:] = 5
        x[1, :n] = 5
        x[2, 45000 - n:45000 + n] = 5
        x[3, rng.integers(0, 90000, n)] = 5
        x[4, ::max(1, 90000 // n)] = 5
        x[5, 8192 * np.arange(1, 10)] = 5
        for rows in (x, x[:, 1:], x[:, :20000].copy()):
            run(np.ascontiguousarray(rows), top=top)


@pytest.mark.parametrize("top", [1, 20, 64])
@pytest.mark.parametrize("dtype", [np.float16, np.float32])
def test_whole_rows_of_one_workgroup(dtype, top):
    """Rows that no other workgroup shares: what has to pass rises along the row, from one pass over it to the next."""
    import bit_quantized_decode_qmv_amd as bq
    torch = torch_mod()
    rng = np.random.default_rng(12)
    V = 151 * 1024 + 3
    x = (rng.standard_normal((8, V)) * 2.5).astype(dtype)
    x[1] = np.linspace(-9, 9, V)
    x[2] = x[1, ::-1]
    x[3, -64:] += 20                                   # the largest at the end
    x[4, 5::8192] += 20                                # all of them one thread's
    x[5] = np.arange(V) // 8192                        # each pass above the last
    x[6] = np.sort(x[6])[::-1]
    x[7, :100000] = -np.inf
    run(x, rng.integers(0, V, (8, 1)), top, workspace=torch.zeros(bq.LOGPROBS_COUNTER_BYTES, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("dtype", [np.float16, np.float32])
def test_masked_infinite_and_missing_values(dtype):
    rng = np.random.default_rng(2)
    V = 20011
    x = (rng.standard_normal((12, V)) * 2).astype(dtype)
    x[0, 100:] = -np.inf                               # a masked tail
    x[1, :-1] = -np.inf                                # all but the last
    x[2] = -np.inf                                     # nothing left
    x[3, 17] = np.nan
    x[4, [5, 19000]] = np.nan, np.inf
    x[5, 9999] = np.inf
    x[6, :] = -np.inf
    x[6, 3] = -65504 if dtype == np.float16 else -3e38  # the lowest value alone
    x[7, :] = -65504 if dtype == np.float16 else -3.4028235e38
    x[8, :] = 65504 if dtype == np.float16 else 3.4028235e38
    x[9, 1::2] = -np.inf
    x[10, :] = np.nan
    x[11, 50:] = -65504                                # masked by the lowest fp16
    tokens = np.tile([0, 17, V - 1, V, -1, 2 ** 31 - 1, -2 ** 31], (12, 1))
    run(x, tokens, top=64)


def test_far_values():
    """Values far from 0, whose differences are small: B's rounding is taken out again."""
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((4, 5000)) + np.array([[30000.0], [-30000.0], [1000.0], [1e6]])).astype(np.float32)
    run(x, [[1, 2]] * 4, top=5)


@pytest.mark.parametrize("dtype", [np.float16, np.float32])
def test_strides_and_starts(dtype):
    """Rows that start anywhere: what lies beside them, NaN here, is not looked at."""
    import bit_quantized_decode_qmv_amd as bq
    torch = torch_mod()
    rng = np.random.default_rng(4)
    for V, stride, start in ((1000, 1001, 1), (777, 1024, 3), (64, 71, 5), (1, 3, 1), (9000, 9007, 7)):
        x = (rng.standard_normal((5, V)) * 3).astype(dtype)
        wide = torch.full((6 * stride + 16,), float("nan"), dtype=up(x).dtype, device="cuda:0")
        view = wide[start:start + 5 * stride].view(5, stride)[:, :V]
        view.copy_(up(x))
        tokens = rng.integers(0, V, (5, 2))
        check(x, tokens, min(V, 9), bq.logprobs(view, up(tokens, np.int32), min(V, 9), True))


def test_tokens_of_one_dimension_and_top_one_as_the_verification_takes_it():
    import bit_quantized_decode_qmv_amd as bq
    torch = torch_mod()
    s = synth.make_spec_inputs(3, 4, 2000, seed=5)
    logits = up(s.logits)
    lp, _, tt, _ = bq.logprobs(logits.view(15, 2000), up(s.planted.ravel(), np.int32), top=1)
    assert lp.shape == (15,)
    _, _, target = bq.spec_decode_verify(logits, up(s.draft))
    assert torch.equal(tt.view(3, 5), target)


@pytest.mark.parametrize("rows,V", [(2, 100000), (40, 60000)])
def test_workspaces(rows, V):
    """None at all, too small a one, one of the attention's: the same tokens, values within the tolerance; the same bits
    on every call; the counters are zero again."""
    import bit_quantized_decode_qmv_amd as bq
    torch = torch_mod()
    rng = np.random.default_rng(6)
    x = (rng.standard_normal((rows, V)) * 3).astype(np.float16)
    tokens = rng.integers(0, V, (rows, 1))
    need = bq.bq_logprobs_workspace(rows, V, bq.DTYPE_F16, 20)
    assert need > bq.LOGPROBS_COUNTER_BYTES
    for size in (0, bq.LOGPROBS_COUNTER_BYTES, bq.LOGPROBS_COUNTER_BYTES + (need - bq.LOGPROBS_COUNTER_BYTES) // 3, need, 32 << 20):
        ws = torch.zeros(size, dtype=torch.uint8, device="cuda:0")
        if size > bq.LOGPROBS_COUNTER_BYTES:
            ws[bq.LOGPROBS_COUNTER_BYTES:] = 255               # contents of the rest do not matter
        a, b = run(x, tokens, 20, workspace=ws), run(x, tokens, 20, workspace=ws)
        assert all(torch.equal(p, q) for p, q in zip(a, b))
        assert size == 0 or int(ws[:bq.LOGPROBS_COUNTER_BYTES].max()) == 0


def test_two_streams():
    import bit_quantized_decode_qmv_amd as bq
    torch = torch_mod()
    rng = np.random.default_rng(7)
    x = [up((rng.standard_normal((3, 150000)) * 3).astype(np.float16)) for _ in range(2)]
    want = [bq.logprobs(t, None, 20, True) for t in x]
    streams, ws = [torch.cuda.Stream() for _ in x], [torch.zeros(1 << 20, dtype=torch.uint8, device="cuda:0") for _ in x]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(bq.logprobs(x[i], None, 20, True, ws[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g[1:], want[i][1:]))


def test_graph():
    import bit_quantized_decode_qmv_amd as bq
    torch = torch_mod()
    rng = np.random.default_rng(8)
    x = up(np.zeros((4, 50000), np.float16))
    tokens = up(np.zeros((4, 2)), np.int32)
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda:0")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = bq.logprobs(x, tokens, 10, True, ws)
    for _ in range(4):
        x.copy_(up((rng.standard_normal((4, 50000)) * 3).astype(np.float16)))
        tokens.copy_(up(rng.integers(0, 50000, (4, 2)), np.int32))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        eager = bq.logprobs(x, tokens, 10, True, ws)
        assert all(torch.equal(a, b) for a, b in zip(out, eager))


def test_rows_past_32_bits():
    """2.6 G logits: the last rows' offsets, in values, do not fit 32 bits."""
    import bit_quantized_decode_qmv_amd as bq
    torch = torch_mod()
    rows, V = 17500, 151936
    x = torch.zeros((rows, V), dtype=torch.float16, device="cuda:0")
    assert x.numel() > 2 ** 31
    rng = np.random.default_rng(9)
    last = (rng.standard_normal((3, V)) * 3).astype(np.float16)
    x[-3:] = up(last)
    got = bq.logprobs(x, up(np.full((rows, 1), 77), np.int32), 5, True)
    check(last, np.full((3, 1), 77), 5, [t[-3:] for t in got])
    assert got[2][0].tolist() == [0, 1, 2, 3, 4] and abs(float(got[1][0]) - np.log(V)) < 1e-3


def test_empty_and_refusals():
    import bit_quantized_decode_qmv_amd as bq
    torch = torch_mod()
    x = torch.zeros((2, 9), dtype=torch.float16, device="cuda:0")
    t = up([1, 2], np.int32)
    lp, ent, tt, tl = bq.logprobs(x[:0], t[:0], 3, True)
    assert lp.shape == (0,) and ent.shape == (0,) and tt.shape == tl.shape == (0, 3)
    for bad in (dict(logits=x.double()), dict(logits=x[0]), dict(logits=x.t()), dict(logits=x[:, ::2]), dict(logits=x[:1].expand(2, 9)),
                dict(tokens=t.long()), dict(tokens=t[:1]), dict(tokens=t[None, None]), dict(tokens=t.cpu()), dict(tokens=[1, 2]), dict(top=65), dict(top=-1),
                dict(tokens=None, top=0, entropy=False), dict(workspace=x), dict(logits=x[:, :0])):
        with pytest.raises((ValueError, TypeError, bq.BQError)):
            bq.logprobs(**{**dict(logits=x, tokens=t, top=2, entropy=True), **bad})
