"""GPU parity of bq_rope against the fp64 oracle.

Tolerance: the result is rounded to fp16 once, 2^-11 |y| (2^-25 below the
normal range); the angle is good to 2^-22 turns (2 pi 2^-22 < 2^-19 rad) and
the hardware sine and cosine to 2^-19, which moves y by at most 2^-17 of the
pair's |x1| + |x2|; the fp32 products by less than that."""
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


def check(y, x, pos, inv, axis, adjacent):
    ref = oracle.rope_f64(x, pos, inv, axis, adjacent)
    rot = 2 * len(inv)
    mass = np.zeros_like(ref)
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if adjacent else (slice(0, rot // 2), slice(rot // 2, rot))
    mass[..., a] = mass[..., b] = np.abs(x[..., a].astype(np.float64)) + np.abs(x[..., b].astype(np.float64))
    tol = 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + 2.0 ** -17 * mass
    worst = np.max(np.abs(y.astype(np.float64) - ref) / tol)
    assert worst <= 1.0, worst


CASES = [  # tokens, heads, D, rot, axes, adjacent
    (1, 1, 64, 64, 1, False), (5, 48, 128, 128, 1, False), (17, 3, 128, 64, 3, False), (33, 8, 256, 128, 3, True),
    (2, 5, 192, 192, 2, False), (7, 2, 80, 32, 1, True), (4099, 2, 64, 48, 3, False), (3, 1, 16, 16, 8, False),
    (6, 4, 128, 0, 1, False),
]


@pytest.mark.parametrize("tokens,heads,D,rot,axes,adjacent", CASES)
def test_rope(tokens, heads, D, rot, axes, adjacent):
    import bit_quantized_decode_qmv_amd as bq
    rng = np.random.default_rng(tokens * 1000 + D + rot)
    x = rng.standard_normal((tokens, heads, D)).astype(np.float16)
    pos = rng.integers(0, 40000, (axes, tokens)).astype(np.int32)
    inv, axis = synth.rope_freqs(rot), rng.integers(0, axes, rot // 2).astype(np.int32)
    y = bq.rope(up(x), up(pos), up(inv), axis=up(axis), adjacent=adjacent).cpu().numpy()
    check(y, x, pos, inv, axis, adjacent)
    # the same bits on a strided view, in place, and on other streams
    torch = torch_mod()
    wide = torch.zeros((tokens, heads * D + 64), dtype=torch.float16, device="cuda:0")
    view = wide[:, 8:8 + heads * D].unflatten(1, (heads, D))
    view.copy_(up(x))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = bq.rope(view, up(pos), up(inv), axis=up(axis), adjacent=adjacent, out=view)
    s.synchronize()
    assert got is view and np.array_equal(view.cpu().numpy(), y)
    assert float(wide[:, :8].abs().max()) == 0 and float(wide[:, 8 + heads * D:].abs().max()) == 0


def test_far_positions():
    """The angle keeps its precision over all of int32; fast pairs are the hard ones."""
    import bit_quantized_decode_qmv_amd as bq
    rng = np.random.default_rng(5)
    x = rng.standard_normal((64, 2, 64)).astype(np.float16)
    pos = np.concatenate([rng.integers(-2 ** 31, 2 ** 31 - 1, 60), [2 ** 31 - 1, -2 ** 31, 2 ** 24 + 1, -1]])[None].astype(np.int32)
    inv = synth.rope_freqs(64)
    check(bq.rope(up(x), up(pos), up(inv)).cpu().numpy(), x, pos, inv, None, False)


def test_axis_out_of_range_is_brought_in():
    import bit_quantized_decode_qmv_amd as bq
    rng = np.random.default_rng(6)
    x = rng.standard_normal((9, 2, 64)).astype(np.float16)
    pos = rng.integers(0, 1000, (2, 9)).astype(np.int32)
    inv = synth.rope_freqs(64)
    axis = rng.integers(-3, 6, 32).astype(np.int32)
    y = bq.rope(up(x), up(pos), up(inv), axis=up(axis)).cpu().numpy()
    check(y, x, pos, inv, np.clip(axis, 0, 1), False)


def test_non_finite_values_stay_in_their_pair():
    import bit_quantized_decode_qmv_amd as bq
    rng = np.random.default_rng(7)
    x = rng.standard_normal((4, 2, 64)).astype(np.float16)
    y0 = bq.rope(up(x), up(np.arange(4)[None], np.int32), up(synth.rope_freqs(64))).cpu().numpy()
    x[1, 0, 5], x[2, 1, 40] = np.inf, np.nan
    y1 = bq.rope(up(x), up(np.arange(4)[None], np.int32), up(synth.rope_freqs(64))).cpu().numpy()
    hit = np.zeros(x.shape, bool)
    hit[1, 0, [5, 37]] = hit[2, 1, [8, 40]] = True
    assert np.array_equal(y0[~hit], y1[~hit]) and not np.isfinite(y1[1, 0, 5]) and np.isnan(y1[2, 1, 40])


def test_empty():
    import bit_quantized_decode_qmv_amd as bq
    torch = torch_mod()
    x = torch.empty((0, 4, 64), dtype=torch.float16, device="cuda:0")
    pos = torch.empty((1, 0), dtype=torch.int32, device="cuda:0")
    assert bq.rope(x, pos, up(synth.rope_freqs(64))).shape == (0, 4, 64)
