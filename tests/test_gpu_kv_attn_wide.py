"""The bounds of the tests of many small terms and of scales far apart, for heads of 128, 192 and 256: their kernels hold
the outputs in other registers.

Tolerance: that of test_gpu_kv_attn_units.py, 2^-11 |o| + 2^-10 mass + 2^-25 (scores: sums of up to 256 products, under
2^-12 of a weight each while scores stay below 2^6)."""
import numpy as np
import pytest

import test_gpu_kv_attn_tail as tail
from gpu_helpers import torch_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = torch_mod()
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import bit_quantized_decode_qmv_amd as bq
    bq.load_library()


@pytest.fixture(params=[128, 192, 256])
def D(request, monkeypatch):
    monkeypatch.setattr(tail, "D", request.param)
    return request.param


def inputs(rng, D, n, fmt, first=0.0, block=None, k0=0.0, far=1.0):
    """q[0] = sqrt(D): a token whose K has k[0] = x there scores x higher.  The first token x = `first` and no value, those
    of `block` x = k0 and `far` times the others' values."""
    top = 127 if fmt == "int8" else 448
    k = rng.standard_normal((n, D))
    k[:, 0] = 0
    blocks = -(-n // 16)
    ks, vs = np.full(blocks, 4.5 / top), rng.uniform(0.75, 1.25, blocks) / top
    v = (60 * rng.choice([-1, 1], D) + 25 * rng.standard_normal((n, D))).clip(-127, 127) / 127
    if first:
        k[0] = 0
        k[0, 0], ks[0], v[0] = first, first / top, 0
    if block is not None:
        k[16 * block:16 * block + 16, 0] = k0
        ks[block] = max(ks[block], abs(k0) / top)
        vs[block] *= far
    return tail.pool(rng, {"k": k, "v": v * np.repeat(vs, 16)[:n, None] * top}, {"k": ks, "v": vs}, fmt)


def check(rng, c, table, n, D, rows, **how):
    q = rng.standard_normal((rows, D))
    q[:, 0] = D ** 0.5
    q = q.astype(np.float16)
    ref, mass, _ = tail.reference(c, table, n, q, D ** -0.5, **how)
    tol = 2.0 ** -11 * np.abs(ref) + 2.0 ** -10 * mass + 2.0 ** -25
    for split in (False, True):
        worst = np.max(np.abs(tail.attn(c, table, n, q, split=split, **how) - ref) / tol)
        print(D, rows, how, split, worst, flush=True)
        assert worst <= 1, (rows, how, split, worst)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_weight_on_the_first_token(D, fmt):
    """97% of it, one early block of V 30 times the others, over 30000 tokens."""
    rng = np.random.default_rng(D)
    n = 30000
    c, table = inputs(rng, D, n, fmt, first=np.log(0.97 / 0.03 * n) + 0.5, block=5, far=30.0)
    for rows in (1, 40):
        check(rng, c, table, n, D, rows)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("far", [14, 26])
def test_large_blocks_of_no_weight_or_unseen(D, far, fmt):
    rng = np.random.default_rng(D + far)
    for block, k0, window in ((1, -60, False), (30, -60, False), (8, 0, True)):
        c, table = inputs(rng, D, 500, fmt, block=block, k0=k0, far=2.0 ** far)
        for rows in (1, 20, 64):
            check(rng, c, table, 500, D, rows, window=500 - rows + 1 - 148 if window else 0)
