"""Attention over blocks of V whose scales lie far apart: a block that no row
attends to, or sees, must not cost the others their bits.

Tolerance, with mass = sum p |v| / sum p over what a row sees: the output's
rounding, 2^-11 |o| + 2^-25; the probabilities' rounding to fp16, 2^-11 mass;
scores in fp32 (sums of 64 products, weights of some tokens: 2^-12 of each
weight), 2^-11 mass once more.  Terms below the normal range of fp16 are off by
2^-32 of the unit, which is at most 2^6 times the scale of a term's own block
where no row attends to larger ones: 500 terms lose less than 2^-17 of the
largest value, under 2^-25 + 2^-12 mass here."""
import numpy as np
import pytest

import oracle
from gpu_helpers import torch_mod
from test_gpu_kv_attn_tail import D, attn, pool, reference

pytestmark = pytest.mark.gpu

N = 500


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = torch_mod()
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import bit_quantized_decode_qmv_amd as bq
    bq.load_library()


def inputs(rng, fmt, block, k0, far):
    """One sequence; the tokens of `block` have K's first dimension k0 (0 elsewhere), so that a row with q[0] = 8 scores
    them k0 higher, and V `far` times the others'."""
    top = 127 if fmt == "int8" else 448
    k = rng.standard_normal((N, D))
    k[:, 0] = 0
    blocks = -(-N // 16)
    ks, vs = np.full(blocks, 4.0 / top), rng.uniform(0.75, 1.25, blocks) / top
    k[16 * block:16 * block + 16, 0] = k0
    ks[block] = max(abs(k0), 4) / top
    vs[block] *= far
    v = (60 * rng.choice([-1, 1], D) + 25 * rng.standard_normal((N, D))).clip(-127, 127) / 127
    return pool(rng, {"k": k, "v": v * np.repeat(vs, 16)[:N, None] * top}, {"k": ks, "v": vs}, fmt)


def check(c, table, q, **how):
    ref, mass, _ = reference(c, table, N, q, 0.125, **how)
    tol = 2.0 ** -11 * np.abs(ref) + 2.0 ** -10 * mass + 2.0 ** -25
    for split in (False, True):
        worst = np.max(np.abs(attn(c, table, N, q, split=split, **how) - ref) / tol)
        print(len(q), how, split, worst, flush=True)
        assert worst <= 1, (len(q), how, split, worst)


def queries(rng, rows):
    q = rng.standard_normal((rows, D))
    q[:, 0] = 8
    return q.astype(np.float16)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("far", [14, 20, 26, 40])
@pytest.mark.parametrize("block", [1, 30])
def test_a_large_block_of_no_weight(block, far, fmt):
    """Scores 60 below the others'; on the first page and on one of the last."""
    rng = np.random.default_rng(far + block)
    c, table = inputs(rng, fmt, block, -60, 2.0 ** far)
    for rows in (1, 20, 64):
        check(c, table, queries(rng, rows))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("far", [14, 26, 40])
def test_a_large_block_ahead_of_the_window(far, fmt):
    """In the page that the window of the first row begins in, 4 tokens ahead of it."""
    rng = np.random.default_rng(far)
    c, table = inputs(rng, fmt, 8, 0, 2.0 ** far)
    for rows in (1, 20, 64):
        check(c, table, queries(rng, rows), window=N - rows + 1 - 148)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_a_large_block_that_half_of_the_rows_attend_to(fmt):
    """Scores of its tokens 20 higher for every second row, 20 lower for the others; values 2^10 times the others'."""
    rng = np.random.default_rng(3)
    c, table = inputs(rng, fmt, 9, 20, 2.0 ** 10)
    for rows in (2, 20, 64):
        q = queries(rng, rows)
        q[1::2, 0] = -8
        check(c, table, q)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("spread", [8, 14, 24])
def test_the_winner_comes_from_any_block(spread, fmt):
    """One token takes nearly all of a row's weight, its V's scale anywhere within 2^spread of the largest."""
    rng = np.random.default_rng(spread)
    top = 127 if fmt == "int8" else 448
    signs = rng.choice([-1.0, 1.0], (N, D))
    blocks = -(-N // 16)
    vs = 2.0 ** (10 - rng.uniform(0, spread, blocks)) / top
    v = (60 * rng.choice([-1, 1], D) + 25 * rng.standard_normal((N, D))).clip(-127, 127) / 127
    c, table = pool(rng, {"k": signs, "v": v * np.repeat(vs, 16)[:N, None] * top}, {"k": np.full(blocks, 1.0 / top), "v": vs}, fmt)
    # a token's own signs score 64 under 8 / 8; others' 0 +- 8, a margin of 30 and more for each row taken
    rows = 64 if spread < 24 else 1
    for take in range(3):
        q = np.concatenate([8 * signs[rng.integers(0, N - rows, 1)] for _ in range(rows)]).astype(np.float16)
        check(c, table, q)
        if rows > 1:
            check(c, table, q[:16])


def test_blocks_without_values():
    """Scales that are zero, here and there and on whole pages, beside blocks with a part of the weight."""
    rng = np.random.default_rng(5)
    for fmt in ("int8", "e4m3"):
        c, table = inputs(rng, fmt, 2, 1, 1.0)
        hit = rng.random(c["vs"].shape) < 0.4
        hit[0, table[0, [0, 3]]] = True
        c["vs"][hit] = 0
        for rows in (1, 20, 64):
            check(c, table, queries(rng, rows))
