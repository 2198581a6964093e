"""Norms where the reciprocal root, or its product with a weight, is at the ends of fp32's range: an eps below its normal
numbers, weights of any size beside values of 0.  Tolerances: those of the tests of the norms."""
import numpy as np
import pytest

import oracle
import synth
from gpu_helpers import torch_mod
from kv_helpers import cu_of, download_cache, up, upload_cache
from test_gpu_norm import check, check_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = torch_mod()
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import bit_quantized_decode_qmv_amd as bq
    bq.load_library()


def both(x, w, eps, D):
    """Rows x [tokens][1][D] normed alone, and on the way into a cache."""
    import bit_quantized_decode_qmv_amd as bq
    n = x.shape[0]
    pos, inv = np.zeros((1, n), np.int32), synth.rope_freqs(0)
    y = bq.norm_rope(up(x), up(w), eps).cpu().numpy()
    check(y, x, w, eps, pos, inv, None, False)
    rng = np.random.default_rng(n)
    for fmt in ("int8", "e4m3"):
        table, pages = synth.make_kv_table(rng, [n])
        before = synth.make_kv_pool(rng, 2, pages, 1, D, fmt)
        cache, cu = upload_cache(before), cu_of([n])
        out = bq.kv_append_norm(cache, 1, up(x), up(x), up(cu), up([n], np.int32), up(table), q=up(x), k_weight=up(w), q_weight=up(w), eps=eps)
        assert np.array_equal(out.cpu().numpy(), y)
        z = oracle.norm_f64(x, w, eps)
        check_cache(download_cache(cache), before, fmt, 1, table, [0], [n], cu, z, x.astype(np.float64), 2.0 ** -18 * float(np.abs(z).max()))
    return y


@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("eps", [1e-6, 2.0 ** -126, 2.0 ** -127, 1e-40, 2.0 ** -149])
def test_rows_of_zeros(D, eps):
    """0 / sqrt(eps) is 0 for any eps above 0; a row that holds anything is far above it."""
    x = np.zeros((20, 1, D), np.float16)
    x[5, 0, 3] = 2.0 ** -24
    x[6] = np.random.default_rng(D).standard_normal((1, D))
    y = both(x, np.linspace(0.5, 2, D).astype(np.float32), eps, D)
    assert not y[:5].any() and not y[7:].any()


@pytest.mark.parametrize("D", [64, 128, 192, 256])
def test_large_weights_beside_zeros(D):
    """A weight that takes the reciprocal root of a small row past fp32's range: where the row is 0, so is the result."""
    x = np.full((20, 1, D), 2.0 ** -24, np.float16)
    x[3] = 6e-5
    x[:, :, :4] = 0
    w = np.linspace(0.5, 2, D).astype(np.float32)
    w[:4] = 1e32, -3e38, 1e36, 2.0 ** 127
    both(x, w, 0.0, D)
    both(x, w, 1e-38, D)
