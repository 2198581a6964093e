"""bq_kv_read of more rows than a 31-bit count of their 16-byte units."""
import numpy as np
import pytest

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


@pytest.mark.parametrize("D,rows", [(64, 77), (128, 300), (192, 1001), (256, 40), (256, 1 << 26)])
def test_rows_ahead_of_the_first_token_are_zero(D, rows):
    """A sequence of 70 tokens asked for more: the rows ahead of them are zeros, the others theirs, and nothing is
    written past either."""
    import bit_quantized_decode_qmv_amd as bq
    torch = torch_mod()
    gen = torch.Generator(device="cuda:0")
    gen.manual_seed(D)
    cache = bq.KVCache.empty(1, 3, 1, D)
    for t in (cache.k, cache.v):
        t.random_(1, 256, generator=gen)
    cache.k_scales.fill_(0.5)
    cache.v_scales.fill_(0.25)
    table, lens = up([[2, 0]], np.int32), up([70], np.int32)
    k, v = (torch.full((rows + 1, D), 7.0, dtype=torch.float16, device="cuda:0") for _ in range(2))
    cu = up([0, rows], np.int32)
    bq.bq_kv_read(cache.desc, 0, k.data_ptr(), v.data_ptr(), cu.data_ptr(), lens.data_ptr(), table.data_ptr(), 1, 2, rows,
                  torch.cuda.current_stream().cuda_stream)
    held = min(rows, 70)
    want = bq.kv_read(cache, 0, up([0, held], np.int32), lens, table, held)
    for got, w in zip((k, v), want):
        assert bool((got[rows] == 7).all())
        assert torch.equal(got[rows - held:rows], w[:, 0])
        step = 1 << 22
        for at in range(0, rows - held, step):
            assert not bool(got[at:min(at + step, rows - held)].any()), at
    del k, v
    torch.cuda.empty_cache()
