"""Attention with its weight spread over a long context: the outputs are
averages, far smaller than the values, and what does not average out shows.

Tolerance, as the root mean square of the error over that of the output.  The
output's rounding to fp16 and the rounding of a probability to fp16 (many
rows) are each uniform within half of a last place, 2^-11 of values spread over
a binade: 2^-11 / sqrt(3) * 0.72 = 2.0e-4 of it, and probabilities of
independent V leave 2.0e-4 of the output as well.  Together 2.9e-4 for many
rows; 2.0e-4 for few, whose probabilities keep 22 bits.  Sums in fp32 of terms of one sign
lose at most 2^-24 of a 4096-token run's total at each of its 256 additions,
randomly: 16 * 2^-24 of 128 times the weight, where the run's own output is 36
/ sqrt(4096) = 0.56 of it: 2.2e-4 at the most, a third of that where roundings
are uniform.  Limits: 3.2e-4 for many rows and 2.4e-4 for few."""
import numpy as np
import pytest

import synth
from gpu_helpers import torch_mod
from kv_helpers import up

pytestmark = pytest.mark.gpu

D = 64


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = torch_mod()
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import bit_quantized_decode_qmv_amd as bq
    bq.load_library()


@pytest.mark.parametrize("n,rows,limit", [(131072, 64, 3.2e-4), (1 << 20, 8, 2.4e-4)])
def test_even_weights(n, rows, limit):
    """`rows` query heads of one token (up to 16: few rows; more: many) over n tokens, without a workspace: one workgroup
    takes them all."""
    import bit_quantized_decode_qmv_amd as bq
    torch = torch_mod()
    gen = torch.Generator(device="cuda:0")
    gen.manual_seed(n)
    rng = np.random.default_rng(n)
    table, pages = synth.make_kv_table(rng, [n])
    # all blocks alike: any order of a page's bytes would do, and the 64-bit form takes them in the one below
    k, v = (((torch.randn((1, pages, 1, 64 * D), generator=gen, device="cuda:0") * 36).round().clamp(-127, 127) + 128)
            .to(torch.uint8) for _ in range(2))
    scales = torch.full((1, pages, 1, 4), 1 / 36, device="cuda:0")
    cache = bq.KVCache(k, v, scales, scales.clone(), "int8")
    q = (torch.randn((1, rows, D), generator=gen, device="cuda:0") * 0.1).half()
    none = torch.zeros(0, dtype=torch.uint8, device="cuda:0")
    out = bq.kv_attn(cache, 0, q, up([0, 1], np.int32), up([n], np.int32), up(table), workspace=none)[0].double()
    ids = up(table[0, :n // 64]).long()
    # K [i][c = 0][g][t][j]: token 16i + t, dim 16g + j; V [n][g][d][i][j]: token 16i + 4g + j, dim 16n + d
    kk = (k[0, ids, 0].view(-1, 4, 4, 16, 16).permute(0, 1, 3, 2, 4).reshape(n, D).double() - 128) / 36
    vv = (v[0, ids, 0].view(-1, 4, 4, 16, 4, 4).permute(0, 4, 2, 5, 1, 3).reshape(n, D).double() - 128) / 36
    ref = torch.softmax(q[0].double() @ kk.T.contiguous() * D ** -0.5, 1) @ vv
    err = float((out - ref).square().mean().sqrt() / ref.square().mean().sqrt())
    print(n, rows, "rms", err, flush=True)
    assert err <= limit, err
