"""Attention whose output is the sum of many small probabilities: the first
token holds most of the weight and has no value, so what is left of the others
is the result.

Tolerance, with mass = sum p |v| / sum p: the output's own rounding, 2^-11
|o| <= 2^-11 mass, and the rounding of the probabilities to fp16, 2^-11 of
each.  Below the normal range of fp16 a term is off by up to half a step, to
either side: steps of 2^-24 under a factor of 2^7 are 2^-31 of the largest
weight times the largest scale of V.  The smallest weights here are near 2^-22
of the largest and V's scales up to 2^5 apart (2^6 with the unit's power of
two), so a term keeps at least three bits, and the sum over tens of thousands
of terms averages their errors to far less than 2^-12.  Together 2^-10 mass."""
import numpy as np
import pytest

import oracle
import synth
from gpu_helpers import torch_mod
from kv_helpers import up, upload_cache

pytestmark = pytest.mark.gpu

D = 64


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = torch_mod()
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import bit_quantized_decode_qmv_amd as bq
    bq.load_library()


def pool(rng, values, scales, fmt):
    """(cache, table) of one sequence of one head that holds the values [n][D] (a dict of k and v) under the scales of
    its blocks [n / 16]."""
    n = len(values["k"])
    table, pages = synth.make_kv_table(rng, [n])
    ids = table[0, :-(-n // 64)]
    c = {"format": fmt}
    for w in ("k", "v"):
        per = np.zeros(4 * len(ids))
        per[:len(scales[w])] = scales[w]
        x = np.zeros((64 * len(ids), D))
        x[:n] = values[w]
        codes = oracle.kv_encode(x / np.repeat(np.where(per > 0, per, 1), 16)[:, None], fmt)
        c[w] = np.full((1, pages, 1, 64 * D), 128 if fmt == "int8" else 0, np.uint8)
        page = np.empty((len(ids), 64 * D), np.uint8)
        page[:, oracle.kv_places(w, D).ravel()] = codes.reshape(len(ids), -1)
        c[w][0, ids, 0] = page
        c[w + "s"] = np.zeros((1, pages, 1, 4), np.float32)
        c[w + "s"][0, ids, 0] = per.reshape(-1, 4)
    return c, table


def reference(c, table, n, q, scale, causal=True, window=0):
    """(out, mass, sum of p over the largest p) of rows q [rows][D] in 64 bits, all tokens of a row at once."""
    k, v = (oracle.kv_sequence(c, 0, table[0], n, w)[:, 0] for w in ("k", "v"))
    s = q.astype(np.float64) @ k.T * scale
    at, pos = np.arange(n), n - len(q) + np.arange(len(q))[:, None]
    if causal:
        s = np.where((at <= pos) & ((at > pos - window) | (window == 0)), s, -np.inf)
    p = np.exp(s - s.max(1, keepdims=True))
    total = p.sum(1, keepdims=True)
    return p @ v / total, p @ np.abs(v) / total, total


def attn(c, table, n, q, causal=True, window=0, split=True):
    """out [rows][D]; split False: no workspace, one workgroup takes all of a tile's tokens."""
    import bit_quantized_decode_qmv_amd as bq
    torch = torch_mod()
    ws = None if split else torch.zeros(0, dtype=torch.uint8, device="cuda:0")
    out = bq.kv_attn(upload_cache(c), 0, up(q[:, None].astype(np.float16)), up([0, len(q)], np.int32), up([n], np.int32),
                     up(table), causal=causal, window=window, workspace=ws)
    return out.cpu().numpy()[:, 0].astype(np.float64)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("n,share,far", [(32768, 0.9, 8), (32768, 0.97, 30), (131072, 0.9, 8), (131072, 0.97, 8),
                                         (131072, 0.9, 30), (131072, 0.97, 30)])
def test_weight_on_the_first_token(n, share, far, fmt):
    """One token with `share` of the weight, scores of the others normal, the V of one early block `far` times the others'."""
    rng = np.random.default_rng(n + far)
    top = 127 if fmt == "int8" else 448
    k = rng.standard_normal((n, D))
    k[:, 0], k[0] = 0, 0
    k[0, 0] = np.log(share / (1 - share) * (n - 1)) + 0.5     # q[0] = 8 under a scale of 1 / 8
    v = (60 * rng.choice([-1, 1], D) + 25 * rng.standard_normal((n, D))).clip(-127, 127) / 127
    v[0] = 0
    ks, vs = np.full(n // 16, 3.8 / top), rng.uniform(0.75, 1.25, n // 16) / top
    ks[0] = k[0, 0] / top
    vs[5] *= far
    c, table = pool(rng, {"k": k, "v": v * np.repeat(vs, 16)[:, None] * top}, {"k": ks, "v": vs}, fmt)
    q = rng.standard_normal((64, D))
    q[:, 0] = 8
    q = q.astype(np.float16)
    for rows in (1, 64):
        ref, mass, _ = reference(c, table, n, q[:rows], 0.125)
        for split in (False, True):
            err = np.abs(attn(c, table, n, q[:rows], split=split) - ref) / mass
            print(n, share, far, fmt, rows, split, err.max(), flush=True)
            assert err.max() <= 2.0 ** -10, (rows, split, err.max())
