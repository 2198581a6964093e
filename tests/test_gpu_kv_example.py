"""The example decoder: its calls work together, sharing and moving pages do
not change a bit of its results, and its attention is that of the values that
its cache holds."""
import os
import sys

import numpy as np
import pytest

import oracle
from gpu_helpers import torch_mod
from kv_helpers import download_cache

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def ex():
    torch = torch_mod()
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import speculative_decode
    return speculative_decode


@pytest.fixture(scope="module")
def model(ex):
    return ex.Decoder()


def prompt(n):
    torch = torch_mod()
    return torch.from_numpy(np.random.default_rng(n).integers(0, 1024, n).astype(np.int32)).to("cuda:0")


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_samples(ex, model, fmt):
    a = ex.Session(model, rows=4, format=fmt)
    out, logits, moved = ex.decode(a, prompt(150), 4, 5, 4)
    assert all(len(t) >= 1 + 5 for t in out) and bool(logits.isfinite().all())
    # pages of freed samples are free, the others' in use once or shared
    refs = a.refs.cpu().numpy()
    table = a.table.cpu().numpy()
    assert np.array_equal(np.bincount(table[table >= 0], minlength=refs.size), refs)
    # the same without compaction: the same tokens and logits, bit for bit
    b = ex.Session(model, rows=4, format=fmt)
    out2, logits2, _ = ex.decode(b, prompt(150), 4, 5, 4, compact=False)
    assert out == out2 and np.array_equal(logits.cpu().numpy(), logits2.cpu().numpy())
    assert moved > 0


def test_a_forked_sample_is_the_sequence_itself(ex, model):
    """A fork that goes on gives what the sequence without forks gives."""
    torch = torch_mod()
    logits = []
    for fork in (False, True):
        s = ex.Session(model, rows=3)
        s.feed(prompt(100), ex.ints([100, 0, 0]))
        if fork:
            s.fork([0, 0], [1, 2])
            s.feed(prompt(7), ex.ints([0, 4, 3]))      # others write to their copies
            s.resize(ex.ints([-1, 30, 0]))
            s.compact()
        logits.append(s.feed(prompt(9), ex.ints([9, 0, 0])).cpu().numpy())
    assert np.array_equal(*logits)


def test_attention_over_what_the_cache_holds(ex, model):
    import bit_quantized_decode_qmv_amd as bq
    torch = torch_mod()
    s = ex.Session(model, rows=2)
    s.feed(prompt(90), ex.ints([70, 20]))
    q = torch.from_numpy(np.random.default_rng(1).standard_normal((6, 8, 64)).astype(np.float16)).to("cuda:0")
    cu = ex.ints([0, 5, 6])
    out = bq.kv_attn(s.cache, 1, q, cu, s.lens, s.table, workspace=s.workspace).cpu().numpy()
    c = download_cache(s.cache)
    table = s.table.cpu().numpy()
    for b, (rows, n) in enumerate(((slice(0, 5), 70), (slice(5, 6), 20))):
        ref, mass = oracle.kv_attn_f64(c, 1, table[b], n, q[rows].cpu().numpy(), 64 ** -0.5)
        # the tolerance of the attention's own tests
        tol = 2.0 ** -11 * np.abs(ref) + 2.0 ** -10 * mass + 2.0 ** -25 * (1 + 256 * 64)
        assert np.max(np.abs(out[rows] - ref) / tol) <= 1
