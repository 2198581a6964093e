"""The helpers of norms, sinks, trees and log probabilities launch on their tensors' device, whichever is current (as
test_device_cpu.py has it for the others)."""
import pytest

import bit_quantized_decode_qmv_amd as bq
from test_device_cpu import calls, far, ints, run  # noqa: F401 (calls: a fixture)

torch = pytest.importorskip("torch")


@pytest.fixture
def cache():
    return bq.KVCache(*(far(2, 4, 2, 64 * 64, dtype=torch.uint8) for _ in range(2)), *(far(2, 4, 2, 4, dtype=torch.float32) for _ in range(2)))


def test_norms(calls, cache):  # noqa: F811
    w = far(64, dtype=torch.float32)
    run(calls, ["bq_norm_rope"], lambda: bq.norm_rope(far(3, 2, 64), w, 1e-6))
    run(calls, ["bq_kv_append_norm"], lambda: bq.kv_append_norm(cache, 0, far(3, 2, 64), far(3, 2, 64), ints(2), ints(1), ints(1, 2),
                                                                q=far(3, 4, 64), k_weight=w, q_weight=w))


def test_attention(calls, cache):  # noqa: F811
    ws = far(64, dtype=torch.uint8)
    args = (cache, 0, far(3, 4, 64), ints(2), ints(1), ints(1, 2))
    run(calls, ["bq_kv_attn_sinks"], lambda: bq.kv_attn(*args, window=4, sinks=2, workspace=ws))
    run(calls, ["bq_kv_attn_tree"], lambda: bq.kv_attn_tree(*args, far(3, 1, dtype=torch.int64), workspace=ws))
    run(calls, ["bq_kv_keep"], lambda: bq.kv_keep(cache, ints(2), ints(1), ints(1, 2), ints(1, 3), ints(1)))


def test_trees_and_log_probabilities(calls):  # noqa: F811
    run(calls, ["bq_tree_plan"], lambda: bq.tree_plan(ints(3), ints(2), ints(1)))
    run(calls, ["bq_tree_accept"], lambda: bq.tree_accept(ints(3), ints(3), ints(3), ints(2), ints(1), 4))
    run(calls, ["bq_logprobs"], lambda: bq.logprobs(far(3, 9), ints(3), top=2, workspace=far(64, dtype=torch.uint8)))
