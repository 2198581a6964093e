"""Sizes that a C int does not hold: the helpers of trees and log probabilities drop no bits of them either."""
import pytest

import bit_quantized_decode_qmv_amd as bq
from test_device_cpu import Far, calls, far, ints, torch  # noqa: F401

PAST = 2 ** 32 + 1                                          # (its low 32 bits are 1)


def wide(rows, dtype):
    return torch.empty_strided((rows, PAST), (PAST, 1), dtype=dtype, device="meta").as_subclass(Far)


@pytest.fixture
def cache():
    codes, scales = far(1, 3, 2, 64 * 64, dtype=torch.uint8), far(1, 3, 2, 4, dtype=torch.float32)
    return bq.KVCache(codes, codes, scales, scales)


def test_words_of_a_mask(calls, cache):  # noqa: F811
    q = far(5, 4, 64)
    with pytest.raises(ValueError, match="words"):
        bq.kv_attn_tree(cache, 0, q, ints(3), ints(2), ints(2, 4), wide(5, torch.int64), out=q, workspace=far(64, dtype=torch.uint8))
    assert not calls.noted


def test_length_of_a_path(calls, cache):  # noqa: F811
    with pytest.raises(ValueError, match="path"):
        bq.kv_keep(cache, ints(3), ints(2), ints(2, 4), wide(2, torch.int32), ints(2))
    assert not calls.noted


def test_tokens_of_a_row(calls):  # noqa: F811
    with pytest.raises(ValueError, match="count"):
        bq.logprobs(far(3, 9), wide(3, torch.int32), workspace=far(64, dtype=torch.uint8))
    assert not calls.noted


def test_what_is_no_tensor(calls, cache):  # noqa: F811
    """Refused as such, whichever argument it is."""
    ok = dict(q=far(5, 4, 64), cu=ints(3), lens=ints(2), table=ints(2, 4), mask=far(5, 1, dtype=torch.int64))
    for name in ok:
        with pytest.raises(TypeError, match=name):
            bq.kv_attn_tree(cache, 0, **{**ok, name: None}, workspace=far(64, dtype=torch.uint8))
    ok = dict(parent=ints(5), cu=ints(3), lens=ints(2))
    for name in ok:
        with pytest.raises(TypeError, match=name):
            bq.tree_plan(**{**ok, name: None})
        with pytest.raises(TypeError, match=name):
            bq.tree_accept(ints(5), ints(5), **{**ok, name: None}, max_path=3)
    assert not calls.noted
