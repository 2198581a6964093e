"""Numbers that a C int does not hold: no bits of them are dropped on the way to the entry points."""
import pytest

import bit_quantized_decode_qmv_amd as bq
from test_device_cpu import calls, far, ints, torch  # noqa: F401


@pytest.fixture
def attn(calls, monkeypatch):  # noqa: F811
    """kv_attn over a small cache; returns the window that arrives."""
    codes, scales = far(2, 3, 2, 64 * 64, dtype=torch.uint8), far(2, 3, 2, 4, dtype=torch.float32)
    cache = bq.KVCache(codes, codes, scales, scales)
    arrived = []

    class Library:
        def __getattr__(self, name):
            def entry(*args):
                arrived.append(args)
                return 0
            return entry
    monkeypatch.setattr(bq, "_lib", Library())

    def run(layer=0, **how):
        q = far(5, 4, 64)
        bq.kv_attn(cache, layer, q, ints(3), ints(2), ints(2, 4), out=q, workspace=far(64, dtype=torch.uint8), **how)
        return arrived[-1][14]
    run.cache = cache
    return run


def test_windows(attn):
    """Longer than any sequence: no window, however long."""
    assert attn(window=5) == 5
    for window in (2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 63 - 1):
        assert attn(window=window) == 2 ** 31 - 1
    with pytest.raises(ValueError, match="window"):
        attn(window=-2 ** 32 + 5)


@pytest.mark.parametrize("layer", [2 ** 32, 2 ** 32 + 1, -2 ** 32])
def test_layers(attn, layer):
    cache, batch = attn.cache, (ints(3), ints(2), ints(2, 4))
    with pytest.raises(ValueError, match="layer"):
        attn(layer)
    with pytest.raises(ValueError, match="layer"):
        bq.kv_append(cache, layer, far(5, 2, 64), far(5, 2, 64), *batch)
    with pytest.raises(ValueError, match="layer"):
        bq.kv_read(cache, layer, *batch, 5)


def test_totals(attn):
    with pytest.raises(ValueError, match="total"):
        bq.kv_read(attn.cache, 0, ints(3), ints(2), ints(2, 4), 2 ** 32)
