"""Calls larger than a launch or an index can be are refused before the GPU is touched."""
from test_kv_abi_cpu import SHAPE, append, attn, desc, lib, read, rope  # noqa: F401


def test_launches_that_do_not_fit(lib):  # noqa: F811
    big = 1 << 28
    assert read(lib, desc(kv_heads=8), total=big) == SHAPE                 # 2^25 workgroups of 256
    assert read(lib, desc(kv_heads=1024), total=big) == SHAPE
    assert append(lib, desc(kv_heads=16), ks=2048, vs=2048, total=big) == SHAPE
    assert rope(lib, tokens=big + 1) == SHAPE


def test_rows_that_31_bits_do_not_count(lib):  # noqa: F811
    assert attn(lib, heads=16, qs=2048, os=2048, total=1 << 28) == SHAPE
    assert attn(lib, desc(kv_heads=1), heads=256, qs=256 * 128, os=256 * 128, total=1 << 23) == SHAPE
