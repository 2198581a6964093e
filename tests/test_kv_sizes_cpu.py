"""Sizes whose sums do not fit the kernels' integers are refused before the GPU is touched."""
from test_kv_abi_cpu import SHAPE, WORKSPACE, compact, fork, lib, resize  # noqa: F401


def test_pages_wanted_that_31_bits_do_not_count(lib):  # noqa: F811
    """All rows may ask for max_pages pages: their sum has to be a number.  (A call that passes is stopped by its missing
    workspace, which is looked at later.)"""
    for rows, pages in ((1 << 20, 1 << 11), (1 << 20, 1 << 24), (1 << 7, 1 << 24)):
        assert resize(lib, rows=rows, pages=pages, ws=None) == SHAPE
    assert resize(lib, rows=1 << 20, pages=(1 << 11) - 1, ws=None) == WORKSPACE
    assert resize(lib, rows=(1 << 7) - 1, pages=1 << 24, ws=None) == WORKSPACE
    # neither adds up what all rows hold
    assert fork(lib, rows=1 << 20, pages=1 << 11, ws=None) == WORKSPACE
    assert compact(lib, rows=1 << 20, pages=1 << 11, ws=None) == WORKSPACE
