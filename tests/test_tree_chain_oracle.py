"""A chain seen as a tree, and as a prompt's rows in a layer with a window and sinks: who sees whom, by the oracle."""
import numpy as np
import pytest

import oracle


@pytest.mark.parametrize("n,base", [(1, 0), (5, 0), (5, 3), (9, 2), (9, 40), (30, 7)])
@pytest.mark.parametrize("window", [0, 1, 4, 9, 100])
@pytest.mark.parametrize("sinks", [0, 2, 3, 50])
def test_a_chain_sees_what_the_rows_see_but_sinks_of_its_own(n, base, window, sinks):
    tree = oracle.tree_context(n, base, oracle.tree_seen(np.arange(-1, n - 1), window), window, sinks)
    rows = oracle.causal_context(n, base, window, sinks)
    i, j = np.mgrid[:n, :base + n]
    only = (window > 0) & (j >= base) & (j < sinks) & (j <= base + i - window)   # rows of the chain ahead of the window
    assert np.array_equal(tree, rows & ~only)
    assert not only.any() or (base < sinks and n > window)
