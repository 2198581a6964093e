"""Seeded trees of drafted tokens.  Holds no arithmetic of the method."""
from __future__ import annotations

import numpy as np


def make_tree(rng, n, levels):
    """parent of each of n rows, level by level behind row 0."""
    if n == 0:
        return np.zeros(0, np.int32)
    level = np.sort(np.concatenate([np.arange(1, min(levels, n - 1) + 1), rng.integers(1, max(min(levels, n - 1), 1) + 1, n)])[:n - 1])
    parent = [-1]
    for at in level:
        above = [0] if at == 1 else [i + 1 for i in range(len(parent) - 1) if level[i] == at - 1]
        parent.append(int(rng.choice(above)))
    return np.array(parent, np.int32)
