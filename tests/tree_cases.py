"""Inputs shared by the tests of trees of drafted tokens."""
import numpy as np


def random_tree(rng, n, spread):
    """Parents of a run of n rows: row 0 begins it, row i hangs below one of the `spread` rows before it."""
    return [-1] + [int(i - 1 - rng.integers(0, min(spread, i))) for i in range(1, n)] if n else []


def random_trees(rng, ns, spread):
    return np.array([p for n in ns for p in random_tree(rng, n, spread)], dtype=np.int32)


def distribution(rng, vocab, sharp=2.0):
    x = rng.standard_normal(vocab) * sharp
    p = np.exp(x - x.max())
    return (p / p.sum()).astype(np.float32)
