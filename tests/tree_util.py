"""Trees for the tests: shapes that a drafting program makes, and some that none should."""
from __future__ import annotations

import numpy as np


def tree(kind, tokens, seed=0):
    """A row of parents."""
    rng = np.random.default_rng(seed)
    if kind == "chain":
        return [t - 1 for t in range(tokens)]
    if kind == "roots":
        return [-1] * tokens
    if kind == "binary":
        return [(t - 1) // 2 if t else -1 for t in range(tokens)]
    if kind == "comb":  # a chain with a leaf at every node
        return [-1 if t < 2 else t - 2 if t % 2 == 0 else t - 1 for t in range(tokens)]
    if kind == "none":
        return [-2] * tokens
    row = [int(rng.integers(-1, t)) for t in range(tokens)]
    if kind == "random":
        return row
    if kind == "short":  # fewer nodes than the call has room for
        live = max(1, tokens * 2 // 3)
        return row[:live] + [-2] * (tokens - live)
    if kind == "holes":  # entries that are no nodes between nodes; nodes after bad ones
        row = [p if rng.random() > 0.2 else int(rng.choice([-2, -9, t, t + 3, 10 ** 6])) for t, p in enumerate(row)]
        return row
    raise KeyError(kind)


def some_path(row, seed=0, node=None):
    """A way from a root on (the longest, or to a random node)."""
    from oracle.tree import ways
    w = [x for x in ways(row) if x]
    if not w:
        return []
    if node is None:
        return list(max(w, key=len))
    return list(w[np.random.default_rng(seed).integers(len(w))])


def pad(paths, tokens):
    return np.asarray([list(p) + [-7] * (tokens - len(p)) for p in paths], np.int32), np.asarray([len(p) for p in paths], np.int32)
