"""The recurrence's closed form in a kernel's roundings: what it loses, and that less is told from it."""
import numpy as np
import pytest

from oracle import tree as T
from oracle.attention import bf16
from tree_util import tree


def inputs(tokens, d, seed, gate, cut):
    rng = np.random.default_rng(seed)
    q, k, v = (rng.standard_normal((tokens, 1, d)) for _ in range(3))
    q, k = (x / np.linalg.norm(x, axis=-1, keepdims=True) for x in (q, k))
    g, beta = -gate * rng.random((tokens, 1, d)), 1 / (1 + np.exp(-rng.standard_normal((tokens, 1))))
    return [cut(x) for x in (q, k, v, g, beta)], rng.standard_normal((1, d, d)).astype(np.float32) / np.sqrt(d)


def rms(x):
    return float(np.sqrt(np.mean(np.square(x))))


@pytest.mark.parametrize("kind,tokens", [("chain", 64), ("binary", 48), ("comb", 33)])
@pytest.mark.parametrize("gate", [0.05, 1.0])
def test_lost_by_the_closed_form(kind, tokens, gate):
    x, S0 = inputs(tokens, 64, 1, gate, bf16)
    ref, _ = T.recur(*x, tree(kind, tokens), S0)
    err = [rms(T.closed_form(*x, tree(kind, tokens), S0, parts) - ref) / rms(ref) for parts in (0, 2, 1)]
    assert err[0] < 2.0 ** -20 and err[1] < 2.0 ** -14 and err[2] > 20 * err[1] > 20 * err[0]
