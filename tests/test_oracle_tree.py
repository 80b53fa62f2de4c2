"""The tree oracle against the chain oracles: a chain is a sequence, a way of a tree too."""
import numpy as np
import pytest

import oracle
from oracle import attention as A
from oracle import conv as C
from oracle import tree as T
from tree_util import some_path, tree


def test_ways_of_good_and_bad_entries():
    assert T.ways([-1, 0, -2, 2, 1, 5, -1, 3]) == [[0], [0, 1], [], None, [0, 1, 4], None, [6], None]


@pytest.mark.parametrize("window,sinks", [(0, 0), (5, 2), (3, 0)])
def test_attention_of_a_chain_is_the_sequence(window, sinks):
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal((6, 4, 64)), rng.standard_normal((15, 2, 64)), rng.standard_normal((15, 2, 64))
    got = T.attend(q, k, v, 9, tree("chain", 6), 0.2, window, sinks)[0]
    want = A.attend(q, k, v, np.arange(9, 15), 0.2, window, sinks)[0]
    assert np.allclose(got, want, rtol=1e-13, atol=1e-14)


@pytest.mark.parametrize("kind", ["chain", "random", "comb"])
def test_recurrence_along_every_way_is_the_token_loop(kind, oracle_lib):
    rng = np.random.default_rng(4)
    n, H, d = 9, 2, 64
    q, k, v, g = (rng.standard_normal((n, H, d)) for _ in range(4))
    k /= np.linalg.norm(k, axis=-1, keepdims=True)
    g, beta, S0 = -np.abs(g) * 0.3, rng.random((n, H)), rng.standard_normal((H, d, d)) / 8
    row = tree(kind, n, 5)
    o, states = T.recur(q, k, v, g, beta, row, S0)
    for t, way in enumerate(T.ways(row)):
        S = S0.copy()
        for s in way:
            S = S * np.exp(g[s])[..., None]
            u = v[s] - np.einsum("hkv,hk->hv", S, k[s])
            S = S + beta[s][:, None, None] * k[s][..., None] * u[:, None]
        assert np.allclose(states[t], S, rtol=1e-13, atol=1e-14)
        assert np.allclose(o[t], np.einsum("hkv,hk->hv", S, q[t]), rtol=1e-12, atol=1e-13)
    size = T.recur_size(q, k, v, g, beta, row, S0)
    assert (size >= np.abs(o)).all()


def test_convolution_along_a_way():
    rng = np.random.default_rng(5)
    x, w, window = rng.standard_normal((8, 3)), rng.standard_normal((3, 4)), rng.standard_normal((3, 3))
    row = tree("random", 8, 2)
    y, _ = T.convolve(x, w, row, window)
    for t, way in enumerate(T.ways(row)):
        line = np.concatenate([window, x[way]])
        assert np.allclose(y[t], sum(w[:, j] * line[len(line) - 4 + j] for j in range(4)))


def test_commit_of_a_prefix_changes_nothing_and_of_one_block_moves_codes():
    rng = np.random.default_rng(6)
    b = A.Int8Blocks(2, 64)
    b.append(rng.standard_normal((5, 2, 64)), 0)
    b.append(rng.standard_normal((7, 2, 64)), 5)
    codes, scales = b.codes.copy(), b.scales.copy()
    T.commit(b, 5, [0, 1, 2])
    assert (b.codes == codes).all() and (b.scales == scales).all()
    T.commit(b, 5, [1, 4, 6])
    assert (b.codes[5:8] == codes[[6, 9, 11]]).all() and (b.codes[:5] == codes[:5]).all() and (b.scales == scales).all()


def test_pages_forked_and_freed_leave_what_was():
    p = T.Pages([1, 1, 0, 0, 0, 2], [[0, 1, -1], [-1, -1, -1]], 4)
    copies, status = p.fork([0], [1], [6])
    assert status == [0] and copies == [[1], [2], [2]] and p.table[1] == [0, 2, -1] and p.refs == [2, 1, 1, 0, 0, 2]
    assert p.reserve([0, 7], [0, 9]) == [0, 0] and p.table[1] == [0, 2, 3]
    p.release([0, 0], [0, 12])
    assert p.table == [[0, 1, -1], [-1, -1, -1]] and p.refs == [1, 1, 0, 0, 0, 2]
    p = T.Pages([0, 1, 0, 2, 1], [[3, 1], [4, 3]], 4)
    assert p.compact() == [(4, 0), (3, 2)] and p.table == [[2, 1], [0, 2]] and p.refs == [1, 1, 2, 0, 0]


def test_some_path_is_a_way():
    row = tree("binary", 15)
    assert some_path(row) == [0, 1, 3, 7]
