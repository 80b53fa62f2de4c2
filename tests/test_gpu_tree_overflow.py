"""The recurrence along trees where finite inputs pass fp32's range on one branch: the nodes that
follow are NaN, and the other branches keep their bits."""
import pytest
import torch

from oracle import tree as T
from test_gpu_tree_state import States
from tree_util import tree

pytestmark = pytest.mark.gpu

SHAPES = [("bf16", 128, 16), ("bf16", 128, 20), ("bf16", 128, 64), ("bf16", 64, 40), ("f32", 128, 16), ("f32", 64, 33), ("f32", 128, 64)]


def others_keep_their_bits(got, clean, row, node, head):
    """Of the first request, the nodes that do not follow `node` and the other heads; all of the other requests."""
    for t, way in enumerate(T.ways(row)):
        for h in range(got.shape[1]):
            if h != head or node not in way:
                assert torch.isfinite(got[t, h]).all() and torch.equal(got[t, h], clean[t, h]), (t, h)
    assert torch.equal(got[len(row):], clean[len(row):])


@pytest.mark.parametrize("dtype,d,tokens", SHAPES)
@pytest.mark.parametrize("gate", [100.0, 3e38])
def test_gates_that_sum_past_the_exponent(dtype, d, tokens, gate):
    """k exp(G) is infinite.  Beside it a gate of -70, past the factored range as well, so that the other
    nodes are summed pair by pair in both runs."""
    row = tree("binary", tokens)
    x = States([row, tree("comb", tokens)], 2, d, dtype, seed=tokens)
    x.x["g"][1, 1, 5] = -70.0
    clean = x.run("f32")
    x.x["g"][1, 1, 5] = gate
    got = x.run("f32")
    others_keep_their_bits(got, clean, row, 1, 1)
    for t, way in enumerate(T.ways(row)):
        if 1 in way:
            assert torch.isnan(got[t, 1]).all(), t


@pytest.mark.parametrize("dtype,d,tokens", SHAPES)
@pytest.mark.parametrize("power,nan", [(100, 3), (60, 7)])
def test_keys_whose_products_pass_the_range(dtype, d, tokens, power, nan):
    """Keys of 2^power on the way 0, 1, 3, 7: a product of two (node 3's row of A) is past 2^128, or that of
    two products (node 7's row of its inverse)."""
    row = tree("binary", tokens)
    x = States([row, tree("comb", tokens)], 2, d, dtype, seed=tokens)
    clean = x.run("f32")
    for t in (1, 3, 7):
        x.x["k"][t, 1] *= 2.0 ** power
    got = x.run("f32")
    others_keep_their_bits(got, clean, row, 1, 1)
    for t, way in enumerate(T.ways(row)):
        if nan in way:
            assert torch.isnan(got[t, 1]).all(), t


def test_a_sum_of_gates_above_zero():
    """exp(70): past the factored range, within fp32's.  Its rounding, 70 * 2^-24 of it a few times, is within
    the 4 * (d + 64) * 2^-24 that check() has for the sums."""
    x = States([tree("binary", 20), tree("chain", 20)], 2, 64, "f32", seed=1)
    x.x["g"][1, 0, 3] = 70.0
    x.check(x.run("f32"), "f32")
