"""How much the recurrence along trees loses over all its rows together, beside the same closed form
in numpy with the same roundings: deep trees, where a bound on each row is far above what is lost."""
import numpy as np
import pytest

from kv_gpu_util import host
from oracle import tree as T
from test_gpu_tree_state import States
from tree_util import tree

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kinds,tokens,d", [(("chain", "binary"), 64, 128), (("random", "chain"), 48, 128), (("comb", "chain"), 32, 128),
                                            (("binary", "comb"), 16, 128), (("chain", "random"), 63, 64), (("comb", "chain"), 31, 64)])
@pytest.mark.parametrize("gate", [0.05, 1.0, 4.0])
def test_lost_over_all_rows(dtype, kinds, tokens, d, gate):
    """The model has a rounding of the same size for each of the kernel's, so the errors' root mean
    squares are alike; twice the model's is allowed, for sums in another order, and for fp32 as much
    again, for its 16-row inverses."""
    x = States([tree(k, tokens, i) for i, k in enumerate(kinds)], 2, d, dtype, seed=tokens, gate=gate)
    y = host(x.run("f32"))
    for r, row in enumerate(x.parents):
        a = [x.row(name, r) for name in ("q", "k", "v", "g", "beta")]
        ref, _ = T.recur(*a, row, x.S0[r].astype(np.float64))
        model = T.closed_form(*a, row, x.S0[r].astype(np.float64), 2 if dtype == "bf16" else 0)
        lost, expected = (np.sqrt(np.mean(np.square(z - ref))) for z in (y[r * tokens: (r + 1) * tokens], model))
        assert lost <= (2 if dtype == "bf16" else 4) * expected, lost / expected
