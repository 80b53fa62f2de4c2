"""int8 caches: tokens a row does not see, and pages it does not need, do not reach it."""
import numpy as np
import pytest
import torch

import hybrid_prefix_cache_amd as K
from kv_gpu_util import Filled, to_dev
from test_gpu_attn import decode, prefill, queries

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
def test_pages_behind_the_window_may_be_freed(d):
    """With a window, pages no row sees may be -1 (or past the pool); the rows that see one are NaN."""
    f = Filled([400, 390], 2, d, 32, "int8")
    q = queries(np.random.default_rng(8), 80, 4, d, "bf16")
    for gone in (-1, f.kb.pages, 1 << 30):
        t = f.table_np.copy()
        t[:, 1:9] = gone  # tokens [32, 288)
        table = torch.from_numpy(t).cuda()
        for tokens in (1, 20):  # 2 and 40 rows a head
            pos = [399 - tokens, 389 - tokens]
            want = decode(f, q[: 2 * tokens], tokens, pos, "bf16", 80, 32)
            assert torch.equal(decode(f, q[: 2 * tokens], tokens, pos, "bf16", 80, 32, table), want)
            assert torch.isfinite(want).all()
            assert torch.isnan(decode(f, q[: 2 * tokens], tokens, pos, "bf16", 0, 0, table)).all()
            assert torch.isnan(decode(f, q[: 2 * tokens], tokens, pos, "bf16", 80, 33, table)).all()
        o = prefill(f, q, [80, 0], [320, 0], "bf16", "bf16", 50, 0, table)
        want = prefill(f, q, [80, 0], [320, 0], "bf16", "bf16", 50, 0)
        see = torch.from_numpy(np.array([max(0, 320 + i - 49) < 288 for i in range(80)]))
        assert torch.isnan(o[see]).all() and torch.equal(o[~see], want[~see])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("where", [0, 1])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_a_block_with_a_scale_that_is_not_finite(bad, where, dtype):
    """One such value makes its block NaN to the rows that see any of it: those before the block and
    those whose window has passed it have the bits they had."""
    H, hq, d, n, window, sinks = 2, 4, 64, 200, 40, 2
    f = Filled([n], H, d, 64, "int8")
    q = queries(np.random.default_rng(10), n, hq, d, dtype)
    want = prefill(f, q, [n], [0], dtype, "f32", window, sinks)
    steps = [(p, tokens) for p in (40, 63, 64, 95, 100, 134, 135, 150) for tokens in (1, 17)]
    was = [decode(f, q[p: p + t], t, [p], "f32", window, sinks) for p, t in steps]
    x = [to_dev(y[70:71].copy(), "f32") for y in f.x]
    x[where][0, 1, 5] = bad  # head 1, block 2: tokens 64..95
    K.kda_kv_append(f.kb.pool, None, x[0], x[1], None, [0, 1], f.table, start_pos=[70])
    p = np.arange(n)
    sees = torch.from_numpy((p >= 64) & (p - window < 95))
    own, other = slice(2, 4), slice(0, 2)  # the query heads of head 1 and of head 0
    got = prefill(f, q, [n], [0], dtype, "f32", window, sinks)
    assert torch.isnan(got[sees][:, own]).all()
    assert torch.equal(got[~sees][:, own], want[~sees][:, own])
    # head 0: the block's new tokens may have re-coded it, no more than that
    assert torch.isfinite(got[:, other]).all()
    for (p0, t), before in zip(steps, was):
        o, s = decode(f, q[p0: p0 + t], t, [p0], "f32", window, sinks), sees[p0: p0 + t]
        assert torch.isnan(o[s][:, own]).all(), p0
        assert torch.equal(o[~s][:, own], before[~s][:, own]), p0
        assert torch.isfinite(o[:, other]).all(), p0
