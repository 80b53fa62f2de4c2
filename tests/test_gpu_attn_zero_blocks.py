"""int8 caches with blocks of zero values (scale 0, as null or sink tokens leave them):
their tokens take their share of the softmax and change nothing else."""
import numpy as np
import pytest

from test_gpu_attn import decode, prefill
from test_gpu_attn_scales import Blocks, both_forms, host, rows_of

import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [1e8, 1.0, 1e-3, 1e-6, 1e-8, 1e-30])
@pytest.mark.parametrize("zeros", [(0,), (0, 3, 4, 10), (1, 2, 3, 4, 5, 6, 7, 8, 9)])
def test_zero_blocks(zeros, size, dtype):
    n = 330
    amp = np.full(11, size)
    amp[list(zeros)] = 0
    both_forms(Blocks(n, 2, 128, 64, amp), dtype, 4, 128, n, windows=((0, 0), (50, 3)), tag=zeros)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [1e20, 1.0, 1e-6])
@pytest.mark.parametrize("zero", [0, 5])
def test_zero_block_with_the_largest_logits(zero, size, dtype):
    """Keys of the zero block lie along the queries: it has most of the softmax."""
    n, d = 330, 64
    amp, lift = np.full(11, size), np.zeros(11)
    amp[zero], lift[zero] = 0, 1.5  # a logit of 12 more
    both_forms(Blocks(n, 1, d, 64, amp, lift), dtype, 4, d, n, common=1.0, windows=((0, 0), (70, 32)), tag=zero)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nothing_but_zeros(dtype):
    n = 200
    f = Blocks(n, 1, 64, 64, np.zeros(7))
    q = rows_of(n, 4, 64, dtype)
    assert (host(prefill(f, q, [n], [0], dtype, "f32")) == 0).all()
    for tokens in (1, 17):
        assert (host(decode(f, q[:tokens], tokens, [n - tokens], "f32")) == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_zero_share_of_a_shared_cache(dtype):
    """One request of 3000 tokens, its cache shared among workgroups, some of which see zeros alone."""
    n = 3000
    amp = np.full(94, 1e-5)
    amp[:50] = 0
    amp[60::3] = 0
    f = Blocks(n, 1, 128, 512, amp)
    q = rows_of(3, 4, 128, dtype)
    for tokens in (1, 3):
        o = decode(f, q[:tokens], tokens, [n - tokens], "f32")
        f.check(o, q[:tokens], n - tokens + np.arange(tokens), dtype, tag=tokens)
    o = prefill(f, q, [3], [n - 3], dtype, "f32")
    f.check(o, q, n - 3 + np.arange(3), dtype, tag="packed")
    assert torch.isfinite(o).all()
