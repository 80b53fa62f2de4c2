"""Attention over int8 caches whose blocks differ in size: value scales many orders
apart, blocks of zero values, scales below the smallest one kept, blocks whose scale is
not finite, and pages that are gone; prompt and step forms against the 64-bit oracle."""
import numpy as np
import pytest
import torch

import hybrid_prefix_cache_amd as K
from kv_gpu_util import KvBuf, host, tables, to_dev, tolerance, ws
from oracle import attention as A
from test_gpu_attn import decode, prefill

pytestmark = pytest.mark.gpu


class Blocks:
    """One request's int8 cache of n tokens: normal keys and values, block b's values times amp[b]
    and its keys plus lift[b] in every channel; codes and scales as the oracle has them."""

    def __init__(self, n, H, d, pt, amp, lift=None, seed=1):
        rng = np.random.default_rng(seed)
        self.kb = KvBuf(-(-n // pt) + 2, H, d, pt, "int8")
        self.lens = [n]
        self.table_np = tables([-(-n // pt)], self.kb.pages, seed)
        self.table = torch.from_numpy(self.table_np).cuda()
        block = np.arange(n) // A.BLOCK
        k = rng.standard_normal((n, H, d)) + (0 if lift is None else np.asarray(lift)[block][:, None, None])
        v = rng.standard_normal((n, H, d)) * np.asarray(amp, np.float64)[block][:, None, None]
        self.x = [A.bf16(k), A.bf16(v)]
        K.kda_kv_append(self.kb.pool, None, *(to_dev(x, "bf16") for x in self.x), None, [0, n], self.table)
        self.k, self.v = A.Int8Blocks(H, d), A.Int8Blocks(H, d)
        self.k.append(self.x[0], 0)
        self.v.append(self.x[1], 0)

    def check(self, o, q, pos, dtype, window=0, sinks=0, tag=None):
        """kv_gpu_util.tolerance, and what unequal scales add.  The fp16 weights carry the value
        scale s and reach at least 2^6, so one below fp16's normal numbers is off by at most half a
        subnormal step, 2^-25 of 2^6: 2^-31 of the row's largest w s, times its code.  The scale's
        logarithm and the sums with it (six roundings of 2^-24 of |log2 s| + 8, times ln 2).  A scale
        below 2^-120 counts as 2^-120: 127 times that of every value."""
        n, qh = self.lens[0], host(q)
        k, v = self.k.values(n), self.v.values(n)
        d, g = qh.shape[2], qh.shape[1] // k.shape[1]
        ref, mag, load = A.attend(qh, k, v, pos, d ** -0.5, window, sinks)
        tol = tolerance(ref, mag, load, n, d, dtype, "f32", "int8") - 1e-30
        s = np.repeat(self.v.scales, A.BLOCK, axis=0)[:n]
        logs = np.abs(np.log2(np.maximum(s[s > 0], 2.0 ** -120))).max() if (s > 0).any() else 0.0
        tol += mag * 8 * 2.0 ** -24 * (logs + 8)
        if ((s > 0) & (s < 2.0 ** -120)).any():
            tol += 2.0 ** -113
        for t, p in enumerate(pos):
            see = A.visible(p, n, window, sinks)
            for h in range(qh.shape[1]):
                x = d ** -0.5 * (k[see, h // g] @ qh[t, h])
                w = np.exp(x - x.max())
                ws_ = (w / w.sum() * s[see, h // g]).max()
                tol[t, h] += 2.0 ** -31 * ws_ * np.abs(self.v.codes[:n][see, h // g]).sum(0)
        got = host(o)
        assert np.isfinite(got).all(), tag
        err = np.abs(got - ref)
        over = err > tol + 1e-38  # the smallest normal fp32: below it results may be 0
        assert not over.any(), (tag, float((err[over] / (tol[over] + 1e-38)).max()), float(err.max() / np.abs(ref).max()))


def rows_of(n, hq, d, dtype, common=0.0, seed=2):
    return to_dev(np.random.default_rng(seed).standard_normal((n, hq, d)) + common, dtype)


def both_forms(f, dtype, hq, d, n, common=0.0, windows=((0, 0),), tag=None):
    """A whole prompt, a resumed one of few rows, and steps of one and of many rows a head."""
    for window, sinks in windows:
        q = rows_of(n, hq, d, dtype, common)
        o = prefill(f, q, [n], [0], dtype, "f32", window, sinks)
        at = np.unique(np.concatenate([[0, 31, 32, 63, n - 1], np.linspace(0, n - 1, 12).astype(int)]))
        f.check(o[torch.from_numpy(at)], q[torch.from_numpy(at)], at, dtype, window, sinks, (tag, window, "prompt"))
        for tokens in (1, 5, 40):
            pos = n - tokens + np.arange(tokens)
            o = decode(f, q[:tokens], tokens, [n - tokens], "f32", window, sinks)
            f.check(o, q[:tokens], pos, dtype, window, sinks, (tag, window, tokens))
        o = prefill(f, q[:3], [3], [n - 3], dtype, "f32", window, sinks)
        f.check(o, q[:3], n - 3 + np.arange(3), dtype, window, sinks, (tag, window, "resumed"))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("small", [1e-4, 1e-8, 1e-10, 1e-30, 1e-38])
def test_small_blocks_among_ordinary_ones(small, dtype):
    """Every second block's values are smaller; their weights count in full."""
    n, hq, H, d = 330, 4, 2, 128
    amp = np.where(np.arange(11) % 2, small, 1.0)
    both_forms(Blocks(n, H, d, 64, amp), dtype, hq, d, n, windows=((0, 0), (50, 3)), tag="odd")
    both_forms(Blocks(n, H, d, 64, amp[::-1]), dtype, hq, d, n, tag="even")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,H,d", [(3, 1, 64), (4, 4, 128)])
def test_scales_over_many_orders(hq, H, d, dtype):
    """Sizes from 1e-22 to 1e+22 in one cache: rising, falling and mixed."""
    n = 400
    e = np.linspace(-22, 22, 13)
    for tag, x in (("rising", e), ("falling", e[::-1]), ("mixed", np.random.default_rng(5).permutation(e))):
        both_forms(Blocks(n, H, d, 96, 10.0 ** x), dtype, hq, d, n, tag=tag)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [1e-38, 1e-36, 1e36])
def test_all_values_at_the_ends_of_the_range(size, dtype):
    n = 200
    both_forms(Blocks(n, 1, 64, 64, np.full(7, size)), dtype, 4, 64, n, tag=size)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_shared_cache_of_unequal_blocks(dtype):
    """One request of 3000 tokens, its cache shared among workgroups whose shares differ in size."""
    n = 3000
    amp = 10.0 ** np.random.default_rng(6).uniform(-12, 0, 94)
    amp[20:60] *= 1e-9
    f = Blocks(n, 1, 128, 512, amp)
    q = rows_of(3, 4, 128, dtype)
    for tokens, form in ((1, "step"), (3, "step"), (3, "packed")):
        pos = n - tokens + np.arange(tokens)
        o = (decode(f, q[:tokens], tokens, [n - tokens], "f32") if form == "step"
             else prefill(f, q[:tokens], [tokens], [n - tokens], dtype, "f32"))
        f.check(o, q[:tokens], pos, dtype, tag=(tokens, form))
