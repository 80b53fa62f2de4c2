"""Helpers for the key/value cache tests: a poisoned pool with page tables, and
the same contents kept as plain arrays for the oracle."""
from __future__ import annotations

import numpy as np
import torch

import hybrid_prefix_cache_amd as K
from oracle import attention as A

TD = {"bf16": torch.bfloat16, "f32": torch.float32}


def to_dev(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda().to(TD[dtype])


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


class KvBuf:
    """A device pool whose every byte is a poison pattern (NaN as bf16, fp32 and scales)."""

    def __init__(self, pages, H, d, page_tokens, cache, pad=0):
        self.dtype = K.KDA_INT8 if cache == "int8" else K.KDA_BF16
        self.H, self.d, self.pt, self.cache, self.pages = H, d, page_tokens, cache, pages
        self.head_bytes = K.kda_kv_head_bytes(d, page_tokens, self.dtype)
        self.page_bytes = -(-H * self.head_bytes // 256) * 256 + pad
        self.buf = torch.full((pages * self.page_bytes // 4,), 0x7FC07FC0, dtype=torch.int32, device="cuda")
        self.pool = K.make_kv_pool(self.buf, self.page_bytes, pages, H, d, page_tokens, self.dtype)
        assert K.kda_kv_pool_check(self.pool) == K.KDA_OK, K.kda_last_error()

    def bytes(self):
        return self.buf.view(torch.uint8).view(self.pages, self.page_bytes).cpu().numpy()


def tables(need, pages, seed=0, width=None):
    """Page tables with the pages of a shuffled free list; -1 past a request's last page."""
    order = np.random.default_rng(seed).permutation(pages).astype(np.int32)
    t, at = np.full((len(need), width or max(max(need), 1)), -1, np.int32), 0
    for r, m in enumerate(need):
        t[r, :m] = order[at: at + m]
        at += m
    return t


def rope_tables(n, rot, seed=3):
    ang = np.arange(n)[:, None] * 10000.0 ** (-np.arange(rot // 2) / (rot // 2))[None]
    return np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)


class Filled:
    """Requests whose caches hold `lens` tokens, appended in one call without rotation."""

    def __init__(self, lens, H, d, page_tokens, cache, seed=1, spare=0, width=None, amp=1.0):
        rng = np.random.default_rng(seed)
        need = [-(-(n + spare) // page_tokens) for n in lens]
        self.kb = KvBuf(sum(need) + 2, H, d, page_tokens, cache)
        self.table_np = tables(need, sum(need) + 2, seed, width)
        self.table = torch.from_numpy(self.table_np).cuda()
        self.lens, T = list(lens), sum(lens)
        # channels of different sizes, values bf16-representable
        gain = amp * (0.3 + 1.4 * rng.random((1, H, d)))
        self.x = [A.bf16(rng.standard_normal((T, H, d)) * gain) for _ in range(2)]
        self.cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
        K.kda_kv_append(self.kb.pool, None, to_dev(self.x[0], "bf16"), to_dev(self.x[1], "bf16"), None, self.cu,
                        self.table, workspace=ws(K.kda_kv_workspace_bytes(len(lens))))
        self.held = []
        for r in range(len(lens)):
            rows = [x[self.cu[r]: self.cu[r + 1]] for x in self.x]
            if cache == "int8":
                blocks = [A.Int8Blocks(H, d) for _ in rows]
                for b, x in zip(blocks, rows):
                    b.append(x, 0)
                rows = [b.values(lens[r]) for b in blocks]
            self.held.append(rows)


def ws(n):
    return torch.empty(max(int(n), 256), dtype=torch.uint8, device="cuda")


def tolerance(ref, mag, load, n, d, in_dtype, out_dtype, cache):
    """|kernel - exact| of one output element, by the roundings on the way:
    the logit: q . k summed in fp32 over d products, its scaling and the exponent's argument
    (d + 8 roundings of 2^-24 relative to the sum of |terms|, `load`), twice, since the
    normaliser has the same error; the weights: rounded to the matrix operand (bf16 beside a
    bf16 cache, fp16 beside an int8 one; two or more parts for fp32 inputs, good to 2^-22);
    the sums over n tokens in fp32; the output's own rounding."""
    operand = 2.0 ** -22 if in_dtype == "f32" else 2.0 ** -11 if cache == "int8" else 2.0 ** -8
    # fp32 q in two fp16 parts beside an int8 cache: 2^-22 of each q
    qpart = 2.0 ** -22 if in_dtype == "f32" and cache == "int8" else 0.0
    logit = 2 * load[..., None] * ((d + 8) * 2.0 ** -24 + qpart)
    tol = mag * (operand + logit + (n + 16) * 2.0 ** -24)
    return tol + np.abs(ref) * (2.0 ** -8 if out_dtype == "bf16" else 2.0 ** -24) + 1e-30
