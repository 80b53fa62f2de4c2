"""GPU parity of the key/value append (rotation, bf16 and int8 caches) and of the
read-back against the numpy oracle: codes, scales and rotated rows are a fixed
function of the inputs, so everything here is compared bit for bit."""
import numpy as np
import pytest
import torch

import hybrid_prefix_cache_amd as K
from kv_gpu_util import KvBuf, TD, host, rope_tables, tables, to_dev, ws
from oracle import attention as A

pytestmark = pytest.mark.gpu


def rounded(x, dtype):
    return A.bf16(A.f32(x)) if dtype == "bf16" else A.f32(x)


class Model:
    """The oracle's copy of one request's cache."""

    def __init__(self, H, d, cache):
        self.cache, self.n = cache, 0
        self.parts = [A.Int8Blocks(H, d) if cache == "int8" else np.zeros((0, H, d)) for _ in range(2)]

    def append(self, k, v, start):
        for i, x in enumerate((k, v)):
            if self.cache == "int8":
                self.parts[i].append(x, start)
            else:
                self.parts[i] = np.concatenate([self.parts[i][:start], A.bf16(A.f32(x))])
        self.n = start + len(k)

    def rows(self, i):
        return self.parts[i].values(self.n) if self.cache == "int8" else self.parts[i]


def data(rng, T, hq, H, d, dtype, spread=True):
    """q, k, v as columns of one projection; token sizes spread so that block scales grow."""
    x = rng.standard_normal((T, (hq + 2 * H) * d))
    if spread:
        x *= np.exp(rng.uniform(-3, 3, (T, 1)))
    t = to_dev(x, dtype)
    cut = [t[:, : hq * d].unflatten(1, (hq, d)) if hq else None, t[:, hq * d: (hq + H) * d].unflatten(1, (H, d)),
           t[:, (hq + H) * d:].unflatten(1, (H, d))]
    return cut, [None if c is None else host(c) for c in cut]


def read(kb, table, lens, dtype="f32", starts=None):
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    k, v = (torch.full((int(cu[-1]), kb.H, kb.d), 7.0, dtype=TD[dtype], device="cuda") for _ in range(2))
    K.kda_kv_read(kb.pool, k, v, cu, table, start_pos=starts, workspace=ws(K.kda_kv_workspace_bytes(len(lens))))
    return host(k), host(v), cu


CASES = [  # cache, dtype, hq, H, d, page_tokens, rot, interleaved, [calls of (start, len) per sequence]
    ("int8", "bf16", 4, 2, 128, 64, 128, False, [[(0, 1)], [(0, 70), (70, 1), (71, 63)], [(0, 0)], [(0, 33), (33, 5)]]),
    ("int8", "f32", 3, 1, 64, 32, 64, True, [[(0, 31), (31, 1), (32, 1), (33, 40)], [(0, 200)]]),
    ("bf16", "bf16", 2, 2, 64, 96, 32, True, [[(0, 95), (95, 2)], [(0, 97), (97, 1)], [(0, 300)]]),
    ("bf16", "f32", 2, 1, 128, 32, 64, False, [[(0, 40), (40, 40)]]),
    ("int8", "bf16", 0, 3, 128, 160, 0, False, [[(0, 161), (161, 30)], [(0, 5)]]),
]


@pytest.mark.parametrize("case", CASES)
def test_append_and_read(case):
    cache, dtype, hq, H, d, pt, rot, inter, plan = case
    rng = np.random.default_rng(len(plan) * 100 + d + H)
    ends = [max(s + n for s, n in p) for p in plan]
    need = [-(-e // pt) for e in ends]
    kb = KvBuf(sum(need) + 3, H, d, pt, cache, pad=512)
    before = kb.bytes().copy()
    tab = tables(need, sum(need) + 3)
    table = torch.from_numpy(tab).cuda()
    rope, cs = None, None
    if rot:
        cs = rope_tables(max(ends), rot)
        dev_cs = [torch.from_numpy(x).cuda() for x in cs]
        rope = K.make_rope(*dev_cs, interleaved=inter)
    models = [Model(H, d, cache) for _ in plan]
    for call in range(max(len(p) for p in plan)):
        part = [p[call] if call < len(p) else (0, 0) for p in plan]
        cu = np.concatenate([[0], np.cumsum([n for _, n in part])]).astype(np.int64)
        T = int(cu[-1])
        (q, k, v), (qh, kh, vh) = data(rng, T, hq, H, d, dtype)
        out = torch.full((T + 2, hq, d), 5.0, dtype=TD[dtype], device="cuda") if hq else None
        K.kda_kv_append(kb.pool, q, k, v, None if out is None else out[:T], cu, table, rope=rope,
                        start_pos=[s for s, _ in part])
        pos = np.concatenate([np.arange(s, s + n) for s, n in part]).astype(int)
        if rot:
            kh = A.rotate(kh, pos, *cs, rot, inter)
            qh = A.rotate(qh, pos, *cs, rot, inter)
        if hq:
            assert np.array_equal(host(out[:T]), rounded(qh, dtype))
            assert (host(out[T:]) == 5.0).all()  # rows behind the last sequence
        for r, (s, n) in enumerate(part):
            if n:
                models[r].append(kh[cu[r]: cu[r + 1]], vh[cu[r]: cu[r + 1]], s)
        lens = [m.n for m in models]
        for out_dtype in ("f32", "bf16"):
            gk, gv, rcu = read(kb, table, lens, out_dtype)
            for r, m in enumerate(models):
                for i, g in ((0, gk), (1, gv)):
                    assert np.array_equal(g[rcu[r]: rcu[r + 1]], rounded(m.rows(i), out_dtype)), (call, r, i)
    # the bytes: every written block in the documented order, every other byte as it was
    want = before.copy()
    elem = 1 if cache == "int8" else 2
    size, hb = 32 * d * elem, kb.head_bytes
    for r, m in enumerate(models):
        for b in range(-(-m.n // 32)):
            page, inner = tab[r, b * 32 // pt], b % (pt // 32)
            n = min(32, m.n - 32 * b)
            for h in range(H):
                base = h * hb + inner * 2 * size
                for i in range(2):
                    rows = np.zeros((32, d))
                    src = m.parts[i].codes if cache == "int8" else m.parts[i]
                    rows[:n] = src[32 * b: 32 * b + n, h]
                    mask = np.zeros((32, d))
                    mask[:n] = 1
                    put = A.block_bytes(rows, i, elem)
                    keep = A.block_bytes(mask, i, elem).view(np.int8 if elem == 1 else np.uint16) == 0
                    keep = np.repeat(keep, elem)
                    span = want[page, base + i * size: base + (i + 1) * size]
                    span[~keep] = put[~keep]
                    if cache == "int8":
                        at = h * hb + (pt // 32) * 2 * size + 8 * inner + 4 * i
                        want[page, at: at + 4] = np.float32(m.parts[i].scales[b, h]).reshape(1).view(np.uint8)
    assert np.array_equal(kb.bytes(), want)


@pytest.mark.parametrize("cache,dtype,tokens", [("int8", "bf16", 1), ("int8", "f32", 7), ("bf16", "bf16", 33),
                                                ("int8", "bf16", 64)])
def test_step_equals_packed(cache, dtype, tokens):
    """The step form gives the bits of the packed form, request by request, and an
    inactive request (negative position) changes nothing."""
    H, hq, d, pt, n = 2, 6, 64, 64, 5
    rng = np.random.default_rng(tokens)
    starts = [0, 31, 64, 100, 5]
    need = [-(-(s + tokens) // pt) for s in starts]
    cs = [torch.from_numpy(x).cuda() for x in rope_tables(200, d)]
    rope = K.make_rope(*cs)
    kbs = [KvBuf(sum(need) + 1, H, d, pt, cache) for _ in range(2)]
    table = torch.from_numpy(tables(need, sum(need) + 1)).cuda()
    (_, k0, v0), _ = data(rng, sum(starts), 0, H, d, dtype)
    (q, k, v), _ = data(rng, n * tokens, hq, H, d, dtype)
    outs = []
    for i, kb in enumerate(kbs):
        K.kda_kv_append(kb.pool, None, k0, v0, None, np.concatenate([[0], np.cumsum(starts)]), table)
        out = torch.full((n * tokens, hq, d), 3.0, dtype=TD[dtype], device="cuda")
        if i == 0:
            lens = [tokens] * 4 + [0]
            K.kda_kv_append(kb.pool, q[: 4 * tokens], k[: 4 * tokens], v[: 4 * tokens], out[: 4 * tokens],
                            np.concatenate([[0], np.cumsum(lens)]), table, rope=rope, start_pos=starts)
            out[4 * tokens:] = 0
        else:
            pos = torch.tensor(starts[:4] + [-1], dtype=torch.int32, device="cuda")
            K.kda_kv_append_step(kb.pool, q, k, v, out, tokens, pos, table, rope=rope)
        outs.append(out)
    assert torch.equal(outs[0], outs[1])
    assert torch.equal(kbs[0].buf, kbs[1].buf)


def test_many_sequences_use_the_workspace_table():
    """Over 128 sequences (and empty ones among them) go through the workspace table."""
    H, d, pt, n = 1, 64, 32, 300
    rng = np.random.default_rng(0)
    lens = [int(x) for x in rng.integers(0, 4, n)]
    lens[-1] = 0
    kb = KvBuf(n + 1, H, d, pt, "int8")
    table = torch.from_numpy(tables([1] * n, n + 1)).cuda()
    (q, k, v), (qh, kh, vh) = data(rng, sum(lens), 1, H, d, "f32")
    cu = np.concatenate([[0], np.cumsum(lens)])
    out = torch.empty((sum(lens), 1, d), device="cuda")
    assert K.kda_kv_workspace_bytes(n) >= 16 * n and K.kda_kv_workspace_bytes(128) == 0
    K.kda_kv_append(kb.pool, q, k, v, out, cu, table, workspace=ws(K.kda_kv_workspace_bytes(n)))
    assert np.array_equal(host(out), qh)
    gk, gv, _ = read(kb, table, lens)
    for r in range(n):
        if lens[r]:
            for g, x in ((gk, kh), (gv, vh)):
                b = A.Int8Blocks(H, d)
                b.append(x[cu[r]: cu[r + 1]], 0)
                assert np.array_equal(g[cu[r]: cu[r + 1]], A.f32(b.values(lens[r]))), r


def test_bad_pages_and_positions_are_not_stored():
    """Tokens of bad pages, past the table or past the rotation table change no page; rows past
    the rotation table are NaN; rows read from a bad page are NaN."""
    H, d, pt = 1, 64, 32
    kb = KvBuf(4, H, d, pt, "bf16")
    table = torch.tensor([[9, 1], [2, -7], [0, 3], [-1, -1]], dtype=torch.int32, device="cuda")
    cs = [torch.from_numpy(x).cuda() for x in rope_tables(60, d)]
    rope = K.make_rope(*cs)
    rng = np.random.default_rng(1)
    (q, k, v), (_, kh, vh) = data(rng, 4 * 8, 1, H, d, "f32")
    out = torch.full((32, 1, d), 3.0, device="cuda")
    before = kb.bytes().copy()
    # 0: page 9 of 4; 1: second page bad; 2: positions 58..65 pass the rotation table (60) and the row (64); 3: inactive
    pos = torch.tensor([0, 28, 58, -5], dtype=torch.int32, device="cuda")
    K.kda_kv_append_step(kb.pool, q, k, v, out, 8, pos, table, rope=rope)
    after = kb.bytes()
    o = host(out)
    assert np.isfinite(o[:18]).all() and np.isnan(o[18:24]).all() and (o[24:] == 0).all()
    assert np.array_equal(after[[0, 1]], before[[0, 1]])
    assert (after[2] != before[2]).any() and (after[3] != before[3]).any()
    gv = read(kb, table[1:2], [4], starts=[28])[1]
    assert np.array_equal(gv, A.bf16(vh[8:12]))
    g = read(kb, table[1:2], [6], starts=[30])[1]
    assert np.isfinite(g[:2]).all() and np.isnan(g[2:]).all()
    assert np.array_equal(read(kb, table[2:3], [2], starts=[58])[1], A.bf16(vh[16:18]))


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_int8_non_finite_values_spoil_their_block_alone(bad):
    H, d, pt = 1, 64, 64
    kb = KvBuf(2, H, d, pt, "int8")
    table = torch.tensor([[1]], dtype=torch.int32, device="cuda")
    rng = np.random.default_rng(2)
    x = rng.standard_normal((64, H, d))
    x[40, 0, 3] = bad
    v = to_dev(rng.standard_normal((64, H, d)), "f32")
    K.kda_kv_append(kb.pool, None, to_dev(x[:35], "f32"), v[:35], None, [0, 35], table)
    K.kda_kv_append(kb.pool, None, to_dev(x[35:], "f32"), v[35:], None, [0, 29], table, start_pos=[35])
    gk, gv, _ = read(kb, table, [64])
    assert np.isfinite(gk[:32]).all() and np.isnan(gk[32:]).all() and np.isfinite(gv).all()


def test_int8_zero_block_and_scale_growth():
    """A block of zeros has scale 0 and reads 0; a later larger token re-codes the older ones."""
    H, d, pt = 1, 64, 32
    kb = KvBuf(1, H, d, pt, "int8")
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    z = torch.zeros((3, H, d), device="cuda")
    K.kda_kv_append(kb.pool, None, z, z, None, [0, 3], table)
    assert (read(kb, table, [3])[0] == 0).all()
    blocks = A.Int8Blocks(H, d)
    blocks.append(np.zeros((3, H, d)), 0)
    rng = np.random.default_rng(3)
    for t in range(3, 32):
        x = rng.standard_normal((1, H, d)) * 2.0 ** (t % 7 - 3)
        K.kda_kv_append(kb.pool, None, to_dev(x, "f32"), to_dev(x, "f32"), None, [0, 1], table, start_pos=[t])
        blocks.append(A.f32(x), t)
    gk, gv, _ = read(kb, table, [32])
    assert np.array_equal(gk, A.f32(blocks.values(32))) and np.array_equal(gv, gk)


def test_far_pages_pass_32_bit_offsets():
    """Pages whose byte offsets pass 2^32 are the ones written and read."""
    H, d, pt = 8, 128, 6144
    hb = K.kda_kv_head_bytes(d, pt, K.KDA_INT8)
    pages = (5 << 30) // (H * hb) + 1
    buf = torch.zeros(pages * H * hb, dtype=torch.uint8, device="cuda")
    pool = K.make_kv_pool(buf, H * hb, pages, H, d, pt, K.KDA_INT8)
    table = torch.tensor([[pages - 1]], dtype=torch.int32, device="cuda")
    x = to_dev(np.random.default_rng(0).standard_normal((40, H, d)), "bf16")
    K.kda_kv_append(pool, None, x, x, None, [0, 40], table, start_pos=[6100])
    k, v = (torch.empty((40, H, d), device="cuda") for _ in range(2))
    K.kda_kv_read(pool, k, v, [0, 40], table, start_pos=[6100])
    assert torch.equal(k, v) and (k - x.float()).abs().max() <= x.float().abs().max() / 127 * 0.5001
    assert not buf[: (pages - 1) * H * hb].any()


def test_append_on_a_stream_and_in_a_graph():
    """A captured append step follows the positions in its device array; replays between eager work."""
    H, hq, d, pt, n = 2, 4, 128, 64, 3
    rng = np.random.default_rng(9)
    kb, kb2 = (KvBuf(2 * n, H, d, pt, "int8") for _ in range(2))
    table = torch.from_numpy(tables([2] * n, 2 * n)).cuda()
    cs = [torch.from_numpy(x).cuda() for x in rope_tables(128, d)]
    rope = K.make_rope(*cs)
    steps = [data(rng, n, hq, H, d, "bf16")[0] for _ in range(5)]
    width = (hq + 2 * H) * d
    qkv = torch.zeros((n, width), dtype=torch.bfloat16, device="cuda")
    cut = [qkv[:, : hq * d].unflatten(1, (hq, d)), qkv[:, hq * d: (hq + H) * d].unflatten(1, (H, d)),
           qkv[:, (hq + H) * d:].unflatten(1, (H, d))]
    out, want = (torch.zeros((n, hq, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pos = torch.tensor([30, 0, 62], dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    (_, k0, v0), _ = data(rng, 92, 0, H, d, "bf16")
    for b in (kb, kb2):
        K.kda_kv_append(b.pool, None, k0, v0, None, [0, 30, 30, 92], table)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        K.kda_kv_append_step(kb.pool, cut[0], cut[1], cut[2], out, 1, pos, table, rope=rope)
    for i, (q, k, v) in enumerate(steps):
        for c, x in zip(cut, (q, k, v)):
            c.copy_(x)
        pos.copy_(torch.tensor([30 + i, i, 62 + i], dtype=torch.int32))
        g.replay()
        K.kda_kv_append_step(kb2.pool, q, k, v, want, 1, pos, table, rope=rope)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(kb.buf, kb2.buf), i
