"""GPU parity of attention over the paged cache (int8 with block scales, bf16;
causal, sliding window, sinks; packed prompts and decode steps) against the
numpy oracle in 64 bits, with tolerances derived from the roundings on the way
(kv_gpu_util.tolerance)."""


import numpy as np
import pytest
import torch

import hybrid_prefix_cache_amd as K
from kv_gpu_util import Filled, KvBuf, TD, host, rope_tables, tables, to_dev, tolerance, ws
from oracle import attention as A

pytestmark = pytest.mark.gpu


def queries(rng, T, hq, d, dtype, wide=True):
    """q rows, cut out of a wider tensor where wide."""
    x = rng.standard_normal((T, hq * d + (64 if wide else 0)))
    t = to_dev(x, dtype)
    return t[:, : hq * d].unflatten(1, (hq, d))


def prefill(f, q, lens, starts, dtype, out_dtype, window=0, sinks=0, table=None, pool=None):
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    o = torch.full((int(cu[-1]) + 1, q.shape[1], q.shape[2]), 9.0, dtype=TD[out_dtype], device="cuda")
    pool = pool or f.kb.pool
    w = ws(K.kda_attn_prefill_workspace_bytes(pool, q.shape[1], cu, start_pos=starts, window=window, sinks=sinks))
    w.fill_(0xFF)
    K.kda_attn_prefill(pool, q, o[:-1], cu, f.table if table is None else table, scale=q.shape[2] ** -0.5,
                       start_pos=starts, window=window, sinks=sinks, workspace=w)
    assert (o[-1] == 9.0).all()
    return o[:-1]


def decode(f, q, tokens, pos, out_dtype, window=0, sinks=0, table=None):
    table = f.table if table is None else table
    n, hq, d = len(pos), q.shape[1], q.shape[2]
    o = torch.full((n * tokens + 1, hq, d), 9.0, dtype=TD[out_dtype], device="cuda")
    w = ws(K.kda_attn_decode_workspace_bytes(f.kb.pool, hq, n, tokens, table.shape[1], window=window, sinks=sinks))
    w.fill_(0xFF)
    K.kda_attn_decode(f.kb.pool, q, o[:-1], tokens, torch.tensor(pos, dtype=torch.int32, device="cuda"), table,
                      scale=d ** -0.5, window=window, sinks=sinks, workspace=w)
    assert (o[-1] == 9.0).all()
    return o[:-1]


def check(got, q, held, pos, dtype, out_dtype, cache, window, sinks, tag):
    qh = host(q)
    ref, mag, load = A.attend(qh, held[0], held[1], pos, qh.shape[2] ** -0.5, window, sinks)
    tol = tolerance(ref, mag, load, len(held[0]), qh.shape[2], dtype, out_dtype, cache)
    err = np.abs(host(got) - ref)
    assert np.isfinite(host(got)).all(), tag
    assert (err <= tol).all(), (tag, float((err / tol).max()))


DECODE = [  # cache, dtype, out, hq, H, d, page_tokens, tokens, lens (tokens cached before the step), window, sinks
    ("int8", "bf16", "bf16", 8, 2, 128, 64, 1, [0, 1, 31, 32, 33, 500], 0, 0),
    ("int8", "bf16", "f32", 3, 1, 64, 32, 1, [700, 2], 0, 0),
    ("bf16", "bf16", "bf16", 16, 1, 128, 96, 1, [95, 96, 200], 0, 0),
    ("bf16", "f32", "f32", 4, 4, 64, 64, 1, [130, 3], 0, 0),
    ("int8", "f32", "f32", 7, 1, 128, 64, 3, [60, 5, 255], 0, 0),
    ("int8", "bf16", "bf16", 10, 2, 64, 160, 5, [0, 158, 40], 0, 0),
    ("bf16", "bf16", "bf16", 12, 3, 128, 32, 9, [90, 1], 0, 0),
    ("int8", "bf16", "bf16", 8, 1, 128, 64, 64, [10, 130], 0, 0),
    ("bf16", "f32", "f32", 4, 1, 64, 64, 40, [100], 0, 0),
    # windows: of one token, shorter than a block, across pages; sinks inside, outside, past the window
    ("bf16", "bf16", "bf16", 4, 2, 128, 64, 1, [300, 5, 0], 1, 0),
    ("int8", "bf16", "bf16", 8, 2, 64, 64, 1, [300, 77], 20, 4),
    ("bf16", "f32", "f32", 2, 1, 64, 32, 6, [257, 3], 33, 35),
    ("int8", "f32", "f32", 8, 4, 128, 64, 4, [500, 90], 100, 200),
    ("bf16", "bf16", "bf16", 32, 1, 128, 64, 7, [400, 64], 64, 1),
]


@pytest.mark.parametrize("case", DECODE)
def test_decode(case):
    cache, dtype, out, hq, H, d, pt, tokens, lens, window, sinks = case
    f = Filled([n + tokens for n in lens], H, d, pt, cache, seed=hq + d + tokens)
    q = queries(np.random.default_rng(5), len(lens) * tokens, hq, d, dtype)
    o = decode(f, q, tokens, lens, out, window, sinks)
    for r, n in enumerate(lens):
        rows = slice(r * tokens, (r + 1) * tokens)
        check(o[rows], q[rows], f.held[r], n + np.arange(tokens), dtype, out, cache, window, sinks, r)


PREFILL = [  # cache, dtype, out, hq, H, d, page_tokens, [(start, len)], window, sinks
    ("int8", "bf16", "bf16", 4, 2, 128, 64, [(0, 1), (0, 300), (0, 0), (64, 65)], 0, 0),
    ("bf16", "bf16", "bf16", 3, 1, 64, 96, [(17, 130), (0, 31)], 0, 0),
    ("bf16", "f32", "f32", 2, 2, 64, 32, [(0, 33), (100, 50)], 0, 0),
    ("int8", "f32", "f32", 5, 1, 128, 160, [(31, 90)], 0, 0),
    ("bf16", "bf16", "f32", 2, 1, 128, 64, [(700, 3), (0, 64)], 0, 0),
    ("int8", "bf16", "bf16", 16, 1, 64, 64, [(512, 40)], 0, 0),
    ("bf16", "bf16", "bf16", 4, 1, 128, 64, [(0, 400), (333, 100)], 1, 0),
    ("bf16", "bf16", "bf16", 4, 2, 64, 64, [(0, 400), (333, 100)], 70, 5),
    ("int8", "bf16", "bf16", 2, 1, 128, 32, [(0, 330), (90, 7)], 33, 64),
    ("bf16", "f32", "f32", 3, 1, 64, 64, [(200, 200)], 150, 300),
    ("int8", "f32", "f32", 1, 1, 64, 64, [(0, 129)], 64, 1),
]


@pytest.mark.parametrize("case", PREFILL)
def test_prefill(case):
    cache, dtype, out, hq, H, d, pt, spans, window, sinks = case
    lens, starts = [n for _, n in spans], [s for s, _ in spans]
    f = Filled([s + n for s, n in spans], H, d, pt, cache, seed=hq + d)
    q = queries(np.random.default_rng(6), sum(lens), hq, d, dtype)
    o = prefill(f, q, lens, starts, dtype, out, window, sinks)
    at = 0
    for r, (s, n) in enumerate(spans):
        if n:
            check(o[at: at + n], q[at: at + n], f.held[r], s + np.arange(n), dtype, out, cache, window, sinks, r)
        at += n


@pytest.mark.parametrize("cache", ["int8", "bf16"])
def test_long_cache_few_rows(cache):
    """One request of 40,000 tokens: the work over the cache is split and joined; a peaked row among flat ones."""
    f = Filled([40000], 1, 128, 512, cache, seed=4, amp=1.0)
    q = queries(np.random.default_rng(7), 2, 4, 128, "bf16")
    q[0, 0] *= 12  # a peaked softmax
    q[0, 1] = 0    # a flat one
    for window, sinks in ((0, 0), (30000, 100)):
        o = decode(f, q, 2, [39998], "bf16", window, sinks)
        check(o, q, f.held[0], np.array([39998, 39999]), "bf16", "bf16", cache, window, sinks, (window, "decode"))
        o = prefill(f, q, [2], [39998], "bf16", "bf16", window, sinks)
        check(o, q, f.held[0], np.array([39998, 39999]), "bf16", "bf16", cache, window, sinks, (window, "prefill"))


def test_pages_behind_the_window_may_be_freed():
    """With a window, pages no row sees may be -1; the same rows without a window are NaN."""
    f = Filled([400, 390], 2, 64, 32, "bf16")
    q = queries(np.random.default_rng(8), 2, 4, 64, "bf16")
    t = f.table_np.copy()
    t[:, 1:9] = -1  # tokens [32, 288); the window covers [300 - ..]
    table = torch.from_numpy(t).cuda()
    want = decode(f, q, 1, [399, 389], "bf16", 100, 32)
    got = decode(f, q, 1, [399, 389], "bf16", 100, 32, table)
    assert torch.equal(want, got) and torch.isfinite(want).all()
    assert torch.equal(prefill(f, q, [1, 1], [399, 389], "bf16", "bf16", 100, 32, table),
                       prefill(f, q, [1, 1], [399, 389], "bf16", "bf16", 100, 32))
    assert torch.isnan(decode(f, q, 1, [399, 389], "bf16", 0, 0, table)).all()
    assert torch.isnan(decode(f, q, 1, [399, 389], "bf16", 100, 33, table)).all()  # one sink on a freed page
    assert torch.isnan(prefill(f, q, [1, 1], [399, 389], "bf16", "bf16", 100, 33, table)).all()
    # only the rows that see a bad page
    q = queries(np.random.default_rng(8), 80, 4, 64, "bf16")
    o = prefill(f, q, [80, 0], [320, 0], "bf16", "bf16", 50, 0, table)
    see = np.array([max(0, 320 + i - 49) < 288 for i in range(80)])
    assert torch.isnan(o[torch.from_numpy(see)]).all() and torch.isfinite(o[torch.from_numpy(~see)]).all()


def test_rows_of_no_request():
    """Inactive requests give zeros; requests past their table row give NaN; their neighbours are right."""
    f = Filled([60, 60, 60], 1, 128, 64, "int8")
    q = queries(np.random.default_rng(9), 6, 4, 128, "bf16")
    o = decode(f, q, 2, [-1, 63, 58], "bf16")
    assert (o[:2] == 0).all() and torch.isnan(o[2:4]).all()
    check(o[4:], q[4:], f.held[2], np.array([58, 59]), "bf16", "bf16", "int8", 0, 0, "active")
    o = decode(f, q, 2, [-(1 << 31), (1 << 31) - 1, 58], "bf16")
    assert (o[:2] == 0).all() and torch.isnan(o[2:4]).all()


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_what_a_row_does_not_see_does_not_reach_it(bad):
    """Non-finite keys and values in a bf16 cache: rows before them (causal) and after them (window)
    are as without them; rows that see them are not finite."""
    H, d, pt, n = 1, 64, 64, 150
    f = Filled([n], H, d, pt, "bf16")
    q = queries(np.random.default_rng(10), n, 2, d, "bf16")
    want = prefill(f, q, [n], [0], "bf16", "bf16", 40, 2)
    for where in (0, 1):
        x = [to_dev(y[90:91].copy(), "f32") for y in f.x]
        x[where][0, 0, 5] = bad
        K.kda_kv_append(f.kb.pool, None, x[0], x[1], None, [0, 1], f.table, start_pos=[90])
        got = prefill(f, q, [n], [0], "bf16", "bf16", 40, 2)
        sees = np.array([90 <= p < 130 for p in range(n)])
        assert torch.equal(got[torch.from_numpy(~sees)], want[torch.from_numpy(~sees)]), where
        if where == 1:
            assert not torch.isfinite(got[torch.from_numpy(sees)][:, :, 5]).any()
            rest = [c for c in range(d) if c != 5]
            assert torch.isfinite(got[torch.from_numpy(sees)][:, :, rest]).all()
        for p in (70, 89, 90, 100, 129, 130, 140):
            one = decode(f, q[p: p + 8], 8, [p], "bf16", 40, 2) if p + 8 <= n else None
            if one is not None:
                s = torch.from_numpy(sees[p: p + 8])
                assert torch.isfinite(one[~s]).all(), (where, p)
                if where == 1:
                    assert not torch.isfinite(one[s][:, :, 5]).any()
        K.kda_kv_append(f.kb.pool, None, to_dev(f.x[0][90:91], "f32"), to_dev(f.x[1][90:91], "f32"), None, [0, 1],
                        f.table, start_pos=[90])


def test_extreme_logits():
    """Logits near the ends of fp32 and equal ones: no overflow, ties shared."""
    f = Filled([100], 1, 64, 64, "bf16", amp=1.0)
    for amp in (0.0, 1e-30, 1e4, 1e30):
        q = queries(np.random.default_rng(11), 1, 2, 64, "bf16")
        q.copy_(A_scale(q, amp))
        o = decode(f, q, 1, [99], "f32")
        qh = host(q)
        ref = A.attend(qh, f.held[0][0], f.held[0][1], np.array([99]), 0.125)[0]
        assert torch.isfinite(o).all(), amp
        if amp <= 1.0:  # all weights equal
            assert np.abs(host(o) - ref).max() <= 2.0 ** -8 * np.abs(f.held[0][1]).mean(0).max() + 1e-6, amp
        else:  # one token has all the weight
            assert np.abs(host(o) - ref).max() <= 2.0 ** -8 * np.abs(f.held[0][1]).max(), amp


def A_scale(q, amp):
    return (q.float() * amp).to(q.dtype)


@pytest.mark.parametrize("cache", ["int8", "bf16"])
def test_resume_and_shared_pages(cache):
    """Prompt, prefix hit on shared pages, decode: appending and attending in chunks gives the
    rows of the whole call; a second request resumes at a boundary of the prefix index on the
    first one's pages and gives the same rows; decode steps continue both."""
    H, hq, d, pt, n, B = 2, 4, 128, 512, 1300, 1024
    rng = np.random.default_rng(12)
    toks = rng.integers(0, 1000, n).astype(np.int32)
    idx = K.kda_index_create(hash_block=512, physical_block=pt)
    kb = KvBuf(8, H, d, pt, cache)
    cs = [torch.from_numpy(x).cuda() for x in rope_tables(2000, d)]
    rope = K.make_rope(*cs)
    qkv = to_dev(rng.standard_normal((n + 4, (hq + 2 * H) * d)), "bf16")

    def cut(a, b):
        x = qkv[a:b]
        return (x[:, : hq * d].unflatten(1, (hq, d)), x[:, hq * d: (hq + H) * d].unflatten(1, (H, d)),
                x[:, (hq + H) * d:].unflatten(1, (H, d)))

    def run(a, b, table):
        q, k, v = cut(a, b)
        qr, o = (torch.empty((b - a, hq, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        K.kda_kv_append(kb.pool, q, k, v, qr, [0, b - a], table, rope=rope, start_pos=[a])
        w = ws(K.kda_attn_prefill_workspace_bytes(kb.pool, hq, [0, b - a], start_pos=[a]))
        K.kda_attn_prefill(kb.pool, qr, o, [0, b - a], table, scale=d ** -0.5, start_pos=[a], workspace=w)
        return o

    first = torch.tensor([[3, 5, 0]], dtype=torch.int32, device="cuda")
    whole = run(0, n, first)
    K.kda_index_register_pages(idx, toks[:1024], [3, 5], step=1)
    K.kda_index_register_ckpt(idx, toks, B, 0, 0, step=1)
    K.kda_index_mark_ready(idx, 1)
    hit = K.kda_index_lookup(idx, toks)
    assert hit["boundary"] == B and hit["pages"][:2] == [3, 5]
    second = torch.tensor([hit["pages"][:2] + [6]], dtype=torch.int32, device="cuda")
    part = run(B, n, second)
    assert torch.equal(part, whole[B:])  # same rows, whatever the call holds beside them
    for t in range(n, n + 4):
        table = torch.cat([first, second])
        q, k, v = (x.expand(2, -1, -1).contiguous() for x in cut(t, t + 1))
        qr, o = (torch.empty((2, hq, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        pos = torch.full((2,), t, dtype=torch.int32, device="cuda")
        K.kda_kv_append_step(kb.pool, q, k, v, qr, 1, pos, table, rope=rope)
        w = ws(K.kda_attn_decode_workspace_bytes(kb.pool, hq, 2, 1, 3))
        K.kda_attn_decode(kb.pool, qr, o, 1, pos, table, scale=d ** -0.5, workspace=w)
        assert torch.equal(o[0], o[1]) and torch.isfinite(o).all()
        # against the cache as it reads back
        kk, vv = (torch.empty((t + 1, H, d), device="cuda") for _ in range(2))
        K.kda_kv_read(kb.pool, kk, vv, [0, t + 1], first)
        check(o[:1], qr[:1], [host(kk), host(vv)], np.array([t]), "bf16", "bf16", cache, 0, 0, t)


def test_decode_in_graphs_with_their_own_workspaces():
    """Two captured steps of different shapes and a growing position array, replayed in turn with
    eager calls between; every replay equals the eager result, and repeated calls are bitwise equal."""
    f = Filled([900, 400, 30], 2, 128, 64, "int8", spare=64)
    rng = np.random.default_rng(13)
    q1, q2 = queries(rng, 3, 8, 128, "bf16", False), queries(rng, 6, 8, 128, "bf16", False)
    pos = torch.tensor([880, 380, 10], dtype=torch.int32, device="cuda")
    outs = [torch.empty_like(q) for q in (q1, q2)]
    wss = [ws(K.kda_attn_decode_workspace_bytes(f.kb.pool, 8, 3, t, f.table.shape[1])) for t in (1, 2)]
    graphs = []
    torch.cuda.synchronize()
    for t, q, o, w in ((1, q1, outs[0], wss[0]), (2, q2, outs[1], wss[1])):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            K.kda_attn_decode(f.kb.pool, q, o, t, pos, f.table, scale=0.09, workspace=w)
        graphs.append(g)
    for i in range(4):
        pos.copy_(torch.tensor([880 + i, 380 + i, 10 + i], dtype=torch.int32))
        for g, t, q, o in ((graphs[0], 1, q1, outs[0]), (graphs[1], 2, q2, outs[1])):
            g.replay()
            e = torch.empty_like(q)
            w = ws(K.kda_attn_decode_workspace_bytes(f.kb.pool, 8, 3, t, f.table.shape[1]))
            K.kda_attn_decode(f.kb.pool, q, e, t, pos, f.table, scale=0.09, workspace=w)
            torch.cuda.synchronize()
            assert torch.equal(o, e), (i, t)


def test_host_validation(monkeypatch):
    """KDA_VALIDATE=1: page tables are read back and checked first; same bits where they pass."""
    f = Filled([200, 100], 1, 64, 64, "bf16", spare=8)
    q = queries(np.random.default_rng(14), 2, 2, 64, "bf16")
    want = decode(f, q, 1, [199, 99], "bf16", 40, 0)
    monkeypatch.setenv("KDA_VALIDATE", "1")
    assert torch.equal(decode(f, q, 1, [199, 99], "bf16", 40, 0), want)
    t = f.table_np.copy()
    t[0, 0] = 99
    bad = torch.from_numpy(t).cuda()
    assert torch.equal(decode(f, q, 1, [199, 99], "bf16", 40, 0, bad), want)  # behind the window
    for call in (lambda: decode(f, q, 1, [199, 99], "bf16", 0, 0, bad),
                 lambda: prefill(f, q, [1, 1], [199, 99], "bf16", "bf16", 0, 0, bad)):
        with pytest.raises(K.KdaError) as e:
            call()
        assert e.value.status == K.KDA_ERR_PAGE_RANGE
    x = to_dev(np.zeros((2, 1, 64)), "bf16")
    t = f.table_np.copy()
    t[1, 1] = t[0, 3]
    with pytest.raises(K.KdaError) as e:
        K.kda_kv_append(f.kb.pool, None, x, x, None, [0, 1, 2], torch.from_numpy(t).cuda(), start_pos=[200, 100])
    assert e.value.status == K.KDA_ERR_PAGE_ALIAS
    before = f.kb.buf.clone()
    with pytest.raises(K.KdaError) as e:
        K.kda_kv_append_step(f.kb.pool, None, x, x, None, 1, torch.tensor([200, 999], dtype=torch.int32, device="cuda"),
                             f.table)
    assert e.value.status == K.KDA_ERR_PAGE_RANGE and torch.equal(before, f.kb.buf)


def _log_uniform(rng, lo, hi):
    return int(round(np.exp(rng.uniform(np.log(lo), np.log(hi)))))


@pytest.mark.parametrize("seed", range(24))
def test_random_calls(seed):
    """Seeded sweep over heads, types, page sizes, windows, sinks and ragged batches, both forms."""
    rng = np.random.default_rng(1000 + seed)
    cache, dtype = rng.choice(["int8", "bf16"]), rng.choice(["bf16", "bf16", "f32"])
    out = rng.choice(["bf16", "f32"])
    d, H = int(rng.choice([64, 128])), int(rng.choice([1, 2, 3]))
    hq = H * int(rng.choice([1, 2, 5, 8, 17]))
    pt = 32 * int(rng.choice([1, 2, 3, 7]))
    window = _log_uniform(rng, 1, 400) if rng.random() < 0.6 else 0
    sinks = int(rng.choice([0, 1, 31, 32, 100]))
    n = int(rng.integers(1, 5))
    step = rng.random() < 0.5
    tokens = int(rng.choice([1, 2, 3, 17]))
    starts = [_log_uniform(rng, 1, 600) - 1 for _ in range(n)]
    lens = [tokens if step else _log_uniform(rng, 1, 120) for _ in range(n)]
    f = Filled([s + m for s, m in zip(starts, lens)], H, d, pt, cache, seed=seed)
    q = queries(rng, sum(lens), hq, d, dtype)
    o = decode(f, q, tokens, starts, out, window, sinks) if step else prefill(f, q, lens, starts, dtype, out, window,
                                                                            sinks)
    at = 0
    for r, (s, m) in enumerate(zip(starts, lens)):
        check(o[at: at + m], q[at: at + m], f.held[r], s + np.arange(m), dtype, out, cache, window, sinks, r)
        at += m


WIDE = [  # cache, out, hq, H, d, page_tokens, sequences, longest call, longest start, window, sinks
    ("int8", "bf16", 6, 2, 128, 64, 140, 70, 300, 0, 0),
    ("bf16", "bf16", 6, 2, 64, 96, 140, 70, 300, 0, 0),
    ("bf16", "f32", 16, 8, 128, 32, 33, 40, 2700, 0, 0),
    ("int8", "f32", 8, 8, 64, 160, 33, 300, 2700, 0, 0),
    ("bf16", "bf16", 8, 8, 128, 64, 33, 300, 900, 75, 5),
    ("int8", "bf16", 24, 8, 128, 64, 33, 90, 2700, 200, 40),
]


@pytest.mark.parametrize("case", WIDE)
def test_wide_batches(case):
    """Batches with a workgroup for every CU: sampled rows against the oracle, and a sequence's rows
    bit for bit as in a call of its own, which is small and cut into other tiles (past 1000 tokens
    such a call is split over the cache and joined, which rounds differently)."""
    cache, out, hq, H, d, pt, n, longest, far, window, sinks = case
    rng = np.random.default_rng(hq + d)
    lens = [int(x) for x in rng.integers(0, longest + 1, n)]
    starts = [int(x) for x in rng.integers(0, far + 1, n)]
    lens[0], starts[0], lens[1], starts[1] = longest, far, 1, 0
    f = Filled([s + m for s, m in zip(starts, lens)], H, d, pt, cache, seed=n + d)
    q = queries(rng, sum(lens), hq, d, "bf16")
    o = prefill(f, q, lens, starts, "bf16", out, window, sinks)
    cu = np.concatenate([[0], np.cumsum(lens)])
    for r in list(range(6)) + [n - 1]:
        if not lens[r]:
            continue
        rows = slice(int(cu[r]), int(cu[r + 1]))
        if starts[r] + lens[r] <= 1000:
            alone = prefill(f, q[rows], [lens[r]], [starts[r]], "bf16", out, window, sinks,
                            f.table[r: r + 1].contiguous())
            assert torch.equal(alone, o[rows]), r
        at = np.unique(np.linspace(0, lens[r] - 1, 9).astype(int))
        check(o[rows][at], q[rows][at], f.held[r], starts[r] + at, "bf16", out, cache, window, sinks, r)


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_wide_batches_and_values_out_of_sight(bad):
    """Non-finite values in a bf16 cache, in a batch with a workgroup for every CU: rows before
    and past the window of them are as without them, a bad page spoils the rows that see it."""
    H, d, pt, n, m = 8, 64, 32, 34, 100
    f = Filled([m] * n, H, d, pt, "bf16", seed=3)
    q = queries(np.random.default_rng(10), n * m, 16, d, "bf16")
    want = prefill(f, q, [m] * n, [0] * n, "bf16", "bf16", 40, 2)
    x = [to_dev(y[50:51].copy(), "f32") for y in f.x]
    x[1][0, :, 5] = bad
    K.kda_kv_append(f.kb.pool, None, x[0], x[1], None, [0, 1], f.table[:1].contiguous(), start_pos=[50])
    t = f.table_np.copy()
    t[1, 1] = -1  # tokens 32..63 of the second sequence
    got = prefill(f, q, [m] * n, [0] * n, "bf16", "bf16", 40, 2, torch.from_numpy(t).cuda())
    p = np.arange(m)
    sees = torch.from_numpy((p >= 50) & (p < 90))
    assert torch.equal(got[2 * m:], want[2 * m:])
    assert torch.equal(got[:m][~sees], want[:m][~sees])
    assert not torch.isfinite(got[:m][sees][:, :, 5]).any()
    assert torch.isfinite(got[:m][sees][:, :, [c for c in range(d) if c != 5]]).all()
    sees = torch.from_numpy((p >= 32) & (p - 39 <= 63))
    assert torch.isnan(got[m: 2 * m][sees]).all() and torch.equal(got[m: 2 * m][~sees], want[m: 2 * m][~sees])


def test_packed_calls_in_a_graph_and_on_two_streams():
    """140 sequences (their table ships through the workspace): append and attention captured together,
    replayed between eager calls; and two streams at once, a workspace each.  All bits as in plain calls."""
    n, H, hq, d, pt = 140, 2, 4, 64, 32
    rng = np.random.default_rng(31)
    lens = [int(x) for x in rng.integers(0, 60, n)]
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    T = int(cu[-1])
    table_np = tables([2] * n, 2 * n)
    table = torch.from_numpy(table_np).cuda()
    k, v = (to_dev(rng.standard_normal((T, H, d)), "bf16") for _ in range(2))
    q = queries(rng, T, hq, d, "bf16", False)
    kbs = [KvBuf(2 * n, H, d, pt, "int8") for _ in range(3)]

    def call(kb, o, w):
        K.kda_kv_append(kb.pool, None, k, v, None, cu, table, workspace=w[0])
        K.kda_attn_prefill(kb.pool, q, o, cu, table, scale=0.11, window=50, sinks=3, workspace=w[1])

    def spaces():
        return (ws(K.kda_kv_workspace_bytes(n)),
                ws(K.kda_attn_prefill_workspace_bytes(kbs[0].pool, hq, cu, window=50, sinks=3)))

    outs, wss = [torch.zeros_like(q) for _ in range(3)], [spaces() for _ in range(3)]
    call(kbs[0], outs[0], wss[0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(kbs[1], outs[1], wss[1])
    for i in range(3):
        k.mul_(-1.5), q.mul_(1.25)
        outs[1].fill_(7.0)
        g.replay()
        call(kbs[0], outs[0], wss[0])
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1]) and torch.equal(kbs[0].buf, kbs[1].buf), i
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for i in range(4):
        for s, kb, o, w in ((streams[0], kbs[1], outs[1], wss[1]), (streams[1], kbs[2], outs[2], wss[2])):
            with torch.cuda.stream(s):
                call(kb, o, w)
    torch.cuda.synchronize()
    assert torch.equal(outs[1], outs[0]) and torch.equal(outs[2], outs[0])
    # pages of the third buffer that no token reached keep their poison
    assert torch.equal(kbs[2].buf, kbs[1].buf)


def test_bindings_refuse():
    """Tensors of another device, type, shape or layout are refused before the library is called."""
    f = Filled([50, 40], 2, 64, 32, "int8", spare=8)
    pool, table, q = f.kb.pool, f.table, queries(np.random.default_rng(5), 2, 4, 64, "bf16", False)
    pos = torch.tensor([50, 40], dtype=torch.int32, device="cuda")
    o, w = torch.zeros_like(q), ws(K.kda_attn_decode_workspace_bytes(pool, 4, 2, 1, table.shape[1]))
    k = to_dev(np.zeros((2, 2, 64)), "bf16")
    before = f.kb.buf.clone()

    def dec(**kw):
        a = dict(q=q, o=o, tokens=1, pos=pos, page_table=table)
        K.kda_attn_decode(pool, **{**a, **kw}, scale=0.1, workspace=w)

    def pre(**kw):
        a = dict(q=q, o=o, cu_seqlens=[0, 1, 2], page_table=table, start_pos=[50, 40])
        K.kda_attn_prefill(pool, **{**a, **kw}, scale=0.1, workspace=w)

    def app(**kw):
        a = dict(q=None, k=k, v=k, q_out=None, tokens=1, pos=pos, page_table=table)
        K.kda_kv_append_step(pool, **{**a, **kw})

    def rd(**kw):
        a = dict(k_out=torch.zeros_like(k), v_out=torch.zeros_like(k), cu_seqlens=[0, 1, 2], page_table=table)
        K.kda_kv_read(pool, **{**a, **kw})

    wide = torch.zeros((2, 8, 64), dtype=torch.bfloat16, device="cuda")
    calls = [
        (dec, dict(q=q.cpu())), (dec, dict(q=q.half())), (dec, dict(q=q[:1])), (dec, dict(q=q[:, :, :32])),
        (dec, dict(q=q.flatten(1))), (dec, dict(q=wide[:, ::2])), (dec, dict(o=wide[:, :4])), (dec, dict(o=o[:1])),
        (dec, dict(o=o.cpu())), (dec, dict(pos=pos.long())), (dec, dict(pos=pos.cpu())), (dec, dict(pos=pos[:1])),
        (dec, dict(page_table=table[:1])), (dec, dict(page_table=table.cpu())), (dec, dict(page_table=table.t())),
        (dec, dict(page_table=table.flatten())), (dec, dict(page_table=table.long())), (dec, dict(tokens=2)),
        (pre, dict(q=q.cpu())), (pre, dict(cu_seqlens=[0, 2])), (pre, dict(cu_seqlens=[0, 1, 3])),
        (pre, dict(start_pos=[50])), (pre, dict(cu_seqlens=[])), (pre, dict(o=o.half())),
        (app, dict(k=k.cpu())), (app, dict(v=k.float())), (app, dict(k=k[:, :1])), (app, dict(q=q)),
        (app, dict(q=q, q_out=wide[:, :4])), (app, dict(v=k.transpose(0, 1))),
        (app, dict(rope=K.kda_rope(0, 0, 8, 16, 0))),
        (rd, dict(k_out=k.float())), (rd, dict(v_out=wide[:, :2])), (rd, dict(cu_seqlens=[0, 1])),
    ]
    for fn, kw in calls:
        with pytest.raises((ValueError, K.KdaError)):
            fn(**kw)
    small = torch.zeros(f.kb.buf.numel() - 64, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        K.make_kv_pool(small, f.kb.page_bytes, f.kb.pages, 2, 64, 32, K.KDA_INT8)
    c = torch.zeros((64, 32), device="cuda")
    for bad in ((c, c[:, :16]), (c, c.cpu()), (c.cpu(), c), (c.t(), c.t()), (c.bfloat16(), c.bfloat16()), (c[0], c[0])):
        with pytest.raises(ValueError):
            K.make_rope(*bad)
    torch.cuda.synchronize()
    assert torch.equal(before, f.kb.buf)


@pytest.mark.parametrize("cache", ["int8", "bf16"])
def test_pages_past_4_gib(cache):
    """The same tokens in the first and in the last pages of a pool of 5 GiB: equal bits from prompts
    (shared among workgroups and not) and decode steps."""
    H, hq, d, pt, n = 2, 8, 128, 64, 1500
    dtype = K.KDA_INT8 if cache == "int8" else K.KDA_BF16
    page = H * K.kda_kv_head_bytes(d, pt, dtype)
    need = -(-n // pt)
    pages = (5 << 30) // page
    buf = torch.zeros(pages * page // 4, dtype=torch.int32, device="cuda")
    pool = K.make_kv_pool(buf, page, pages, H, d, pt, dtype)
    near = torch.arange(need, dtype=torch.int32, device="cuda")[None].contiguous()
    far = pages - 1 - near
    rng = np.random.default_rng(17)
    k, v = (to_dev(rng.standard_normal((n, H, d)), "bf16") for _ in range(2))
    q = queries(rng, n, hq, d, "bf16")
    got = []
    for table in (near, far):
        K.kda_kv_append(pool, None, k, v, None, [0, n], table)
        for length, window in ((n, 0), (40, 0), (n, 100)):
            start = n - length
            w = ws(K.kda_attn_prefill_workspace_bytes(pool, hq, [0, length], start_pos=[start], window=window))
            o = torch.zeros((length, hq, d), dtype=torch.float32, device="cuda")
            K.kda_attn_prefill(pool, q[:length], o, [0, length], table, scale=0.1, start_pos=[start], window=window,
                               workspace=w)
            got.append(o)
        o = torch.zeros((2, hq, d), dtype=torch.float32, device="cuda")
        w = ws(K.kda_attn_decode_workspace_bytes(pool, hq, 1, 2, need))
        K.kda_attn_decode(pool, q[:2], o, 2, torch.tensor([n - 2], dtype=torch.int32, device="cuda"), table, scale=0.1,
                          workspace=w)
        got.append(o)
    assert all(torch.equal(a, b) and a.abs().sum() > 0 for a, b in zip(got[:4], got[4:]))


@pytest.mark.parametrize("hq,H,d,lens,starts", [(8, 2, 128, [16, 1, 5], [300, 900, 0]), (3, 1, 64, [21, 7], [40, 1500]),
                                                (64, 1, 64, [1, 1], [700, 31])])
def test_few_rows_keep_their_weights(hq, H, d, lens, starts):
    """bf16 queries over a bf16 cache, at most 64 rows a sequence and head, in a prompt call and in decode
    steps, fp32 output: a weight in two bf16 parts is off by at most 2^-8 of 2^-8 (half a step of each
    part), so the 2^-8 of one part in kv_gpu_util.tolerance becomes 2^-16; its other terms stand."""
    f = Filled([s + n for s, n in zip(starts, lens)], H, d, 64, "bf16", seed=hq)
    q = queries(np.random.default_rng(41), sum(lens), hq, d, "bf16")
    got = prefill(f, q, lens, starts, "bf16", "f32")
    cu = np.concatenate([[0], np.cumsum(lens)])
    last = torch.stack([q[int(e) - 1] for e in cu[1:]])
    step = decode(f, last, 1, [s + n - 1 for s, n in zip(starts, lens)], "f32")
    for r, (s, n) in enumerate(zip(starts, lens)):
        rows, pos = slice(int(cu[r]), int(cu[r + 1])), s + np.arange(n)
        for o, x, p in ((got[rows], q[rows], pos), (step[r:r + 1], last[r:r + 1], pos[-1:])):
            ref, mag, load = A.attend(host(x), f.held[r][0], f.held[r][1], p, d ** -0.5, 0, 0)
            tol = tolerance(ref, mag, load, s + n, d, "bf16", "f32", "bf16") - mag * (2.0 ** -8 - 2.0 ** -16)
            err = np.abs(host(o) - ref)
            assert (err <= tol).all(), (r, float((err / tol).max()))
