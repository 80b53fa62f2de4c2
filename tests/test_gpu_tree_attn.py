"""GPU parity of trees of drafted tokens over the paged cache (attention, append, the
accepted path kept) against the numpy oracle in 64 bits, with tolerances derived from
the roundings on the way (kv_gpu_util.tolerance)."""
import numpy as np
import pytest
import torch

import hybrid_prefix_cache_amd as K
from kv_gpu_util import TD, Filled, host, rope_tables, to_dev, tolerance, ws
from oracle import attention as A
from oracle import tree as T
from tree_util import pad, some_path, tree

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Draft:
    """Requests with `lens` cached tokens and a tree each, whose keys and values the oracle holds too."""

    def __init__(self, lens, parents, H, hq, d, pt, cache, dtype, rope=None, seed=1, amp=1.0, width=None):
        rng = np.random.default_rng(seed + 100)
        self.n, self.tokens = len(lens), len(parents[0])
        self.f = Filled(lens, H, d, pt, cache, seed=seed, spare=self.tokens, amp=amp, width=width)
        self.lens, self.parents, self.cache, self.dtype = lens, parents, cache, dtype
        rows = self.n * self.tokens
        self.qkv = to_dev(rng.standard_normal((rows, hq * d + 2 * H * d)), dtype)
        cut = self.qkv.split([hq * d, H * d, H * d], 1)
        self.q, self.k, self.v = (x.unflatten(1, (-1, d)) for x in cut)
        self.pos, self.parent = ints(lens), ints(parents)
        self.rope = rope
        if rope:
            rot, inter = rope
            self.tables_np = rope_tables(max(lens) + self.tokens, rot)
            self.rope_desc = K.make_rope(*(torch.from_numpy(x).cuda() for x in self.tables_np), interleaved=inter)

    def append(self):
        out = torch.full_like(self.q, 5.0).contiguous()
        K.kda_kv_append_tree(self.f.kb.pool, self.q, self.k, self.v, out, self.parent, self.pos, self.f.table,
                             rope=self.rope_desc if self.rope else None)
        return out

    def rotated(self, x, r):
        """fp32 values of request r's rows as the cache takes them: zeros for what is stored as none."""
        rows = host(x)[r * self.tokens: (r + 1) * self.tokens]
        w = T.ways(self.parents[r])
        depth = np.array([len(y) - 1 if y else 0 for y in w])
        if self.rope:
            rows = A.rotate(rows, self.lens[r] + depth, *self.tables_np, *self.rope)
        rows = A.f32(rows)
        rows[[not y for y in w]] = 0
        return rows

    def held(self, r, path=None):
        """Request r's cached keys and values (old, draft) after the append, and after a commit."""
        out = []
        f = self.f
        for part, x in ((0, self.k), (1, self.v)):
            new = self.rotated(x, r) if part == 0 else A.f32(np.where(
                np.array([bool(y) for y in T.ways(self.parents[r])])[:, None, None],
                host(x)[r * self.tokens: (r + 1) * self.tokens], 0))
            old = f.x[part][f.cu[r]: f.cu[r + 1]]
            if self.cache == "int8":
                b = A.Int8Blocks(new.shape[1], new.shape[2])
                b.append(old, 0)
                b.append(new, self.lens[r])
                if path is not None:
                    T.commit(b, self.lens[r], path)
                out.append(b.values(self.lens[r] + (self.tokens if path is None else len(path))))
            else:
                new = A.bf16(new)
                out.append(np.concatenate([old, new if path is None else new[path]]))
        return out

    def attend(self, out_dtype, window=0, sinks=0, w=None):
        o = torch.full((self.n * self.tokens + 1, *self.q.shape[1:]), 9.0, dtype=TD[out_dtype], device="cuda")
        if w is None:
            w = ws(K.kda_attn_tree_workspace_bytes(self.f.kb.pool, self.q.shape[1], self.n, self.tokens,
                                                   self.f.table.shape[1], window=window, sinks=sinks))
        w.fill_(0xFF)
        K.kda_attn_tree(self.f.kb.pool, self.q, o[:-1], self.parent, self.pos, self.f.table,
                        scale=self.q.shape[2] ** -0.5, window=window, sinks=sinks, workspace=w)
        assert (o[-1] == 9.0).all()
        return o[:-1]


def check_rows(got, d, r, out_dtype, window, sinks, tag):
    k, v = d.held(r)
    q = host(d.q)[r * d.tokens: (r + 1) * d.tokens]
    ref, mag, load = T.attend(q, k, v, d.lens[r], d.parents[r], q.shape[2] ** -0.5, window, sinks)
    y = host(got)[r * d.tokens: (r + 1) * d.tokens]
    tol = tolerance(ref, mag, load, len(k), q.shape[2], d.dtype, out_dtype, d.cache)
    for t, way in enumerate(T.ways(d.parents[r])):
        if way is None:
            assert np.isnan(y[t]).all(), (tag, r, t)
        elif not way:
            assert (y[t] == 0).all(), (tag, r, t)
        else:
            assert (np.abs(y[t] - ref[t]) <= tol[t]).all(), (tag, r, t, float((np.abs(y[t] - ref[t]) / tol[t]).max()))


ATTEND = [  # cache, dtype, out, hq, H, d, page_tokens, tokens, kinds, lens, window, sinks
    ("int8", "bf16", "bf16", 8, 2, 128, 64, 4, ("binary", "chain", "roots", "short"), [0, 31, 62, 500], 0, 0),
    ("int8", "bf16", "f32", 3, 1, 64, 32, 5, ("random", "holes", "none"), [700, 2, 40], 0, 0),
    ("bf16", "bf16", "bf16", 4, 1, 128, 96, 1, ("chain", "none"), [95, 96], 0, 0),
    ("bf16", "f32", "f32", 4, 4, 64, 64, 7, ("comb", "random"), [130, 3], 0, 0),
    ("int8", "f32", "f32", 7, 1, 128, 64, 3, ("roots", "random", "holes"), [60, 5, 255], 0, 0),
    ("int8", "bf16", "bf16", 8, 1, 128, 64, 64, ("binary", "random"), [10, 130], 0, 0),
    ("bf16", "bf16", "bf16", 12, 3, 128, 32, 21, ("random", "holes"), [90, 1], 0, 0),
    ("bf16", "f32", "f32", 4, 1, 64, 64, 40, ("comb",), [100], 0, 0),
    ("int8", "f32", "f32", 6, 1, 64, 32, 63, ("chain", "short"), [33, 0], 0, 0),
    # windows: one position, shorter than the tree's ways, across pages; sinks in and past the tree
    ("bf16", "bf16", "bf16", 4, 2, 128, 64, 6, ("chain", "random", "comb"), [300, 5, 0], 1, 0),
    ("int8", "bf16", "bf16", 8, 2, 64, 64, 9, ("chain", "binary"), [300, 77], 4, 3),
    ("bf16", "f32", "f32", 2, 1, 128, 32, 33, ("chain", "comb"), [40, 2], 10, 5),
    ("int8", "bf16", "f32", 16, 1, 64, 96, 30, ("comb", "holes"), [200, 7], 20, 40),
    ("bf16", "bf16", "bf16", 5, 1, 64, 64, 64, ("chain",), [9], 12, 0),
]


@pytest.mark.parametrize("case", ATTEND, ids=lambda c: "-".join(str(x) for x in c[:8]) + f"-w{c[10]}")
def test_attend(case):
    cache, dtype, out, hq, H, d, pt, tokens, kinds, lens, window, sinks = case
    parents = [tree(k, tokens, i) for i, k in enumerate(kinds)]
    x = Draft(lens, parents, H, hq, d, pt, cache, dtype)
    x.append()
    got = x.attend(out, window, sinks)
    for r in range(len(lens)):
        check_rows(got, x, r, out, window, sinks, case)


@pytest.mark.parametrize("cache", ["int8", "bf16"])
@pytest.mark.parametrize("tokens,hq", [(6, 4), (20, 8)])
def test_split_caches(cache, tokens, hq):
    """Few rows over long caches: shared among workgroups and joined, with entries that are no nodes and bad ones."""
    lens = [5000, 0, 1300]
    x = Draft(lens, [tree("random", tokens, 1), tree("holes", tokens, 4), tree("holes", tokens, 7)], 1, hq, 64, 64, cache,
              "bf16")
    assert K.kda_attn_tree_workspace_bytes(x.f.kb.pool, hq, 3, tokens, x.f.table.shape[1]) > 256
    x.append()
    got = x.attend("bf16")
    for r in range(3):
        check_rows(got, x, r, "bf16", 0, 0, (cache, tokens))


@pytest.mark.parametrize("cache,dtype", [("int8", "bf16"), ("bf16", "bf16"), ("int8", "f32")])
@pytest.mark.parametrize("n,tokens,hq", [(65, 17, 2), (131, 9, 4), (150, 34, 2), (70, 12, 16)])
def test_many_requests_longest_first(cache, dtype, n, tokens, hq):
    """More requests than a wave orders at once, most of them alike in length, some without part."""
    rng = np.random.default_rng(n)
    lens = [int(x) for x in rng.choice([0, 1, 31, 32, 40, 200], n)]
    d = Draft(lens, [tree(("random", "comb", "roots", "holes")[i % 4], tokens, i) for i in range(n)], 1, hq, 64, 64, cache, dtype,
              seed=n)
    out = [i for i in range(n) if i % 11 == 5]
    d.append()
    d.pos[torch.tensor(out, device="cuda")] = -1
    o = d.attend("f32")
    for r in range(n):
        if r in out:
            assert (host(o)[r * tokens: (r + 1) * tokens] == 0).all()
        else:
            check_rows(o, d, r, "f32", 0, 0, (cache, n))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("tokens,hq", [(5, 2), (24, 8)])
def test_other_branches_do_not_reach_a_row(bad, tokens, hq):
    """bf16 cache: a node's keys or values that are not finite are its descendants' alone."""
    row = tree("roots", tokens)
    row[-1] = 1
    x = Draft([45], [row], 1, hq, 64, 32, "bf16", "bf16")
    x.append()
    clean = x.attend("f32")
    for part in (x.k, x.v):
        part[0] = bad
    x.append()
    got = x.attend("f32")
    assert torch.equal(got[1:], clean[1:]) or np.allclose(host(got[1:]), host(clean[1:]), rtol=1e-6, atol=1e-7)
    assert not torch.isfinite(got[0]).any()


def test_a_chain_is_a_step():
    """A tree that is a chain gives kda_kv_append_step's cache to the bit, and rows that are as near the exact
    ones as kda_attn_decode's (few rows, which one kernel takes in both calls: its bits)."""
    for cache, tokens, hq in (("int8", 5, 4), ("bf16", 40, 4)):
        a, b = (Draft([70, 3], [tree("chain", tokens)] * 2, 1, hq, 64, 32, cache, "bf16", rope=(64, False)) for _ in range(2))
        qa = a.append()
        qb = torch.zeros_like(qa)
        K.kda_kv_append_step(b.f.kb.pool, b.q, b.k, b.v, qb, tokens, b.pos, b.f.table, rope=b.rope_desc)
        assert torch.equal(qa, qb) and torch.equal(a.f.kb.buf, b.f.kb.buf)
        got, o = a.attend("bf16"), torch.zeros((2 * tokens, hq, 64), dtype=torch.bfloat16, device="cuda")
        w = ws(K.kda_attn_decode_workspace_bytes(b.f.kb.pool, hq, 2, tokens, b.f.table.shape[1]))
        K.kda_attn_decode(b.f.kb.pool, b.q, o, tokens, b.pos, b.f.table, scale=64 ** -0.5, workspace=w)
        if tokens * hq <= 32:
            assert torch.equal(got, o)
        for r in range(2):
            check_rows(got, a, r, "bf16", 0, 0, "tree")
            check_rows(o, a, r, "bf16", 0, 0, "step")


APPEND = [  # cache, dtype, hq, H, d, page_tokens, tokens, rot, interleaved, kinds, lens
    ("int8", "bf16", 4, 2, 128, 64, 7, 128, False, ("random", "holes", "short"), [0, 61, 30]),
    ("int8", "f32", 3, 1, 64, 32, 64, 32, True, ("binary", "random"), [31, 100]),
    ("bf16", "bf16", 2, 2, 64, 96, 33, 64, True, ("comb", "holes"), [5, 95]),
    ("bf16", "f32", 5, 1, 128, 32, 1, 16, False, ("chain", "none"), [32, 8]),
    ("int8", "bf16", 2, 1, 64, 64, 64, 64, False, ("chain", "roots"), [17, 64]),
]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: "-".join(str(x) for x in c[:8]))
@pytest.mark.parametrize("longest", [True, False])
def test_append_commit_read(case, longest):
    cache, dtype, hq, H, d, pt, tokens, rot, inter, kinds, lens = case
    parents = [tree(k, tokens, i + 1) for i, k in enumerate(kinds)]
    x = Draft(lens, parents, H, hq, d, pt, cache, dtype, rope=(rot, inter))
    q_out = host(x.append())
    half = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}[dtype]
    for r in range(len(lens)):
        w = T.ways(parents[r])
        want = x.rotated(x.q, r)
        for t in range(tokens):
            y = q_out[r * tokens + t]
            if w[t] is None:
                assert np.isnan(y).all()
            else:
                # one rounding to fp32 and one to the type
                assert (np.abs(y - want[t]) <= np.abs(want[t]) * (half + 2.0 ** -24)).all()

    def read(ends):
        cu = np.concatenate([[0], np.cumsum(ends)])
        out = [torch.zeros((int(cu[-1]), H, d), device="cuda") for _ in range(2)]
        K.kda_kv_read(x.f.kb.pool, *out, cu, x.f.table)
        return cu, [host(y) for y in out]

    # a value: code or bf16 element times scale, in fp32
    cu, got = read([n + tokens for n in lens])
    for r in range(len(lens)):
        for part, want in enumerate(x.held(r)):
            y = got[part][cu[r]: cu[r + 1]]
            assert (np.abs(y - want) <= np.abs(want) * 2.0 ** -24).all(), (r, part)
    paths = [some_path(p, i, node=None if longest else True) for i, p in enumerate(parents)]
    path, count = pad(paths, tokens)
    before = x.f.kb.bytes()
    K.kda_kv_commit(x.f.kb.pool, ints(path), ints(count), x.pos, x.f.table)
    cu, got = read([n + len(p) for n, p in zip(lens, paths)])
    for r in range(len(lens)):
        for part, want in enumerate(x.held(r, paths[r])):
            y = got[part][cu[r]: cu[r + 1]]
            assert (np.abs(y - want) <= np.abs(want) * 2.0 ** -24).all(), (r, part)
    # nothing but the pages of the accepted slots has changed
    after = x.f.kb.bytes()
    pages = {int(x.f.table_np[r, j]) for r, n in enumerate(lens) for j in range(n // pt, (n + max(len(paths[r]), 1) - 1) // pt + 1)}
    for p in range(len(after)):
        assert p in pages or (before[p] == after[p]).all()


@pytest.mark.parametrize("path,count", [([0, 1, 1, -7], 3), ([2, 1, -7, -7], 2), ([0, 4, -7, -7], 2), ([-1, 2, -7, -7], 2),
                                        ([1, 2, 3, -7], 5), ([1, 2, 3, -7], -1), ([0, 1, 2, 3], 4), ([3, 2, 1, 0], 0)])
def test_paths_that_move_nothing(path, count):
    """Bad paths, and paths whose rows are in their places already."""
    x = Draft([40, 40], [tree("random", 4)] * 2, 1, 2, 64, 32, "int8", "bf16")
    x.append()
    before = x.f.kb.buf.clone()
    K.kda_kv_commit(x.f.kb.pool, ints([path] * 2), ints([count] * 2), x.pos, x.f.table)
    assert torch.equal(before, x.f.kb.buf)


def test_commit_where_nothing_may_be_written():
    x = Draft([40, 60, 30], [tree("chain", 8)] * 3, 1, 2, 64, 32, "bf16", "bf16")
    x.append()
    path, count = pad([[1, 3, 5]] * 3, 8)
    before = x.f.kb.buf.clone()
    table = x.f.table.clone()
    table[1, 1], table[2, 0] = -1, 10 ** 6   # a page in which rows begin, and one past the pool
    K.kda_kv_commit(x.f.kb.pool, ints(path), ints(count), ints([-1, 60, 30]), table)
    # the row's end: 3 pages of 32
    K.kda_kv_commit(x.f.kb.pool, ints(path[:1]), ints(count[:1]), ints([89]), x.f.table[:1, :3].contiguous())
    assert torch.equal(before, x.f.kb.buf)


def test_requests_without_part_and_past_their_rows():
    x = Draft([40, 60, 30], [tree("binary", 6)] * 3, 1, 4, 64, 32, "int8", "bf16")
    x.append()
    ref = x.attend("f32")
    before = x.f.kb.buf.clone()
    end = x.f.table.shape[1] * 32
    x.pos = ints([-1, end - 3, 30])
    out = x.append()
    assert (out[:6] == 0).all()
    got = x.attend("f32")
    assert (got[:6] == 0).all() and torch.isnan(got[6:12]).all() and torch.equal(got[12:], ref[12:])
    # the third request's rows again, the second's into its row's last slots, if there are pages
    changed = (before != x.f.kb.buf).view(x.f.kb.pages, -1).any(1)
    allowed = {int(p) for p in x.f.table_np[1, (end - 3) // 32:].tolist() if p >= 0}
    assert {int(p) for p in changed.nonzero()} <= allowed


def test_rotation_ends():
    """Nodes past the rotation table: not stored (zeros), NaN rows; the others as they are."""
    x = Draft([20], [tree("chain", 6)], 1, 2, 64, 32, "bf16", "bf16", rope=(64, False))
    cos, sin = (torch.from_numpy(t[:23].copy()).cuda() for t in x.tables_np)
    out = torch.zeros_like(x.q).contiguous()
    K.kda_kv_append_tree(x.f.kb.pool, x.q, x.k, x.v, out, x.parent, x.pos, x.f.table, rope=K.make_rope(cos, sin))
    assert torch.isfinite(out[:3]).all() and torch.isnan(out[3:]).all()
    k = [torch.zeros((6, 1, 64), device="cuda") for _ in range(2)]
    K.kda_kv_read(x.f.kb.pool, *k, [0, 6], x.f.table, start_pos=[20])
    assert (k[0][3:] == 0).all() and (k[1][3:] == 0).all() and (k[0][:3] != 0).any()


def test_a_step_in_graphs_and_on_two_streams():
    """Append, attend and commit captured and replayed with other trees, each graph with its own workspace."""
    a = Draft([70, 300], [tree("binary", 12), tree("random", 12)], 2, 8, 64, 32, "int8", "bf16", rope=(64, False))
    b = Draft([70, 300], [tree("binary", 12), tree("random", 12)], 2, 8, 64, 32, "int8", "bf16", rope=(64, False))
    need = K.kda_attn_tree_workspace_bytes(a.f.kb.pool, 8, 2, 12, a.f.table.shape[1])
    state = []
    for x in (a, b):
        path, count = pad([some_path(p) for p in x.parents], 12)
        state.append(dict(o=torch.zeros((24, 8, 64), dtype=torch.bfloat16, device="cuda"), q=torch.zeros_like(x.q).contiguous(),
                          w=ws(need), path=ints(path), count=ints(count)))

    def step(x, s):
        K.kda_kv_append_tree(x.f.kb.pool, x.q, x.k, x.v, s["q"], x.parent, x.pos, x.f.table, rope=x.rope_desc)
        K.kda_attn_tree(x.f.kb.pool, s["q"], s["o"], x.parent, x.pos, x.f.table, scale=0.125, workspace=s["w"])
        K.kda_kv_commit(x.f.kb.pool, s["path"], s["count"], x.pos, x.f.table)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step(a, state[0])
    torch.cuda.current_stream().wait_stream(side)
    for i in range(4):
        parents = [tree("random", 12, i), tree("holes", 12, i)]
        path, count = pad([some_path(p) for p in parents], 12)
        for x, s in ((a, state[0]), (b, state[1])):
            x.parent.copy_(ints(parents))
            s["path"].copy_(ints(path))
            s["count"].copy_(ints(count))
            s["w"].fill_(0xFF)
        g.replay()
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.current_stream())
            step(b, state[1])
        torch.cuda.synchronize()
        assert torch.equal(state[0]["o"].view(torch.int16), state[1]["o"].view(torch.int16)), i
        assert torch.equal(a.f.kb.buf, b.f.kb.buf), i


def test_pages_past_4_gib():
    """The same draft in the first and in the last pages of a pool of 5 GiB."""
    H, hq, d, pt, n, tokens = 2, 8, 128, 64, 300, 20
    page = H * K.kda_kv_head_bytes(d, pt, K.KDA_INT8)
    need, pages = -(-(n + tokens) // pt), (5 << 30) // page
    pool = K.make_kv_pool(torch.zeros(pages * page // 4, dtype=torch.int32, device="cuda"), page, pages, H, d, pt, K.KDA_INT8)
    near = torch.arange(need, dtype=torch.int32, device="cuda")[None].contiguous()
    far = pages - 1 - near
    rng = np.random.default_rng(3)
    old = [to_dev(rng.standard_normal((n, H, d)), "bf16") for _ in range(2)]
    q, k, v = (to_dev(rng.standard_normal((tokens, h, d)), "bf16") for h in (hq, H, H))
    parent, pos = ints([tree("random", tokens)]), ints([n])
    path, count = pad([some_path(tree("random", tokens))], tokens)
    got = []
    for table in (near, far):
        K.kda_kv_append(pool, None, *old, None, [0, n], table)
        K.kda_kv_append_tree(pool, None, k, v, None, parent, pos, table)
        o, w = torch.zeros_like(q), ws(K.kda_attn_tree_workspace_bytes(pool, hq, 1, tokens, need))
        K.kda_attn_tree(pool, q, o, parent, pos, table, scale=0.1, workspace=w)
        K.kda_kv_commit(pool, ints(path), ints(count), pos, table)
        r = [torch.zeros((n + int(count[0]), H, d), device="cuda") for _ in range(2)]
        K.kda_kv_read(pool, *r, [0, n + int(count[0])], table)
        got.append([o, *r])
    for x, y in zip(*got):
        assert torch.equal(x, y) and (x != 0).any()


def test_host_validation(monkeypatch):
    monkeypatch.setenv("KDA_VALIDATE", "1")
    x = Draft([40, 60], [tree("binary", 6)] * 2, 1, 4, 64, 32, "int8", "bf16")
    x.append()
    x.attend("f32")
    good = x.parent.clone()
    for bad in (6, 2):  # an entry past the tree, and a child of no node
        x.parent.copy_(good)
        x.parent[1, 3] = bad
        x.parent[1, 2] = -2 if bad == 2 else 0
        for call in (x.append, lambda: x.attend("f32")):
            with pytest.raises(K.KdaError) as e:
                call()
            assert e.value.status == K.KDA_ERR_SEQ
    x.parent.copy_(good)
    x.parent[:, 4:] = -2
    x.attend("f32")
    for path, count in (([[0, 0, 0, 0, 0, 0]] * 2, [2, 0]), ([[0, 1, 3, 0, 0, 0]] * 2, [3, 7])):
        with pytest.raises(K.KdaError) as e:
            K.kda_kv_commit(x.f.kb.pool, ints(path), ints(count), x.pos, x.f.table)
        assert e.value.status == K.KDA_ERR_SEQ
    table = x.f.table.clone()
    table[1] = table[0]
    with pytest.raises(K.KdaError) as e:
        K.kda_kv_append_tree(x.f.kb.pool, None, x.k, x.v, None, x.parent, x.pos, table)
    assert e.value.status == K.KDA_ERR_PAGE_ALIAS


def test_bindings_refuse():
    x = Draft([40, 60], [tree("binary", 6)] * 2, 1, 4, 64, 32, "int8", "bf16")
    pool, table, p = x.f.kb.pool, x.f.table, x.parent
    o, w = torch.zeros((12, 4, 64), dtype=torch.bfloat16, device="cuda"), ws(1 << 20)
    path, count = ints([[0] * 6] * 2), ints([1, 1])
    before = x.f.kb.buf.clone()
    bad = [
        lambda: K.kda_attn_tree(pool, x.q, o, p.long(), x.pos, table, scale=0.1, workspace=w),
        lambda: K.kda_attn_tree(pool, x.q, o, p[0], x.pos, table, scale=0.1, workspace=w),
        lambda: K.kda_attn_tree(pool, x.q, o, p[:, :5], x.pos, table, scale=0.1, workspace=w),
        lambda: K.kda_attn_tree(pool, x.q, o, p.cpu(), x.pos, table, scale=0.1, workspace=w),
        lambda: K.kda_attn_tree(pool, x.q, o[:11], p, x.pos, table, scale=0.1, workspace=w),
        lambda: K.kda_attn_tree(pool, x.q, o, p, x.pos[:1], table, scale=0.1, workspace=w),
        lambda: K.kda_attn_tree(pool, x.q, o, p, x.pos, table[:1], scale=0.1, workspace=w),
        lambda: K.kda_attn_tree(pool, x.q, o, p, x.pos, table, scale=0.1, workspace=None),
        lambda: K.kda_kv_append_tree(pool, x.q, x.k, x.v, None, p, x.pos, table),
        lambda: K.kda_kv_append_tree(pool, None, x.k[:6], x.v, None, p, x.pos, table),
        lambda: K.kda_kv_append_tree(pool, None, x.k, x.v.float(), None, p, x.pos, table),
        lambda: K.kda_kv_commit(pool, path, count[:1], x.pos, table),
        lambda: K.kda_kv_commit(pool, path.t().contiguous(), count, x.pos, table),
        lambda: K.kda_kv_commit(pool, path, count, x.pos.long(), table),
    ]
    for call in bad:
        with pytest.raises((ValueError, K.KdaError)):
            call()
    torch.cuda.synchronize()
    assert torch.equal(before, x.f.kb.buf)


@pytest.mark.parametrize("seed", range(12))
def test_random_calls(seed):
    rng = np.random.default_rng(1000 + seed)
    H, g, d = int(rng.choice([1, 2, 3])), int(rng.choice([1, 2, 4, 7])), int(rng.choice([64, 128]))
    cache, dtype = str(rng.choice(["int8", "bf16"])), str(rng.choice(["bf16", "bf16", "f32"]))
    tokens, n, pt = int(rng.integers(1, 65)), int(rng.integers(1, 4)), int(rng.choice([32, 64, 160]))
    lens = [int(x) for x in rng.integers(0, 260, n)]
    kinds = ["random", "holes", "comb", "short", "binary"]
    parents = [tree(kinds[int(rng.integers(5))], tokens, seed + i) for i in range(n)]
    window = int(rng.choice([0, 0, 3, 50]))
    x = Draft(lens, parents, H, H * g, d, pt, cache, dtype, seed=seed)
    x.append()
    got = x.attend(dtype, window, 2)
    for r in range(n):
        check_rows(got, x, r, dtype, window, 2, seed)
