"""GPU parity of the recurrence and the short convolution along trees of drafted tokens,
and of their commits, against the numpy oracle in 64 bits and against the calls for
single tokens."""
import numpy as np
import pytest
import torch

import hybrid_prefix_cache_amd as K
from kda_gpu_util import PoolBuf
from kv_gpu_util import TD, host, to_dev
from oracle import tree as T
from oracle.attention import bf16
from tree_util import pad, some_path, tree

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class States:
    def __init__(self, parents, H, d, dtype, seed=0, gate=0.05, scale=1.0):
        rng = np.random.default_rng(seed)
        self.n, self.tokens, self.H, self.d, self.dtype, self.parents = len(parents), len(parents[0]), H, d, dtype, parents
        rows = self.n * self.tokens
        q, k, v = (rng.standard_normal((rows, H, d)) for _ in range(3))
        q, k = (x / np.linalg.norm(x, axis=-1, keepdims=True) for x in (q, k))
        g, beta = -gate * rng.random((rows, H, d)), 1 / (1 + np.exp(-rng.standard_normal((rows, H))))
        self.x = {name: to_dev(y, dtype) for name, y in dict(q=q, k=k, v=scale * v, g=g, beta=beta).items()}
        self.pb = PoolBuf(2 * self.n + 1, H, d, page_bytes=H * d * d * 4 + 256)
        self.page_in, self.page_out = rng.permutation(self.n), self.n + rng.permutation(self.n)
        self.S0 = [scale * rng.standard_normal((H, d, d)).astype(np.float32) / np.sqrt(d) for _ in range(self.n)]
        for p, s in zip(self.page_in, self.S0):
            self.pb.set_states(int(p), s)
        self.parent = ints(parents)

    def row(self, name, r):
        return host(self.x[name])[r * self.tokens: (r + 1) * self.tokens]

    def run(self, out):
        o = torch.full((self.n * self.tokens + 1, self.H, self.d), 9.0, dtype=TD[out], device="cuda")
        x = self.x
        K.kda_decode_tree(self.pb.pool, x["q"], x["k"], x["v"], x["g"], x["beta"], o[:-1], self.parent, ints(self.page_in))
        assert (o[-1] == 9.0).all()
        return o[:-1]

    def check(self, o, out, tag=None):
        """Sums of up to d + 64 terms, four of them one in another (the gated products, the triangular
        system, its product with the values, the state's), with 2^-24 a term; gates summed and
        exponentiated (2^-24 of the sum each); bf16 inputs: two-part operands, 2^-15 a product of four.
        The sums' size is recur_size's."""
        y = host(o)
        for r in range(self.n):
            a = [self.row(name, r) for name in ("q", "k", "v", "g", "beta")]
            w = T.ways(self.parents[r])
            for i in range(3):
                a[i][[not z for z in w]] = 0
            ref, _ = T.recur(*a, self.parents[r], self.S0[r].astype(np.float64))
            size = T.recur_size(*a, self.parents[r], self.S0[r].astype(np.float64))
            gates = max([-np.maximum(a[3][z], -104).sum(0).min() for z in w if z] + [0])
            eps = (4 * (self.d + 64) + 4 * min(gates, 120) + 40) * 2.0 ** -24 + (4 * 2.0 ** -15 if self.dtype == "bf16" else 0)
            tol = eps * size + np.abs(ref) * (2.0 ** -8 if out == "bf16" else 2.0 ** -24) + 1e-35
            for t, way in enumerate(w):
                z = y[r * self.tokens + t]
                if way is None:
                    assert np.isnan(z).all(), (tag, r, t)
                elif not way:
                    assert (z == 0).all(), (tag, r, t)
                else:
                    assert (np.abs(z - ref[t]) <= tol[t]).all(), (tag, r, t, float((np.abs(z - ref[t]) / tol[t]).max()))


CASES = [  # kinds, tokens, H, d, dtype, out
    (("chain",), 1, 1, 128, "bf16", "bf16"),
    (("binary", "random"), 7, 3, 128, "bf16", "f32"),
    (("roots", "comb"), 16, 2, 128, "f32", "f32"),
    (("random", "holes"), 17, 2, 128, "bf16", "bf16"),
    (("chain", "short"), 33, 2, 128, "f32", "bf16"),
    (("comb", "binary"), 48, 1, 128, "bf16", "f32"),
    (("chain", "random"), 64, 2, 128, "bf16", "bf16"),
    (("chain", "holes"), 64, 1, 128, "f32", "f32"),
    (("random",), 2, 5, 64, "f32", "f32"),
    (("holes", "none"), 15, 2, 64, "bf16", "f32"),
    (("binary", "chain"), 32, 1, 64, "bf16", "bf16"),
    (("random", "comb"), 47, 2, 64, "f32", "f32"),
    (("chain", "roots"), 63, 2, 64, "bf16", "f32"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:1][0] + c[1:])))
@pytest.mark.parametrize("gate", [0.05, 1.0, 0.0])
def test_tree(case, gate):
    kinds, tokens, H, d, dtype, out = case
    x = States([tree(k, tokens, i) for i, k in enumerate(kinds)], H, d, dtype, seed=tokens, gate=gate)
    before = x.pb.buf.clone()
    x.check(x.run(out), out, case)
    assert torch.equal(before, x.pb.buf)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
@pytest.mark.parametrize("gate", [3.0, 40.0, 400.0])
def test_gates_that_forget_at_once(dtype, d, gate):
    """Sums of gates past the factored form: pair by pair; past fp32's exponent: forgotten."""
    x = States([tree("chain", 40), tree("comb", 40)], 2, d, dtype, seed=3, gate=gate)
    x.check(x.run("f32"), "f32", gate)


def test_a_gate_of_minus_infinity_forgets():
    x = States([tree("chain", 6), tree("binary", 6)], 1, 64, "bf16", seed=4)
    x.x["g"][2] = -float("inf")
    x.check(x.run("f32"), "f32")


@pytest.mark.parametrize("name,bad", [("k", float("nan")), ("v", float("inf")), ("beta", float("nan")), ("g", float("nan")),
                                      ("g", float("inf")), ("k", -float("inf"))])
@pytest.mark.parametrize("tokens", [9, 40])
def test_values_that_are_not_finite_are_their_descendants_alone(name, bad, tokens):
    row = tree("binary", tokens)
    x = States([row, row], 2, 64, "bf16", seed=5)
    clean = x.run("f32")
    y = x.x[name]
    (y[1] if y.dim() == 2 else y[1, :, 5]).fill_(bad)  # node 1 of the first request
    got = x.run("f32")
    for t, way in enumerate(T.ways(row)):
        if 1 in way:
            assert torch.isnan(got[t]).all(), t
        else:
            assert torch.equal(got[t], clean[t]), t
    assert torch.equal(got[tokens:], clean[tokens:])


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 128), ("bf16", 64)])
@pytest.mark.parametrize("tokens", [16, 20, 48, 64])
@pytest.mark.parametrize("gate", [0.05, 40.0])
def test_values_that_are_not_finite_beside_gates_that_forget(dtype, d, tokens, gate):
    """The same where A and Q are summed pair by pair, in every size of the kernels, in a tree with holes."""
    row = tree("holes", tokens, 2)
    ways = T.ways(row)
    x = States([row, tree("comb", tokens)], 2, d, dtype, seed=tokens, gate=gate)
    clean = x.run("f32")
    nodes = [t for t, way in enumerate(ways) if way]
    spoilt = nodes[1::5]
    for i, t in enumerate(spoilt):
        y = x.x[("k", "v", "beta")[i % 3]]
        (y[t, 1:] if y.dim() == 2 else y[t, 1:, 3 * i % d]).fill_((float("nan"), float("inf"), -float("inf"))[i // 3 % 3])
    got = x.run("f32")
    assert torch.equal(got[:, 0].nan_to_num(7.0), clean[:, 0].nan_to_num(7.0))
    for t, way in enumerate(ways):
        if way and set(way) & set(spoilt):
            assert torch.isnan(got[t, 1]).all(), t
        else:
            assert torch.equal(got[t, 1].nan_to_num(7.0), clean[t, 1].nan_to_num(7.0)), t
    assert torch.equal(got[tokens:], clean[tokens:])


def test_rows_of_no_node_are_not_read():
    row = tree("holes", 20, 3)
    x = States([row], 2, 64, "f32", seed=6)
    clean = x.run("f32")
    for t, way in enumerate(T.ways(row)):
        if not way:
            for y in x.x.values():
                y[t] = float("nan")
    got = x.run("f32")
    assert torch.equal(got.isnan(), clean.isnan()) and torch.equal(got.nan_to_num(), clean.nan_to_num())


def test_bad_pages():
    x = States([tree("binary", 5)] * 3, 2, 64, "bf16", seed=7)
    ref = x.run("f32")
    x.page_in[0], x.page_in[2] = -1, 7
    got = x.run("f32")
    assert torch.isnan(got[:5]).all() and torch.equal(got[5:10], ref[5:10]) and torch.isnan(got[10:]).all()
    before = x.pb.buf.clone()
    path, count = pad([[0, 1]] * 3, 5)
    a = x.x
    K.kda_decode_commit(x.pb.pool, a["k"], a["v"], a["g"], a["beta"], ints(path), ints(count), ints([-1, x.page_in[1], 3]),
                        ints([3, 99, -2]))
    for p, c in (([2, 1, 0, 0, 0], 2), ([1, 1, 0, 0, 0], 2), ([0, 5, 0, 0, 0], 2), ([0, 1, 2, 3, 4], 6), ([0] * 5, -1)):
        K.kda_decode_commit(x.pb.pool, a["k"], a["v"], a["g"], a["beta"], ints([p] * 3), ints([c] * 3), ints([0, 1, 2]), ints([3, 4, 5]))
    assert torch.equal(before, x.pb.buf)


@pytest.mark.parametrize("dtype,d,tokens", [("bf16", 128, 9), ("f32", 128, 3), ("bf16", 64, 40), ("f32", 64, 64)])
@pytest.mark.parametrize("in_place", [True, False])
def test_commit_gives_the_decode_steps_bits(dtype, d, tokens, in_place):
    parents = [tree("random", tokens, 1), tree("chain", tokens), tree("comb", tokens), tree("roots", tokens)]
    x = States(parents, 2, d, dtype, seed=8)
    paths = [some_path(parents[0]), some_path(parents[1]), some_path(parents[2], 3, True), []]
    path, count = pad(paths, tokens)
    a, out = x.x, x.page_in if in_place else x.page_out
    want = []
    for r in range(4):
        p = PoolBuf(1, 2, d)
        p.set_states(0, x.S0[r])
        for t in paths[r]:
            row = slice(r * tokens + t, r * tokens + t + 1)
            K.kda_decode_step(p.pool, *(a[name][row] for name in ("q", "k", "v", "g", "beta")),
                              torch.empty((1, 2, d), dtype=torch.float32, device="cuda"), ints([0]), ints([0]))
        want.append(p.states(0))
    before = x.pb.snapshot().reshape(2 * x.n + 1, -1)
    K.kda_decode_commit(x.pb.pool, a["k"], a["v"], a["g"], a["beta"], ints(path), ints(count), ints(x.page_in), ints(out))
    for r in range(4):
        assert np.array_equal(x.pb.states(int(out[r])), want[r]), r
    after = x.pb.snapshot().reshape(2 * x.n + 1, -1)
    words = 2 * d * d
    for p in range(2 * x.n + 1):
        same = before[p] == after[p]
        assert (same if p not in out else same[words:]).all()


def test_a_chain_is_a_verification():
    """Rows of a chain agree with kda_decode_verify's to both calls' roundings, states to the bit."""
    x = States([tree("chain", 12)] * 2, 2, 128, "f32", seed=9)
    got = x.run("f32")
    a = x.x
    v = PoolBuf(26, 2, 128)
    for r in range(2):
        v.set_states(r, x.S0[r])
    o = torch.empty_like(got)
    K.kda_decode_verify(v.pool, a["q"], a["k"], a["v"], a["g"], a["beta"], o, 12, ints([0, 1]), ints(list(range(2, 26))))
    x.check(got, "f32")
    x.check(o, "f32")
    K.kda_decode_commit(x.pb.pool, a["k"], a["v"], a["g"], a["beta"], ints([list(range(12))] * 2), ints([12, 5]), ints(x.page_in),
                        ints(x.page_out))
    assert np.array_equal(x.pb.states(int(x.page_out[0])), v.states(13)) and np.array_equal(x.pb.states(int(x.page_out[1])), v.states(18))


def test_state_far_in_the_pool():
    """Pages past 4 GiB."""
    H, d, pages = 32, 128, 2100
    pool = torch.zeros(pages * H * d * d, device="cuda")
    x = States([tree("binary", 10)], H, d, "bf16", seed=10)
    ref = x.run("f32")
    pool[(pages - 1) * H * d * d:] = torch.from_numpy(x.S0[0]).reshape(-1).cuda()
    o, a = torch.empty_like(ref), x.x
    p = K.make_pool(pool, H * d * d * 4, pages, H, d)
    K.kda_decode_tree(p, a["q"], a["k"], a["v"], a["g"], a["beta"], o, x.parent, ints([pages - 1]))
    assert torch.equal(o, ref)
    path, count = pad([[0, 2, 5]], 10)
    for where, page in ((x.pb.pool, int(x.page_in[0])), (p, pages - 1)):
        K.kda_decode_commit(where, a["k"], a["v"], a["g"], a["beta"], ints(path), ints(count), ints([page]), ints([page]))
    assert np.array_equal(pool[(pages - 1) * H * d * d:].cpu().numpy().reshape(H, d, d), x.pb.states(int(x.page_in[0])).astype(np.float32))


class Conv:
    def __init__(self, parents, C, W, dtype, seed=0):
        rng = np.random.default_rng(seed)
        self.n, self.tokens, self.C, self.W, self.dtype, self.parents = len(parents), len(parents[0]), C, W, dtype, parents
        self.x = to_dev(rng.standard_normal((self.n * self.tokens, C)), dtype)
        self.w = to_dev(rng.standard_normal((C, W)), "f32")
        e = 2 if dtype == "bf16" else 4
        self.page = -(-(W - 1) * C * e // 256) * 256 + 256
        self.buf = torch.full((2 * self.n * self.page,), 0xFF, dtype=torch.uint8, device="cuda")
        self.pool = K.make_conv_pool(self.buf, self.page, 2 * self.n, C, W, K.KDA_BF16 if dtype == "bf16" else K.KDA_F32)
        self.page_in, self.page_out = rng.permutation(self.n), self.n + rng.permutation(self.n)
        self.windows = to_dev(rng.standard_normal((self.n, W - 1, C)), dtype)
        for p, w in zip(self.page_in, self.windows):
            self.rows(p).copy_(w)
        self.parent = ints(parents)

    def rows(self, p):
        e = 2 if self.dtype == "bf16" else 4
        return self.buf[int(p) * self.page: int(p) * self.page + (self.W - 1) * self.C * e].view(TD[self.dtype]).view(self.W - 1, self.C)

    def run(self, out):
        y = torch.full((self.n * self.tokens + 1, self.C), 9.0, dtype=TD[out], device="cuda")
        K.kda_short_conv_tree(self.pool, self.x, self.w, y[:-1], self.parent, ints(self.page_in))
        assert (y[-1] == 9.0).all()
        return y[:-1]


CONV = [(("random", "binary"), 7, 1024, 4, "bf16", "bf16"), (("chain", "holes"), 64, 264, 4, "bf16", "f32"),
        (("comb", "none"), 9, 2056, 3, "f32", "f32"), (("roots", "short"), 1, 8, 2, "bf16", "bf16"),
        (("chain", "random"), 17, 4, 4, "f32", "bf16"), (("random", "holes"), 33, 520, 2, "f32", "f32")]


@pytest.mark.parametrize("case", CONV, ids=lambda c: "-".join(map(str, c[0] + c[1:])))
def test_conv_tree(case):
    kinds, tokens, C, W, dtype, out = case
    c = Conv([tree(k, tokens, i) for i, k in enumerate(kinds)], C, W, dtype, seed=tokens)
    before = c.buf.clone()
    y = c.run(out)
    assert torch.equal(before, c.buf)
    for r in range(c.n):
        x = host(c.x)[r * tokens: (r + 1) * tokens]
        ref, mag = T.convolve(x, host(c.w), c.parents[r], host(c.windows[r]))
        got = host(y)[r * tokens: (r + 1) * tokens]
        tol = mag * (W + 1) * 2.0 ** -24 + np.abs(ref) * (2.0 ** -8 if out == "bf16" else 0)
        for t, way in enumerate(T.ways(c.parents[r])):
            if way is None:
                assert np.isnan(got[t]).all()
            elif not way:
                assert (got[t] == 0).all()
            else:
                assert (np.abs(got[t] - ref[t]) <= tol[t]).all(), (r, t)
        # the update's bits: each way, token by token, from a copy of the window
        for way in [w for w in T.ways(c.parents[r]) if w][:6]:
            one = Conv([[-1]], C, W, dtype)
            one.rows(one.page_in[0]).copy_(c.windows[r])
            z = torch.empty((1, C), dtype=TD[out], device="cuda")
            for t in way:
                K.kda_short_conv_update(one.pool, c.x[r * tokens + t: r * tokens + t + 1], c.w, z, ints(one.page_in), ints(one.page_in))
            assert torch.equal(z[0], y[r * tokens + way[-1]]), (r, way)


@pytest.mark.parametrize("W,dtype,C", [(4, "bf16", 1024), (3, "f32", 12), (2, "bf16", 4104)])
@pytest.mark.parametrize("in_place", [True, False])
def test_conv_commit(W, dtype, C, in_place):
    tokens = 9
    parents = [tree("chain", tokens)] * 5
    c = Conv(parents, C, W, dtype, seed=W)
    paths = [[], [0], [0, 1], [2, 5, 6], list(range(9))]
    path, count = pad(paths, tokens)
    out = c.page_in if in_place else c.page_out
    before = c.buf.clone()
    K.kda_short_conv_commit(c.pool, c.x, ints(path), ints(count), ints(c.page_in), ints(out))
    for r in range(5):
        line = torch.cat((c.windows[r], c.x[r * tokens: (r + 1) * tokens][paths[r]]))
        assert torch.equal(c.rows(out[r]), line[-(W - 1):]), r
    mask = torch.ones_like(before, dtype=torch.bool)
    for p in out:
        mask[int(p) * c.page: int(p) * c.page + (W - 1) * C * (2 if dtype == "bf16" else 4)] = False
    assert torch.equal(before[mask], c.buf[mask])
    after = c.buf.clone()
    for p, n in (([1, 1, 0, 0, 0, 0, 0, 0, 0], 2), ([0] * 9, 10), ([0] * 9, -1), ([0, 9] + [0] * 7, 2)):
        K.kda_short_conv_commit(c.pool, c.x, ints([p] * 5), ints([n] * 5), ints(c.page_in), ints(c.page_out))
    K.kda_short_conv_commit(c.pool, c.x, ints(path), ints(count), ints([-1, 10, 0, 0, 0]), ints([5, 5, -1, 10, 11]))
    assert torch.equal(after, c.buf)


def test_conv_bad_pages_and_values():
    c = Conv([tree("binary", 7)] * 3, 520, 4, "bf16", seed=3)
    ref = c.run("bf16")
    c.page_in[0] = 6
    c.x[7 + 1] = float("nan")
    got = c.run("bf16")
    assert torch.isnan(got[:7]).all() and torch.equal(got[14:], ref[14:])
    for t, way in enumerate(T.ways(tree("binary", 7))):
        assert torch.isnan(got[7 + t]).all() if 1 in way[-4:] else torch.equal(got[7 + t], ref[7 + t])


def test_a_hybrid_layer_pair_in_a_graph():
    """Convolution, recurrence and both commits in one captured step, replayed with other trees and paths."""
    n, tokens, H, d = 3, 11, 2, 64
    runs = []
    for _ in range(2):
        x, c = States([tree("binary", tokens)] * n, H, d, "bf16", seed=1), Conv([tree("binary", tokens)] * n, H * d, 4, "bf16", seed=2)
        path, count = pad([[0, 1]] * n, tokens)
        runs.append((x, c, ints(path), ints(count), torch.zeros((n * tokens, H * d), dtype=torch.bfloat16, device="cuda"),
                     torch.zeros((n * tokens, H, d), dtype=torch.bfloat16, device="cuda"), ints(x.page_in), ints(c.page_in)))

    def step(x, c, path, count, y, o, pages, windows):
        K.kda_short_conv_tree(c.pool, c.x, c.w, y, x.parent, windows)
        v = y.view(n * tokens, H, d)
        a = x.x
        K.kda_decode_tree(x.pb.pool, a["q"], a["k"], v, a["g"], a["beta"], o, x.parent, pages)
        K.kda_decode_commit(x.pb.pool, a["k"], v, a["g"], a["beta"], path, count, pages, pages)
        K.kda_short_conv_commit(c.pool, c.x, path, count, windows, windows)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(*runs[0])
    for i in range(4):
        parents = [tree(k, tokens, i) for k in ("random", "short", "holes")]
        path, count = pad([some_path(p) for p in parents], tokens)
        for x, c, p, m, *_ in runs:
            x.parent.copy_(ints(parents))
            p.copy_(ints(path))
            m.copy_(ints(count))
        g.replay()
        step(*runs[1])
        torch.cuda.synchronize()
        for a, b in zip((runs[0][0].pb.buf, runs[0][1].buf, runs[0][4], runs[0][5]), (runs[1][0].pb.buf, runs[1][1].buf, runs[1][4], runs[1][5])):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16)), i


def test_host_validation(monkeypatch):
    monkeypatch.setenv("KDA_VALIDATE", "1")
    x = States([tree("binary", 5)] * 2, 1, 64, "bf16")
    x.run("f32")
    a, path, count = x.x, ints([[0] * 5] * 2), ints([1, 1])
    for pin, pout, status in (([0, 9], [2, 3], K.KDA_ERR_PAGE_RANGE), ([0, 1], [2, 2], K.KDA_ERR_PAGE_ALIAS),
                              ([0, 1], [1, 2], K.KDA_ERR_PAGE_ALIAS), ([0, 1], [2, -1], K.KDA_ERR_PAGE_RANGE)):
        with pytest.raises(K.KdaError) as e:
            K.kda_decode_commit(x.pb.pool, a["k"], a["v"], a["g"], a["beta"], path, count, ints(pin), ints(pout))
        assert e.value.status == status
    with pytest.raises(K.KdaError):
        K.kda_decode_tree(x.pb.pool, a["q"], a["k"], a["v"], a["g"], a["beta"], torch.empty_like(a["v"]), x.parent, ints([0, 5]))
    c = Conv([tree("binary", 5)] * 2, 64, 4, "bf16")
    with pytest.raises(K.KdaError):
        K.kda_short_conv_tree(c.pool, c.x, c.w, torch.empty_like(c.x), c.parent, ints([0, 4]))
    with pytest.raises(K.KdaError):
        K.kda_short_conv_commit(c.pool, c.x, path, count, ints([0, 1]), ints([1, 0]))


def test_bindings_refuse():
    x = States([tree("binary", 5)] * 2, 1, 64, "bf16")
    a, o, pages = x.x, torch.empty_like(x.x["v"]), ints([0, 1])
    path, count = ints([[0] * 5] * 2), ints([1, 1])
    c = Conv([tree("binary", 5)] * 2, 64, 4, "bf16")
    y = torch.empty_like(c.x)
    tree_args = dict(q=a["q"], k=a["k"], v=a["v"], g=a["g"], beta=a["beta"], o=o, parent=x.parent, page_in=pages)
    commit = dict(k=a["k"], v=a["v"], g=a["g"], beta=a["beta"], path=path, count=count, page_in=pages, page_out=pages)
    conv = dict(x=c.x, w=c.w, y=y, parent=c.parent, page_in=pages)
    cc = dict(x=c.x, path=path, count=count, page_in=pages, page_out=pages)
    for fn, pool, args, bad in (
            (K.kda_decode_tree, x.pb.pool, tree_args, dict(q=a["q"].float(), k=a["k"][:9], v=a["v"].cpu(), g=a["g"].transpose(0, 1),
                                                           beta=a["beta"][:, :0], o=o[:9], parent=x.parent.long(), page_in=pages[:1])),
            (K.kda_decode_commit, x.pb.pool, commit, dict(k=a["k"].half(), v=a["v"][::2], beta=a["beta"].float(), path=path[:1],
                                                          count=count.cpu(), page_out=pages.long())),
            (K.kda_short_conv_tree, c.pool, conv, dict(x=c.x.float(), w=c.w[:, :3], y=y[:9], parent=c.parent[0], page_in=pages.cpu())),
            (K.kda_short_conv_commit, c.pool, cc, dict(x=c.x[:9], path=path.long(), count=count[:1], page_in=pages[:1]))):
        for name, value in bad.items():
            with pytest.raises((ValueError, K.KdaError)):
                fn(pool, **{**args, name: value})
        fn(pool, **args)


def test_bf16_round_trip_of_the_helper():
    assert np.array_equal(bf16([1.0, 1 / 3]), host(to_dev([1.0, 1 / 3], "bf16")))
