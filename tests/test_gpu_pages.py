"""The upkeep of pages on the GPU (reserve, free, fork, compact, copy) against plain loops:
counts, tables and lists are equal, and a cache's contents follow them."""
import numpy as np
import pytest
import torch

import hybrid_prefix_cache_amd as K
from kv_gpu_util import Filled, KvBuf, host, ws
from oracle import tree as T

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Book:
    """The same counts and table on the GPU and as plain lists."""

    def __init__(self, refs, table, pt):
        self.plain = T.Pages(refs, table, pt)
        self.refs, self.table, self.pt = ints(refs), ints(table), pt
        self.map = K.make_page_map(self.refs, self.table, pt)
        assert K.kda_page_map_check(self.map) == K.KDA_OK
        self.ws = ws(K.kda_pages_workspace_bytes(self.map))

    def same(self, tag=None):
        assert self.refs.tolist() == self.plain.refs, tag
        assert self.table.tolist() == self.plain.table, tag

    def reserve(self, first, last):
        self.ws.fill_(0xFF)
        status = torch.full((len(first),), 77, dtype=torch.int32, device="cuda")
        K.kda_pages_reserve(self.map, ints(first), ints(last), status, workspace=self.ws)
        assert status.tolist() == self.plain.reserve(first, last)
        self.same()

    def free(self, first, last):
        K.kda_pages_free(self.map, ints(first), ints(last))
        self.plain.release(first, last)
        self.same()

    def fork(self, src, dst, tokens):
        self.ws.fill_(0xFF)
        out = [torch.full((len(src),), 77, dtype=torch.int32, device="cuda") for _ in range(4)]
        K.kda_pages_fork(self.map, ints(src), ints(dst), ints(tokens), *out, workspace=self.ws)
        copies, status = self.plain.fork(src, dst, tokens)
        assert [x.tolist() for x in out[:3]] == copies and out[3].tolist() == status
        self.same()
        return out[:3]

    def compact(self):
        self.ws.fill_(0xFF)
        out = [torch.full((len(self.plain.refs),), 77, dtype=torch.int32, device="cuda") for _ in range(2)]
        K.kda_pages_compact(self.map, *out, workspace=self.ws)
        moves = self.plain.compact()
        moves += [(-1, -1)] * (len(self.plain.refs) - len(moves))
        assert [x.tolist() for x in out] == [list(x) for x in zip(*moves)]
        self.same()
        return out


def book(pages, rows, width, pt, seed, fill=0.5, shared=True):
    """Rows with pages at the front, some of them shared, some held by others too."""
    rng = np.random.default_rng(seed)
    refs, table = np.zeros(pages, int), np.full((rows, width), -1)
    order = list(rng.permutation(pages))
    for r in range(rows):
        for j in range(int(rng.integers(0, max(1, int(width * fill)) + 1))):
            p = int(rng.integers(pages)) if shared and rng.random() < 0.2 and refs.max() > 0 else -1
            if p < 0 or refs[p] == 0:
                if not order:
                    break
                p = int(order.pop())
            if p in table[r]:
                continue
            table[r, j] = p
            refs[p] += 1
    refs[rng.random(pages) < 0.05] += 1
    return Book(refs, table, pt)


@pytest.mark.parametrize("pages,rows,width,pt", [(1, 1, 1, 1), (40, 5, 8, 64), (700, 9, 130, 32), (5000, 1100, 3, 32), (9001, 70, 65, 96),
                                                 (20000, 2, 3000, 16)])
@pytest.mark.parametrize("seed", [0, 1, 2])
def test_reserve_free_fork_compact(pages, rows, width, pt, seed):
    b, rng, end = book(pages, rows, width, pt, seed), np.random.default_rng(seed + 50), width * pt
    for _ in range(2):
        lo = rng.integers(-5, end + 3, rows)
        hi = lo + rng.integers(-2, max(2, end // 3), rows)
        b.reserve(lo.tolist(), hi.tolist())
        # some rows end, some are cut back, some lose a middle
        lo = rng.integers(0, end + 1, rows) * (rng.random(rows) < 0.7)
        hi = np.where(rng.random(rows) < 0.5, end, rng.integers(0, end + 1, rows))
        hi = np.where(rng.random(rows) < 0.4, 0, hi)
        b.free(lo.tolist(), hi.tolist())
        ends = rng.permutation(rows)[: rows // 2]
        first, last = np.zeros(rows, int), np.zeros(rows, int)
        last[ends] = 2 ** 31 - 1
        b.free(first.tolist(), last.tolist())
        src = [int(x) for x in rng.choice(np.setdiff1d(np.arange(rows), ends), max(0, len(ends)))]
        tokens = [int(x) for x in rng.integers(-1, end + 2, len(ends))]
        if len(ends):
            b.fork(src, ends.tolist(), tokens)
        b.compact()


def test_as_many_rows_as_a_map_may_have():
    rows, pages = 1 << 24, 1000
    refs, table = torch.zeros(pages, dtype=torch.int32, device="cuda"), torch.full((rows, 1), -1, dtype=torch.int32, device="cuda")
    m = K.make_page_map(refs, table, 1)
    work = torch.empty(K.kda_pages_workspace_bytes(m), dtype=torch.uint8, device="cuda")
    first, last, status = (torch.zeros(rows, dtype=torch.int32, device="cuda") for _ in range(3))
    some = torch.arange(5, rows, 17000, device="cuda")  # 987 rows
    last[some] = 1
    K.kda_pages_reserve(m, first, last, status, workspace=work)
    assert torch.equal(table[some, 0], torch.arange(len(some), dtype=torch.int32, device="cuda")) and not status.any()
    assert int((table >= 0).sum()) == len(some) == int(refs.sum())
    last[some[: len(some) // 2]] = 0
    K.kda_pages_free(m, first, last)
    kept = some[: len(some) // 2]
    assert int((table >= 0).sum()) == len(kept) == int(refs.sum()) and (table[kept, 0] >= 0).all()
    copies = torch.empty((2, pages), dtype=torch.int32, device="cuda")
    last.fill_(2)
    K.kda_pages_free(m, first, torch.where(torch.arange(rows, device="cuda") == kept[0], last, 0).int())
    K.kda_pages_compact(m, copies[0], copies[1], workspace=work)
    assert copies[:, 0].tolist() == [len(kept) - 1, 0] and (copies[:, 1:] == -1).all()
    assert table[kept[-1]].item() == 0 and int(refs.sum()) == len(kept) - 1


def test_reserve_when_pages_run_out():
    b = Book([0, 1, 0, 2, 0], [[1, -1, -1, -1], [-1, 3, -1, -1], [3, -1, -1, -1]], 8)
    b.reserve([0, 4, 8], [24, 9, 33])  # two, one, and three of which none is left
    assert b.table.tolist() == [[1, 0, 2, -1], [4, 3, -1, -1], [3, -1, -1, -1]]
    b.reserve([0, 0, 0], [0, -3, 2 ** 31 - 1])


def test_fork_refusals_and_no_page_for_the_tail():
    b = Book([1, 1, 0, 3, 1], [[0, 1, 3], [-1, -1, -1], [-1, -1, -1], [3, 4, -1], [-1, -1, -1], [3, -1, -1], [-1, -1, -1]], 4)
    out = b.fork([0, 0, 9, 0, 0, 0, 3], [1, 2, 4, 3, 4, -1, 6], [5, 9, 3, 3, 13, 2, 8])
    assert out[0].tolist() == [1, -1, -1, -1, -1, -1, -1]
    b.fork([0, 0], [4, 4 + 10], [-1, 4])


def test_entries_and_rows_out_of_range_are_passed_over():
    b = Book([1, 0, 1], [[0, 2, -1], [-1, -1, -1]], 4)
    b.table[0, 1] = b.plain.table[0][1] = 55  # no page of the pool
    before = b.refs.clone()
    K.kda_pages_free(b.map, ints([4, 0]), ints([8, 0]))
    assert torch.equal(before, b.refs) and b.table[0].tolist() == [0, -1, -1]


@pytest.mark.parametrize("cache", ["int8", "bf16"])
@pytest.mark.parametrize("H,d,pt", [(2, 64, 32), (1, 128, 96), (3, 64, 160)])
def test_copies(cache, H, d, pt):
    kb = KvBuf(9, H, d, pt, cache, pad=256)
    kb.buf.copy_(torch.randint(-2 ** 31, 2 ** 31 - 1, kb.buf.shape, dtype=torch.int32, device="cuda"))
    before = kb.bytes().copy()
    tokens = [pt, 1, 33 if pt > 32 else 32, 0]
    src, dst = [0, 7, 3, 3], [8, 1, 2, 5]
    K.kda_kv_copy_pages(kb.pool, ints([-1] + src + [-3]), ints([4] + dst + [6]), tokens=ints([pt] + tokens + [pt]))
    part = 2 * 32 * d * (1 if cache == "int8" else 2)

    def copied(want, s, t, n):
        for h in range(H):
            o = h * kb.head_bytes
            blocks = -(-n // 32)
            want[t, o: o + blocks * part] = want[s, o: o + blocks * part]
            if cache == "int8":
                o += pt // 32 * part
                want[t, o: o + 8 * blocks] = want[s, o: o + 8 * blocks]

    for s, t, n in zip(src, dst, tokens):
        copied(before, s, t, n)
    after = kb.bytes()
    assert np.array_equal(before, after)
    K.kda_kv_copy_pages(kb.pool, ints([0, 9, 2, 6]), ints([4, 5, -1, 7]))  # pairs out of range are passed over
    copied(before, 0, 4, pt)
    copied(before, 6, 7, pt)
    assert np.array_equal(before, kb.bytes())


def test_copies_past_4_gib_and_many():
    H, d, pt = 2, 128, 512
    page = H * K.kda_kv_head_bytes(d, pt, K.KDA_INT8)
    pages = (5 << 30) // page
    buf = torch.zeros((pages, page), dtype=torch.uint8, device="cuda")
    buf[:700] = torch.randint(0, 255, (700, page), dtype=torch.uint8, device="cuda")
    pool = K.make_kv_pool(buf, page, pages, H, d, pt, K.KDA_INT8)
    used = K.kda_kv_head_bytes(d, pt, K.KDA_INT8)
    K.kda_kv_copy_pages(pool, ints(list(range(700))), ints([pages - 1 - i for i in range(700)]))
    body = 2 * pt * d + pt // 32 * 8
    for h in range(H):
        a = buf[:700, h * used: h * used + body]
        assert torch.equal(a, buf[pages - 700:, h * used: h * used + body].flip(0))


@pytest.mark.parametrize("n,every", [(1, 1), (1500, 3), (9000, 29), (70001, 90), (12000, 13000)])
def test_copies_of_a_list_with_gaps(n, every):
    """Pairs spread over lists of one gathering and of many; the last entry of a list is one of them."""
    H, d, pt, pages = 1, 64, 64, 1700
    page = 256 + K.kda_kv_head_bytes(d, pt, K.KDA_INT8)
    buf = torch.randint(0, 255, (pages, page), dtype=torch.uint8, device="cuda")
    pool = K.make_kv_pool(buf, page, pages, H, d, pt, K.KDA_INT8)
    rng = np.random.default_rng(n)
    src, dst, tokens = np.full(n, -1), rng.integers(-5, pages + 5, n), rng.integers(-3, pt + 70, n)
    at = np.arange(n - 1, -1, -every)
    order = rng.permutation(pages)
    src[at], dst[at] = order[rng.integers(0, 800, len(at))], order[800: 800 + len(at)]
    want, part = buf.clone(), 2 * 32 * d
    for i in at:
        blocks = max(0, min(pt // 32, -(-int(tokens[i]) // 32)))
        for lo, size in ((0, part), (pt // 32 * part, 8)):
            want[dst[i], lo: lo + blocks * size] = buf[src[i], lo: lo + blocks * size]
    K.kda_kv_copy_pages(pool, ints(src), ints(dst), tokens=ints(tokens))
    assert torch.equal(buf, want)


@pytest.mark.parametrize("cache", ["int8", "bf16"])
def test_samples_forked_from_a_running_request(cache):
    """Fork, copy, reserve, append: the samples hold the source's tokens and their own, the source what it held."""
    H, d, pt, n = 2, 64, 64, 150
    f = Filled([n, 20], H, d, pt, cache, seed=3, spare=0, width=4)
    pages = f.kb.pages
    kb = KvBuf(pages + 8, H, d, pt, cache)
    kb.buf[: f.kb.buf.numel()] = f.kb.buf
    table = np.full((5, 5), -1)
    table[:2, :4] = f.table_np
    refs = np.bincount(table[table >= 0], minlength=pages + 8)
    b = Book(refs, table, pt)
    forks = [(0, 2, 150), (0, 3, 100), (1, 4, 20)]
    copies = b.fork(*(list(x) for x in zip(*forks)))
    K.kda_kv_copy_pages(kb.pool, copies[0], copies[1], tokens=copies[2])
    b.reserve([0, 0, 150, 100, 20], [0, 0, 190, 140, 60])
    rng = np.random.default_rng(5)
    k, v = (torch.from_numpy(rng.standard_normal((120, H, d))).cuda().to(torch.bfloat16) for _ in range(2))
    K.kda_kv_append(kb.pool, None, k, v, None, [0, 40, 80, 120], b.table[2:].contiguous(), start_pos=[150, 100, 20])

    def read(row, length, buf=None, tab=None):
        out = [torch.zeros((length, H, d), device="cuda") for _ in range(2)]
        K.kda_kv_read((buf or kb).pool, *out, [0, length], (b.table if tab is None else tab)[row: row + 1].contiguous())
        return out

    for row, length in ((0, n), (1, 20)):
        for x, y in zip(read(row, length), read(row, length, f.kb, f.table)):
            assert torch.equal(x, y)
    for s, t, length in forks:
        # complete blocks are the source's bits
        for x, y in zip(read(t, length // 32 * 32), read(s, length // 32 * 32)):
            assert torch.equal(x, y)
        own = read(t, length + 40)
        for x, new in zip(own, (k, v)):
            want = host(new)[40 * (t - 2): 40 * (t - 1)]
            err = np.abs(host(x[length:]) - want)
            assert (err <= (0 if cache == "bf16" else np.abs(want).max() / 100)).all()
    moves = b.compact()
    before = [read(t, length + 40) for _, t, length in forks]
    # (the table is the compacted one: contents follow once the copies are made)
    K.kda_kv_copy_pages(kb.pool, *moves)
    for (s, t, length), old in zip(forks, before):
        for x, new in zip(read(t, length + 40), (k, v)):
            want = host(new)[40 * (t - 2): 40 * (t - 1)]
            assert (np.abs(host(x[length:]) - want) <= (0 if cache == "bf16" else np.abs(want).max() / 100)).all()
    for row, length in ((0, n), (1, 20)):
        for x, y in zip(read(row, length), read(row, length, f.kb, f.table)):
            assert torch.equal(x, y)


def test_upkeep_in_a_graph():
    """Free, fork, reserve and compact captured once, replayed on changing rows."""
    n, width, pt, pages = 12, 9, 32, 150
    books = [book(pages, n, width, pt, 4) for _ in range(2)]
    a = [dict(first=ints([0] * n), last=ints([0] * n), lo=ints([0] * n), hi=ints([0] * n), src=ints([0] * 4), dst=ints([0] * 4),
              tok=ints([-1] * 4), cs=ints([0] * 4), cd=ints([0] * 4), ct=ints([0] * 4), st=ints([0] * 4), rs=ints([0] * n),
              ms=ints([0] * pages), md=ints([0] * pages)) for _ in books]

    def step(b, x):
        K.kda_pages_free(b.map, x["first"], x["last"])
        K.kda_pages_fork(b.map, x["src"], x["dst"], x["tok"], x["cs"], x["cd"], x["ct"], x["st"], workspace=b.ws)
        K.kda_pages_reserve(b.map, x["lo"], x["hi"], x["rs"], workspace=b.ws)
        K.kda_pages_compact(b.map, x["ms"], x["md"], workspace=b.ws)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(books[0], a[0])
    for i in range(5):
        rng = np.random.default_rng(i)
        rows = rng.permutation(n)
        last = np.zeros(n, int)
        last[rows[:4]] = width * pt
        lo = rng.integers(0, width * pt, n)
        new = dict(last=last, lo=lo, hi=lo + 40, src=rows[4:8], dst=rows[:4], tok=rng.integers(0, width * pt, 4))
        for x in a:
            for name, value in new.items():
                x[name].copy_(ints(value))
        g.replay()
        step(books[1], a[1])
        torch.cuda.synchronize()
        assert torch.equal(books[0].refs, books[1].refs) and torch.equal(books[0].table, books[1].table), i
        for name in a[0]:
            assert torch.equal(a[0][name], a[1][name]), (i, name)


def test_host_validation(monkeypatch):
    monkeypatch.setenv("KDA_VALIDATE", "1")
    b = Book([1, 0, 0], [[0], [-1], [-1]], 4)
    out = [ints([0, 0]) for _ in range(4)]
    for src, dst, status in (([0, 0], [1, 1], K.KDA_ERR_PAGE_ALIAS), ([0, 1], [1, 2], K.KDA_ERR_PAGE_ALIAS),
                             ([0, 3], [1, 2], K.KDA_ERR_PAGE_RANGE)):
        with pytest.raises(K.KdaError) as e:
            K.kda_pages_fork(b.map, ints(src), ints(dst), ints([2, 2]), *out, workspace=b.ws)
        assert e.value.status == status
    kb = KvBuf(4, 1, 64, 32, "bf16")
    for src, dst, status in (([0, 1], [2, 2], K.KDA_ERR_PAGE_ALIAS), ([0, 1], [1, 2], K.KDA_ERR_PAGE_ALIAS),
                             ([0, 4], [1, 2], K.KDA_ERR_PAGE_RANGE)):
        with pytest.raises(K.KdaError) as e:
            K.kda_kv_copy_pages(kb.pool, ints(src), ints(dst))
        assert e.value.status == status
    K.kda_kv_copy_pages(kb.pool, ints([0, -1, -9]), ints([1, 1, 1]))


def test_bindings_refuse():
    b = Book([1, 0, 0], [[0], [-1], [-1]], 4)
    x = ints([0, 0, 0])
    for refs, table in ((b.refs.long(), b.table), (b.refs.cpu(), b.table), (b.refs, b.table[0]), (b.refs, b.table.cpu()),
                        (b.refs.cpu(), b.table.cpu()), (b.refs.view(1, 3), b.table)):
        with pytest.raises(ValueError):
            K.make_page_map(refs, table, 4)
    for call in (lambda: K.kda_pages_free(b.map, x[:2], x), lambda: K.kda_pages_free(b.map, x, x.long()),
                 lambda: K.kda_pages_reserve(b.map, x, x, x.cpu(), workspace=b.ws),
                 lambda: K.kda_pages_reserve(b.map, x, x, x), lambda: K.kda_pages_reserve(b.map, x, x, x, workspace=b.ws[:256]),
                 lambda: K.kda_pages_fork(b.map, x, x[:2], x, x, x, x, x, workspace=b.ws),
                 lambda: K.kda_pages_compact(b.map, x[:2], x, workspace=b.ws)):
        with pytest.raises((ValueError, K.KdaError)):
            call()
