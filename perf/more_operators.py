"""Cases for timing and checking speculative decoding with a tree of drafted
tokens over the hybrid cache, and the upkeep of the cache's pages: attention
for a tree over the paged key/value cache, appending a tree to that cache and
keeping its accepted path, the gated delta-rule recurrence and the short
convolution along a tree, and forking, freeing, reserving, compacting and
copying pages.

Every operator has a plain form here (elementary torch, 32 bits) beside the
library's calls, so the same inputs go through both.

A tree of up to 64 drafted tokens per request is an int32 row `parent`: entry t
is -1 for a node that follows the last cached token, s < t for a child of node s,
-2 for no node (a request that drafted fewer).  Node t sits in cache slot
pos + t, at position pos + depth(t).  The accepted path is a row of node
indices from the root on and their count.

Cache pages (bytes, per include/kda.h): head after head; a head is its 32-token
blocks, each a K part then a V part of 32 * d elements in matrix-operand order,
then (int8) two fp32 scales per block (K, V).
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

BLOCK = 32  # tokens per cache block (one scale each for K and V)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _case(name, op, **kw):
    c = dict(name=name, op=op, dtype="bf16", n=1, tokens=8, roots=2, branch=2, d=128, mix=1)
    if op in ("attend", "draft"):
        c.update(cache="int8", hq=32, hkv=8, page_tokens=512, start_lo=0, start_hi=0, window=0, sinks=0, rot=128,
                 interleaved=False)
    elif op == "state":
        c.update(heads=32)
    elif op == "conv":
        c.update(channels=4096, width=4)
    elif op in ("fork", "compact"):
        c.update(hkv=4, page_tokens=64, start_lo=1, start_hi=1000, spare=50, cut=2)
        for k in ("tokens", "roots", "branch", "dtype"):
            del c[k]
    c.update(kw)
    return c


def listed():
    return [
        # attention for a tree: one request with a small draft, where latency counts; a
        # serving batch over an int8 cache; odd head groups and a wide tree beside a
        # sliding window with sinks, bf16 cache
        _case("tree_one_request", "attend", start_lo=700, start_hi=700),
        _case("tree_64_requests", "attend", n=64, tokens=16, start_lo=512, start_hi=8191, mix=2),
        _case("tree_wide_window", "attend", cache="bf16", hq=28, hkv=4, n=12, tokens=61, roots=5, page_tokens=96,
              start_lo=100, start_hi=6000, window=1024, sinks=4, mix=3),
        # a draft in the cache: the tail pages are copied (shared pages stay as they are),
        # the tree's keys and values stored with rotation, the accepted path kept and read
        # back; a serving batch, int8; three requests of odd sizes, fp32 into bf16
        _case("draft_64_requests", "draft", n=64, tokens=32, roots=4, start_lo=512, start_hi=8191, mix=4),
        _case("draft_three_requests", "draft", dtype="f32", cache="bf16", hq=8, hkv=2, d=64, n=3, tokens=7,
              page_tokens=64, start_lo=1, start_hi=1000, rot=32, interleaved=True, mix=5),
        # the recurrence along a tree, then along its accepted path: one request with few
        # heads in fp32; a serving batch of 16-node trees; trees as large as they get
        _case("state_one_request", "state", dtype="f32", tokens=5, d=64, heads=8),
        _case("state_64_requests", "state", n=64, tokens=16, mix=6),
        _case("state_large_trees", "state", n=24, tokens=63, roots=3, mix=7),
        # the short convolution before it: q, k and v of 32 heads in one call; odd sizes in fp32
        _case("conv_64_requests", "conv", n=64, tokens=16, channels=12288, mix=8),
        _case("conv_three_requests", "conv", dtype="f32", n=3, tokens=7, channels=520, width=3, mix=9),
        # pages: finished samples leave, new ones fork from 64 running requests and get
        # room for their next tokens; a pool with holes is compacted
        _case("fork_32_samples", "fork", hkv=8, n=64, page_tokens=32, start_lo=100, start_hi=1900, mix=10),
        _case("compact_pool", "compact", n=40, start_lo=60, start_hi=1500, mix=11),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "draft", "state", "state", "conv", "fork", "compact"])
    c = _case("", op)
    del c["name"]
    c["mix"] = rng.randrange(1 << 20)
    if op in ("fork", "compact"):
        c["d"] = rng.choice([64, 128])
        c["hkv"] = rng.choice([1, 2, 4])
        c["page_tokens"] = 32 * rng.choice([1, 2, 3, 8])
        c["n"] = _log_int(rng, 2, 90)
        c["start_hi"] = _log_int(rng, 40, 3000)
        c["start_lo"] = c["start_hi"] // rng.choice([1, 3, 100])
        c["spare"] = _log_int(rng, 1, 200)
        c["cut"] = rng.choice([2, 3, 5])
        return c
    c["dtype"] = "f32" if rng.random() < 0.25 else "bf16"
    c["tokens"] = _log_int(rng, 1, 64)
    c["roots"] = rng.choice([1, 1, 2, 4])
    c["branch"] = rng.choice([1, 2, 2, 3])
    if op == "conv":
        c["n"] = _log_int(rng, 1, max(1, 1000 // c["tokens"]))
        c["width"] = rng.choice([2, 3, 4])
        c["channels"] = 8 * _log_int(rng, 1, 1500)
        return c
    c["d"] = rng.choice([64, 128, 128])
    if op == "state":
        c["heads"] = rng.choice([1, 3, 8, 32])
        c["n"] = _log_int(rng, 1, max(1, 24 * 32 * 63 // (c["tokens"] * c["heads"]) // 2))
        c["n"] = min(c["n"], 100)
        return c
    c["cache"] = rng.choice(["int8", "bf16"])
    c["hkv"] = rng.choice([1, 2, 4, 8])
    c["hq"] = c["hkv"] * rng.choice([g for g in (1, 2, 3, 4, 7, 8, 16) if g * c["hkv"] <= 32])
    c["page_tokens"] = 32 * rng.choice([1, 2, 3, 5, 16])
    if op == "draft":
        c["rot"] = rng.choice([c["d"], c["d"], c["d"] // 2, 32])
        c["interleaved"] = rng.random() < 0.3
        c["n"] = _log_int(rng, 1, max(1, 1500 // c["tokens"]))
        c["start_hi"] = _log_int(rng, 1, 5000)
    else:
        if rng.random() < 0.4:
            c["window"] = _log_int(rng, 1, 3000)
            c["sinks"] = rng.choice([0, 1, 4, 33, 200])
        c["n"] = _log_int(rng, 1, max(1, 800 // c["tokens"]))
        c["start_hi"] = _log_int(rng, 1, min(100000, 200000 // (c["n"] * max(1, c["tokens"] // 16))))
    c["start_lo"] = c["start_hi"] // rng.choice([1, 3, 100])
    return c


def _spans(c):
    """Per request: tokens already cached."""
    r = random.Random(c["mix"])
    return [r.randint(c["start_lo"], c["start_hi"]) for _ in range(c["n"])]


def _trees(c):
    """(parent, path [n, tokens], count [n]) as lists: most nodes follow breadth first, a few
    anywhere before; in a batch some requests drafted fewer nodes."""
    r = random.Random(c["mix"] + 1)
    parents, paths, counts = [], [], []
    for _ in range(c["n"]):
        live = c["tokens"] - (r.randint(0, c["tokens"] // 4) if c["n"] > 1 else 0)
        p = []
        for t in range(live):
            if t < c["roots"]:
                p.append(-1)
            else:
                p.append((t - c["roots"]) // c["branch"] if r.random() < 0.85 else r.randrange(t))
        at, way = r.randrange(-1, live), []
        while at >= 0:
            way.insert(0, at)
            at = p[at]
        parents.append(p + [-2] * (c["tokens"] - live))
        counts.append(len(way))
        paths.append(way + [-1] * (c["tokens"] - len(way)))
    return parents, paths, counts


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _tdtype(c):
    return torch.float32 if c["dtype"] == "f32" else torch.bfloat16


def _elem(c):
    return 1 if c["cache"] == "int8" else 2


def _head_bytes(c):
    blocks = c["page_tokens"] // BLOCK
    b = blocks * 2 * BLOCK * c["d"] * _elem(c)
    return b if c["cache"] == "bf16" else -(-(b + blocks * 8) // 256) * 256


def _quantise(x):
    """x: [..., 32 tokens, d] fp32 -> codes (int8), scale [...] by the block rule."""
    s = x.abs().amax(dim=(-1, -2)) / 127
    q = torch.where(s[..., None, None] > 0, torch.round(x / s[..., None, None]), torch.zeros_like(x))
    return q.clamp(-127, 127).to(torch.int8), s


def _pack_k(x, elem):
    """[..., 32, d] -> K part order, flattened."""
    e, d = 16 // elem, x.shape[-1]
    lead = x.shape[:-2]
    return x.reshape(*lead, 2, 16, d // e, e).transpose(-3, -2).reshape(*lead, -1)


def _pack_v(x, elem):
    g, d = 2 // elem, x.shape[-1]
    lead, m = x.shape[:-2], len(x.shape) - 2
    y = x.reshape(*lead, 2, 4, 4, d // (16 * g), g, 16)  # half, group, t%4 | d group, G, channel
    p = list(range(m)) + [m + i for i in (3, 1, 5, 4, 0, 2)]
    return y.permute(*p).reshape(*lead, -1)


def _fill_pool(c, pool, gen):
    """Every page filled as a running program's cache is: block by block."""
    h, d, e = c["hkv"], c["d"], _elem(c)
    blocks, part = c["page_tokens"] // BLOCK, BLOCK * c["d"] * _elem(c)
    step = max(1, (1 << 27) // (h * c["page_tokens"] * d))
    for p0 in range(0, pool.shape[0], step):
        rows = pool[p0: p0 + step]
        n = rows.shape[0]
        heads = rows[:, : h * _head_bytes(c)].reshape(n, h, -1)
        x = torch.randn((2, n, h, blocks, BLOCK, d), generator=gen, device="cuda")
        # heads and channels of different sizes, as trained projections have
        x *= 0.3 + 1.4 * torch.rand((2, 1, h, 1, 1, d), generator=gen, device="cuda")
        out = heads.clone()
        body = out[..., : blocks * 2 * part].view(n, h, blocks, 2, part)
        if c["cache"] == "int8":
            q, s = _quantise(x)
            body[..., 0, :] = _pack_k(q[0], e).view(torch.uint8)
            body[..., 1, :] = _pack_v(q[1], e).view(torch.uint8)
            out[..., blocks * 2 * part: blocks * 2 * part + blocks * 8] = (
                torch.stack((s[0], s[1]), -1).reshape(n, h, -1).view(torch.uint8))
        else:
            xb = x.to(torch.bfloat16)
            body[..., 0, :] = _pack_k(xb[0], e).contiguous().view(torch.uint8).view(n, h, blocks, part)
            body[..., 1, :] = _pack_v(xb[1], e).contiguous().view(torch.uint8).view(n, h, blocks, part)
        rows[:, : h * _head_bytes(c)] = out.reshape(n, -1)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _prepare_cache(c, s, gen, rnd):
    """The cache and the projections of an attention layer's step."""
    starts = _spans(c)
    pt, hq, hkv, d, n, T = c["page_tokens"], c["hq"], c["hkv"], c["d"], c["n"], c["tokens"]
    need = [-(-(a + T) // pt) for a in starts]
    # a draft goes into a copy of the tail page: where tokens end inside a page, that
    # page stays another holder's too
    tails = [int(c["op"] == "draft" and a % pt > 0) for a in starts]
    max_pages, pages = max(need), sum(need) + sum(tails) + 1
    page_bytes = -(-hkv * _head_bytes(c) // 256) * 256
    pool = torch.zeros((pages, page_bytes), dtype=torch.uint8, device="cuda")
    _fill_pool(c, pool, gen)
    # pages in the order a free list gives them; entries past a request's last page are -1
    order = rnd.permutation(pages).astype(np.int32)
    table, at = np.full((n, max_pages), -1, np.int32), 0
    for r, m in enumerate(need):
        table[r, :m] = order[at: at + m]
        at += m
    cps, cpd, cpt = [], [], []
    for r, a in enumerate(starts):
        if tails[r]:
            cps.append(int(order[at]))
            cpd.append(int(table[r, a // pt]))
            cpt.append(a % pt)
            at += 1
    # q, k and v as rows of one fused projection, as a layer has them
    width = (hq + 2 * hkv) * d
    qkv = torch.randn((n * T, width), generator=gen, device="cuda").to(_tdtype(c))
    s.update(pool=pool, page_bytes=page_bytes, table=torch.from_numpy(table).cuda(), pos=_ints(starts),
             q=qkv[:, : hq * d].unflatten(1, (hq, d)), k=qkv[:, hq * d: (hq + hkv) * d].unflatten(1, (hkv, d)),
             v=qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d)),
             out=torch.empty((n * T, hq, d), dtype=_tdtype(c), device="cuda"), scale=1.0 / math.sqrt(d))
    if c["op"] == "draft":
        s.update(copy_src=_ints(cps + [-1]), copy_dst=_ints(cpd + [-1]), copy_tokens=_ints(cpt + [0]))
        half = c["rot"] // 2
        angle = (torch.arange(max(starts) + T, dtype=torch.float64)[:, None]
                 * 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)[None])
        s["cos"], s["sin"] = angle.cos().float().cuda(), angle.sin().float().cuda()
        # read back: from the block of the first new token to the last accepted one
        count = _trees(c)[2]
        lo = [a // BLOCK * BLOCK if c["cache"] == "int8" else a for a in starts]
        s["read_lo"] = np.asarray(lo, np.int64)
        s["read_cu"] = np.concatenate([[0], np.cumsum([a + k - x for a, k, x in zip(starts, count, lo)])]).astype(np.int64)
        m = int(s["read_cu"][-1])
        s["k_out"] = torch.empty((m, hkv, d), dtype=_tdtype(c), device="cuda")
        s["v_out"] = torch.empty((m, hkv, d), dtype=_tdtype(c), device="cuda")


def _prepare_state(c, s, gen, rnd):
    """One recurrent layer's step: q and k normalised, gates that forget at a rate of each
    channel's own, states in the pages a free list gave; the accepted states go to fresh pages."""
    n, T, H, d, dt = c["n"], c["tokens"], c["heads"], c["d"], _tdtype(c)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    def unit(x):
        return (x / x.square().sum(-1, keepdim=True).sqrt()).to(dt)

    def spread(*shape):
        return torch.rand(shape, generator=gen, device="cuda")

    rate = 10.0 ** (-2.3 + 2.3 * spread(1, H, d))
    s.update(q=unit(normal(n * T, H, d)), k=unit(normal(n * T, H, d)), v=normal(n * T, H, d).to(dt),
             g=(-rate * spread(n * T, H, d)).to(dt), beta=torch.sigmoid(normal(n * T, H)).to(dt),
             o=torch.empty((n * T, H, d), dtype=dt, device="cuda"))
    pool = torch.zeros((2 * n, H, d, d), device="cuda")
    pool[:n] = normal(n, H, d, d) / math.sqrt(d)
    s.update(pool=pool, page_in=torch.from_numpy(rnd.permutation(n).astype(np.int32)).cuda(),
             page_out=torch.from_numpy((n + rnd.permutation(n)).astype(np.int32)).cuda())


def _prepare_conv(c, s, gen, rnd):
    n, T, C, W, dt = c["n"], c["tokens"], c["channels"], c["width"], _tdtype(c)
    page = -(-(W - 1) * C * dt.itemsize // 256) * 256 // dt.itemsize
    pool = torch.zeros((2 * n, page), dtype=dt, device="cuda")
    pool[:n, : (W - 1) * C] = torch.randn((n, (W - 1) * C), generator=gen, device="cuda").to(dt)
    s.update(pool=pool, x=torch.randn((n * T, C), generator=gen, device="cuda").to(dt),
             w=torch.randn((C, W), generator=gen, device="cuda") / math.sqrt(W),
             y=torch.empty((n * T, C), dtype=dt, device="cuda"),
             page_in=torch.from_numpy(rnd.permutation(n).astype(np.int32)).cuda(),
             page_out=torch.from_numpy((n + rnd.permutation(n)).astype(np.int32)).cuda())


def _prepare_pages(c, s, gen, rnd):
    """n running requests; n // cut rows beside them hold samples that have ended.  Some
    requests share their first pages, some pages are held outside of the tables (a prefix
    cache's)."""
    n, pt, hkv, d = c["n"], c["page_tokens"], c["hkv"], c["d"]
    starts = np.asarray(_spans(c))
    m = max(1, n // c["cut"])
    lens = np.concatenate([starts, np.random.RandomState(c["mix"]).permutation(starts)[:m]])
    need = -(-lens // pt)
    rows, max_pages = n + m, int(need.max()) + -(-c["spare"] // pt) + 1
    total = int(need.sum())
    pages = total + total // 3 + m * (2 + c["spare"] // pt) + 8
    order = rnd.permutation(pages).astype(np.int32)
    j = np.arange(max_pages)[None]
    held = j < need[:, None]
    table = np.full((rows, max_pages), -1, np.int32)
    table[held] = order[:total]
    # every third running request begins with the pages of the one before it
    share = np.minimum(need[:-1], need[1:])[: n - 1] // 2
    for r in range(1, n, 3):
        table[r, : share[r - 1]] = table[r - 1, : share[r - 1]]
    refs = np.bincount(table[table >= 0], minlength=pages).astype(np.int32)
    refs[rnd.permutation(pages)[: pages // 16]] += 1
    pool = torch.zeros((pages, hkv * pt * d * 2), dtype=torch.bfloat16, device="cuda")
    pool.normal_(generator=gen)
    # forks: a sample for each of m running requests, at its whole length or a part of it
    src = rnd.permutation(n)[:m] if m > 1 else np.array([0])
    whole = rnd.rand(m) < 0.6
    at = np.where(whole, starts[src], 1 + (rnd.rand(m) * (starts[src] - 1)).astype(np.int64))
    first, last = np.zeros(rows, np.int32), np.zeros(rows, np.int32)
    last[n:] = max_pages * pt
    new_lo, new_hi = np.zeros(rows, np.int32), np.zeros(rows, np.int32)
    new_lo[n:], new_hi[n:] = at, at + c["spare"]
    s.update(pool=pool, refs=torch.from_numpy(refs).cuda(), table=torch.from_numpy(table).cuda(),
             src=_ints(src.tolist()), dst=_ints(list(range(n, n + m))), at=_ints(at.tolist()),
             first=torch.from_numpy(first).cuda(), last=torch.from_numpy(last).cuda(),
             new_lo=torch.from_numpy(new_lo).cuda(), new_hi=torch.from_numpy(new_hi).cuda(),
             status=torch.zeros(rows, dtype=torch.int32, device="cuda"),
             fork_status=torch.zeros(m, dtype=torch.int32, device="cuda"))
    lists = m if c["op"] == "fork" else pages
    for name in ("copy_src", "copy_dst", "copy_tokens"):
        s[name] = torch.zeros(lists, dtype=torch.int32, device="cuda")
    if c["op"] == "compact":
        # the ended samples have left: their pages are the holes
        gone = torch.from_numpy(table[n:][table[n:] >= 0]).cuda().long()
        s["refs"].index_add_(0, gone, -torch.ones_like(gone, dtype=torch.int32))
        s["table"][n:] = -1
        s["refs0"], s["table0"] = s["refs"].clone(), s["table"].clone()


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 2 + 1)
    rnd = np.random.RandomState(int(seed) % (1 << 31))
    s = {"case": c}
    if c["op"] in ("fork", "compact"):
        _prepare_pages(c, s, gen, rnd)
        return s
    parent, path, count = _trees(c)
    s.update(parent=_ints(parent), path=_ints(path), count=_ints(count))
    {"attend": _prepare_cache, "draft": _prepare_cache, "state": _prepare_state, "conv": _prepare_conv}[c["op"]](c, s, gen, rnd)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _ancestors(parent):
    """[n, T, T] truth values: node s is on the way from the root to node t (t itself too); and
    whether t is a node."""
    n, T = parent.shape
    node = parent >= -1
    up = torch.zeros((n, T, T + 1), device="cuda")
    up.scatter_(2, torch.where(parent >= 0, parent.long(), T)[..., None], 1.0)
    a = up[..., :T] + torch.eye(T, device="cuda")
    for _ in range(6):  # paths of up to 64 nodes
        a = (torch.bmm(a, a) > 0).float()
    return (a > 0) & node[..., None], node


def _unpack(c, pool):
    """The cache of every page as fp32: two [pages, H, page_tokens, d]."""
    pages, h, d, e = pool.shape[0], c["hkv"], c["d"], _elem(c)
    blocks, part = c["page_tokens"] // BLOCK, BLOCK * c["d"] * _elem(c)
    heads = pool[:, : h * _head_bytes(c)].reshape(pages, h, -1)
    body = heads[..., : blocks * 2 * part].reshape(pages, h, blocks, 2, part)
    body = body.view(torch.int8 if c["cache"] == "int8" else torch.bfloat16)
    k, v = body[..., 0, :], body[..., 1, :]
    ek, g = 16 // e, 2 // e
    k = k.reshape(pages, h, blocks, 2, d // ek, 16, ek).transpose(-3, -2).reshape(pages, h, blocks, BLOCK, d).float()
    v = v.reshape(pages, h, blocks, d // (16 * g), 4, 16, g, 2, 4).permute(0, 1, 2, 7, 4, 8, 3, 6, 5)
    v = v.reshape(pages, h, blocks, BLOCK, d).float()
    if c["cache"] == "int8":
        sc = heads[..., blocks * 2 * part: blocks * 2 * part + blocks * 8].contiguous().view(torch.float32)
        sc = sc.reshape(pages, h, blocks, 2)
        k, v = k * sc[..., 0, None, None], v * sc[..., 1, None, None]
    return k.reshape(pages, h, -1, d), v.reshape(pages, h, -1, d)


def _plain_attend(s):
    c = s["case"]
    n, T, hkv, d, g = c["n"], c["tokens"], c["hkv"], c["d"], c["hq"] // c["hkv"]
    k, v = _unpack(c, s["pool"])
    table = s["table"].long().clamp(min=0)
    k = k[table].transpose(1, 2).reshape(n, hkv, -1, d)  # [n, H, L, d]
    v = v[table].transpose(1, 2).reshape(n, hkv, -1, d)
    q = s["q"].float().reshape(n, T, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, g * T, d)
    x = torch.matmul(q * s["scale"], k.transpose(-1, -2).contiguous()).view(n, hkv, g, T, -1)
    del k
    anc, node = _ancestors(s["parent"])
    depth = anc.sum(-1) - 1
    pos = s["pos"].long()
    j = torch.arange(x.shape[-1], device="cuda")
    slot = j[None] - pos[:, None]  # [n, L]: the node in a cache slot
    drafted = (slot >= 0) & (slot < T)
    slot = slot.clamp(0, T - 1)
    at = torch.where(drafted, pos[:, None] + depth.gather(1, slot), j[None])[:, None]  # positions of the slots
    see = torch.where(drafted[:, None], anc.gather(2, slot[:, None].expand(n, T, -1)), (j[None] < pos[:, None])[:, None])
    if c["window"]:
        p = (pos[:, None] + depth)[..., None]
        see &= (at > p - c["window"]) | (at < c["sinks"])
    see = see & node[..., None]
    x.masked_fill_(~see[:, None, None], -math.inf)
    x -= x.amax(-1, keepdim=True)
    x.exp_()
    x /= x.sum(-1, keepdim=True)
    x.masked_fill_(~node[:, None, None, :, None], 0.0)
    o = torch.matmul(x.view(n, hkv, g * T, -1), v).view(n, hkv, g, T, d)
    return o.permute(0, 3, 1, 2, 4).reshape(n * T, c["hq"], d).to(_tdtype(c))


def _plain_rotate(c, x, pos, cos, sin):
    half = c["rot"] // 2
    co, si = cos[pos].double()[:, None], sin[pos].double()[:, None]
    y = x.double()
    r = y[..., : c["rot"]]
    a, b = (r[..., 0::2], r[..., 1::2]) if c["interleaved"] else (r[..., :half], r[..., half:])
    ra, rb = a * co - b * si, b * co + a * si
    r = torch.stack((ra, rb), -1).flatten(-2) if c["interleaved"] else torch.cat((ra, rb), -1)
    return torch.cat((r, y[..., c["rot"]:]), -1).float()


def _plain_rows(c, pool, page, slot, part):
    """Elements (codes or values) of single cached rows [M, H, d] and their block scales [M, H]."""
    e, d, h = _elem(c), c["d"], c["hkv"]
    blocks, size = c["page_tokens"] // BLOCK, BLOCK * d
    b, t = slot // BLOCK, slot % BLOCK
    ch = torch.arange(d, device="cuda")
    if part == 0:
        ek = 16 // e
        off = (t // 16)[:, None] * (16 * d) + (ch // ek)[None] * (16 * ek) + (t % 16)[:, None] * ek + (ch % ek)[None]
    else:
        g = 2 // e
        off = ((ch // (16 * g))[None] * (512 * g) + ((t % 16) // 4)[:, None] * (128 * g) + (ch % 16)[None] * (8 * g)
               + ((ch // 16) % g)[None] * 8 + (t % 4 + 4 * (t // 16))[:, None])
    flat = pool.view(-1).view(torch.int8 if e == 1 else torch.bfloat16)
    head = torch.arange(h, device="cuda") * (_head_bytes(c) // e)
    base = page * (pool.shape[1] // e) + (2 * b + part) * size
    rows = flat[base[:, None, None] + head[None, :, None] + off[:, None, :]].float()
    if c["cache"] == "bf16":
        return rows, None
    at = (page[:, None] * (pool.shape[1] // 4) + torch.arange(h, device="cuda")[None] * (_head_bytes(c) // 4)
          + (blocks * 2 * size) // 4 + 2 * b[:, None] + part)
    return rows, pool.view(-1).view(torch.float32)[at]


def _code(x, scale):
    return torch.where(scale > 0, torch.round(x / scale), torch.zeros_like(x)).clamp(-127, 127)


def _plain_draft(s):
    """What a cache holds after the tree was appended and its path kept: the rows from the
    block of the first new token to the last accepted one, block by block."""
    c = s["case"]
    n, T, hkv, d, pt = c["n"], c["tokens"], c["hkv"], c["d"], c["page_tokens"]
    anc, node = _ancestors(s["parent"])
    start = s["pos"].long()
    pos = (start[:, None] + anc.sum(-1) - 1).clamp(min=0).reshape(-1)
    live = node.reshape(-1, 1, 1)
    q = torch.where(live, _plain_rotate(c, s["q"], pos, s["cos"], s["sin"]), 0.0)
    k = torch.where(live, _plain_rotate(c, s["k"], pos, s["cos"], s["sin"]), 0.0)
    v = torch.where(live, s["v"].float(), 0.0)
    out = [q.to(_tdtype(c))]
    # rows read back: the request, the position, the slot the row was appended to
    lens = np.diff(s["read_cu"])
    seq = torch.from_numpy(np.repeat(np.arange(n), lens)).cuda()
    at = torch.from_numpy(np.arange(int(s["read_cu"][-1])) - np.repeat(s["read_cu"][:-1], lens)
                          + np.repeat(s["read_lo"], lens)).cuda()
    step = at - start[seq]
    fresh = step >= 0
    came = torch.where(fresh, start[seq] + s["path"].long()[seq, step.clamp(0, T - 1)], at)  # source slot
    if c["cache"] == "bf16":
        for new in (k, v):
            rows = new.view(n, T, hkv, d)[seq, (came - start[seq]).clamp(min=0)]
            out.append(rows.to(torch.bfloat16).float().to(_tdtype(c)))
        return out
    lo = start // BLOCK * BLOCK  # the first block's start, per request
    nb = (T + 2 * BLOCK - 2) // BLOCK  # blocks a tree can touch
    # the block's older rows come from the page that was copied for the draft
    old_page = s["table"].long().clamp(min=0)[torch.arange(n, device="cuda"), (start // pt).clamp(max=s["table"].shape[1] - 1)].clone()
    held = start % pt > 0
    old_page[held] = s["copy_src"].long()[:-1]
    slots = (lo % pt)[:, None] + torch.arange(BLOCK, device="cuda")[None]
    kept = (lo[:, None] + torch.arange(BLOCK, device="cuda")[None]) < start[:, None]  # [n, 32]
    node_at = (start - lo)[:, None] + torch.arange(T, device="cuda")[None]  # place of node t from lo on
    for part, new in ((0, k), (1, v)):
        codes, scales = _plain_rows(c, s["pool"], old_page[:, None].expand(n, BLOCK).reshape(-1), slots.reshape(-1), part)
        codes = torch.where(kept[..., None, None], codes.view(n, BLOCK, hkv, d), 0.0)
        before = torch.zeros((n, nb, hkv), device="cuda")
        before[:, 0] = torch.where(kept.any(1)[:, None], scales.view(n, BLOCK, hkv)[:, 0], 0.0)
        x = torch.zeros((n, nb * BLOCK, hkv, d), device="cuda")
        x.scatter_(1, node_at[..., None, None].expand(n, T, hkv, d), new.view(n, T, hkv, d))
        amax = x.view(n, nb, BLOCK, hkv, d).abs().amax((2, 4))
        scale = torch.maximum(before, amax / torch.full_like(amax, 127))  # tensor by tensor: the IEEE quotient
        full = scale.repeat_interleave(BLOCK, 1)[..., None]
        cx = _code(x, full)
        older = torch.where((scale[:, :1] > before[:, :1])[..., None], _code(codes * before[:, :1, :, None], scale[:, :1, :, None]), codes)
        cx[:, :BLOCK] = torch.where(kept[..., None, None], older, cx[:, :BLOCK])
        # the accepted path: a block takes the largest scale of the blocks its rows come
        # from (and its own, where it holds older rows); rows of a smaller scale are coded again
        src = came - lo[seq]
        to = at - lo[seq]
        row_scale = scale[seq, src // BLOCK]
        last = torch.zeros_like(scale)
        last.view(n * nb, hkv).index_reduce_(0, seq * nb + to // BLOCK, row_scale, "amax")
        sn, so = last[seq, to // BLOCK][..., None], row_scale[..., None]
        row = cx[seq, src]
        row = torch.where(sn > so, _code(row * so, sn), row)
        out.append((row * sn).to(_tdtype(c)))
    return out


def _plain_state(s):
    """The recurrence node by node from each parent's state, then the path's last state."""
    c = s["case"]
    n, T, H, d = c["n"], c["tokens"], c["heads"], c["d"]
    q, k, v, g, beta = (s[x].float().view(n, T, H, -1) for x in ("q", "k", "v", "g", "beta"))
    node = s["parent"] >= -1
    q, k, v, g, beta = (torch.where(node[..., None, None], x, 0.0) for x in (q, k, v, g, beta))
    states = torch.empty((n, T + 1, H, d, d), device="cuda")  # the entering state last
    states[:, T] = s["pool"][s["page_in"].long()]
    r = torch.arange(n, device="cuda")
    up = torch.where(s["parent"] >= 0, s["parent"].long(), T)
    o = torch.empty((n, T, H, d), device="cuda")
    for t in range(T):
        S = states[r, up[:, t]] * torch.exp(g[:, t])[..., None]
        u = v[:, t] - (S * k[:, t][..., None]).sum(-2)
        S = S + (beta[:, t] * k[:, t])[..., None] * u[..., None, :]
        o[:, t] = (S * q[:, t][..., None]).sum(-2)
        states[:, t] = S
    end = s["path"].long().gather(1, (s["count"].long() - 1).clamp(min=0)[:, None])[:, 0]
    kept = states[r, torch.where(s["count"] > 0, end, T)]
    done = torch.empty_like(kept)
    done[s["page_out"].long() - n] = kept
    return [o.view(n * T, H, d).to(_tdtype(c)), done]


def _plain_conv(s):
    c = s["case"]
    n, T, C, W = c["n"], c["tokens"], c["channels"], c["width"]
    before = s["pool"][s["page_in"].long(), : (W - 1) * C].view(n, W - 1, C).float()
    node = s["parent"] >= -1
    x = torch.where(node[..., None], s["x"].float().view(n, T, C), 0.0)
    every = torch.cat((x, before.flip(1)), 1)  # T + i: i + 1 tokens before the tree
    line = torch.cat((torch.where(s["parent"] >= 0, s["parent"].long(), T),
                      (T + 1 + torch.arange(W - 1, device="cuda")).clamp(max=T + W - 2).expand(n, W - 1)), 1)
    at = torch.arange(T, device="cuda").expand(n, T)
    y = torch.zeros((n, T, C), device="cuda")
    for j in range(W - 1, -1, -1):
        y += every.gather(1, at[..., None].expand(n, T, C)) * s["w"][:, j]
        at = line.gather(1, at)
    y = torch.where(node[..., None], y, 0.0)
    # the window after the path: its last W - 1 inputs, the oldest first
    end = s["path"].long().gather(1, (s["count"].long() - 1).clamp(min=0)[:, None])
    at = torch.where(s["count"][:, None] > 0, end, T)
    kept = torch.empty((n, W - 1, C), device="cuda")
    for j in range(W - 2, -1, -1):
        kept[:, j] = every.gather(1, at[..., None].expand(n, 1, C))[:, 0]
        at = line.gather(1, at)
    done = torch.zeros_like(s["pool"][n:])
    done[s["page_out"].long() - n, : (W - 1) * C] = kept.view(n, -1).to(_tdtype(c))
    return [y.view(n * T, C).to(_tdtype(c)), done]


def _plain_release(s, refs, table, first, last):
    pt = s["case"]["page_tokens"]
    j = torch.arange(table.shape[1], device="cuda")[None] * pt
    out = (j >= first[:, None]) & (j + pt <= last[:, None]) & (table >= 0)
    gone = table[out].long()
    refs.index_add_(0, gone, -torch.ones_like(gone, dtype=torch.int32))
    table[out] = -1


def _plain_copy(s, src, dst, tokens=None):
    """Whole pages, or the blocks that hold their first tokens."""
    c = s["case"]
    blocks = c["page_tokens"] // BLOCK
    pool = s["pool"].view(s["pool"].shape[0], c["hkv"], blocks, -1)
    new = pool[src]
    if tokens is not None:
        b = torch.arange(blocks, device="cuda")[None] * BLOCK < tokens[:, None]
        new = torch.where(b[:, None, :, None], new, pool[dst])
    pool[dst] = new


def _plain_fork(s):
    c = s["case"]
    pt, refs, table = c["page_tokens"], s["refs"], s["table"]
    _plain_release(s, refs, table, s["first"], s["last"])
    src, dst, at = s["src"].long(), s["dst"].long(), s["at"].long()
    j = torch.arange(table.shape[1], device="cuda")[None]
    rows = torch.where(j < (at // pt)[:, None], table[src], -1)
    shared = rows[rows >= 0].long()
    refs.index_add_(0, shared, torch.ones_like(shared, dtype=torch.int32))
    tail = table[src, at // pt]
    need = (at % pt > 0) & (tail >= 0)
    free = (refs <= 0).nonzero()[:, 0].int()
    m = int(need.sum())
    fresh = free[:m]
    rows[need, (at // pt)[need]] = fresh
    table[dst] = rows
    refs[fresh.long()] = 1
    for name, x, pad in (("copy_src", tail[need], -1), ("copy_dst", fresh, -1), ("copy_tokens", (at % pt)[need].int(), 0)):
        s[name].fill_(pad)
        s[name][:m] = x
    s["fork_status"].zero_()
    # room for the next tokens: the free pages of lowest number, row by row
    j = j * pt
    want = (j + pt > s["new_lo"][:, None]) & (j < s["new_hi"][:, None]) & (table < 0)
    free = (refs <= 0).nonzero()[:, 0].int()
    k = int(want.sum())
    table[want] = free[:k]
    refs[free[:k].long()] = 1
    s["status"].zero_()
    _plain_copy(s, tail[need].long(), fresh.long(), (at % pt)[need])
    return [refs, table, s["copy_src"], s["copy_dst"], s["copy_tokens"], s["fork_status"], s["status"], s["pool"]]


def _plain_compact(s):
    refs, table = s["refs"], s["table"]
    refs.copy_(s["refs0"])
    table.copy_(s["table0"])
    held = torch.bincount(table[table >= 0].long(), minlength=refs.numel())
    holes = (refs <= 0).nonzero()[:, 0]
    movable = ((refs > 0) & (held == refs)).nonzero()[:, 0].flip(0)
    m = min(holes.numel(), movable.numel())
    m = int((holes[:m] < movable[:m]).sum())
    src, dst = movable[:m], holes[:m]
    place = torch.arange(refs.numel(), device="cuda", dtype=torch.int32)
    place[src] = dst.int()
    table.copy_(torch.where(table >= 0, place[table.long().clamp(min=0)], table))
    refs[dst] = refs[src]
    refs[src] = 0
    for name, x in (("copy_src", src), ("copy_dst", dst)):
        s[name].fill_(-1)
        s[name][:m] = x.int()
    _plain_copy(s, src, dst)
    return [refs, table, s["copy_src"], s["copy_dst"], s["pool"]]


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def _plan(s):
    """What a serving program keeps between calls: descriptors and workspaces."""
    if "plan" in s:
        return s["plan"]
    import hybrid_prefix_cache_amd as K
    c = s["case"]
    p = {"K": K}
    if c["op"] in ("attend", "draft"):
        p["pool"] = K.make_kv_pool(s["pool"], s["page_bytes"], s["pool"].shape[0], c["hkv"], c["d"], c["page_tokens"],
                                   K.KDA_INT8 if c["cache"] == "int8" else K.KDA_BF16)
        if c["op"] == "draft":
            p["rope"] = K.make_rope(s["cos"], s["sin"], interleaved=c["interleaved"])
            need = K.kda_kv_workspace_bytes(c["n"])
        else:
            need = K.kda_attn_tree_workspace_bytes(p["pool"], c["hq"], c["n"], c["tokens"], s["table"].shape[1],
                                                   window=c["window"], sinks=c["sinks"])
        p["ws"] = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    elif c["op"] == "state":
        p["pool"] = K.make_pool(s["pool"], c["heads"] * c["d"] * c["d"] * 4, 2 * c["n"], c["heads"], c["d"])
    elif c["op"] == "conv":
        p["pool"] = K.make_conv_pool(s["pool"], s["pool"].shape[1] * s["pool"].element_size(), 2 * c["n"], c["channels"],
                                     c["width"], K.KDA_F32 if c["dtype"] == "f32" else K.KDA_BF16)
    else:
        p["pool"] = K.make_kv_pool(s["pool"], s["pool"].shape[1] * 2, s["pool"].shape[0], c["hkv"], c["d"], c["page_tokens"],
                                   K.KDA_BF16)
        p["map"] = K.make_page_map(s["refs"], s["table"], c["page_tokens"])
        p["ws"] = torch.empty(K.kda_pages_workspace_bytes(p["map"]), dtype=torch.uint8, device="cuda")
    s["plan"] = p
    return p


def _own_run(s):
    c, p = s["case"], _plan(s)
    K, pool = p["K"], p["pool"]
    if c["op"] == "attend":
        K.kda_attn_tree(pool, s["q"], s["out"], s["parent"], s["pos"], s["table"], scale=s["scale"], window=c["window"],
                        sinks=c["sinks"], workspace=p["ws"])
        return s["out"]
    if c["op"] == "draft":
        K.kda_kv_copy_pages(pool, s["copy_src"], s["copy_dst"], tokens=s["copy_tokens"])
        K.kda_kv_append_tree(pool, s["q"], s["k"], s["v"], s["out"], s["parent"], s["pos"], s["table"], rope=p["rope"])
        K.kda_kv_commit(pool, s["path"], s["count"], s["pos"], s["table"])
        K.kda_kv_read(pool, s["k_out"], s["v_out"], s["read_cu"], s["table"], start_pos=s["read_lo"], workspace=p["ws"])
        return [s["out"], s["k_out"], s["v_out"]]
    if c["op"] == "state":
        K.kda_decode_tree(pool, s["q"], s["k"], s["v"], s["g"], s["beta"], s["o"], s["parent"], s["page_in"])
        K.kda_decode_commit(pool, s["k"], s["v"], s["g"], s["beta"], s["path"], s["count"], s["page_in"], s["page_out"])
        return [s["o"], s["pool"][c["n"]:]]
    if c["op"] == "conv":
        K.kda_short_conv_tree(pool, s["x"], s["w"], s["y"], s["parent"], s["page_in"])
        K.kda_short_conv_commit(pool, s["x"], s["path"], s["count"], s["page_in"], s["page_out"])
        return [s["y"], s["pool"][c["n"]:]]
    if c["op"] == "fork":
        K.kda_pages_free(p["map"], s["first"], s["last"])
        K.kda_pages_fork(p["map"], s["src"], s["dst"], s["at"], s["copy_src"], s["copy_dst"], s["copy_tokens"],
                         s["fork_status"], workspace=p["ws"])
        K.kda_pages_reserve(p["map"], s["new_lo"], s["new_hi"], s["status"], workspace=p["ws"])
        K.kda_kv_copy_pages(pool, s["copy_src"], s["copy_dst"], tokens=s["copy_tokens"])
        return [s["refs"], s["table"], s["copy_src"], s["copy_dst"], s["copy_tokens"], s["fork_status"], s["status"], s["pool"]]
    s["refs"].copy_(s["refs0"])
    s["table"].copy_(s["table0"])
    K.kda_pages_compact(p["map"], s["copy_src"], s["copy_dst"], workspace=p["ws"])
    K.kda_kv_copy_pages(pool, s["copy_src"], s["copy_dst"])
    return [s["refs"], s["table"], s["copy_src"], s["copy_dst"], s["pool"]]


def run(state):
    if own:
        return _own_run(state)
    plain = {"attend": _plain_attend, "draft": _plain_draft, "state": _plain_state, "conv": _plain_conv,
             "fork": _plain_fork, "compact": _plain_compact}
    return plain[state["case"]["op"]](state)


def work(case):
    c = case
    if c["op"] in ("fork", "compact"):
        # the tables and counts read and written once; the copied pages read and written
        n, pt = c["n"], c["page_tokens"]
        starts = _spans(c)
        m = max(1, n // c["cut"])
        pages = sum(-(-a // pt) for a in starts)
        book = 2 * 4 * (pages * (1 + 1 / c["cut"]) * 2)
        tail = m * 0.5 if c["op"] == "fork" else pages / c["cut"] / 2
        return {"bytes": book + 2 * tail * c["hkv"] * pt * c["d"] * 4, "flops": 0}
    e, d, n, T = (4 if c["dtype"] == "f32" else 2), c["d"], c["n"], c["tokens"]
    parent, _, count = _trees(c)
    nodes = sum(sum(p >= -1 for p in row) for row in parent)
    depth = []
    for row in parent:
        at = []
        for p in row:
            at.append(0 if p == -2 else 1 + (at[p] if p >= 0 else 0))
        depth.append(at)
    pairs = sum(map(sum, depth))
    if c["op"] == "conv":
        rows = 2 * nodes * c["channels"] * e + 2 * n * (c["width"] - 1) * c["channels"] * e
        return {"bytes": rows + 4 * c["channels"] * c["width"], "flops": 2 * nodes * c["channels"] * c["width"]}
    if c["op"] == "state":
        H = c["heads"]
        # the entering state read once, the accepted one written once; a node needs two
        # products with the state, and two and an update with each ancestor
        return {"bytes": 2 * n * H * d * d * 4 + nodes * H * (5 * d + 1) * e, "flops": H * (4 * nodes * d * d + 8 * pairs * d)}
    starts, ec = _spans(c), _elem(c)
    if c["op"] == "draft":
        back = sum(a % BLOCK if c["cache"] == "int8" else 0 for a in starts)
        kept = sum(count)
        tail = sum(-(-(a % c["page_tokens"]) // BLOCK) * BLOCK for a in starts)
        return {"bytes": nodes * d * (2 * c["hq"] * e + 2 * c["hkv"] * (e + ec)) + 2 * kept * c["hkv"] * d * 2 * ec
                + 2 * (back + kept) * c["hkv"] * d * (e + ec) + 2 * tail * c["hkv"] * 2 * d * ec,
                "flops": nodes * d * 4 * (c["hq"] + c["hkv"])}
    seen, keys = 0, 0
    for a, row, at in zip(starts, parent, depth):
        live = sum(p >= -1 for p in row)
        far = min(a, c["window"] + c["sinks"]) if c["window"] else a
        seen += live * far + sum(at)
        keys += far + live
    return {"bytes": 2 * keys * c["hkv"] * d * ec + 2 * nodes * c["hq"] * d * e, "flops": 4 * seen * c["hq"] * d}


# ---------------------------------------------------------------------------
# 64 bits, written apart from the plain forms
# ---------------------------------------------------------------------------
def _bytes_of(c, part, t, ch):
    """Byte offset, within a block, of channel ch of token t (numpy arrays)."""
    size = BLOCK * c["d"] * _elem(c)
    if c["cache"] == "bf16":
        if part == 0:
            return 2 * ((t >> 4) * 16 * c["d"] + (ch >> 3) * 128 + (t & 15) * 8 + (ch & 7))
        return size + 2 * ((ch >> 4) * 512 + ((t & 15) >> 2) * 128 + (ch & 15) * 8 + (t & 3) + 4 * (t >> 4))
    if part == 0:
        return (t >> 4) * 16 * c["d"] + (ch >> 4) * 256 + (t & 15) * 16 + (ch & 15)
    return size + (ch >> 5) * 1024 + ((t & 15) >> 2) * 256 + (ch & 15) * 16 + ((ch >> 4) & 1) * 8 + (t & 3) + 4 * (t >> 4)


def _exact_rows(c, pool, pages, part, n, first=0):
    """Tokens [first, n) of a sequence (its page ids; first a multiple of the block), every head, in 64 bits:
    codes or values [heads, n - first, d], and the scales [heads, n - first] or None."""
    hb, size = _head_bytes(c), 2 * BLOCK * c["d"] * _elem(c)
    blocks = c["page_tokens"] // BLOCK
    t, ch = np.meshgrid(np.arange(BLOCK), np.arange(c["d"]), indexing="ij")
    inside = torch.from_numpy(_bytes_of(c, part, t, ch)).cuda()
    b = torch.arange(first // BLOCK, -(-n // BLOCK), device="cuda")
    head = torch.arange(c["hkv"], device="cuda")[:, None] * hb
    page = pages[b // blocks].long() * pool.shape[1]
    at = (page + (b % blocks) * size + head)[:, :, None, None] + inside
    raw = pool.view(-1)
    if c["cache"] == "bf16":
        x = raw.view(torch.bfloat16)[at // 2].double()
        return x.flatten(1, 2)[:, : n - first], None
    code = raw.view(torch.int8)[at].double().flatten(1, 2)[:, : n - first]
    sat = page + blocks * size + (b % blocks) * 8 + 4 * part + head
    return code, raw.view(torch.float32)[sat // 4].double().repeat_interleave(BLOCK, 1)[:, : n - first]


def _ways(row):
    """Per node the nodes from its root to itself (empty: no node)."""
    out = []
    for t, p in enumerate(row):
        out.append([] if p < -1 else (out[p] if p >= 0 else []) + [t])
    return out


def _exact_attend(c, s):
    n, T, g, hkv = c["n"], c["tokens"], c["hq"] // c["hkv"], c["hkv"]
    out = torch.zeros((n * T, c["hq"], c["d"]), dtype=torch.float64, device="cuda")
    for r, (a, row) in enumerate(zip(_spans(c), _trees(c)[0])):
        k, ks = _exact_rows(c, s["pool"], s["table"][r], 0, a + T)
        v, vs = _exact_rows(c, s["pool"], s["table"][r], 1, a + T)
        if ks is not None:
            k, v = k * ks[..., None], v * vs[..., None]
        see = np.zeros((T, a + T), bool)
        for t, way in enumerate(_ways(row)):
            if not way:
                continue
            p = a + len(way) - 1
            where = np.concatenate([np.arange(a), a + np.arange(len(way))])
            slots = np.concatenate([np.arange(a), a + np.asarray(way)])
            ok = np.ones(len(where), bool)
            if c["window"]:
                ok = (p - where < c["window"]) | (where < c["sinks"])
            see[t, slots[ok]] = True
        live = [t for t in range(T) if row[t] >= -1]
        see = torch.from_numpy(see[live]).cuda()
        for h in range(hkv):
            q = s["q"][r * T: (r + 1) * T, h * g: (h + 1) * g].double()[live]
            x = (q.transpose(0, 1).reshape(-1, c["d"]) @ k[h].T * s["scale"]).view(g, len(live), -1)
            x = x.masked_fill(~see, -math.inf)
            w = torch.exp(x - x.amax(2, keepdim=True))
            y = (w / w.sum(2, keepdim=True)).view(g * len(live), -1) @ v[h]
            rows = r * T + torch.tensor(live, device="cuda")
            out[rows, h * g: (h + 1) * g] = y.view(g, len(live), -1).transpose(0, 1)
    return out


def _f32(x):
    return x.float().double()


def _exact_rotate(c, x, pos, cos, sin):
    """x: [rows, heads, d] in 64 bits at positions pos."""
    half, at = c["rot"] // 2, torch.arange(c["d"], device="cuda")
    if c["interleaved"]:
        other, pair, first = at ^ 1, at // 2, at % 2 == 0
    else:
        other, pair, first = torch.where(at < half, at + half, at - half), at % half, at < half
    turned = at < c["rot"]
    pair, other = torch.where(turned, pair, 0), torch.where(turned, other, at)
    co, si = (m[pos].double()[:, pair][:, None] for m in (cos, sin))
    return torch.where(turned, x * co + x[..., other] * torch.where(first, -si, si), x)


def _exact_draft(c, s):
    n, T, hkv, d, pt = c["n"], c["tokens"], c["hkv"], c["d"], c["page_tokens"]
    out = [torch.zeros((n * T, c["hq"], d), dtype=torch.float64, device="cuda")]
    out += [torch.zeros((int(s["read_cu"][-1]), hkv, d), dtype=torch.float64, device="cuda") for _ in range(2)]
    parent, path, count = _trees(c)
    tails = iter(s["copy_src"].tolist())
    for r, a in enumerate(_spans(c)):
        ways = _ways(parent[r])
        live = [t for t in range(T) if ways[t]]
        rows = r * T + torch.tensor(live, device="cuda")
        pos = torch.tensor([a + len(ways[t]) - 1 for t in live], device="cuda")
        out[0][rows] = _exact_rotate(c, s["q"][rows].double(), pos, s["cos"], s["sin"])
        lo, way = int(s["read_lo"][r]), path[r][: count[r]]
        tail = next(tails) if a % pt else -1
        for part, x in ((0, _exact_rotate(c, s["k"][rows].double(), pos, s["cos"], s["sin"])), (1, s["v"][rows].double())):
            to = out[1 + part][int(s["read_cu"][r]): int(s["read_cu"][r + 1])]
            new = torch.zeros((T, hkv, d), dtype=torch.float64, device="cuda")
            new[live] = x
            if c["cache"] == "bf16":
                to.copy_(new[way].float().to(torch.bfloat16))
                continue
            # codes are a rule on fp32 numbers: quotients in 64 bits, rounded to fp32 as IEEE division gives them
            held, nb = a - lo, -(-(a + T - lo) // BLOCK)
            line = torch.zeros((nb * BLOCK, hkv, d), dtype=torch.float64, device="cuda")
            line[held: held + T] = _f32(new)
            top = _f32(line.view(nb, BLOCK, hkv, d).abs().amax((1, 3)) / 127.0)
            if held:
                pages = s["table"][r].clone()
                pages[a // pt] = tail
                old, before = _exact_rows(c, s["pool"], pages, part, a, lo)
                old, before = old.transpose(0, 1), before[:, 0]
                grown = top[0] > before
                top[0] = torch.maximum(top[0], before)
            sc = top.repeat_interleave(BLOCK, 0)[..., None]
            div = torch.where(sc > 0, sc, 1.0)
            code = torch.round(_f32(line / div)).clamp(-127, 127)
            if held:
                again = torch.round(_f32(_f32(old * before[:, None]) / div[:held])).clamp(-127, 127)
                code[:held] = torch.where(grown[:, None], again, old)
            src = list(range(held)) + [held + t for t in way]
            for b in range(-(-len(src) // BLOCK)):
                mine = torch.tensor(src[b * BLOCK: (b + 1) * BLOCK], device="cuda")
                big = sc[mine].amax(0)  # [heads, 1]
                again = torch.round(_f32(_f32(code[mine] * sc[mine]) / torch.where(big > 0, big, 1.0))).clamp(-127, 127)
                kept = torch.where(sc[mine] < big, again, code[mine])
                to[b * BLOCK: b * BLOCK + len(mine)] = kept * big
    return out


def _exact_state(c, s):
    """The closed form: with G the gates summed along each way, u solves a unit triangular
    system over the ancestors, and outputs and states are sums over them."""
    n, T, H, d = c["n"], c["tokens"], c["heads"], c["d"]
    parent, path, count = _trees(c)
    anc = np.zeros((n, T, T))
    for r in range(n):
        for t, way in enumerate(_ways(parent[r])):
            anc[r, t, way] = 1.0
    node = torch.from_numpy(anc.any(2)).cuda()
    anc = torch.from_numpy(anc).cuda()
    done = torch.zeros((n, H, d, d), dtype=torch.float64, device="cuda")
    out = torch.zeros((n, T, H, d), dtype=torch.float64, device="cuda")
    strict = anc * (1 - torch.eye(T, device="cuda", dtype=torch.float64))
    for h in range(H):
        q, k, v, g, beta = (s[x].double().view(n, T, H, -1)[:, :, h] for x in ("q", "k", "v", "g", "beta"))
        q, k, v, g, beta = (torch.where(node[..., None], x, 0.0) for x in (q, k, v, g, beta))
        S = s["pool"][s["page_in"].long(), h].double()
        G = torch.bmm(anc, g)
        kb = beta * k
        A, Q = (torch.zeros((n, T, T), dtype=torch.float64, device="cuda") for _ in range(2))
        for t in range(T):
            f = torch.exp(torch.where(anc[:, t, :, None] > 0, G[:, t, None] - G, -math.inf)) * kb
            A[:, t] = torch.bmm(f, k[:, t, :, None])[..., 0]
            Q[:, t] = torch.bmm(f, q[:, t, :, None])[..., 0]
        eye = torch.eye(T, device="cuda", dtype=torch.float64)
        u = torch.linalg.solve_triangular(A * strict + eye, v - torch.bmm(k * torch.exp(G), S), upper=False)
        out[:, :, h] = torch.bmm(q * torch.exp(G), S) + torch.bmm(Q, u)
        for r in range(n):
            way = path[r][: count[r]]
            if not way:
                done[r, h] = S[r]
                continue
            last = G[r, way[-1]]
            done[r, h] = torch.exp(last)[:, None] * S[r] + (torch.exp(last - G[r, way]) * kb[r, way]).T.contiguous() @ u[r, way]
    kept = torch.empty_like(done)
    kept[s["page_out"].long() - n] = done
    return [out.view(n * T, H, d), kept]


def _exact_conv(c, s):
    n, T, C, W = c["n"], c["tokens"], c["channels"], c["width"]
    parent, path, count = _trees(c)
    y = torch.zeros((n * T, C), dtype=torch.float64, device="cuda")
    done = torch.zeros(s["pool"][n:].shape, dtype=torch.float64, device="cuda")
    w = s["w"].double()
    for r in range(n):
        before = s["pool"][int(s["page_in"][r]), : (W - 1) * C].view(W - 1, C).double()
        x = s["x"][r * T: (r + 1) * T].double()
        for t, way in enumerate(_ways(parent[r])):
            if way:
                y[r * T + t] = (torch.cat((before, x[way]))[-W:] * w.T).sum(0)
        kept = torch.cat((before, x[path[r][: count[r]]]))[-(W - 1):]
        done[int(s["page_out"][r]) - n, : (W - 1) * C] = kept.reshape(-1)
    return [y, done]


def exact(case, seed):
    if case["op"] in ("fork", "compact"):
        return None  # whole numbers and copies
    s = prepare(case, seed)
    c = s["case"]
    return {"attend": _exact_attend, "draft": _exact_draft, "state": _exact_state, "conv": _exact_conv}[c["op"]](c, s)
