"""Argument checks of the tree and page calls that need no GPU: every call here is
refused (or has nothing to do) before the device is touched."""
import ctypes

import pytest

import hybrid_prefix_cache_amd as K

F = 1 << 20  # stands for a device pointer
BF, F32 = K.KDA_BF16, K.KDA_F32


def pool(**kw):
    d = dict(base=F, page_bytes=2 * 64 * 64 * 4, num_pages=8, num_heads=2, d_k=64, d_v=64)
    d.update(kw)
    return K.kda_pool(*d.values())


def cpool(**kw):
    d = dict(base=F, page_bytes=4096, num_pages=8, channels=256, width=4, dtype=BF)
    d.update(kw)
    return K.kda_conv_pool(*d.values())


def kv(**kw):
    d = dict(base=F, page_bytes=2 * K.kda_kv_head_bytes(64, 64, BF), num_pages=8, num_heads=2, head_dim=64, page_tokens=64,
             dtype=BF)
    d.update(kw)
    return K.kda_kv_pool(*d.values())


def page_map(**kw):
    d = dict(refs=F, table=2 * F, num_pages=16, rows=4, max_pages=8, page_tokens=64)
    d.update(kw)
    return K.kda_page_map(*d.values())


def call(name, first, defaults, kw):
    a = {**defaults, **kw}
    return K.raw_call(name, None if first is None else ctypes.byref(first), *a.values(), None)


def told(status):
    assert (K.kda_last_error() == "") == (status == K.KDA_OK)


TREE = dict(q=F, k=2 * F, v=3 * F, g=4 * F, beta=5 * F, ind=BF, o=6 * F, outd=BF, n=3, tokens=7, parent=7 * F, page_in=8 * F)


@pytest.mark.parametrize("p,kw,status", [
    (None, {}, K.KDA_ERR_NULL), (pool(base=0), {}, K.KDA_ERR_POOL), (pool(page_bytes=256), {}, K.KDA_ERR_POOL),
    (pool(d_k=96, d_v=96), {}, K.KDA_ERR_SHAPE), (pool(), dict(ind=K.KDA_INT8), K.KDA_ERR_DTYPE),
    (pool(), dict(outd=9), K.KDA_ERR_DTYPE), (pool(), dict(n=-1), K.KDA_ERR_SHAPE), (pool(), dict(tokens=0), K.KDA_ERR_SHAPE),
    (pool(), dict(tokens=65), K.KDA_ERR_SHAPE), (pool(), dict(n=1 << 22), K.KDA_ERR_SHAPE),
    (pool(), dict(q=F + 8), K.KDA_ERR_SHAPE), (pool(), dict(o=F + 2), K.KDA_ERR_SHAPE),
    *[(pool(), {x: None}, K.KDA_ERR_NULL) for x in ("q", "k", "v", "g", "beta", "o", "parent", "page_in")],
    (pool(), dict(n=0, q=None), K.KDA_OK),
])
def test_decode_tree(p, kw, status):
    assert call("kda_decode_tree", p, TREE, kw) == status
    told(status)


COMMIT = dict(k=2 * F, v=3 * F, g=4 * F, beta=5 * F, ind=BF, n=3, tokens=7, path=F, count=F, page_in=F, page_out=F)


@pytest.mark.parametrize("p,kw,status", [
    (None, {}, K.KDA_ERR_NULL), (pool(num_pages=0), {}, K.KDA_ERR_POOL), (pool(), dict(ind=5), K.KDA_ERR_DTYPE),
    (pool(), dict(tokens=-2), K.KDA_ERR_SHAPE), (pool(), dict(n=-4), K.KDA_ERR_SHAPE), (pool(), dict(v=F + 4), K.KDA_ERR_SHAPE),
    *[(pool(), {x: None}, K.KDA_ERR_NULL) for x in ("k", "v", "g", "beta", "path", "count", "page_in", "page_out")],
    (pool(), dict(n=0, path=None), K.KDA_OK),
])
def test_decode_commit(p, kw, status):
    assert call("kda_decode_commit", p, COMMIT, kw) == status
    told(status)


CONV = dict(x=F, w=2 * F, y=3 * F, outd=BF, n=3, tokens=7, parent=F, page_in=F)


@pytest.mark.parametrize("p,kw,status", [
    (None, {}, K.KDA_ERR_NULL), (cpool(width=5), {}, K.KDA_ERR_SHAPE), (cpool(channels=12), {}, K.KDA_ERR_SHAPE),
    (cpool(), dict(outd=2), K.KDA_ERR_DTYPE), (cpool(), dict(tokens=65), K.KDA_ERR_SHAPE), (cpool(), dict(n=-1), K.KDA_ERR_SHAPE),
    (cpool(), dict(x=F + 8), K.KDA_ERR_SHAPE), (cpool(), dict(y=F), K.KDA_ERR_SHAPE),
    (cpool(channels=1 << 20, page_bytes=3 << 21), dict(n=1 << 16), K.KDA_ERR_SHAPE),
    *[(cpool(), {x: None}, K.KDA_ERR_NULL) for x in ("x", "w", "y", "parent", "page_in")], (cpool(), dict(n=0), K.KDA_OK),
])
def test_conv_tree(p, kw, status):
    assert call("kda_short_conv_tree", p, CONV, kw) == status
    told(status)


CONV_COMMIT = dict(x=F, n=3, tokens=7, path=F, count=F, page_in=F, page_out=F)


@pytest.mark.parametrize("p,kw,status", [
    (None, {}, K.KDA_ERR_NULL), (cpool(base=None), {}, K.KDA_ERR_POOL), (cpool(), dict(tokens=0), K.KDA_ERR_SHAPE),
    (cpool(), dict(x=F + 4), K.KDA_ERR_SHAPE),
    *[(cpool(), {x: None}, K.KDA_ERR_NULL) for x in ("x", "path", "count", "page_in", "page_out")], (cpool(), dict(n=0), K.KDA_OK),
])
def test_conv_commit(p, kw, status):
    assert call("kda_short_conv_commit", p, CONV_COMMIT, kw) == status
    told(status)


APPEND = dict(rope=None, q=F, k=2 * F, v=3 * F, ind=BF, q_ld=256, k_ld=128, v_ld=128, q_out=5 * F, hq=4, n=2, tokens=7,
              pos=F, parent=F, table=F, max_pages=4)


@pytest.mark.parametrize("p,kw,status", [
    (None, {}, K.KDA_ERR_NULL), (kv(dtype=F32), {}, K.KDA_ERR_DTYPE), (kv(), dict(parent=None), K.KDA_ERR_NULL),
    (kv(), dict(tokens=65), K.KDA_ERR_SHAPE), (kv(), dict(pos=None), K.KDA_ERR_NULL), (kv(), dict(k_ld=64), K.KDA_ERR_SHAPE),
    (kv(), dict(q_out=F + 512), K.KDA_ERR_SHAPE), (kv(), dict(table=None), K.KDA_ERR_NULL),
    (kv(), dict(max_pages=0), K.KDA_ERR_SHAPE), (kv(), dict(n=0, parent=None), K.KDA_OK),
])
def test_append_tree(p, kw, status):
    assert call("kda_kv_append_tree", p, APPEND, kw) == status
    told(status)


ATTEND = dict(q=F, ind=BF, q_ld=256, o=2 * F, outd=BF, hq=4, scale=ctypes.c_float(0.1), window=0, sinks=0, n=2, tokens=7,
              pos=F, parent=F, table=F, max_pages=4, ws=F, wsb=ctypes.c_size_t(1 << 20))


@pytest.mark.parametrize("p,kw,status", [
    (None, {}, K.KDA_ERR_NULL), (kv(), dict(hq=3), K.KDA_ERR_SHAPE), (kv(), dict(scale=ctypes.c_float(-1)), K.KDA_ERR_SHAPE),
    (kv(), dict(window=-1), K.KDA_ERR_SHAPE), (kv(), dict(parent=None), K.KDA_ERR_NULL), (kv(), dict(tokens=0), K.KDA_ERR_SHAPE),
    (kv(), dict(ws=None), K.KDA_ERR_WORKSPACE), (kv(), dict(ws=F + 16), K.KDA_ERR_WORKSPACE),
    (kv(), dict(wsb=ctypes.c_size_t(255)), K.KDA_ERR_WORKSPACE), (kv(), dict(o=F), K.KDA_ERR_SHAPE),
    (kv(), dict(max_pages=1 << 25), K.KDA_ERR_SHAPE), (kv(), dict(n=0), K.KDA_OK),
])
def test_attn_tree(p, kw, status):
    assert call("kda_attn_tree", p, ATTEND, kw) == status
    told(status)


def test_attn_tree_workspace():
    p = kv()
    assert K.kda_attn_tree_workspace_bytes(p, 4, 2, 7, 4) == K.kda_attn_decode_workspace_bytes(p, 4, 2, 7, 4) >= 256
    assert K.kda_attn_tree_workspace_bytes(p, 3, 2, 7, 4) == 0 and K.kda_attn_tree_workspace_bytes(p, 4, 2, 65, 4) == 0


KV_COMMIT = dict(n=2, tokens=7, pos=F, path=F, count=F, table=F, max_pages=4)


@pytest.mark.parametrize("p,kw,status", [
    (None, {}, K.KDA_ERR_NULL), (kv(head_dim=32), {}, K.KDA_ERR_SHAPE), (kv(), dict(tokens=0), K.KDA_ERR_SHAPE),
    (kv(), dict(path=None), K.KDA_ERR_NULL), (kv(), dict(count=None), K.KDA_ERR_NULL), (kv(), dict(pos=None), K.KDA_ERR_NULL),
    (kv(), dict(table=None), K.KDA_ERR_NULL), (kv(), dict(n=1 << 23), K.KDA_ERR_SHAPE), (kv(), dict(n=0), K.KDA_OK),
])
def test_kv_commit(p, kw, status):
    assert call("kda_kv_commit", p, KV_COMMIT, kw) == status
    told(status)


@pytest.mark.parametrize("kw,status", [
    ({}, K.KDA_OK), (dict(refs=None), K.KDA_ERR_NULL), (dict(table=None), K.KDA_ERR_NULL), (dict(refs=F + 2), K.KDA_ERR_SHAPE),
    (dict(num_pages=0), K.KDA_ERR_SHAPE), (dict(num_pages=(1 << 24) + 1), K.KDA_ERR_SHAPE), (dict(rows=0), K.KDA_ERR_SHAPE),
    (dict(max_pages=0), K.KDA_ERR_SHAPE), (dict(page_tokens=0), K.KDA_ERR_SHAPE),
    (dict(max_pages=1 << 20, page_tokens=1 << 11), K.KDA_ERR_SHAPE), (dict(rows=1 << 20, max_pages=1 << 11), K.KDA_ERR_SHAPE),
])
def test_page_map(kw, status):
    m = page_map(**kw)
    assert K.kda_page_map_check(m) == status
    told(status)
    assert (K.kda_pages_workspace_bytes(m) > 0) == (status == K.KDA_OK)


def test_page_map_null():
    assert K.raw_call("kda_page_map_check", None) == K.KDA_ERR_NULL


WS = dict(ws=F, wsb=ctypes.c_size_t(1 << 20))
NO_WS = [(dict(ws=None), K.KDA_ERR_WORKSPACE), (dict(ws=F + 128), K.KDA_ERR_WORKSPACE),
         (dict(wsb=ctypes.c_size_t(1023)), K.KDA_ERR_WORKSPACE)]


@pytest.mark.parametrize("kw,status", [*[({x: None}, K.KDA_ERR_NULL) for x in ("first", "last", "status")], *NO_WS])
def test_reserve(kw, status):
    assert call("kda_pages_reserve", page_map(), dict(first=F, last=F, status=F, **WS), kw) == status
    assert call("kda_pages_reserve", page_map(rows=0), dict(first=F, last=F, status=F, **WS), {}) == K.KDA_ERR_SHAPE


def test_free():
    for kw in (dict(first=None), dict(last=None)):
        assert call("kda_pages_free", page_map(), dict(first=F, last=F), kw) == K.KDA_ERR_NULL
    assert call("kda_pages_free", None, dict(first=F, last=F), {}) == K.KDA_ERR_NULL


FORK = dict(n=3, src=F, dst=F, tokens=F, cs=F, cd=F, ct=F, status=F, **WS)


@pytest.mark.parametrize("kw,status", [
    *[({x: None}, K.KDA_ERR_NULL) for x in ("src", "dst", "tokens", "cs", "cd", "ct", "status")], *NO_WS,
    (dict(n=-1), K.KDA_ERR_SHAPE), (dict(n=5), K.KDA_ERR_SHAPE), (dict(n=0, src=None), K.KDA_OK),
])
def test_fork(kw, status):
    assert call("kda_pages_fork", page_map(), FORK, kw) == status
    told(status)


@pytest.mark.parametrize("kw,status", [(dict(cs=None), K.KDA_ERR_NULL), (dict(cd=None), K.KDA_ERR_NULL), *NO_WS])
def test_compact(kw, status):
    assert call("kda_pages_compact", page_map(), dict(cs=F, cd=F, **WS), kw) == status


@pytest.mark.parametrize("p,kw,status", [
    (None, {}, K.KDA_ERR_NULL), (kv(num_pages=0), {}, K.KDA_ERR_POOL), (kv(), dict(n=-1), K.KDA_ERR_SHAPE),
    (kv(), dict(src=None), K.KDA_ERR_NULL), (kv(), dict(dst=None), K.KDA_ERR_NULL), (kv(), dict(n=0, src=None), K.KDA_OK),
])
def test_copy_pages(p, kw, status):
    assert call("kda_kv_copy_pages", p, dict(n=4, src=F, dst=F, tokens=None), kw) == status
    told(status)
