"""Argument checks of the key/value cache operators that need no GPU: every call
here is refused (or has nothing to do) before the device is touched."""
import ctypes

import numpy as np
import pytest

import hybrid_prefix_cache_amd as K

FAKE = 1 << 20
P = ctypes.c_void_p


def pool(**kw):
    d = dict(base=FAKE, num_pages=16, num_heads=2, head_dim=128, page_tokens=64, dtype=K.KDA_INT8)
    d.update(kw)
    if "page_bytes" not in d:
        d["page_bytes"] = d["num_heads"] * max(K.kda_kv_head_bytes(d["head_dim"], d["page_tokens"], d["dtype"]), 256)
    return K.make_kv_pool(d["base"], d["page_bytes"], d["num_pages"], d["num_heads"], d["head_dim"],
                          d["page_tokens"], d["dtype"])


def test_head_bytes():
    assert K.kda_kv_head_bytes(128, 64, K.KDA_BF16) == 64 * 128 * 4
    assert K.kda_kv_head_bytes(64, 32, K.KDA_BF16) == 32 * 64 * 4
    assert K.kda_kv_head_bytes(128, 6144, K.KDA_INT8) == 6144 * 256 + 192 * 8
    assert K.kda_kv_head_bytes(64, 32, K.KDA_INT8) == 32 * 128 + 256  # scales padded to 256
    for bad in ((96, 64, K.KDA_BF16), (128, 48, K.KDA_BF16), (128, 0, K.KDA_INT8), (128, 64, K.KDA_F32),
                (128, (1 << 20) + 32, K.KDA_INT8), (128, -32, K.KDA_BF16)):
        assert K.kda_kv_head_bytes(*bad) == -1, bad


@pytest.mark.parametrize("kw,status", [
    ({}, K.KDA_OK), (dict(dtype=K.KDA_BF16), K.KDA_OK), (dict(base=0), K.KDA_ERR_POOL),
    (dict(base=FAKE + 128), K.KDA_ERR_POOL), (dict(num_pages=0), K.KDA_ERR_POOL), (dict(num_heads=0), K.KDA_ERR_POOL),
    (dict(dtype=K.KDA_F32), K.KDA_ERR_DTYPE), (dict(dtype=9), K.KDA_ERR_DTYPE), (dict(head_dim=96), K.KDA_ERR_SHAPE),
    (dict(page_tokens=48), K.KDA_ERR_SHAPE), (dict(page_tokens=0), K.KDA_ERR_SHAPE),
    (dict(page_bytes=2 * K.kda_kv_head_bytes(128, 64, K.KDA_INT8) - 256), K.KDA_ERR_POOL),
    (dict(page_bytes=2 * K.kda_kv_head_bytes(128, 64, K.KDA_INT8) + 8), K.KDA_ERR_POOL),
    (dict(page_bytes=2 * K.kda_kv_head_bytes(128, 64, K.KDA_INT8) + 256), K.KDA_OK),
])
def test_pool_check(kw, status):
    assert K.kda_kv_pool_check(pool(**kw)) == status
    assert (K.kda_last_error() == "") == (status == K.KDA_OK)


def test_null_pool():
    assert K.raw_call("kda_kv_pool_check", None) == K.KDA_ERR_NULL


def i64(x):
    return (ctypes.c_int64 * len(x))(*x)


def append(p=None, rope=None, q=FAKE, k=2 * FAKE, v=3 * FAKE, dt=K.KDA_BF16, q_ld=512, k_ld=256, v_ld=256,
           q_out=5 * FAKE, hq=4, cu=(0, 10), start=None, table=FAKE, max_pages=4, ws=None, wsb=0):
    return K.raw_call("kda_kv_append", ctypes.byref(p or pool()), None if rope is None else ctypes.byref(rope), q, k, v,
                      dt, q_ld, k_ld, v_ld, q_out, hq, len(cu) - 1, i64(cu), None if start is None else i64(start),
                      table, max_pages, ws, wsb, None)


def step(p=None, rope=None, k_ld=256, hq=4, n=2, tokens=1, pos=FAKE, table=FAKE, max_pages=4, q_out=5 * FAKE):
    return K.raw_call("kda_kv_append_step", ctypes.byref(p or pool()), None if rope is None else ctypes.byref(rope),
                      FAKE, 2 * FAKE, 3 * FAKE, K.KDA_BF16, 512, k_ld, 256, q_out, hq, n, tokens, pos, table, max_pages,
                      None)


def rope(cos=FAKE, sin=FAKE, num_pos=100, rot=128, inter=0):
    return K.kda_rope(cos, sin, num_pos, rot, inter)


@pytest.mark.parametrize("kw,status", [
    (dict(p=pool(dtype=K.KDA_F32)), K.KDA_ERR_DTYPE), (dict(dt=K.KDA_INT8), K.KDA_ERR_DTYPE), (dict(dt=7), K.KDA_ERR_DTYPE),
    (dict(k=None), K.KDA_ERR_NULL), (dict(v=None), K.KDA_ERR_NULL), (dict(q=None), K.KDA_ERR_NULL),
    (dict(q_out=None), K.KDA_ERR_NULL), (dict(hq=0), K.KDA_ERR_SHAPE), (dict(hq=-1), K.KDA_ERR_SHAPE),
    (dict(k=2 * FAKE + 8), K.KDA_ERR_SHAPE), (dict(k_ld=260), K.KDA_ERR_SHAPE), (dict(k_ld=248), K.KDA_ERR_SHAPE),
    (dict(v_ld=0), K.KDA_ERR_SHAPE), (dict(v_ld=-256), K.KDA_ERR_SHAPE), (dict(q_ld=504), K.KDA_ERR_SHAPE),
    (dict(q_out=FAKE), K.KDA_ERR_SHAPE), (dict(q_out=2 * FAKE + 1024), K.KDA_ERR_SHAPE),
    (dict(table=None), K.KDA_ERR_NULL), (dict(max_pages=0), K.KDA_ERR_SHAPE), (dict(max_pages=1 << 25), K.KDA_ERR_SHAPE),
    (dict(cu=(1, 4)), K.KDA_ERR_SEQ), (dict(cu=(0, 4, 2)), K.KDA_ERR_SEQ), (dict(cu=(0, 257)), K.KDA_ERR_SEQ),
    (dict(start=(250,)), K.KDA_ERR_SEQ), (dict(start=(-1,)), K.KDA_ERR_SEQ), (dict(start=(1 << 62,)), K.KDA_ERR_SEQ),
    (dict(rope=rope(num_pos=9)), K.KDA_ERR_SEQ), (dict(rope=rope(cos=None)), K.KDA_ERR_NULL),
    (dict(rope=rope(rot=8)), K.KDA_ERR_SHAPE), (dict(rope=rope(rot=144)), K.KDA_ERR_SHAPE),
    (dict(rope=rope(rot=40)), K.KDA_ERR_SHAPE), (dict(rope=rope(sin=FAKE + 4)), K.KDA_ERR_SHAPE),
    (dict(rope=rope(inter=2)), K.KDA_ERR_SHAPE), (dict(rope=rope(num_pos=0)), K.KDA_ERR_SHAPE),
    (dict(cu=tuple(range(131))), K.KDA_ERR_WORKSPACE),
    (dict(cu=tuple(range(131)), ws=FAKE + 16, wsb=1 << 20), K.KDA_ERR_WORKSPACE),
    (dict(cu=tuple(range(131)), ws=FAKE, wsb=2047), K.KDA_ERR_WORKSPACE),
    (dict(cu=(0,)), K.KDA_OK), (dict(cu=(0, 0, 0), k=None), K.KDA_OK),
])
def test_append_refusals(kw, status):
    assert append(**kw) == status
    assert (K.kda_last_error() == "") == (status == K.KDA_OK)


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=0), K.KDA_ERR_SHAPE), (dict(tokens=65), K.KDA_ERR_SHAPE), (dict(n=-1), K.KDA_ERR_SHAPE),
    (dict(pos=None), K.KDA_ERR_NULL), (dict(table=None), K.KDA_ERR_NULL), (dict(max_pages=-3), K.KDA_ERR_SHAPE),
    (dict(k_ld=128), K.KDA_ERR_SHAPE), (dict(q_out=FAKE + 512), K.KDA_ERR_SHAPE), (dict(rope=rope(rot=24)), K.KDA_ERR_SHAPE),
    (dict(n=0, pos=None), K.KDA_OK),
])
def test_step_refusals(kw, status):
    assert step(**kw) == status


def read(p=None, k=FAKE, v=2 * FAKE, dt=K.KDA_F32, cu=(0, 10), start=None, table=FAKE, max_pages=4, ws=None, wsb=0):
    return K.raw_call("kda_kv_read", ctypes.byref(p or pool()), k, v, dt, len(cu) - 1, i64(cu),
                      None if start is None else i64(start), table, max_pages, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), K.KDA_ERR_NULL), (dict(v=FAKE + 64), K.KDA_ERR_SHAPE), (dict(dt=K.KDA_INT8), K.KDA_ERR_DTYPE),
    (dict(k=FAKE + 8), K.KDA_ERR_SHAPE), (dict(table=None), K.KDA_ERR_NULL), (dict(cu=(0, 300)), K.KDA_ERR_SEQ),
    (dict(start=(247,)), K.KDA_ERR_SEQ), (dict(cu=tuple(range(140))), K.KDA_ERR_WORKSPACE), (dict(cu=(0,)), K.KDA_OK),
])
def test_read_refusals(kw, status):
    assert read(**kw) == status


def prefill(p=None, q=FAKE, dt=K.KDA_BF16, q_ld=512, o=4 * FAKE, odt=K.KDA_BF16, hq=4, scale=0.1, window=0, sinks=0,
            cu=(0, 10), start=None, table=FAKE, max_pages=4, ws=FAKE, wsb=1 << 30):
    return K.raw_call("kda_attn_prefill", ctypes.byref(p or pool()), q, dt, q_ld, o, odt, hq, scale, window, sinks,
                      len(cu) - 1, i64(cu), None if start is None else i64(start), table, max_pages, ws, wsb, None)


def decode(p=None, q=FAKE, dt=K.KDA_BF16, q_ld=512, o=4 * FAKE, odt=K.KDA_BF16, hq=4, scale=0.1, window=0, sinks=0,
           n=2, tokens=1, pos=FAKE, table=FAKE, max_pages=4, ws=FAKE, wsb=1 << 30):
    return K.raw_call("kda_attn_decode", ctypes.byref(p or pool()), q, dt, q_ld, o, odt, hq, scale, window, sinks,
                      n, tokens, pos, table, max_pages, ws, wsb, None)


SHARED = [
    (dict(q=None), K.KDA_ERR_NULL), (dict(o=None), K.KDA_ERR_NULL), (dict(q=FAKE + 8), K.KDA_ERR_SHAPE),
    (dict(q_ld=508), K.KDA_ERR_SHAPE), (dict(q_ld=504), K.KDA_ERR_SHAPE), (dict(o=FAKE), K.KDA_ERR_SHAPE),
    (dict(dt=K.KDA_INT8), K.KDA_ERR_DTYPE), (dict(odt=5), K.KDA_ERR_DTYPE), (dict(hq=3), K.KDA_ERR_SHAPE),
    (dict(hq=0), K.KDA_ERR_SHAPE), (dict(scale=0.0), K.KDA_ERR_SHAPE), (dict(scale=-1.0), K.KDA_ERR_SHAPE),
    (dict(scale=float("nan")), K.KDA_ERR_SHAPE), (dict(scale=float("inf")), K.KDA_ERR_SHAPE),
    (dict(window=-1), K.KDA_ERR_SHAPE), (dict(sinks=-1), K.KDA_ERR_SHAPE), (dict(table=None), K.KDA_ERR_NULL),
    (dict(max_pages=0), K.KDA_ERR_SHAPE), (dict(ws=None), K.KDA_ERR_WORKSPACE), (dict(ws=FAKE + 32), K.KDA_ERR_WORKSPACE),
    (dict(wsb=0), K.KDA_ERR_WORKSPACE), (dict(p=pool(head_dim=64, num_heads=3)), K.KDA_ERR_SHAPE),
]


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(cu=(0, 300)), K.KDA_ERR_SEQ), (dict(cu=(2, 3)), K.KDA_ERR_SEQ), (dict(start=(-1,)), K.KDA_ERR_SEQ),
    (dict(start=(247,)), K.KDA_ERR_SEQ), (dict(cu=(0,)), K.KDA_OK), (dict(cu=(0, 0)), K.KDA_OK)])
def test_prefill_refusals(kw, status):
    assert prefill(**kw) == status


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(pos=None), K.KDA_ERR_NULL), (dict(tokens=0), K.KDA_ERR_SHAPE), (dict(tokens=65), K.KDA_ERR_SHAPE),
    (dict(n=-1), K.KDA_ERR_SHAPE), (dict(n=0, pos=None), K.KDA_OK)])
def test_decode_refusals(kw, status):
    assert decode(**kw) == status


def test_workspace_bytes():
    p = pool()
    assert K.kda_kv_workspace_bytes(0) == 0 and K.kda_kv_workspace_bytes(128) == 0
    assert K.kda_kv_workspace_bytes(129) >= 16 * 129 and K.kda_kv_workspace_bytes(-1) == -1
    assert K.kda_attn_prefill_workspace_bytes(p, 4, [0, 100]) > 0
    assert K.kda_attn_prefill_workspace_bytes(p, 3, [0, 100]) == 0
    assert K.kda_attn_prefill_workspace_bytes(p, 4, [0, 100], window=-1) == 0
    assert K.kda_attn_decode_workspace_bytes(p, 4, 8, 1, 100) > 0
    for args in ((3, 8, 1, 100), (4, -1, 1, 100), (4, 8, 0, 100), (4, 8, 65, 100), (4, 8, 1, 0)):
        assert K.kda_attn_decode_workspace_bytes(p, *args) == 0, args


def step_only(heads, n, tokens):
    return K.raw_call("kda_kv_append_step", ctypes.byref(pool(num_heads=heads)), None, None, FAKE, 2 * FAKE, K.KDA_BF16,
                      0, heads * 128, heads * 128, None, 0, n, tokens, FAKE, FAKE, 4, None)


@pytest.mark.parametrize("call,kw", [
    (append, dict(p=pool(num_heads=64, page_tokens=32), k_ld=8192, v_ld=8192, q=None, q_out=None, hq=0,
                  cu=(0, 1 << 22), max_pages=1 << 17)),
    (step_only, dict(heads=4, n=1 << 21, tokens=1)),
    (step_only, dict(heads=1, n=3 << 20, tokens=64)),
    (read, dict(p=pool(num_heads=1), cu=(0, 1 << 29), max_pages=1 << 23, v=FAKE << 28)),
    (decode, dict(p=pool(num_heads=32), n=1 << 19, q_ld=4096, hq=32, o=FAKE << 20)),
])
def test_calls_past_the_launch_limit(call, kw):
    """2^24 workgroups and more are refused, before anything is enqueued."""
    assert call(**kw) == K.KDA_ERR_SHAPE and "too much work" in K.kda_last_error()


@pytest.mark.parametrize("call", [prefill, decode])
def test_scale_past_fp32(call):
    assert call(scale=3e38) == K.KDA_ERR_SHAPE


def test_block_order_of_the_oracle_covers_every_slot():
    """The documented element order is a permutation of the block, for both parts and types."""
    from oracle import attention as A
    for d in (64, 128):
        x = np.arange(32 * d).reshape(32, d) % 251 - 125
        for elem in (1, 2):
            for part in (0, 1):
                b = A.block_bytes(x.astype(float), part, elem)
                assert len(b) == 32 * d * elem
                got = np.sort(b.view(np.int8)) if elem == 1 else np.sort(b.view(np.uint16))
                want = x.astype(np.int8).ravel() if elem == 1 else (
                    (A.bf16(x.astype(float)).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16).ravel())
                assert np.array_equal(got, np.sort(want))
