"""Tree attention past what one launch can count (2^32 threads): refused before anything is enqueued."""
import ctypes

import pytest

import hybrid_prefix_cache_amd as K

F = 1 << 20  # stands for a device pointer


@pytest.mark.parametrize("dtype,cache,n,heads,per", [
    (K.KDA_BF16, K.KDA_INT8, 128, 1 << 16, 1),   # 64 rows a head: 2^23 workgroups of 512 threads
    (K.KDA_BF16, K.KDA_BF16, 256, 1 << 15, 2),   # 128 rows: the same
    (K.KDA_F32, K.KDA_INT8, 256, 1 << 15, 2),
    (K.KDA_BF16, K.KDA_BF16, 256, 1 << 16, 1),   # 64 rows: 2^24 of 256
    (K.KDA_F32, K.KDA_INT8, 256, 1 << 16, 1),
])
def test_too_many_workgroups(dtype, cache, n, heads, per):
    d, hq = 64, heads * per
    pool = K.kda_kv_pool(F, heads * K.kda_kv_head_bytes(d, 32, cache), 8, heads, d, 32, cache)
    assert K.kda_kv_pool_check(pool) == K.KDA_OK
    status = K.raw_call("kda_attn_tree", ctypes.byref(pool), F, dtype, hq * d, 1 << 44, K.KDA_BF16, hq, ctypes.c_float(0.1), 0, 0,
                        n, 64, F, F, F, 4, F, ctypes.c_size_t(1 << 40), None)
    assert status == K.KDA_ERR_SHAPE and "too much work" in K.kda_last_error()
