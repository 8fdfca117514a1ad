"""Host-side checks of the 16-bit cache mode: row size, refusals, exports."""
import ctypes

import pytest

from test_abi import K, _cache, _paging  # noqa: F401


def test_row_bytes_and_workspace(K):  # noqa: F811
    assert K.kvq_row_bytes(K.KVQ_BF16_CACHE, 128) == 256 and K.kvq_row_bytes(K.KVQ_BF16_CACHE, 64) == 128
    assert K.kvq_row_bytes(K.KVQ_BF16_CACHE, 96) == 0
    n, s = ctypes.c_size_t(0), ctypes.c_int32(0)
    L, ref = K.lib(), ctypes.byref
    c = _cache(K, mode=K.KVQ_BF16_CACHE)
    assert L.kvq_decode_workspace_size(ref(c), ref(_paging(K)), 8, 0, ref(n), ref(s)) == K.KVQ_OK
    assert n.value > 0 and s.value >= 1


def test_refusals(K):  # noqa: F811
    L, ref = K.lib(), ctypes.byref
    signs = _cache(K, mode=K.KVQ_BF16_CACHE, rht_signs=4096)
    c = _cache(K, mode=K.KVQ_BF16_CACHE)
    assert L.kvq_write(ref(signs), ref(_paging(K)), 16, 16, 1, 16, 1, None, None) == K.KVQ_ERR_INVALID_ARG
    assert b"RHT" in L.kvq_last_error()
    assert L.kvq_write(ref(_cache(K, mode=7)), ref(_paging(K)), 16, 16, 1, 16, 1, None, None) == K.KVQ_ERR_UNSUPPORTED
    assert L.kvq_prefill_attn(ref(c), ref(_paging(K)), 256, 1, 8, 256, 4, 4, 0.1, 256, None, None) == K.KVQ_ERR_UNSUPPORTED
    assert b"kvq_prefill_dense_attn" in L.kvq_last_error()
    assert L.kvq_decode_attn(ref(c), ref(_paging(K)), 256, 1, 8, 0.1, 256, 256, 16, 0, None, None) == K.KVQ_ERR_WORKSPACE
    assert L.kvq_decode_attn(ref(c), ref(_paging(K)), 256, 1, 18, 0.1, 256, 256, 1 << 30, 0, None, None) == K.KVQ_ERR_UNSUPPORTED
    big = _cache(K, mode=K.KVQ_BF16_CACHE, num_blocks=0x7FFFFFFF, num_kv_heads=2)
    assert L.kvq_decode_attn(ref(big), ref(_paging(K)), 256, 1, 8, 0.1, 256, 256, 1 << 30, 0, None, None) == K.KVQ_ERR_UNSUPPORTED
    wide = _paging(K, max_blocks=0x7FFFFFF)
    c64 = _cache(K, mode=K.KVQ_BF16_CACHE, block_size=64)
    assert L.kvq_decode_attn(ref(c64), ref(wide), 256, 1, 8, 0.1, 256, 256, 1 << 30, 0, None, None) == K.KVQ_ERR_UNSUPPORTED
    many = _paging(K, batch=60000, max_blocks=20000)
    assert L.kvq_decode_attn(ref(c), ref(many), 256, 1, 8, 0.1, 256, 256, 1 << 40, 0, None, None) == K.KVQ_ERR_UNSUPPORTED
    assert L.kvq_write_decode_attn(ref(c), ref(_paging(K)), None, 4096, 1, 4096, 2, 256, 1, 8, 0.1, 256, 256, 1 << 30, 0,
                                   None, None) == K.KVQ_ERR_INVALID_ARG


def test_python_cache_shapes(K):  # noqa: F811
    c = K.PagedCache(K.KVQ_BF16_CACHE, 3, 2, 16, 64, device="cpu")
    assert tuple(c.k_pages.shape) == (3, 2, 16, 128)
    with pytest.raises(ValueError):
        K.PagedCache(K.KVQ_BF16_CACHE, 3, 2, 16, 80, device="cpu")


def test_a_step_of_more_tokens_than_one_write_takes(K):  # noqa: F811
    """The bound of kvq_write holds for the write inside a 16-bit step."""
    L, ref = K.lib(), ctypes.byref
    c = _cache(K, mode=K.KVQ_BF16_CACHE, num_kv_heads=8)
    many = 0x7FFFFFFF
    assert L.kvq_write(ref(c), ref(_paging(K)), 4096, 4096, 1, 4096, many, None, None) == K.KVQ_ERR_UNSUPPORTED
    assert L.kvq_write_decode_attn(ref(c), ref(_paging(K)), 4096, 4096, 1, 4096, many, 256, 1, 8, 0.1, 256, 256, 1 << 40, 0,
                                   None, None) == K.KVQ_ERR_UNSUPPORTED
    assert b"too many tokens" in L.kvq_last_error()
