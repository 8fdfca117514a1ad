"""Cross attention without a GPU: the refusals of the calls and the sizes of their scratch."""
import ctypes

import pytest

from test_abi import K, _cache, _paging  # noqa: F401  (K: the fixture)


def test_cross_refusals(K):  # noqa: F811
    L, ref = K.lib(), ctypes.byref
    ok, bad, no = K.KVQ_OK, K.KVQ_ERR_INVALID_ARG, K.KVQ_ERR_UNSUPPORTED

    def cross(cache=None, paging=None, q=256, dtype=1, hq=8, cu=256, total=4, most=4, out=256, ws=256, n=1 << 30):
        return L.kvq_cross_attn(ref(cache or _cache(K)), ref(paging or _paging(K)), q, dtype, hq, cu, total, most, 0.1, out,
                                ws, n, None, None)
    for mode in (K.KVQ_INT4_TOKEN_HEAD, K.KVQ_BF16_CACHE, K.KVQ_FP8_TOKEN_HEAD):
        c = _cache(K, mode=mode)
        assert cross(c, _paging(K, window_per_kv_head=4096)) == no
        assert b"window" in L.kvq_last_error()
        assert cross(c, q=None) == bad and cross(c, out=None) == bad and cross(c, cu=None) == bad
        assert cross(c, q=264) == bad and cross(c, out=264) == bad and cross(c, dtype=3) == no
        assert cross(c, hq=7) == bad and cross(c, hq=18) == no and cross(c, hq=0) == bad
        assert cross(c, total=-1) == bad and cross(c, most=-1) == bad
        assert cross(c, total=0) == ok and cross(c, most=0) == ok and cross(c, paging=_paging(K, batch=0)) == ok
        assert cross(c, most=1, ws=None) == K.KVQ_ERR_WORKSPACE and cross(c, most=1, n=16) == K.KVQ_ERR_WORKSPACE
        assert cross(c, paging=_paging(K, max_blocks=1 << 28)) == no                      # positions past 31 bits
        assert cross(c, paging=_paging(K, block_tables=None)) == bad
        assert cross(_cache(K, mode=mode, num_kv_heads=70000), hq=70000, most=100) == no  # heads past the launch's
    big = _cache(K, mode=K.KVQ_BF16_CACHE, num_blocks=1 << 26, num_kv_heads=2)
    assert cross(big, most=100, hq=2) == no                                               # rows past 31 bits


def test_cross_dense_refusals(K):  # noqa: F811
    L, ref = K.lib(), ctypes.byref
    ok, bad, no = K.KVQ_OK, K.KVQ_ERR_INVALID_ARG, K.KVQ_ERR_UNSUPPORTED
    pg = _paging(K, block_tables=None)

    def dense(k=512, v=512, cukv=256, rows=64, hkv=2, d=128, paging=pg, q=256, dtype=1, hq=8, cu=256, total=4, most=4,
              out=256, ws=256, n=1 << 30):
        return L.kvq_cross_dense_attn(k, v, cukv, rows, hkv, d, None if paging is None else ref(paging), q, dtype, hq, cu,
                                      total, most, 0.1, out, ws, n, None, None)
    assert dense(paging=None) == bad and dense(paging=_paging(K)) == bad
    assert dense(paging=_paging(K, block_tables=None, window_per_kv_head=4096)) == no
    for name in ("k", "v", "cukv", "q", "cu", "out"):
        assert dense(**{name: None}) == bad, name
    assert dense(k=520) == bad and dense(v=520) == bad and dense(q=264) == bad and dense(out=264) == bad
    assert dense(d=96) == no and dense(hkv=0) == bad and dense(rows=-1) == bad and dense(rows=0) == bad
    assert dense(hq=7) == bad and dense(hq=18) == no and dense(dtype=2) == no
    assert dense(total=-1) == bad and dense(most=-1) == bad
    assert dense(rows=2 ** 31 - 1) == no and dense(hkv=70000, hq=70000) == no
    assert dense(paging=_paging(K, block_tables=None, batch=70000)) == no
    assert dense(paging=_paging(K, block_tables=None, seq_lens=None)) == bad
    assert dense(rows=100000, ws=None) == K.KVQ_ERR_WORKSPACE and dense(rows=100000, ws=264) == bad
    assert dense(total=0) == ok and dense(most=0) == ok and dense(paging=_paging(K, block_tables=None, batch=0)) == ok


@pytest.mark.parametrize("mode", ["INT4_TOKEN_HEAD", "BF16_CACHE"])
def test_cross_scratch_does_not_go_by_the_type(K, mode):  # noqa: F811
    """One size serves bf16 and fp32 queries; few queries over long sources need records, many over short ones none."""
    L, ref = K.lib(), ctypes.byref
    n = ctypes.c_size_t(0)
    c = _cache(K, mode=getattr(K, "KVQ_" + mode))

    def size(most, blocks=4, batch=2):
        assert L.kvq_cross_workspace_size(ref(c), ref(_paging(K, max_blocks=blocks, batch=batch)), 8, most,
                                          ref(n)) == K.KVQ_OK
        return n.value
    assert size(0) == 0 and size(1) > 0
    assert size(40, blocks=4096, batch=1) >= 2 * 2 * 128 * 130 * 4     # two parts of two heads' tile, at least
    assert size(4096, blocks=4, batch=64) == 0                         # CTAs enough without parts
    assert L.kvq_cross_workspace_size(ref(c), ref(_paging(K, window_per_kv_head=4096)), 8, 4, ref(n)) == K.KVQ_ERR_UNSUPPORTED
    assert L.kvq_cross_workspace_size(ref(c), ref(_paging(K)), 8, -1, ref(n)) == K.KVQ_ERR_INVALID_ARG
    assert L.kvq_cross_workspace_size(ref(c), ref(_paging(K)), 7, 4, ref(n)) == K.KVQ_ERR_INVALID_ARG
    assert L.kvq_cross_workspace_size(ref(c), ref(_paging(K)), 8, 4, None) == K.KVQ_ERR_INVALID_ARG
    assert L.kvq_cross_dense_workspace_size(64, 2, 128, 2, 8, 4, None) == K.KVQ_ERR_INVALID_ARG
    assert L.kvq_cross_dense_workspace_size(64, 2, 80, 2, 8, 4, ref(n)) == K.KVQ_ERR_UNSUPPORTED
