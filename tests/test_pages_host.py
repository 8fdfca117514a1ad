"""Host-side checks of the page calls: sizes and refusals, before anything is launched."""
import copy
import ctypes
import pickle

import pytest
import torch

from test_abi import K, _cache, _paging  # noqa: F401


def arr(K, *cs):  # noqa: F811
    return (K.KvqCache * len(cs))(*cs)


def test_workspace_sizes(K):  # noqa: F811
    L, ref, n = K.lib(), ctypes.byref, ctypes.c_size_t(0)
    cs = arr(K, _cache(K), _cache(K, mode=K.KVQ_BF16_CACHE, head_dim=64))
    assert L.kvq_copy_workspace_size(cs, 2, 2048, 0, ref(n)) == K.KVQ_OK and n.value == 0
    assert L.kvq_copy_workspace_size(cs, 2, 2049, 0, ref(n)) == K.KVQ_OK and n.value >= 40
    assert L.kvq_copy_workspace_size(cs, 2, 2049, 1, ref(n)) == K.KVQ_OK and n.value >= 80
    assert L.kvq_fork_workspace_size(cs, 2, ref(_paging(K)), ref(_paging(K, batch=7)), ref(n)) == K.KVQ_OK and n.value > 0
    assert L.kvq_fork_workspace_size(cs, 2, None, ref(_paging(K, batch=7)), ref(n)) == K.KVQ_OK
    assert L.kvq_compact_workspace_size(cs, 2, ref(_paging(K)), ref(n)) == K.KVQ_OK and n.value > 0


def test_cache_lists(K):  # noqa: F811
    L, ref, n = K.lib(), ctypes.byref, ctypes.c_size_t(0)
    for kw in (dict(num_blocks=11), dict(num_kv_heads=1), dict(block_size=32)):
        assert L.kvq_copy_workspace_size(arr(K, _cache(K), _cache(K, **kw)), 2, 5, 0, ref(n)) == K.KVQ_ERR_INVALID_ARG
    assert L.kvq_copy_workspace_size(arr(K, _cache(K), _cache(K, mode=9)), 2, 5, 0, ref(n)) == K.KVQ_ERR_UNSUPPORTED
    assert L.kvq_copy_workspace_size(arr(K, _cache(K)), 0, 5, 0, ref(n)) == K.KVQ_ERR_INVALID_ARG
    assert L.kvq_copy_workspace_size(None, 1, 5, 0, ref(n)) == K.KVQ_ERR_INVALID_ARG
    assert L.kvq_copy_workspace_size(arr(K, *[_cache(K)] * 129), 129, 5, 0, ref(n)) == K.KVQ_ERR_UNSUPPORTED
    big = _cache(K, num_blocks=0x40000000, num_kv_heads=4)
    assert L.kvq_copy_workspace_size(arr(K, big), 1, 5, 0, ref(n)) == K.KVQ_ERR_UNSUPPORTED


def test_copy_refusals(K):  # noqa: F811
    L, cs = K.lib(), arr(K, _cache(K))
    assert L.kvq_copy_pages(cs, 1, 4096, None, 3, 0, 4096, 1 << 20, None, None) == K.KVQ_ERR_INVALID_ARG
    assert L.kvq_copy_pages(cs, 1, 4096, 8192, -1, 0, 4096, 1 << 20, None, None) == K.KVQ_ERR_INVALID_ARG
    assert L.kvq_copy_pages(cs, 1, 4096, 8192, 3000, 0, 4096, 16, None, None) == K.KVQ_ERR_WORKSPACE
    assert L.kvq_copy_pages(cs, 1, 4096, 8192, 3000, 0, None, 0, None, None) == K.KVQ_ERR_WORKSPACE
    assert L.kvq_copy_pages(cs, 1, 4096, 8192, 3000, 0, 4100, 1 << 20, None, None) == K.KVQ_ERR_INVALID_ARG
    assert L.kvq_copy_pages(cs, 1, None, None, 0, 0, None, 0, None, None) == K.KVQ_OK   # nothing to do


def _fork(K, cs, old, new, parents=1 << 20, keep=None, more=None, pins=None, refs=2 << 20, ws=3 << 20, size=1 << 20):  # noqa: F811
    ref = ctypes.byref
    return K.lib().kvq_fork(cs, len(cs), None if old is None else ref(old), parents, keep, more, pins,
                            None if new is None else ref(new), refs, ws, size, None, None)


def test_fork_refusals(K):  # noqa: F811
    cs = arr(K, _cache(K))
    old = _paging(K)                                                   # tables and lengths at 4096
    new = lambda **kw: _paging(K, **{**dict(block_tables=1 << 16, seq_lens=1 << 17), **kw})  # noqa: E731
    bad = K.KVQ_ERR_INVALID_ARG
    assert _fork(K, cs, old, None) == bad
    assert _fork(K, cs, old, new(batch=0)) == bad
    assert _fork(K, cs, old, new(max_blocks=5)) == bad
    assert _fork(K, cs, old, new(block_tables=None, block_tables_headwise=1 << 16)) == bad
    assert _fork(K, cs, old, new(), parents=None) == bad
    assert _fork(K, cs, old, new(), refs=None) == bad
    assert _fork(K, cs, old, new(), ws=(3 << 20) + 8) == bad
    assert _fork(K, cs, old, new(), size=64) == K.KVQ_ERR_WORKSPACE
    for kw in (dict(block_tables=4096), dict(block_tables=4096 + 16), dict(seq_lens=4096), dict(block_tables=1 << 17),
               dict(seq_lens=1 << 20), dict(seq_lens=(2 << 20) + 4)):
        assert _fork(K, cs, old, new(**kw)) == bad, kw
        assert b"overlap" in K.lib().kvq_last_error()
    assert _fork(K, cs, None, new(batch=65535, max_blocks=40000)) == K.KVQ_ERR_UNSUPPORTED
    assert _fork(K, cs, old, new(), pins=2 << 20) == bad
    assert _fork(K, cs, old, new(), more=2 << 20) == bad


def test_compact_refusals(K):  # noqa: F811
    cs, p, ref = arr(K, _cache(K)), _paging(K, seq_lens=1 << 14), ctypes.byref
    L, bad = K.lib(), K.KVQ_ERR_INVALID_ARG
    ok = dict(pins=None, table=4096, map=1 << 16, refs=2 << 16, used=3 << 16, ws=4 << 16, size=1 << 20)

    def call(paging=p, **kw):
        a = {**ok, **kw}
        return L.kvq_compact(cs, 1, ref(paging), a["pins"], a["table"], a["map"], a["refs"], a["used"], a["ws"], a["size"],
                             None, None)
    for kw in (dict(table=None), dict(map=None), dict(refs=None), dict(used=None), dict(table=4096 + 4), dict(map=4096),
               dict(refs=1 << 16), dict(used=(2 << 16) + 4), dict(pins=1 << 16), dict(refs=1 << 14), dict(ws=(4 << 16) + 4)):
        assert call(**kw) == bad, kw
    assert call(size=64) == K.KVQ_ERR_WORKSPACE
    assert call(paging=_paging(K, batch=0)) == bad
    assert call(paging=_paging(K, block_tables=None)) == bad


def test_python_refusals(K):  # noqa: F811
    c = K.PagedCache(K.KVQ_BF16_CACHE, 8, 2, 16, 64, device="cpu")
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        K.kvq_copy_pages([], i(1), i(1))
    with pytest.raises(ValueError):
        K.kvq_copy_pages([c], i(2), i(1))
    with pytest.raises(ValueError):                                   # a row too few in the table
        K.kvq_fork([c], K.Paging(i(3), block_tables=i(2, 4)), i(3), out=K.Paging(i(3), block_tables=i(3, 4)))
    with pytest.raises(ValueError):
        K.kvq_fork([c], None, i(3))
    with pytest.raises(ValueError):
        K.kvq_compact([c], K.Paging(i(3)))
    # a handle follows its pools: a new tensor gives a new struct
    old = K.PagedCache(K.KVQ_BF16_CACHE, 8, 2, 16, 64, device="cpu")
    old._build = lambda: K.KvqCache(old.k_pages.data_ptr(), old.v_pages.data_ptr())
    first = old.struct()
    assert old.struct() is first
    old.k_pages = torch.zeros_like(old.k_pages)
    assert old.struct().k_pages == old.k_pages.data_ptr()


def test_handles_copy_and_pickle(K):  # noqa: F811
    c = K.PagedCache(K.KVQ_BF16_CACHE, 3, 2, 16, 64, device="cpu")
    c._build = lambda: K.KvqCache(c.k_pages.data_ptr())
    c.struct()
    del c.__dict__["_build"]
    c.k_pages[1] = 5
    for d in (copy.copy(c), copy.deepcopy(c), pickle.loads(pickle.dumps(c))):
        assert d.num_blocks == 3 and torch.equal(d.k_pages, c.k_pages) and d._struct is None
    p = copy.deepcopy(K.Paging(torch.zeros(2, dtype=torch.int32), block_tables=torch.zeros((2, 3), dtype=torch.int32)))
    assert p.max_blocks == 3 and p.block_tables.shape == (2, 3)
