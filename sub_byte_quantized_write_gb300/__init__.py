"""Python binding of libkvq: a paged KV cache in dynamic low-bit form on GB300.

Argument marshalling only: tensors are checked for device, dtype and
contiguity, turned into raw pointers and handed to the C ABI declared in
``include/kvq.h``.  Every step of the write and attention paths runs in the
library's CUDA kernels; there is no fallback.  If ``libkvq.so`` has not been
built, importing this package raises ImportError.

Names mirror the C calls: ``kvq_write``, ``kvq_gather``, ``kvq_prefill_dense_attn``, ``kvq_decode_attn``,
``kvq_write_decode_attn``,
``kvq_decode_attn_noalloc``, ``kvq_prefill_attn``, ``kvq_decode_workspace_size``,
``kvq_row_bytes``, ``kvq_copy_pages``, ``kvq_fork``, ``kvq_compact`` and their ``_workspace_size``.

A call runs on the device of its cache, on `stream` if one is given, else on
that device's current stream; what it allocates belongs to that stream.
"""
from __future__ import annotations

import ctypes
import itertools
import os
from typing import Optional, Sequence, Tuple, Union

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# KVQ_BOUNDS_CHECK=1 loads the debug library: the same kernels with device-side
# bounds checks on their computed indices (a failure sets KVQ_DEVERR_BOUNDS).
BOUNDS_CHECK = os.environ.get("KVQ_BOUNDS_CHECK", "0") == "1"
LIB_NAME = "libkvq_debug.so" if BOUNDS_CHECK else "libkvq.so"
LIB_PATH = os.path.join(_HERE, LIB_NAME)

if not os.path.exists(LIB_PATH):
    raise ImportError("%s is not built: run `python sub_byte_quantized_write_gb300/build_lib.py` "
                      "(or __graft_entry__.build()) first" % LIB_NAME)

_lib = ctypes.CDLL(LIB_PATH)

KVQ_OK, KVQ_ERR_INVALID_ARG, KVQ_ERR_UNSUPPORTED, KVQ_ERR_CUDA, KVQ_ERR_WORKSPACE = 0, 1, 2, 3, 4
KVQ_INT4_TOKEN_HEAD, KVQ_INT2_TOKEN_HEAD, KVQ_INT8_CHANNEL, KVQ_INT4_STEGO = 0, 1, 2, 3
KVQ_INT8_TOKEN_HEAD, KVQ_FP8_TOKEN_HEAD, KVQ_BF16_CACHE = 4, 5, 6
KVQ_F32, KVQ_BF16 = 0, 1
KVQ_DEVERR_BLOCK_RANGE, KVQ_DEVERR_TABLE_RANGE, KVQ_DEVERR_SEQ_LEN, KVQ_DEVERR_TIMEOUT = 1, 2, 4, 8
KVQ_DEVERR_BOUNDS = 16  # debug library only
KVQ_DEVERR_ROW_RANGE, KVQ_DEVERR_NO_PAGES, KVQ_DEVERR_PAGE_CONFLICT = 32, 64, 128


class KvqCache(ctypes.Structure):
    _fields_ = [("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p),
                ("num_blocks", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("mode", ctypes.c_int32), ("rht_signs", ctypes.c_void_p),
                ("ch_amax", ctypes.c_void_p), ("ch_amax_ready", ctypes.c_void_p)]


class KvqPaging(ctypes.Structure):
    _fields_ = [("block_tables", ctypes.c_void_p), ("block_tables_headwise", ctypes.c_void_p),
                ("max_blocks", ctypes.c_int32), ("batch", ctypes.c_int32),
                ("seq_lens", ctypes.c_void_p), ("window_per_kv_head", ctypes.c_void_p),
                ("sink_size", ctypes.c_int32)]


_P, _I = ctypes.c_void_p, ctypes.c_int32
_CP, _PP = ctypes.POINTER(KvqCache), ctypes.POINTER(KvqPaging)
_lib.kvq_row_bytes.argtypes, _lib.kvq_row_bytes.restype = [_I, _I], _I
_lib.kvq_abi_version.argtypes, _lib.kvq_abi_version.restype = [], _I
_lib.kvq_status_string.argtypes, _lib.kvq_status_string.restype = [_I], ctypes.c_char_p
_lib.kvq_last_error.argtypes, _lib.kvq_last_error.restype = [], ctypes.c_char_p
_lib.kvq_write.argtypes = [_CP, _PP, _P, _P, _I, _P, _I, _P, _P]
_lib.kvq_write.restype = _I
_lib.kvq_gather.argtypes = [_CP, _PP, _P, _I, _P, _P, _I, _P, _P]
_lib.kvq_gather.restype = _I
_lib.kvq_gather_chunk.argtypes = [_CP, _PP, _P, _I, _P, _P, _I, _P, _P, _P, _I, _P, _P]
_lib.kvq_gather_chunk.restype = _I
_lib.kvq_decode_workspace_size.argtypes = [_CP, _PP, _I, _I, ctypes.POINTER(ctypes.c_size_t),
                                           ctypes.POINTER(ctypes.c_int32)]
_lib.kvq_decode_workspace_size.restype = _I
_lib.kvq_decode_attn.argtypes = [_CP, _PP, _P, _I, _I, ctypes.c_float, _P, _P, ctypes.c_size_t, _I, _P, _P]
_lib.kvq_decode_attn.restype = _I
_lib.kvq_write_decode_attn.argtypes = [_CP, _PP, _P, _P, _I, _P, _I, _P, _I, _I, ctypes.c_float, _P, _P,
                                       ctypes.c_size_t, _I, _P, _P]
_lib.kvq_write_decode_attn.restype = _I
_lib.kvq_decode_attn_noalloc.argtypes = [_CP, _PP, _P, _I, _I, ctypes.c_float, _P, _I, _P, _P]
_lib.kvq_decode_attn_noalloc.restype = _I
_lib.kvq_prefill_attn.argtypes = [_CP, _PP, _P, _I, _I, _P, _I, _I, ctypes.c_float, _P, _P, _P]
_lib.kvq_prefill_attn.restype = _I
_lib.kvq_prefill_dense_attn.argtypes = [_P, _P, _P, _I, _I, _I, _PP, _P, _I, _I, _P, _I, _I, ctypes.c_float, _P, _P,
                                        _P]
_lib.kvq_prefill_dense_attn.restype = _I
_SZ = ctypes.POINTER(ctypes.c_size_t)
_lib.kvq_copy_workspace_size.argtypes = [_CP, _I, _I, _I, _SZ]
_lib.kvq_copy_workspace_size.restype = _I
_lib.kvq_copy_pages.argtypes = [_CP, _I, _P, _P, _I, _I, _P, ctypes.c_size_t, _P, _P]
_lib.kvq_copy_pages.restype = _I
_lib.kvq_fork_workspace_size.argtypes = [_CP, _I, _PP, _PP, _SZ]
_lib.kvq_fork_workspace_size.restype = _I
_lib.kvq_fork.argtypes = [_CP, _I, _PP, _P, _P, _P, _P, _PP, _P, _P, ctypes.c_size_t, _P, _P]
_lib.kvq_fork.restype = _I
_lib.kvq_compact_workspace_size.argtypes = [_CP, _I, _PP, _SZ]
_lib.kvq_compact_workspace_size.restype = _I
_lib.kvq_compact.argtypes = [_CP, _I, _PP, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P, _P]
_lib.kvq_compact.restype = _I


class KvqError(RuntimeError):
    def __init__(self, status: int):
        self.status = status
        super().__init__("%s: %s" % (_lib.kvq_status_string(status).decode(), _lib.kvq_last_error().decode()))


def _check(status: int):
    if status != KVQ_OK:
        raise KvqError(status)


def lib() -> ctypes.CDLL:
    return _lib


def kvq_row_bytes(mode: int, head_dim: int) -> int:
    return _lib.kvq_row_bytes(mode, head_dim)


def _dev_ptr(t: Optional[torch.Tensor], dtype=None, name="tensor", dev: Optional[int] = None):
    """Device pointer of a contiguous tensor, on device `dev` where that is given."""
    if t is None:
        return None
    if dev is not None:
        if t.get_device() != dev:
            raise ValueError("%s must be on the cache's device" % name)
    elif not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


# The current stream of a device as a raw cudaStream_t; building a torch.cuda.Stream for it costs more than the
# rest of a call's checks together.
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _stream_ptr(stream) -> Optional[int]:
    if stream is None:
        return _current_raw_stream(torch.cuda.current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _as_stream(stream, device):
    """A torch stream object for `stream` (a torch stream or a raw cudaStream_t)."""
    return stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream), device=device)


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """torch.empty for a call on `stream`: the memory belongs to the stream that uses it, so that the allocator
    neither hands out what other work still holds nor takes it back too early."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(_as_stream(stream, device)):
        return torch.empty(shape, dtype=dtype, device=device)


def _copy(to: torch.Tensor, t: torch.Tensor, stream) -> None:
    """to = t, on `stream`."""
    if stream is None:
        to.copy_(t)
    else:
        with torch.cuda.stream(_as_stream(stream, t.device)):
            to.copy_(t)


def _run(device: torch.device, stream, fn, *args) -> None:
    """fn(*args, stream) with `device` current."""
    index = device.index
    if index == torch.cuda.current_device():
        status = fn(*args, _current_raw_stream(index) if stream is None else _stream_ptr(stream))
    else:
        with torch.cuda.device(device):
            status = fn(*args, _stream_ptr(stream))
    if status != KVQ_OK:
        raise KvqError(status)


def _qdtype(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return KVQ_F32
    if t.dtype == torch.bfloat16:
        return KVQ_BF16
    raise ValueError("q/k/v must be float32 or bfloat16")


class _Handle:
    """Holds tensors and, in `_struct`, the C struct made of them; setting an attribute drops the struct, and copies
    and pickles leave it out."""

    def __setattr__(self, name, value):
        self.__dict__[name] = value
        self.__dict__["_struct"] = None

    def __getstate__(self):
        return {k: v for k, v in self.__dict__.items() if k not in ("_struct", "_group")}

    def __setstate__(self, state):
        self.__dict__.update(state, _struct=None)


_serial = itertools.count()


class _Kept:
    """What a handle's C struct was made of, the struct, a number of its own, and that of the paging state that a
    cache was last checked against."""
    __slots__ = ("tensors", "pointers", "shapes", "struct", "devices", "serial", "paired")

    def __init__(self, tensors, struct, by_shape):
        self.tensors, self.struct, self.serial = tensors, struct, next(_serial)
        self.pointers = [t.data_ptr() for t in tensors]
        self.shapes = [t.shape for t in tensors] if by_shape else None
        self.devices = {t.device for t in tensors}
        self.paired = None


def _kept_struct(handle, tensors, by_shape):
    """A handle's C struct, rebuilt (with its checks) unless the tensors it was made of are where they were and, where
    the struct takes numbers from their shapes (by_shape), as large."""
    kept = handle._struct
    if (kept is None or [t.data_ptr() for t in kept.tensors] != kept.pointers
            or by_shape and [t.shape for t in kept.tensors] != kept.shapes):
        kept = handle.__dict__["_struct"] = _Kept([t for t in tensors(handle) if t is not None], handle._build(), by_shape)
    return kept.struct


def _cache_tensors(c):
    return c.k_pages, c.v_pages, c.rht_signs, c.ch_amax, c.ch_amax_ready


def _paging_tensors(p):
    return p.seq_lens, p.block_tables, p.block_tables_headwise, p.window_per_kv_head


class PagedCache(_Handle):
    """One layer's paged cache: uint8 K and V pools of shape
    [num_blocks, num_kv_heads, block_size, row_bytes] (allocated here, as
    torch.uint8, unless given), the RHT sign vector and, for INT8, the
    per-channel amax state."""

    def __init__(self, mode: int, num_blocks: int, num_kv_heads: int, block_size: int, head_dim: int,
                 rht_signs: Optional[torch.Tensor] = None, device="cuda", k_pages=None, v_pages=None,
                 ch_amax=None, ch_amax_ready=None):
        row_bytes = kvq_row_bytes(mode, head_dim)
        if row_bytes == 0:
            raise ValueError("unsupported mode/head_dim")
        shape = (num_blocks, num_kv_heads, block_size, row_bytes)
        if k_pages is None:
            k_pages = torch.zeros(shape, dtype=torch.uint8, device=device)
        if v_pages is None:
            v_pages = torch.zeros(shape, dtype=torch.uint8, device=device)
        if mode != KVQ_INT8_CHANNEL:
            ch_amax = ch_amax_ready = None
        else:
            if ch_amax is None:
                ch_amax = torch.zeros((2, num_kv_heads, head_dim), dtype=torch.float32, device=device)
            if ch_amax_ready is None:
                ch_amax_ready = torch.zeros(1, dtype=torch.int32, device=device)
        self.__dict__.update(mode=mode, num_blocks=num_blocks, num_kv_heads=num_kv_heads, block_size=block_size,
                             head_dim=head_dim, k_pages=k_pages, v_pages=v_pages,
                             rht_signs=rht_signs, ch_amax=ch_amax, ch_amax_ready=ch_amax_ready, _struct=None)

    @property
    def row_bytes(self) -> int:
        return kvq_row_bytes(self.mode, self.head_dim)

    def struct(self) -> KvqCache:
        """The C struct: built once, and again when an attribute was set or a tensor's memory changed."""
        return _kept_struct(self, _cache_tensors, False)

    def _build(self) -> KvqCache:
        need = self.num_blocks * self.num_kv_heads * self.block_size * self.row_bytes
        if self.k_pages.numel() < need or self.v_pages.numel() < need:
            raise ValueError("k_pages / v_pages hold fewer than num_blocks blocks")
        for t, name, least in ((self.rht_signs, "rht_signs", self.head_dim),
                               (self.ch_amax, "ch_amax", 2 * self.num_kv_heads * self.head_dim),
                               (self.ch_amax_ready, "ch_amax_ready", 1)):
            if t is not None and 0 < t.numel() < least:  # (none at all is NULL, which the library judges)
                raise ValueError("%s must have %d elements, got %d" % (name, least, t.numel()))
        return KvqCache(_dev_ptr(self.k_pages, torch.uint8, "k_pages"), _dev_ptr(self.v_pages, torch.uint8, "v_pages"),
                        self.num_blocks, self.num_kv_heads, self.block_size, self.head_dim, self.mode,
                        _dev_ptr(self.rht_signs, torch.int8, "rht_signs"),
                        _dev_ptr(self.ch_amax, torch.float32, "ch_amax"),
                        _dev_ptr(self.ch_amax_ready, torch.int32, "ch_amax_ready"))


class Paging(_Handle):
    """Block table (uniform [batch, max_blocks] or head-wise
    [batch * num_kv_heads, max_blocks], int32, -1 = evicted), seq_lens [batch]
    and the optional per-kv-head sliding window plus sink size.  max_blocks is
    the width of the table that is set."""

    def __init__(self, seq_lens: torch.Tensor, block_tables: Optional[torch.Tensor] = None,
                 block_tables_headwise: Optional[torch.Tensor] = None,
                 window_per_kv_head: Optional[torch.Tensor] = None, sink_size: int = 0):
        self.__dict__.update(seq_lens=seq_lens, block_tables=block_tables,
                             block_tables_headwise=block_tables_headwise, window_per_kv_head=window_per_kv_head,
                             sink_size=int(sink_size), _struct=None)

    @property
    def max_blocks(self) -> int:
        t = self.block_tables if self.block_tables is not None else self.block_tables_headwise
        return 0 if t is None else int(t.shape[-1])

    def struct(self) -> KvqPaging:
        """The C struct: built once, and again when an attribute was set or a tensor's memory or shape changed."""
        return _kept_struct(self, _paging_tensors, True)

    def _build(self) -> KvqPaging:
        for t in (self.block_tables, self.block_tables_headwise):
            if t is None:
                continue
            if t.dim() != 2:
                raise ValueError("a block table has two dimensions, got %d" % t.dim())
            if t.shape[0] < self.seq_lens.shape[0]:
                raise ValueError("the block table has fewer rows than seq_lens")
        return KvqPaging(_dev_ptr(self.block_tables, torch.int32, "block_tables"),
                         _dev_ptr(self.block_tables_headwise, torch.int32, "block_tables_headwise"),
                         self.max_blocks, int(self.seq_lens.shape[0]),
                         _dev_ptr(self.seq_lens, torch.int32, "seq_lens"),
                         _dev_ptr(self.window_per_kv_head, torch.int32, "window_per_kv_head"),
                         self.sink_size)


def _structs(cache: PagedCache, paging: Paging) -> Tuple[KvqCache, KvqPaging]:
    """The C structs of a cache and of a paging state that fits it."""
    cs, ps = cache.struct(), paging.struct()
    kept, other = cache._struct, paging._struct
    if kept.paired != other.serial:
        Hkv, t, w = cache.num_kv_heads, paging.block_tables_headwise, paging.window_per_kv_head
        if len(kept.devices) != 1 or other.devices != kept.devices:
            raise ValueError("the cache and the paging state must be on one device")
        if t is not None and t.shape[0] < ps.batch * Hkv:
            raise ValueError("a head-wise block table needs batch * num_kv_heads = %d rows" % (ps.batch * Hkv))
        if w is not None and w.numel() < Hkv:
            raise ValueError("window_per_kv_head must have %d elements, got %d" % (Hkv, w.numel()))
        kept.paired = other.serial
    return cs, ps


# Sizes.  Buffers may be larger than the call needs (those of a captured step are sized for its largest batch), and a
# token's rows may come flat: what is refused is what would be read or written past its end, or at another stride.

def _check_rows(cache: PagedCache, t: torch.Tensor, name: str) -> None:
    """t is [tokens, num_kv_heads, head_dim], or [tokens, num_kv_heads * head_dim]."""
    if t.dim() == 0 or t.numel() != t.shape[0] * cache.num_kv_heads * cache.head_dim:
        raise ValueError("%s must be [tokens, %d, %d], got %s" % (name, cache.num_kv_heads, cache.head_dim,
                                                                  tuple(t.shape)))


def _check_cu(cu: Optional[torch.Tensor], batch: int, name: str) -> None:
    if cu is not None and cu.numel() <= batch:
        raise ValueError("%s must have batch + 1 = %d elements, got %d" % (name, batch + 1, cu.numel()))


def _check_q(cache: PagedCache, ps: KvqPaging, q: torch.Tensor, out: Optional[torch.Tensor]) -> None:
    """q is [batch or more, num_q_heads, head_dim]; out, if given, holds the batch's rows."""
    shape = q.shape
    if len(shape) != 3 or shape[0] < ps.batch or shape[2] != cache.head_dim:
        raise ValueError("q must be [%d, num_q_heads, %d], got %s" % (ps.batch, cache.head_dim, tuple(shape)))
    if out is not None and out.numel() < ps.batch * shape[1] * shape[2]:
        raise ValueError("out must hold [%d, %d, %d]" % (ps.batch, shape[1], shape[2]))


def _check_prefill(q: torch.Tensor, head_dim: int, cu_q: Optional[torch.Tensor], batch: int,
                   out: Optional[torch.Tensor]) -> None:
    """q is [total_q, num_q_heads, head_dim] and out, if given, as large at least."""
    if q.shape[2] != head_dim:
        raise ValueError("q must be [total_q, num_q_heads, %d], got %s" % (head_dim, tuple(q.shape)))
    if out is not None and out.numel() < q.numel():
        raise ValueError("out must hold %s" % (list(q.shape),))
    _check_cu(cu_q, batch, "cu_q")


def kvq_write(cache: PagedCache, paging: Paging, k: torch.Tensor, v: torch.Tensor,
              cu_new_tokens: torch.Tensor, dev_error: Optional[torch.Tensor] = None, stream=None) -> None:
    """Quantise k, v [num_tokens, num_kv_heads, head_dim] and scatter them into the pages (16-bit caches: as bf16)."""
    if k.shape != v.shape or k.dtype != v.dtype:
        raise ValueError("k and v must have the same shape and dtype")
    cs, ps = _structs(cache, paging)
    dev = cache.k_pages.get_device()
    _check_rows(cache, k, "k")
    _check_cu(cu_new_tokens, ps.batch, "cu_new_tokens")
    _run(cache.k_pages.device, stream, _lib.kvq_write, ctypes.byref(cs), ctypes.byref(ps),
         _dev_ptr(k, None, "k", dev), _dev_ptr(v, None, "v", dev), _qdtype(k),
         _dev_ptr(cu_new_tokens, torch.int32, "cu_new_tokens", dev), int(k.shape[0]),
         _dev_ptr(dev_error, torch.int32, "dev_error", dev))


def kvq_gather(cache: PagedCache, paging: Paging, cu_tokens: torch.Tensor, num_tokens: int,
               out_dtype: torch.dtype = torch.float32, k_out: Optional[torch.Tensor] = None,
               v_out: Optional[torch.Tensor] = None, dev_error: Optional[torch.Tensor] = None, stream=None,
               k_chunk: Optional[torch.Tensor] = None, v_chunk: Optional[torch.Tensor] = None,
               cu_chunk: Optional[torch.Tensor] = None):
    """Dense dequantised (k, v) [num_tokens, num_kv_heads, head_dim] of the
    positions cu_tokens names (kvq_write's position map); -1 rows are zeros.
    With k_chunk / v_chunk / cu_chunk (kvq_gather_chunk) the last positions
    of each sequence come from those full-precision rows instead."""
    shape = (num_tokens, cache.num_kv_heads, cache.head_dim)
    device = cache.k_pages.device
    if k_out is None:
        k_out = _empty(shape, out_dtype, device, stream)
    if v_out is None:
        v_out = _empty(shape, out_dtype, device, stream)
    if k_out.dtype != v_out.dtype:
        raise ValueError("k_out and v_out must have the same dtype")
    cs, ps = _structs(cache, paging)
    dev = cache.k_pages.get_device()
    for t, name in ((k_out, "k_out"), (v_out, "v_out")):
        if t.numel() < num_tokens * cache.num_kv_heads * cache.head_dim:
            raise ValueError("%s must hold [%d, %d, %d], got %s" % (name, *shape, tuple(t.shape)))
    _check_cu(cu_tokens, ps.batch, "cu_tokens")
    if k_chunk is None:
        _run(device, stream, _lib.kvq_gather, ctypes.byref(cs), ctypes.byref(ps),
             _dev_ptr(cu_tokens, torch.int32, "cu_tokens", dev), int(num_tokens), _dev_ptr(k_out, None, "k_out", dev),
             _dev_ptr(v_out, None, "v_out", dev), _qdtype(k_out), _dev_ptr(dev_error, torch.int32, "dev_error", dev))
    else:
        if v_chunk is None or k_chunk.dtype != v_chunk.dtype or k_chunk.numel() != v_chunk.numel():
            raise ValueError("k_chunk and v_chunk must be given together, with one dtype and size")
        _check_rows(cache, k_chunk, "k_chunk")
        _check_cu(cu_chunk, ps.batch, "cu_chunk")
        _run(device, stream, _lib.kvq_gather_chunk, ctypes.byref(cs), ctypes.byref(ps),
             _dev_ptr(cu_tokens, torch.int32, "cu_tokens", dev), int(num_tokens),
             _dev_ptr(k_chunk, None, "k_chunk", dev), _dev_ptr(v_chunk, None, "v_chunk", dev), _qdtype(k_chunk),
             _dev_ptr(cu_chunk, torch.int32, "cu_chunk", dev),
             _dev_ptr(k_out, None, "k_out", dev), _dev_ptr(v_out, None, "v_out", dev), _qdtype(k_out),
             _dev_ptr(dev_error, torch.int32, "dev_error", dev))
    return k_out, v_out


def kvq_decode_workspace_size(cache: PagedCache, paging: Paging, num_q_heads: int, num_splits: int = 0):
    """(bytes, splits) the decode call needs for its split-KV partials."""
    cs, ps = _structs(cache, paging)
    nbytes, splits = ctypes.c_size_t(0), ctypes.c_int32(0)
    _check(_lib.kvq_decode_workspace_size(ctypes.byref(cs), ctypes.byref(ps), num_q_heads, num_splits,
                                          ctypes.byref(nbytes), ctypes.byref(splits)))
    return nbytes.value, splits.value


def kvq_decode_attn(cache: PagedCache, paging: Paging, q: torch.Tensor, softmax_scale: float,
                    out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                    num_splits: int = 0, dev_error: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Decode attention of q [batch, num_q_heads, head_dim]; returns fp32 out."""
    B, Hq, D = q.shape
    given = out
    if out is None:
        out = _empty((B, Hq, D), torch.float32, q.device, stream)
    if workspace is None:
        nbytes, _ = kvq_decode_workspace_size(cache, paging, Hq, num_splits)
        workspace = _empty(max(nbytes, 256), torch.uint8, q.device, stream)
    cs, ps = _structs(cache, paging)
    dev = cache.k_pages.get_device()
    _check_q(cache, ps, q, given)
    _run(cache.k_pages.device, stream, _lib.kvq_decode_attn, ctypes.byref(cs), ctypes.byref(ps),
         _dev_ptr(q, None, "q", dev), _qdtype(q), Hq, float(softmax_scale), _dev_ptr(out, torch.float32, "out", dev),
         _dev_ptr(workspace, None, "workspace", dev), workspace.numel() * workspace.element_size(), num_splits,
         _dev_ptr(dev_error, torch.int32, "dev_error", dev))
    return out


def kvq_write_decode_attn(cache: PagedCache, paging: Paging, k: torch.Tensor, v: torch.Tensor,
                          cu_new_tokens: torch.Tensor, q: torch.Tensor, softmax_scale: float,
                          out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                          num_splits: int = 0, dev_error: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """One decode step in one call: kvq_write of k, v [num_tokens, num_kv_heads, head_dim] (the step's new
    tokens), then decode attention of q [batch, num_q_heads, head_dim]; returns fp32 out.  The pages and
    the output are those of kvq_write followed by kvq_decode_attn."""
    if k.shape != v.shape or k.dtype != v.dtype:
        raise ValueError("k and v must have the same shape and dtype")
    B, Hq, D = q.shape
    given = out
    if out is None:
        out = _empty((B, Hq, D), torch.float32, q.device, stream)
    if workspace is None:
        nbytes, _ = kvq_decode_workspace_size(cache, paging, Hq, num_splits)
        workspace = _empty(max(nbytes, 256), torch.uint8, q.device, stream)
    cs, ps = _structs(cache, paging)
    dev = cache.k_pages.get_device()
    _check_rows(cache, k, "k")
    _check_cu(cu_new_tokens, ps.batch, "cu_new_tokens")
    _check_q(cache, ps, q, given)
    _run(cache.k_pages.device, stream, _lib.kvq_write_decode_attn, ctypes.byref(cs), ctypes.byref(ps),
         _dev_ptr(k, None, "k", dev), _dev_ptr(v, None, "v", dev), _qdtype(k),
         _dev_ptr(cu_new_tokens, torch.int32, "cu_new_tokens", dev), int(k.shape[0]), _dev_ptr(q, None, "q", dev),
         _qdtype(q), Hq, float(softmax_scale), _dev_ptr(out, torch.float32, "out", dev),
         _dev_ptr(workspace, torch.uint8, "workspace", dev), workspace.numel(), int(num_splits),
         _dev_ptr(dev_error, torch.int32, "dev_error", dev))
    return out


def kvq_decode_attn_noalloc(cache: PagedCache, paging: Paging, q: torch.Tensor, softmax_scale: float,
                            out: Optional[torch.Tensor] = None, num_splits: int = 0,
                            dev_error: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """kvq_decode_attn without a caller workspace: for callers that cannot
    allocate device memory at call time.  Uses the library's one static
    device scratch array (KVQ_NOALLOC_SCRATCH_BYTES per GPU); calls that
    overlap on the GPU race on it, so serialise them.  The first call on a
    device must come before any stream capture."""
    B, Hq, D = q.shape
    given = out
    if out is None:
        out = _empty((B, Hq, D), torch.float32, q.device, stream)
    cs, ps = _structs(cache, paging)
    dev = cache.k_pages.get_device()
    _check_q(cache, ps, q, given)
    _run(cache.k_pages.device, stream, _lib.kvq_decode_attn_noalloc, ctypes.byref(cs), ctypes.byref(ps),
         _dev_ptr(q, None, "q", dev), _qdtype(q), Hq, float(softmax_scale), _dev_ptr(out, torch.float32, "out", dev),
         num_splits, _dev_ptr(dev_error, torch.int32, "dev_error", dev))
    return out


def kvq_prefill_attn(cache: PagedCache, paging: Paging, q: torch.Tensor, cu_q: torch.Tensor, max_q_per_seq: int,
                     softmax_scale: float, out: Optional[torch.Tensor] = None,
                     dev_error: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Causal chunked-prefill attention of q [total_q, num_q_heads, head_dim]; returns fp32 out."""
    T, Hq, D = q.shape
    cs, ps = _structs(cache, paging)
    dev = cache.k_pages.get_device()
    _check_prefill(q, cache.head_dim, cu_q, ps.batch, out)
    if out is None:
        out = _empty((T, Hq, D), torch.float32, q.device, stream)
    _run(cache.k_pages.device, stream, _lib.kvq_prefill_attn, ctypes.byref(cs), ctypes.byref(ps),
         _dev_ptr(q, None, "q", dev), _qdtype(q), Hq, _dev_ptr(cu_q, torch.int32, "cu_q", dev), T, int(max_q_per_seq),
         float(softmax_scale), _dev_ptr(out, torch.float32, "out", dev),
         _dev_ptr(dev_error, torch.int32, "dev_error", dev))
    return out


def kvq_prefill_dense_attn(k: torch.Tensor, v: torch.Tensor, cu_kv: torch.Tensor, seq_lens: torch.Tensor,
                           q: torch.Tensor, cu_q: torch.Tensor, max_q_per_seq: int, softmax_scale: float,
                           window_per_kv_head: Optional[torch.Tensor] = None, sink_size: int = 0,
                           out: Optional[torch.Tensor] = None, dev_error: Optional[torch.Tensor] = None,
                           stream=None) -> torch.Tensor:
    """Causal chunked-prefill attention of q [total_q, num_q_heads, head_dim]
    over dense bf16 k, v [rows, num_kv_heads, head_dim] (sequence b's key j at
    row cu_kv[b] + j, e.g. kvq_gather's output); returns fp32 out."""
    if k.dtype != torch.bfloat16 or v.dtype != torch.bfloat16 or k.shape != v.shape:
        raise ValueError("k and v must be bfloat16 tensors of one shape")
    T, Hq, D = q.shape
    if k.dim() != 3:
        raise ValueError("k and v must be [rows, num_kv_heads, head_dim], got %s" % (tuple(k.shape),))
    dev, batch = k.get_device(), int(seq_lens.shape[0])
    _check_prefill(q, k.shape[2], cu_q, batch, out)
    _check_cu(cu_kv, batch, "cu_kv")
    if window_per_kv_head is not None and window_per_kv_head.numel() < k.shape[1]:
        raise ValueError("window_per_kv_head must have %d elements, got %d" % (k.shape[1], window_per_kv_head.numel()))
    if out is None:
        out = _empty((T, Hq, D), torch.float32, q.device, stream)
    ps = KvqPaging(None, None, 0, batch, _dev_ptr(seq_lens, torch.int32, "seq_lens", dev),
                   _dev_ptr(window_per_kv_head, torch.int32, "window_per_kv_head", dev), int(sink_size))
    _run(k.device, stream, _lib.kvq_prefill_dense_attn, _dev_ptr(k, None, "k", dev), _dev_ptr(v, None, "v", dev),
         _dev_ptr(cu_kv, torch.int32, "cu_kv", dev), int(k.shape[0]), int(k.shape[1]), int(k.shape[2]),
         ctypes.byref(ps), _dev_ptr(q, None, "q", dev), _qdtype(q), Hq, _dev_ptr(cu_q, torch.int32, "cu_q", dev), T,
         int(max_q_per_seq), float(softmax_scale), _dev_ptr(out, torch.float32, "out", dev),
         _dev_ptr(dev_error, torch.int32, "dev_error", dev))
    return out


# ---------------------------------------------------------------------------
# pages

Caches = Union[PagedCache, Sequence[PagedCache]]


def _cache_array(caches: Caches):
    """(ctypes array, number, device, num_kv_heads, num_blocks) of the caches that share page numbers; kept with the
    first cache as long as the caches' structs are the same (by their numbers and pointers: nothing here keeps another
    cache's memory alive)."""
    cs = (caches,) if isinstance(caches, PagedCache) else caches
    if not cs:
        raise ValueError("no caches")
    first = cs[0].__dict__
    group = first.get("_group")
    structs = [c._struct for c in cs]
    if (group is not None and None not in structs and [k.serial for k in structs] == group[0]
            and [t.data_ptr() for k in structs for t in k.tensors] == group[1]):
        return group[2]
    dev = cs[0].k_pages.device
    array = (KvqCache * len(cs))(*[c.struct() for c in cs])
    structs = [c._struct for c in cs]
    if any(k.devices != {dev} for k in structs):
        raise ValueError("the caches of one call must be on one device")
    first["_group"] = group = ([k.serial for k in structs], [p for k in structs for p in k.pointers],
                               (array, len(cs), dev, array[0].num_kv_heads, array[0].num_blocks))
    return group[2]


def _page_tensor(t: Optional[torch.Tensor], name: str, dev: torch.device, numel: Optional[int] = None):
    """Device pointer of an int32 tensor of the caches' device, with `numel` elements where that is given."""
    if t is None:
        return None
    if t.get_device() != dev.index or t.dtype is not torch.int32 or not t.is_contiguous():
        if t.device != dev:
            raise ValueError("%s must be on the caches' device" % name)
        return _dev_ptr(t, torch.int32, name)  # says what is wrong
    if numel is not None and t.numel() != numel:
        raise ValueError("%s must have %d elements, got %d" % (name, numel, t.numel()))
    return t.data_ptr()


def _page_paging(p: "Paging", name: str, dev: torch.device, num_kv_heads: int) -> Tuple[KvqPaging, bool, int]:
    """(struct, head-wise, rows) of a paging state of the caches' device."""
    headwise = p.block_tables_headwise is not None
    t = p.block_tables_headwise if headwise else p.block_tables
    if t is None:
        raise ValueError("%s needs a block table" % name)
    struct = p.struct()
    if p._struct.devices != {dev}:
        raise ValueError("%s must be on the caches' device" % name)
    rows = struct.batch
    if len(t) != (rows * num_kv_heads if headwise else rows):
        raise ValueError("%s: the table's rows do not match seq_lens" % name)
    return struct, headwise, rows


def _page_scratch(workspace, size, dev, stream, *args):
    if workspace is None:
        workspace = _empty(max(size(*args), 256), torch.uint8, dev, stream)
    elif workspace.get_device() != dev.index:
        raise ValueError("workspace must be on the caches' device")
    return _dev_ptr(workspace, torch.uint8, "workspace"), workspace.numel(), workspace


def kvq_copy_workspace_size(caches: Caches, num_pairs: int, headwise: bool = False) -> int:
    """Bytes of scratch that kvq_copy_pages needs (0 for short lists)."""
    cs, n, _, _, _ = _cache_array(caches)
    size = ctypes.c_size_t(0)
    _check(_lib.kvq_copy_workspace_size(cs, n, int(num_pairs), int(headwise), ctypes.byref(size)))
    return size.value


def kvq_copy_pages(caches: Caches, src: torch.Tensor, dst: torch.Tensor, headwise: bool = False,
                   workspace: Optional[torch.Tensor] = None, dev_error: Optional[torch.Tensor] = None,
                   stream=None) -> None:
    """Page src[i] into page dst[i] (int32 tensors), K and V of every cache.  headwise: the numbers count
    (block, head) pages, block * num_kv_heads + head.  Sources are read as they were before the call; pairs
    that conflict are skipped and set KVQ_DEVERR_PAGE_CONFLICT."""
    cs, n, dev, _, _ = _cache_array(caches)
    pairs = int(src.numel())
    ps, pd = _page_tensor(src, "src", dev), _page_tensor(dst, "dst", dev, pairs)
    ws, nbytes = None, 0
    if workspace is not None or kvq_copy_workspace_size(caches, pairs, headwise) > 0:  # short lists need none
        ws, nbytes, _keep = _page_scratch(workspace, kvq_copy_workspace_size, dev, stream, caches, pairs, headwise)
    _run(dev, stream, _lib.kvq_copy_pages, cs, n, ps, pd, pairs, int(headwise), ws, nbytes,
         _page_tensor(dev_error, "dev_error", dev))


def _fork_out(caches: Caches, paging: Optional[Paging], rows: int, dev, stream) -> Paging:
    if paging is None:
        raise ValueError("without old rows, `out` gives the new table's kind and width")
    headwise = paging.block_tables_headwise is not None
    first = caches if isinstance(caches, PagedCache) else caches[0]
    table = _empty((rows * (first.num_kv_heads if headwise else 1), paging.max_blocks), torch.int32, dev, stream)
    kw = {"block_tables_headwise" if headwise else "block_tables": table}
    return Paging(_empty(rows, torch.int32, dev, stream), window_per_kv_head=paging.window_per_kv_head,
                  sink_size=paging.sink_size, **kw)


def kvq_fork_workspace_size(caches: Caches, paging: Optional[Paging], rows: int, out: Optional[Paging] = None) -> int:
    """Bytes of scratch that kvq_fork needs for `rows` new rows."""
    cs, n, _, _, _ = _cache_array(caches)
    like = (out or paging)._build()  # (the size goes by the new rows' number, the table's kind and its width)
    like.batch = int(rows)
    size = ctypes.c_size_t(0)
    _check(_lib.kvq_fork_workspace_size(cs, n, None, ctypes.byref(like), ctypes.byref(size)))
    return size.value


def kvq_fork(caches: Caches, paging: Optional[Paging], parents: torch.Tensor,
             new_tokens: Optional[torch.Tensor] = None, keep_tokens: Optional[torch.Tensor] = None,
             pins: Optional[torch.Tensor] = None, out: Optional[Paging] = None,
             page_refs: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
             dev_error: Optional[torch.Tensor] = None, stream=None) -> Tuple[Paging, torch.Tensor]:
    """New table rows from old ones: row i continues old row parents[i] (int32; negative: starts empty), keeps its
    first keep_tokens[i] tokens and gets pages for new_tokens[i] more.  Full pages are shared, a shared partly
    filled last page is copied in every cache, rows that nobody continues are freed.  Returns the new paging state
    (`out` if given: its table and seq_lens are written) and page_refs [spaces, num_blocks], the uses of every page
    (0: free).  paging None: there are no old rows yet (`out` is needed)."""
    cs, n, dev, Hkv, blocks = _cache_array(caches)
    rows = int(parents.numel())
    if out is None:
        out = _fork_out(caches, paging, rows, dev, stream)
    new, headwise, got = _page_paging(out, "out", dev, Hkv)
    if got != rows:
        raise ValueError("out must have one row per parent")
    old = None if paging is None else _page_paging(paging, "paging", dev, Hkv)[0]
    spaces = Hkv if headwise else 1
    if page_refs is None:
        page_refs = _empty((spaces, blocks), torch.int32, dev, stream)
    ws, nbytes, _keep = _page_scratch(workspace, kvq_fork_workspace_size, dev, stream, caches, paging, rows, out)
    _run(dev, stream, _lib.kvq_fork, cs, n, None if old is None else ctypes.byref(old),
         _page_tensor(parents, "parents", dev), _page_tensor(keep_tokens, "keep_tokens", dev, rows),
         _page_tensor(new_tokens, "new_tokens", dev, rows), _page_tensor(pins, "pins", dev, spaces * blocks),
         ctypes.byref(new), _page_tensor(page_refs, "page_refs", dev, spaces * blocks), ws, nbytes,
         _page_tensor(dev_error, "dev_error", dev))
    return out, page_refs


def kvq_compact_workspace_size(caches: Caches, paging: Paging) -> int:
    """Bytes of scratch that kvq_compact needs."""
    cs, n, _, _, _ = _cache_array(caches)
    ps = paging.struct()
    size = ctypes.c_size_t(0)
    _check(_lib.kvq_compact_workspace_size(cs, n, ctypes.byref(ps), ctypes.byref(size)))
    return size.value


def kvq_compact(caches: Caches, paging: Paging, pins: Optional[torch.Tensor] = None, out: Optional[Paging] = None,
                page_map: Optional[torch.Tensor] = None, page_refs: Optional[torch.Tensor] = None,
                num_used: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                dev_error: Optional[torch.Tensor] = None, stream=None):
    """The used pages of each space moved to its lowest numbers, in every cache.  Returns (paging state with the
    rewritten table, page_map [spaces, num_blocks] (old number -> new, -1: unused), page_refs [spaces, num_blocks]
    by new number, num_used [spaces]).  `out` gives the table to write; it may be `paging` itself, and gets its
    lengths where it has a tensor of its own for them.  Pages with a positive `pins` stay where they are."""
    cs, n, dev, Hkv, blocks = _cache_array(caches)
    old, headwise, rows = _page_paging(paging, "paging", dev, Hkv)
    kind = "block_tables_headwise" if headwise else "block_tables"
    table = getattr(paging, kind)
    if out is None:
        out = Paging(paging.seq_lens, window_per_kv_head=paging.window_per_kv_head, sink_size=paging.sink_size,
                     **{kind: _empty(tuple(table.shape), torch.int32, dev, stream)})
    to = getattr(out, kind)
    if to is None or to.shape != table.shape:
        raise ValueError("out must have a table of the same kind and shape")
    own_lens = _page_tensor(out.seq_lens, "out.seq_lens", dev, rows) not in (None, paging.seq_lens.data_ptr())
    spaces = Hkv if headwise else 1
    if page_map is None:
        page_map = _empty((spaces, blocks), torch.int32, dev, stream)
    if page_refs is None:
        page_refs = _empty((spaces, blocks), torch.int32, dev, stream)
    if num_used is None:
        num_used = _empty(spaces, torch.int32, dev, stream)
    ws, nbytes, _keep = _page_scratch(workspace, kvq_compact_workspace_size, dev, stream, caches, paging)
    _run(dev, stream, _lib.kvq_compact, cs, n, ctypes.byref(old), _page_tensor(pins, "pins", dev, spaces * blocks),
         _page_tensor(to, "out", dev), _page_tensor(page_map, "page_map", dev, spaces * blocks),
         _page_tensor(page_refs, "page_refs", dev, spaces * blocks), _page_tensor(num_used, "num_used", dev, spaces),
         ws, nbytes, _page_tensor(dev_error, "dev_error", dev))
    if own_lens:
        _copy(out.seq_lens, paging.seq_lens, stream)
    return out, page_map, page_refs, num_used
