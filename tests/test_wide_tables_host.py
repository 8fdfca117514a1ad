"""Tables whose positions pass 32 bits are refused by every attention call over pages, whatever the mode."""
import ctypes

import pytest

from test_abi import K, _cache, _paging  # noqa: F401

MODES = ["INT4_TOKEN_HEAD", "INT2_TOKEN_HEAD", "INT8_CHANNEL", "INT4_STEGO", "INT8_TOKEN_HEAD", "FP8_TOKEN_HEAD", "BF16_CACHE"]


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("bs", [16, 32, 64])
def test_positions_past_32_bits(K, mode, bs):  # noqa: F811
    L, ref = K.lib(), ctypes.byref
    extra = dict(ch_amax=4096, ch_amax_ready=4096) if mode == "INT8_CHANNEL" else {}
    c = _cache(K, mode=getattr(K, "KVQ_" + mode), block_size=bs, **extra)
    wide = _paging(K, max_blocks=(1 << 31) // bs)
    assert L.kvq_decode_attn(ref(c), ref(wide), 256, 1, 8, 0.1, 256, 256, 1 << 40, 0, None, None) == K.KVQ_ERR_UNSUPPORTED
    assert b"32-bit" in L.kvq_last_error()
    if mode != "INT8_CHANNEL":
        assert L.kvq_write_decode_attn(ref(c), ref(wide), 4096, 4096, 1, 4096, 2, 256, 1, 8, 0.1, 256, 256, 1 << 40, 0, None,
                                       None) == K.KVQ_ERR_UNSUPPORTED
    if mode != "BF16_CACHE":
        assert L.kvq_prefill_attn(ref(c), ref(wide), 256, 1, 8, 256, 4, 4, 0.1, 256, None, None) == K.KVQ_ERR_UNSUPPORTED
        assert b"32-bit" in L.kvq_last_error()
