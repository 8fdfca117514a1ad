"""Buffers larger than a call needs, and rows given flat: what the library takes, the binding passes on."""
import numpy as np
import pytest
import torch

import decode16_ref as ref
from harness import kvq

pytestmark = pytest.mark.gpu


def padded(t, rows, fill):
    out = torch.full((t.shape[0] + rows, *t.shape[1:]), fill, dtype=t.dtype, device=t.device)
    out[:t.shape[0]] = t
    return out


@pytest.mark.parametrize("mode", ["BF16_CACHE", "INT4_TOKEN_HEAD"])
def test_buffers_sized_for_a_larger_batch(mode):
    """cu longer than batch + 1, q with more rows than the batch, out larger than q: as a captured step keeps them."""
    K = kvq()
    c = ref.make(3, 2, 4, 128, 16, [40, 70, 5], seed=3)
    a, b = (K.PagedCache(getattr(K, "KVQ_" + mode), c["cache"].num_blocks, 2, 16, 128) for _ in range(2))
    K.kvq_write(a, c["pag"], c["k"], c["v"], c["cu"])
    want = K.kvq_decode_attn(a, c["pag"], c["q"], c["scale"])
    cu, q = padded(c["cu"], 5, 115), padded(c["q"], 2, 7)
    K.kvq_write(b, c["pag"], c["k"], c["v"], cu)
    assert torch.equal(a.k_pages, b.k_pages) and torch.equal(a.v_pages, b.v_pages)
    n = want.numel()
    for kw in ({}, dict(num_splits=3)):
        exact = K.kvq_decode_attn(a, c["pag"], c["q"], c["scale"], **kw)
        for call in (lambda o: K.kvq_decode_attn(b, c["pag"], q, c["scale"], out=o, **kw),
                     lambda o: K.kvq_decode_attn_noalloc(b, c["pag"], q, c["scale"], out=o, **kw),
                     lambda o: K.kvq_write_decode_attn(b, c["pag"], c["k"], c["v"], cu, q, c["scale"], out=o, **kw)):
            out = torch.full((6, 8, 128), -3.0, device="cuda")     # larger than q
            assert call(out) is out
            assert torch.equal(out[:3], exact) and bool((out[3:] == -3).all())
            out = torch.full((3, 8, 128), -3.0, device="cuda")     # as large as the batch needs, smaller than q
            assert torch.equal(call(out), exact)
    assert K.kvq_decode_attn(b, c["pag"], q, c["scale"])[:3].numel() == n
    k, v = K.kvq_gather(a, c["pag"], c["cu"], 115)
    ko, vo = torch.full((130, 2, 128), -3.0, device="cuda"), torch.full((130 * 256,), -3.0, device="cuda")
    K.kvq_gather(a, c["pag"], cu, 115, k_out=ko, v_out=vo)
    assert torch.equal(ko[:115], k) and torch.equal(vo[:115 * 256].view(115, 2, 128), v)
    assert bool((ko[115:] == -3).all()) and bool((vo[115 * 256:] == -3).all())


def test_rows_given_flat():
    """k, v, the chunk and the outputs as [tokens, heads * dim]: the same memory."""
    K = kvq()
    c = ref.make(3, 2, 4, 128, 16, [40, 70, 5], seed=4)
    flat = K.PagedCache(K.KVQ_BF16_CACHE, c["cache"].num_blocks, 2, 16, 128)
    K.kvq_write(flat, c["pag"], c["k"].view(115, 256), c["v"].view(115, 256), c["cu"])
    out = [K.kvq_gather(x, c["pag"], c["cu"], 115) for x in (c["cache"], flat)]
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
    new = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda")
    rows = torch.randn((2, 3, 2, 128), device="cuda").bfloat16()
    a = K.kvq_write_decode_attn(c["cache"], c["pag"], rows[0], rows[1], new, c["q"], c["scale"])
    b = K.kvq_write_decode_attn(flat, c["pag"], rows[0].view(3, 256), rows[1].view(3, 256), new, c["q"], c["scale"])
    assert torch.equal(a, b)
    want = K.kvq_gather(c["cache"], c["pag"], c["cu"], 115, k_chunk=rows[0], v_chunk=rows[1], cu_chunk=new)
    ko, vo = torch.empty((115, 256), device="cuda"), torch.empty((115, 256), device="cuda")
    K.kvq_gather(c["cache"], c["pag"], c["cu"], 115, k_out=ko, v_out=vo, k_chunk=rows[0].view(3, 256),
                 v_chunk=rows[1].view(3, 256), cu_chunk=padded(new, 3, 3))
    assert torch.equal(ko.view(115, 2, 128), want[0]) and torch.equal(vo.view(115, 2, 128), want[1])


def test_what_would_pass_the_end_is_still_refused():
    K = kvq()
    c = ref.make(3, 2, 4, 128, 16, [40, 70, 5], seed=5)
    cache, pag, cu = c["cache"], c["pag"], c["cu"]
    f = lambda *s: torch.empty(s, device="cuda")  # noqa: E731
    bad = [lambda: K.kvq_write(cache, pag, c["k"].view(-1), c["v"].view(-1), cu),
           lambda: K.kvq_write(cache, pag, c["k"].view(230, 128), c["v"].view(230, 128), cu),
           lambda: K.kvq_write(cache, pag, c["k"], c["v"], cu[:3].contiguous()),
           lambda: K.kvq_gather(cache, pag, cu[:3].contiguous(), 115),
           lambda: K.kvq_gather(cache, pag, cu, 115, k_out=f(114, 256), v_out=f(115, 256)),
           lambda: K.kvq_gather(cache, pag, cu, 115, k_out=f(115, 256), v_out=f(115 * 256 - 1)),
           lambda: K.kvq_gather(cache, pag, cu, 115, k_chunk=c["k"][:3], v_chunk=c["v"][:2], cu_chunk=cu),
           lambda: K.kvq_decode_attn(cache, pag, c["q"][:2], 0.1),
           lambda: K.kvq_decode_attn(cache, pag, c["q"], 0.1, out=f(2, 8, 128)),
           lambda: K.kvq_decode_attn(cache, pag, padded(c["q"], 2, 0), 0.1, out=f(2, 8, 128))]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for call in (lambda: K.kvq_write(cache, pag, c["k"], c["v"], None),      # refused by the library, as ever
                 lambda: K.kvq_gather(cache, pag, None, 115),
                 lambda: K.kvq_gather(cache, pag, cu, 115, k_chunk=c["k"], v_chunk=c["v"])):
        with pytest.raises(K.KvqError, match="KVQ_ERR_INVALID_ARG"):
            call()
    assert np.array_equal(K.kvq_decode_attn(cache, pag, c["q"], c["scale"]).cpu(),
                          K.kvq_decode_attn_noalloc(cache, pag, c["q"], c["scale"]).cpu())
