"""Prefill calls whose counts do not fit their tensors: what is not there is skipped and reported."""
import numpy as np
import pytest
import torch

import kvq_inputs as gen
import oracle
from harness import ATOL, build_case, kvq, max_err, prefill_oracle, q_host, to_dev_input, to_orc_input, write_step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [1, 20, 33, 64])
@pytest.mark.parametrize("dense", [False, True])
def test_queries_past_the_rows_that_were_given(rows, dense):
    """cu_q names 70 + 33 rows; q and out hold fewer, with guards behind them."""
    K = kvq()
    wl = gen.custom(gen.MODE_INT4, 8, 2, 128, 16, "bf16", seq_lens=[200, 33], n_new=[70, 33], step="prefill", seed=6)
    c = build_case(wl)
    write_step(c)
    q = q_host(wl)
    want = prefill_oracle(c, q)
    cu = torch.from_numpy(wl.cu(wl.n_new)).cuda()
    buf = torch.full((110, 8, 128), -3.0, device="cuda")
    dq, err = to_dev_input(q, wl.dtype)[:rows], torch.zeros(1, dtype=torch.int32, device="cuda")
    if dense:
        cu_kv = torch.tensor([0, 200, 233], dtype=torch.int32, device="cuda")
        k, v = K.kvq_gather(c.gcache, c.gpag, cu_kv, 233, out_dtype=torch.bfloat16)
        full = K.kvq_prefill_dense_attn(k, v, cu_kv, c.gpag.seq_lens, to_dev_input(q, wl.dtype), cu, 70, 128 ** -0.5)
        K.kvq_prefill_dense_attn(k, v, cu_kv, c.gpag.seq_lens, dq, cu, 70, 128 ** -0.5, out=buf, dev_error=err)
        assert torch.equal(buf[:rows], full[:rows])
    else:
        K.kvq_prefill_attn(c.gcache, c.gpag, dq, cu, 70, 128 ** -0.5, out=buf, dev_error=err)
        assert max_err(buf[:rows].cpu().numpy(), want[:rows]) <= ATOL
    assert bool((buf[rows:] == -3).all())
    assert int(err.item()) == K.KVQ_DEVERR_SEQ_LEN


@pytest.mark.parametrize("mode", [gen.MODE_INT4, gen.MODE_INT8])
@pytest.mark.parametrize("sink", [0, 20, 70])
def test_windows_of_lengths_past_the_table(mode, sink):
    """The windows of a length far past its table row hold no key there; the sinks stay."""
    K = kvq()
    wl = gen.custom(mode, 8, 2, 128, 16, "bf16", seq_lens=[300, 150], n_new=[40, 30], step="prefill", seed=9)
    c = build_case(wl)
    write_step(c)
    q = q_host(wl)
    lens, window = np.array([5000, 150], np.int32), np.array([16, 0], np.int32)
    pag = K.Paging(torch.from_numpy(lens).cuda(), block_tables=torch.from_numpy(wl.table).cuda(),
                   window_per_kv_head=torch.from_numpy(window).cuda(), sink_size=sink)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = torch.from_numpy(wl.cu(wl.n_new)).cuda()
    # only the pages that were written, so that the rows past token 300 of the last page are not seen
    table = wl.table.copy()
    table[0, 300 // 16:] = -1
    pag.block_tables.copy_(torch.from_numpy(table))
    g = K.kvq_prefill_attn(c.gcache, pag, to_dev_input(q, wl.dtype), cu, 40, 128 ** -0.5, dev_error=err).cpu().numpy()
    o, bits = oracle.attention(c.ocache, oracle.Paging(table, False, lens, window, sink), to_orc_input(q, wl.dtype),
                               128 ** -0.5, cu_q=wl.cu(wl.n_new))
    assert bits == K.KVQ_DEVERR_TABLE_RANGE and int(err.item()) == K.KVQ_DEVERR_TABLE_RANGE
    assert g[:40, :4].any() == (sink > 0)
    assert max_err(g, o) <= ATOL
