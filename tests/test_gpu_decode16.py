"""16-bit (bf16) pages on the GPU: the write, the gather and the decode
attention against plain 64-bit code.  Every pool starts as 0xFF bytes, so that
a slot that was never written holds a NaN row."""
import numpy as np
import pytest
import torch

import decode16_ref as ref
from harness import kvq

pytestmark = pytest.mark.gpu


def decode(c, **kw):
    out = kvq().kvq_decode_attn(c["cache"], c["pag"], c["q"], c["scale"], dev_error=c["err"], **kw)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 7, 8])
def test_decode16_groups_dims_types(G, D, dtype):
    c = ref.make(6, 2, G, D, (16, 32, 64)[G % 3], [1, 31, 0, 33, 250, 700], dtype, seed=G + D)
    ref.check(decode(c), ref.attention64(c))
    assert int(c["err"].item()) == 0


@pytest.mark.parametrize("bs", [16, 32, 64])
@pytest.mark.parametrize("headwise", [False, True])
def test_decode16_lengths(bs, headwise):
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 0, 1000]
    c = ref.make(len(lens), 3, 4, 128, bs, lens, headwise=headwise, seed=bs)
    ref.check(decode(c), ref.attention64(c))
    assert int(c["err"].item()) == 0


@pytest.mark.parametrize("window", [[0, 1], [16, 40], [300, 5000]])
@pytest.mark.parametrize("sink", [0, 3, 20])
def test_decode16_windows_sinks_and_evicted_pages(window, sink):
    lens = [900, 75, 17, 300]
    c = ref.make(4, 2, 5, 128, 16, lens, headwise=True, window=window, sink=sink, seed=sink + window[0])
    t = c["pag"].block_tables_headwise.view(4, 2, -1)
    t[0, 1, 1:4] = -1       # a hole inside the sequence
    t[2, 0] = -1            # a row that leaves nothing
    t[3, 1, -1] = -1
    c["table"] = t.cpu().numpy()
    out = decode(c)
    ref.check(out, ref.attention64(c))
    assert not out[2, :5].any()
    assert int(c["err"].item()) == 0


@pytest.mark.parametrize("splits", [1, 2, 7, 100, 100000])
def test_decode16_forced_splits(splits):
    c = ref.make(3, 2, 4, 128, 32, [3000, 5, 640], seed=splits)
    ref.check(decode(c, num_splits=splits), ref.attention64(c))


def test_decode16_many_pairs_and_empty_sequences():
    r = np.random.Generator(np.random.PCG64(5))
    lens = r.integers(0, 40, 900)
    lens[::7] = 0
    c = ref.make(900, 5, 2, 64, 16, lens, seed=9)   # 4500 pairs: several pairs to a run of the prefix sums
    out = decode(c)
    ref.check(out, ref.attention64(c))
    assert not out[torch.from_numpy(lens == 0)].any()
    same = decode(c)
    assert torch.equal(out, same)


def test_decode16_large_logits_and_late_maximum():
    """A maximum that keeps growing along the sequence moves the reference again and again."""
    c = ref.make(2, 1, 4, 128, 16, [2000, 333], seed=3, write=False)
    n = c["k"].shape[0]
    ramp = torch.linspace(0.01, 6.0, n, device="cuda")[:, None, None]
    c["k"] = (c["k"].float() * ramp).to(torch.bfloat16)
    kvq().kvq_write(c["cache"], c["pag"], c["k"], c["v"], c["cu"])
    ref.check(decode(c), ref.attention64(c))


def test_decode16_bad_pages_and_lengths_set_their_bits():
    K = kvq()
    c = ref.make(4, 2, 4, 128, 16, [100, 60, 200, 30], seed=1, max_blocks=13)
    t = c["pag"].block_tables
    t[0, 2] = 10 ** 6       # past the pool: skipped
    t[1, 1] = -5            # any negative entry is an evicted page
    c["pag"].seq_lens[3] = -2
    c["table"] = t.view(4, 1, -1).cpu().numpy().copy()
    c["table"][0, 0, 2] = -1
    lens = np.array([100, 60, 200, 0])
    out = decode(c)
    ref.check(out, ref.attention64(c, lens=lens))
    assert int(c["err"].item()) == K.KVQ_DEVERR_BLOCK_RANGE | K.KVQ_DEVERR_SEQ_LEN
    c["err"].zero_()
    c["pag"].seq_lens.copy_(torch.tensor([100, 60, 5000, 30]))   # longer than its table row
    lens = np.array([100, 60, 208, 30])
    c["lens"] = np.array([100, 60, 200, 30])
    t[2, 12] = -1           # (the row's last page holds only 8 written rows)
    c["table"][2, 0, 12] = -1
    ref.check(decode(c), ref.attention64(c, lens=lens))
    assert int(c["err"].item()) == K.KVQ_DEVERR_BLOCK_RANGE | K.KVQ_DEVERR_TABLE_RANGE


@pytest.mark.parametrize("sink", [0, 20])
def test_decode16_windows_of_lengths_past_the_table(sink):
    """The window of a length that passes its table row by more than the window holds no key; the sinks stay."""
    K = kvq()
    c = ref.make(3, 2, 4, 128, 16, [90, 208, 40], headwise=True, window=[16, 0], sink=sink, seed=12, max_blocks=13)
    c["pag"].seq_lens.copy_(torch.tensor([90, 5000, 40]))
    out = decode(c)
    ref.check(out, ref.attention64(c, lens=np.array([90, 5000, 40])))
    assert out[1, :4].any() == (sink > 0) and int(c["err"].item()) == K.KVQ_DEVERR_TABLE_RANGE


@pytest.mark.parametrize("mode", ["INT4_TOKEN_HEAD", "INT8_CHANNEL"])
def test_low_bit_windows_of_lengths_past_the_table(mode):
    import kvq_inputs as gen
    from harness import ATOL, build_case, decode_gpu, q_host, write_step
    K = kvq()
    wl = gen.custom({"INT4_TOKEN_HEAD": gen.MODE_INT4, "INT8_CHANNEL": gen.MODE_INT8}[mode], 8, 2, 128, 16, "bf16",
                    seq_lens=[300, 64, 130], n_new=[1, 1, 1], seed=6)
    c = build_case(wl)
    write_step(c)
    q = q_host(wl)
    want = decode_gpu(c, q)
    pag = K.Paging(torch.tensor([300, 100000, 130], dtype=torch.int32, device="cuda"), block_tables=c.gpag.block_tables,
                   window_per_kv_head=torch.tensor([16, 0], dtype=torch.int32, device="cuda"))
    out = decode_gpu(c, q, paging=pag)
    assert not out[1, :4].any()         # no key of the window is in the table, and there is no sink
    # the head without a window sees the same keys, in other slices (entries past the 64 tokens are -1)
    assert np.abs(out[:, 4:] - want[:, 4:]).max() <= ATOL
    assert int(c.dev_err.item()) == K.KVQ_DEVERR_TABLE_RANGE


@pytest.mark.parametrize("splits", [0, 3, 200])
@pytest.mark.parametrize("lens", [[60, 33], [9000, 700], [1, 9000]])
def test_decode16_visible_nans_reach_their_outputs_alone(lens, splits):
    """A NaN in a visible key: the outputs of its kv head's q heads; in a visible value: its dim of them."""
    c = ref.make(2, 2, 4, 128, 16, lens, seed=13)
    want = decode(c, num_splits=splits)
    kp, vp = c["cache"].k_pages.view(torch.bfloat16), c["cache"].v_pages.view(torch.bfloat16)
    for key in sorted({0, min(32, lens[0] - 1), lens[0] - 1}):
        page = int(c["table"][0, 0, key // 16])
        held = kp[page, 1, key % 16, 5].clone()
        kp[page, 1, key % 16, 5] = float("nan")
        out = decode(c, num_splits=splits)
        assert torch.isnan(out[0, 4:]).all()
        out[0, 4:] = want[0, 4:]
        assert torch.equal(out, want)
        kp[page, 1, key % 16, 5] = held
        held = vp[page, 1, key % 16, 77].clone()
        vp[page, 1, key % 16, 77] = float("nan")
        out = decode(c, num_splits=splits)
        assert torch.isnan(out[0, 4:, 77]).all()
        out[0, 4:, 77] = want[0, 4:, 77]
        assert torch.equal(out, want)
        vp[page, 1, key % 16, 77] = held


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 128])
def test_write16_gather16_round_trip(D, dtype):
    K = kvq()
    lens = [5, 0, 77, 16, 300]
    c = ref.make(5, 3, 1, D, 16, lens, dtype, headwise=True, seed=D)
    n = sum(lens)
    for out_dtype in (torch.float32, torch.bfloat16):
        k, v = K.kvq_gather(c["cache"], c["pag"], c["cu"], n, out_dtype=out_dtype, dev_error=c["err"])
        assert torch.equal(k, c["k"].to(torch.bfloat16).to(out_dtype)) and torch.equal(v, c["v"].to(torch.bfloat16).to(out_dtype))
    # rows behind the last token of each sequence were left as they were
    pages = c["cache"].k_pages.view(torch.bfloat16)
    assert int(torch.isnan(pages).sum()) == pages.numel() - n * 3 * D
    # an evicted page drops its rows and reads back as zeros
    t = c["pag"].block_tables_headwise
    t.view(5, 3, -1)[2, 1, 0] = -1
    before = c["cache"].k_pages.clone()
    K.kvq_write(c["cache"], c["pag"], c["k"], c["v"], c["cu"], dev_error=c["err"])
    assert torch.equal(before, c["cache"].k_pages)
    k, _ = K.kvq_gather(c["cache"], c["pag"], c["cu"], n, dev_error=c["err"])
    assert not k[5:21, 1].any() and torch.equal(k[21:, 1], c["k"][21:, 1].to(torch.bfloat16).float())
    # the last rows as given
    cu = torch.tensor([0, 2, 2, 5, 5, 105], dtype=torch.int32, device="cuda")
    chunk = torch.randn((2, 105, 3, D), device="cuda")
    k, v = K.kvq_gather(c["cache"], c["pag"], c["cu"], n, k_chunk=chunk[0], v_chunk=chunk[1], cu_chunk=cu, dev_error=c["err"])
    assert torch.equal(k[3:5], chunk[0, :2]) and torch.equal(v[-100:], chunk[1, 5:])
    assert torch.equal(v[5:79], c["v"][5:79].to(torch.bfloat16).float().index_put(
        (torch.arange(16, device="cuda"), torch.ones(16, dtype=torch.long, device="cuda")), torch.zeros((), device="cuda")))
    assert int(c["err"].item()) == 0


@pytest.mark.parametrize("new", [[1, 1, 1], [3, 1, 20]])
def test_write_decode16_is_the_write_then_the_decode(new):
    K = kvq()
    a = ref.make(3, 2, 4, 128, 16, [40, 1, 333], seed=2, write=False)
    b = ref.make(3, 2, 4, 128, 16, [40, 1, 333], seed=2)
    lens = np.minimum(new, a["lens"])
    pre = torch.cat([torch.arange(s, s + n - m) for s, n, m in zip(a["cu"].tolist(), a["lens"], lens)]).cuda()
    fin = torch.cat([torch.arange(s + n - m, s + n) for s, n, m in zip(a["cu"].tolist(), a["lens"], lens)]).cuda()
    pag = K.Paging(a["pag"].seq_lens - torch.from_numpy(lens.astype(np.int32)).cuda(), block_tables=a["pag"].block_tables)
    cu = lambda x: torch.from_numpy(np.concatenate([[0], np.cumsum(x)]).astype(np.int32)).cuda()  # noqa: E731
    K.kvq_write(a["cache"], pag, a["k"][pre], a["v"][pre], cu(a["lens"] - lens))
    out = K.kvq_write_decode_attn(a["cache"], a["pag"], a["k"][fin], a["v"][fin], cu(lens), a["q"], a["scale"])
    assert torch.equal(a["cache"].k_pages, b["cache"].k_pages) and torch.equal(a["cache"].v_pages, b["cache"].v_pages)
    assert torch.equal(out, decode(b))
    assert torch.equal(K.kvq_decode_attn_noalloc(b["cache"], b["pag"], b["q"], b["scale"]), out)


def test_decode16_pages_past_four_gigabytes():
    K = kvq()
    blocks, Hkv, bs, D = 150000, 8, 16, 128     # 4.9 GB a pool
    cache = K.PagedCache(K.KVQ_BF16_CACHE, blocks, Hkv, bs, D, k_pages=torch.empty((blocks, Hkv, bs, 2 * D), dtype=torch.uint8, device="cuda"),
                         v_pages=torch.empty((blocks, Hkv, bs, 2 * D), dtype=torch.uint8, device="cuda"))
    c = ref.make(2, Hkv, 4, D, bs, [50, 33], seed=4)
    t = c["pag"].block_tables
    t[t >= 0] = (blocks - 1 - t[t >= 0])
    K.kvq_write(cache, c["pag"], c["k"], c["v"], c["cu"], dev_error=c["err"])
    c["cache"] = cache
    ref.check(decode(c), ref.attention64(c))
    k, _ = K.kvq_gather(cache, c["pag"], c["cu"], 83)
    assert torch.equal(k, c["k"].float()) and int(c["err"].item()) == 0


def test_decode16_captured_and_on_another_stream():
    K = kvq()
    c = ref.make(3, 2, 4, 128, 16, [500, 20, 90], seed=8)
    want = decode(c)
    n, _ = K.kvq_decode_workspace_size(c["cache"], c["pag"], 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws, out = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty_like(want)
    with torch.cuda.stream(side):
        K.kvq_decode_attn(c["cache"], c["pag"], c["q"], c["scale"], out=out, workspace=ws)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    out.zero_()
    with torch.cuda.graph(graph):
        K.kvq_decode_attn(c["cache"], c["pag"], c["q"], c["scale"], out=out, workspace=ws)
    for _ in range(3):
        ws.fill_(0xFF)      # what the workspace holds does not matter
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_decode16_after_the_dense_prefill_of_its_gathered_prompt():
    """The run of them together: the prompt written, gathered and attended densely, its last query by the decode."""
    K = kvq()
    c = ref.make(2, 2, 4, 128, 16, [70, 129], seed=11)
    q = torch.randn((199, 8, 128), device="cuda").to(torch.bfloat16)
    k, v = K.kvq_gather(c["cache"], c["pag"], c["cu"], 199, out_dtype=torch.bfloat16)
    dense = K.kvq_prefill_dense_attn(k, v, c["cu"], c["pag"].seq_lens, q, c["cu"], 129, c["scale"])
    c["q"] = q[[69, 198]].contiguous()
    out = decode(c)
    ref.check(out, ref.attention64(c))
    assert float((out - dense[[69, 198]]).abs().max()) <= 2e-3


@pytest.mark.parametrize("mode", ["INT4_TOKEN_HEAD", "INT8_CHANNEL"])
def test_low_bit_decode_with_more_splits_than_tiles(mode):
    """A forced split count above the number of tiles: every record the merge reads was written by this call."""
    import kvq_inputs as gen
    from harness import ATOL, build_case, decode_gpu, decode_oracle, max_err, q_host, write_step
    wl = gen.custom({"INT4_TOKEN_HEAD": gen.MODE_INT4, "INT8_CHANNEL": gen.MODE_INT8}[mode], 8, 2, 128, 16, "bf16",
                    seq_lens=[700, 3, 130], n_new=[1, 1, 1], seed=6)
    c = build_case(wl)
    write_step(c)
    q = q_host(wl)
    assert max_err(decode_gpu(c, q, num_splits=100000), decode_oracle(c, q)) <= ATOL


def test_binding_refuses_tensors_of_other_shapes():
    K = kvq()
    c = ref.make(2, 2, 4, 128, 16, [20, 3], seed=1)
    bad = [c["q"][:1], c["q"][:, :, :64].contiguous(), c["q"][0], c["q"].cpu()]
    for q in bad:
        with pytest.raises(ValueError):
            K.kvq_decode_attn(c["cache"], c["pag"], q, 0.1)
    with pytest.raises(ValueError):
        K.kvq_decode_attn(c["cache"], c["pag"], c["q"], 0.1, out=torch.empty(2, 7, 128, device="cuda"))
    for k in (c["k"][:, :1].contiguous(), c["k"][:, :, :64].contiguous()):
        with pytest.raises(ValueError):
            K.kvq_write(c["cache"], c["pag"], k, k, c["cu"])
    with pytest.raises(ValueError):
        K.kvq_write(c["cache"], c["pag"], c["k"], c["v"], c["cu"][:2].contiguous())
    with pytest.raises(ValueError):
        K.kvq_gather(c["cache"], c["pag"], c["cu"], 23, k_out=torch.empty(22, 2, 128, device="cuda"))
    K.kvq_decode_attn(c["cache"], c["pag"], c["q"], c["scale"])


def test_binding_refuses_pagings_that_do_not_fit_the_cache():
    K = kvq()
    c = ref.make(2, 2, 4, 128, 16, [20, 3], headwise=True, window=[8, 0], seed=1)
    pag, ws = c["pag"], torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    new = c["k"][:2].contiguous()
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")

    def calls(p, **kw):
        yield lambda: K.kvq_decode_attn(c["cache"], p, c["q"], 0.1, workspace=ws, **kw)
        yield lambda: K.kvq_decode_attn_noalloc(c["cache"], p, c["q"], 0.1, **kw)
        yield lambda: K.kvq_write_decode_attn(c["cache"], p, new, new, cu, c["q"], 0.1, workspace=ws, **kw)
        yield lambda: K.kvq_write(c["cache"], p, c["k"], c["v"], c["cu"], **kw)
        yield lambda: K.kvq_gather(c["cache"], p, c["cu"], 23, **kw)

    short = K.Paging(pag.seq_lens, block_tables_headwise=pag.block_tables_headwise[:2].contiguous())
    narrow = K.Paging(pag.seq_lens, block_tables_headwise=pag.block_tables_headwise,
                      window_per_kv_head=pag.window_per_kv_head[:1].contiguous())
    for p, kw in ((short, {}), (narrow, {}), (pag, dict(dev_error=torch.zeros(1, dtype=torch.int32)))):
        for call in calls(p, **kw):
            with pytest.raises(ValueError):
                call()
    pag.window_per_kv_head = narrow.window_per_kv_head     # a paging state that fitted, changed
    with pytest.raises(ValueError):
        decode(c)
    pag.window_per_kv_head = torch.tensor([8, 0], dtype=torch.int32, device="cuda")
    ref.check(decode(c), ref.attention64(c))
