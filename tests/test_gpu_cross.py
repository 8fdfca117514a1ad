"""Cross attention on the GPU against plain 64-bit code, over every mode's pages (their rows read back with
kvq_gather, which other tests pin) and over dense rows."""
import numpy as np
import pytest
import torch

import cross_ref as ref
from harness import kvq
from test_gpu_rope import cu_of, i32, make_cache, paging, rows

pytestmark = pytest.mark.gpu
MODES = ["INT4_TOKEN_HEAD", "INT2_TOKEN_HEAD", "INT4_STEGO", "INT8_TOKEN_HEAD", "FP8_TOKEN_HEAD", "BF16_CACHE",
         "INT8_CHANNEL"]


def filled(mode, lens, H, D, bs, headwise, seed=0, rht=True, stale=0xFF):
    """A cache whose unwritten bytes are `stale`, with rows of `lens` tokens; the rows as fp32; the paging state."""
    K = kvq()
    pag, blocks = paging(lens, H, bs, headwise, seed=seed)
    c = make_cache(mode, H, D, bs, blocks, seed, rht and mode != "INT8_CHANNEL")
    c.k_pages.fill_(stale)
    c.v_pages.fill_(stale)
    T = sum(lens)
    if T:
        k, v = rows(seed + 1, T, H, D), rows(seed + 2, T, H, D)
        k[:, :, D // 3] *= 6  # an outlier channel
        v[:, :, 5] += 0.5     # values whose mean is not zero
        K.kvq_write(c, pag, k, v, cu_of(lens))
        k, v = K.kvq_gather(c, pag, cu_of(lens), T)
    else:
        k = v = torch.zeros((0, H, D), device="cuda")
    return c, pag, k, v


def run(c, pag, q, n, scale, most=None, **kw):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full(q.shape, 7.0, device="cuda")
    got = kvq().kvq_cross_attn(c, pag, q, cu_of(n), max(n) if most is None else most, scale, out=out, dev_error=err, **kw)
    torch.cuda.synchronize()
    assert got is out
    return out, int(err.item())


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("D,bs,headwise,dtype", [(128, 16, False, torch.bfloat16), (64, 64, True, torch.float32),
                                                 (128, 32, True, torch.float32), (64, 16, False, torch.bfloat16)])
@pytest.mark.parametrize("G,n", [(1, (1, 0, 1, 1, 1)), (4, (2, 1, 0, 2, 1)), (3, (5, 1, 9, 0, 2)), (8, (1, 1, 1, 1, 1)),
                                 (5, (30, 100, 1, 0, 26)), (2, (0, 64, 65, 129, 3))])
def test_cross_modes(mode, D, bs, headwise, dtype, G, n):
    """Few queries (the decode kernels) and many, lengths of none to several tiles, ends inside a page."""
    H, lens = 2, [300, 17, 64, 1, 0]
    c, pag, k, v = filled(mode, lens, H, D, bs, headwise, seed=G)
    q = rows(20 + G, sum(n) + 2, H * G, D, dtype=dtype)  # two rows behind the last sequence
    out, err = run(c, pag, q, n, D ** -0.5)
    ref.check(out, q, k, v, n, lens, D ** -0.5)
    assert err == 0 and (out[sum(n):] == 7).all()
    at = sum(n[:4])
    assert not out[at:sum(n)].any()  # a source of length 0


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("G,n", [(4, (1, 2, 1)), (4, (70, 1, 33))])
def test_cross_evicted_pages(mode, G, n):
    """Holes, a last page without an entry, and a row whose mask leaves nothing: what they held is never seen."""
    H, D, bs, lens = 2, 128, 16, [200, 150, 90]
    c, pag, k, v = filled(mode, lens, H, D, bs, True, seed=3)
    t = pag.block_tables_headwise.view(3, H, -1)
    t[0, 0, 2:5] = -1
    t[0, 1, 12] = -1
    t[1, 0] = -1
    t[2, 1, 0] = -1
    tab = t.cpu().numpy()
    q = rows(4, sum(n), H * G, D)
    out, err = run(c, pag, q, n, D ** -0.5)
    ref.check(out, q, k, v, n, lens, D ** -0.5, seen=lambda b: np.stack([tab[b, h][np.arange(lens[b]) // bs] >= 0 for h in range(H)]))
    assert err == 0
    assert not out[n[0]:n[0] + n[1], :G].any()


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("D", [64, 128])
def test_cross_ragged_batch(mode, D):
    """More query tiles than the card runs at once, sources of many key tiles whose last is partly filled."""
    H, G, bs, lens, n = 4, 4, 32, [1500, 900, 33, 4500, 700, 1281, 2305], [330, 70, 300, 128, 64, 401, 95]
    c, pag, k, v = filled(mode, lens, H, D, bs, False, seed=31)
    q = rows(32, sum(n), H * G, D)
    out, err = run(c, pag, q, n, D ** -0.5)
    ref.check(out, q, k, v, n, lens, D ** -0.5)
    assert err == 0


@pytest.mark.parametrize("mode", ["INT4_TOKEN_HEAD", "INT2_TOKEN_HEAD", "FP8_TOKEN_HEAD", "BF16_CACHE"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [(2,), (40,), (300,)])
def test_cross_one_long_source(mode, dtype, n):
    """Keys cut into parts over the whole card, and joined."""
    H, G, D, lens = 1, 4, 128, [20011]
    c, pag, k, v = filled(mode, lens, H, D, 64, False, seed=9)
    q = rows(5, sum(n), H * G, D, dtype=dtype)
    out, err = run(c, pag, q, n, D ** -0.5)
    ref.check(out, q, k, v, n, lens, D ** -0.5)
    assert err == 0


@pytest.mark.parametrize("mode", ["INT8_TOKEN_HEAD", "FP8_TOKEN_HEAD"])
@pytest.mark.parametrize("n", [(2, 1), (60, 9)])
@pytest.mark.parametrize("size", [1e-20, 1e-3, 1.0, 3000.0])
def test_cross_value_sizes(mode, n, size):
    """8-bit rows whose scales are far from 1, growing along the sequence by eight orders."""
    K = kvq()
    H, G, D, bs, lens = 1, 3, 64, 16, [400, 70]
    pag, blocks = paging(lens, H, bs, False)
    c = make_cache(mode, H, D, bs, blocks, rht=False)
    T = sum(lens)
    k, v = rows(1, T, H, D), rows(2, T, H, D) * size
    v[:200] *= torch.logspace(-8, 0, 200, device="cuda")[:, None, None]
    v[390:400] = 0  # rows of zeros: a scale of 0
    K.kvq_write(c, pag, k, v, cu_of(lens))
    k, v = K.kvq_gather(c, pag, cu_of(lens), T)
    q = rows(3, sum(n), H * G, D)
    out, err = run(c, pag, q, n, D ** -0.5)
    ref.check(out / size, q, k, v / size, n, lens, D ** -0.5)
    assert err == 0


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
@pytest.mark.parametrize("mode", ["INT4_TOKEN_HEAD", "BF16_CACHE"])
def test_cross_scales(mode, scale):
    H, G, D, lens, n = 1, 2, 64, [200, 31], (40, 3)
    c, pag, k, v = filled(mode, lens, H, D, 16, False, seed=2)
    q = rows(6, sum(n), H * G, D)
    out, err = run(c, pag, q, n, scale)
    ref.check(out, q, k, v, n, lens, scale)
    assert err == 0


@pytest.mark.parametrize("mode", ["INT4_TOKEN_HEAD", "BF16_CACHE"])
@pytest.mark.parametrize("n", [(1, 2, 1), (50, 20, 9)])
def test_cross_flags(mode, n):
    K = kvq()
    H, G, D, lens = 1, 4, 128, [100, 40, 33]
    c, pag, k, v = filled(mode, lens, H, D, 16, False, seed=4)
    q = rows(7, sum(n), H * G, D)
    good, err = run(c, pag, q, n, 0.1)
    assert err == 0
    # more queries than max_q_per_seq: the first ones are served
    if max(n) == 50:
        out, err = run(c, pag, q, n, 0.1, most=20)
        assert err == K.KVQ_DEVERR_SEQ_LEN
        for a, m in ((0, 50), (50, 20), (70, 9)):
            assert torch.allclose(out[a:a + min(m, 20)], good[a:a + min(m, 20)], rtol=1e-4, atol=1e-5)
        assert (out[20:50] == 7).all()
    # rows of q that are not there
    e = torch.zeros(1, dtype=torch.int32, device="cuda")
    part = torch.full((sum(n) - 1, H * G, D), 7.0, device="cuda")
    K.kvq_cross_attn(c, pag, q[:-1].contiguous(), cu_of(n), max(n), 0.1, out=part, dev_error=e)
    assert int(e.item()) == K.KVQ_DEVERR_SEQ_LEN and torch.equal(part, good[:-1])
    # a negative length, one past the table, an entry past the pool
    for lens2, entry, bit in (([100, -3, 33], None, K.KVQ_DEVERR_SEQ_LEN), ([100, 40, 5000], None, K.KVQ_DEVERR_TABLE_RANGE),
                              ([100, 40, 33], 10 ** 6, K.KVQ_DEVERR_BLOCK_RANGE)):
        t = pag.block_tables.clone()
        if entry:
            t[1, 1] = entry
        p2 = K.Paging(i32(lens2), block_tables=t)
        out, err = run(c, p2, q, n, 0.1)
        assert err == bit
        assert torch.equal(out[:n[0]], good[:n[0]])
        if lens2[1] < 0:
            assert not out[n[0]:n[0] + n[1]].any()


def dense(k, v, start, lens, q, n, scale, most=None, **kw):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full(q.shape, 7.0, device="cuda")
    kvq().kvq_cross_dense_attn(k, v, i32(start), i32(lens), q, cu_of(n), max(n) if most is None else most, scale, out=out,
                               dev_error=err, **kw)
    torch.cuda.synchronize()
    return out, int(err.item())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("G,n", [(1, (1, 1, 0, 2, 1, 1)), (8, (1, 3, 16, 0, 17, 2)), (3, (42, 43, 85, 86, 1, 0)),
                                 (4, (300, 1, 64, 65, 0, 7))])
def test_dense(D, dtype, G, n):
    """Lengths about the tile's 128 keys, rows behind each sequence that hold NaN."""
    H, lens = 2, [127, 1, 128, 0, 129, 500]
    room = [x + 3 for x in lens]
    start = np.concatenate([[0], np.cumsum(room)]).tolist()
    k, v = (rows(s, start[-1], H, D, dtype=torch.bfloat16) for s in (1, 2))
    k[:, :, 9] *= 6
    for b, L in enumerate(lens):
        k[start[b] + L:start[b + 1]] = float("nan")
        v[start[b] + L:start[b + 1]] = float("nan")
    q = rows(3, sum(n) + 3, H * G, D, dtype=dtype)
    out, err = dense(k, v, start, lens, q, n, D ** -0.5)
    ref.check(out, q, k, v, n, lens, D ** -0.5, start=start)
    assert err == 0 and (out[sum(n):] == 7).all()


@pytest.mark.parametrize("n", [(1,), (130,), (513,)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_dense_long(n, dtype):
    H, G, D, lens = 2, 2, 128, [30011]
    k, v = (rows(s, lens[0], H, D, dtype=torch.bfloat16) for s in (1, 2))
    q = rows(3, sum(n), H * G, D, dtype=dtype)
    out, err = dense(k, v, [0, lens[0]], lens, q, n, D ** -0.5)
    ref.check(out, q, k, v, n, lens, D ** -0.5)
    assert err == 0


def test_dense_skipped_sequences():
    """Rows that are not there: fewer than the length, before the first, past the last."""
    K = kvq()
    H, G, D = 1, 4, 64
    k = rows(1, 300, H, D, dtype=torch.bfloat16)
    q = rows(2, 12, H * G, D)
    good, err = dense(k, k, [0, 100, 200, 300], [100, 100, 100], q, (4, 4, 4), 0.1)
    assert err == 0
    for start, lens in (([0, 100, 200, 300], [100, 101, 100]), ([0, 250, 250, 350], [100, 0, 100])):
        out, err = dense(k, k, start, lens, q, (4, 4, 4), 0.1)
        assert err == K.KVQ_DEVERR_SEQ_LEN and torch.equal(out[:4], good[:4])
    out, err = dense(k, k, [-50, 100, 200, 300], [100, 100, 100], q, (4, 4, 4), 0.1)
    assert err == K.KVQ_DEVERR_SEQ_LEN and (out[:4] == 7).all() and torch.equal(out[4:], good[4:])
    out, err = dense(k, k, [0, 100, 200, 300], [100, -1, 100], q, (4, 4, 4), 0.1)
    assert err == K.KVQ_DEVERR_SEQ_LEN and not out[4:8].any()


def test_dense_and_pages_agree():
    """The same rows by pages, by a gather, and dense: one encoder's states, several ways to them."""
    K = kvq()
    H, G, D, lens, n = 2, 4, 128, [700, 90, 33], (60, 5, 0)
    c, pag, _, _ = filled("BF16_CACHE", lens, H, D, 16, False, seed=8)
    q = rows(9, sum(n), H * G, D, dtype=torch.bfloat16)
    cu = cu_of(lens)
    kd, vd = K.kvq_gather(c, pag, cu, sum(lens), torch.bfloat16)
    paged, _ = run(c, pag, q, n, 0.09)
    flat, _ = dense(kd, vd, cu.tolist(), lens, q, n, 0.09)
    ref.check(paged, q, kd, vd, n, lens, 0.09)
    ref.check(flat, q, kd, vd, n, lens, 0.09)


def test_encoder_decoder_as_used():
    """An encoder's states written once; a prompt's queries, then captured decode steps of two beams per source, on a
    stream of their own while another call with a workspace of its own runs."""
    K = kvq()
    H, G, D, lens = 2, 4, 64, [333, 48]
    c, pag, k, v = filled("INT4_TOKEN_HEAD", lens, H, D, 16, False, seed=6)
    q0 = rows(1, 70, H * G, D, dtype=torch.bfloat16)
    out, _ = run(c, pag, q0, (30, 40), D ** -0.5)
    ref.check(out, q0, k, v, (30, 40), lens, D ** -0.5)
    q = rows(2, 4, H * G, D, dtype=torch.bfloat16)
    cu = cu_of((2, 2))
    ws = [torch.empty(K.kvq_cross_workspace_size(c, pag, H * G, 2), dtype=torch.uint8, device="cuda") for _ in range(2)]
    res = [torch.empty((4, H * G, D), device="cuda") for _ in range(2)]
    K.kvq_cross_attn(c, pag, q, cu, 2, D ** -0.5, out=res[0], workspace=ws[0])
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            K.kvq_cross_attn(c, pag, q, cu, 2, D ** -0.5, out=res[i], workspace=ws[i])
        graphs.append(g)
    s = torch.cuda.Stream()
    for step in range(3):
        q.copy_(rows(30 + step, 4, H * G, D, dtype=torch.bfloat16))
        s.wait_stream(torch.cuda.current_stream())
        graphs[0].replay()
        with torch.cuda.stream(s):
            graphs[1].replay()
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        ref.check(res[0], q, k, v, (2, 2), lens, D ** -0.5)
        assert torch.equal(res[0], res[1])


@pytest.mark.parametrize("mode", ["INT4_TOKEN_HEAD", "INT8_CHANNEL", "BF16_CACHE"])
@pytest.mark.parametrize("n", [(2, 1), (90, 33)])
def test_cross_captured_over_a_cache_that_changes(mode, n):
    """A captured call answers with the lengths, tables, rows and queries of each replay, its parts' records in a
    workspace of its own; the step after it writes into the pages that it reads."""
    K = kvq()
    H, G, D, lens = 2, 4, 128, [1500, 700]
    c, pag, k, v = filled(mode, lens, H, D, 16, False, seed=12)
    q = rows(3, sum(n), H * G, D, dtype=torch.bfloat16)
    cu = cu_of(n)
    ws = torch.empty(max(1, K.kvq_cross_workspace_size(c, pag, H * G, max(n))), dtype=torch.uint8, device="cuda")
    res = torch.empty((sum(n), H * G, D), device="cuda")
    K.kvq_cross_attn(c, pag, q, cu, max(n), D ** -0.5, out=res, workspace=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        K.kvq_cross_attn(c, pag, q, cu, max(n), D ** -0.5, out=res, workspace=ws)
    for step in range(3):
        now = [lens[0] - 129 * step, lens[1] - 333 * step]
        pag.seq_lens.copy_(i32(now))
        q.copy_(rows(40 + step, sum(n), H * G, D, dtype=torch.bfloat16))
        kk, vv = K.kvq_gather(c, pag, cu_of(now), sum(now))
        g.replay()
        if mode != "INT8_CHANNEL":  # behind it, into its last rows
            one = rows(50 + step, 2, H, D), rows(60 + step, 2, H, D)
            K.kvq_write_decode_attn(c, pag, *one, i32([0, 1, 2]), rows(70, 2, H * G, D), D ** -0.5)
        torch.cuda.synchronize()
        ref.check(res, q, kk, vv, n, now, D ** -0.5)


def test_dense_captured_beside_itself():
    """Two captured calls, each with its own workspace, on two streams at once, over lengths that change."""
    K = kvq()
    H, G, D, n, lens = 2, 4, 64, (70, 5), [900, 1400]
    k, v = (rows(5 + i, sum(lens), H, D, dtype=torch.bfloat16) for i in range(2))
    q, cu, ck = rows(9, sum(n), H * G, D, dtype=torch.bfloat16), cu_of(n), cu_of(lens)
    L = i32(lens)
    ws = [torch.empty(max(1, K.kvq_cross_dense_workspace_size(k, L, H * G, max(n))), dtype=torch.uint8, device="cuda") for _ in range(2)]
    res = [torch.empty((sum(n), H * G, D), device="cuda") for _ in range(2)]
    K.kvq_cross_dense_attn(k, v, ck, L, q, cu, max(n), D ** -0.5, out=res[0], workspace=ws[0])
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i, g in enumerate(graphs):
        with torch.cuda.graph(g):
            K.kvq_cross_dense_attn(k, v, ck, L, q, cu, max(n), D ** -0.5, out=res[i], workspace=ws[i])
    s = torch.cuda.Stream()
    for step in range(3):
        now = [lens[0] - 300 * step, lens[1] - 17 * step]
        L.copy_(i32(now))
        s.wait_stream(torch.cuda.current_stream())
        graphs[0].replay()
        with torch.cuda.stream(s):
            graphs[1].replay()
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        ref.check(res[0], q, k, v, n, now, D ** -0.5, start=[0, lens[0]])
        assert torch.equal(res[0], res[1])


def test_cross_binding_refusals():
    K = kvq()
    c, pag, _, _ = filled("BF16_CACHE", [20], 1, 64, 16, False)
    q = rows(1, 4, 2, 64)
    cu = cu_of((4,))
    with pytest.raises(ValueError, match="cu_q"):
        K.kvq_cross_attn(c, pag, q, cu[:1], 4, 0.1)
    with pytest.raises(ValueError, match="64"):
        K.kvq_cross_attn(c, pag, rows(1, 4, 2, 128), cu, 4, 0.1)
    with pytest.raises(ValueError, match="out"):
        K.kvq_cross_attn(c, pag, q, cu, 4, 0.1, out=torch.empty((2, 2, 64), device="cuda"))
    with pytest.raises(ValueError, match="q must"):
        K.kvq_cross_attn(c, pag, q.view(4, 128), cu, 4, 0.1)
    win = K.Paging(pag.seq_lens, block_tables=pag.block_tables, window_per_kv_head=i32([8]))
    with pytest.raises(K.KvqError, match="window"):
        K.kvq_cross_attn(c, win, q, cu, 4, 0.1)
    k = rows(1, 20, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="bfloat16"):
        K.kvq_cross_dense_attn(k.float(), k.float(), cu, pag.seq_lens, q, cu, 4, 0.1)
    with pytest.raises(ValueError, match="cu_kv"):
        K.kvq_cross_dense_attn(k, k, cu[:1], pag.seq_lens, q, cu, 4, 0.1)
