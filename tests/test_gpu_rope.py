"""Rotary positions on the GPU: kvq_rope against 64 bits, kvq_rope_write and kvq_rope_write_decode_attn against the
separate calls on the same rows (whose arithmetic they share, so every byte is the same; the step's outputs over 2-bit
and 8-bit rows, whose sums are closer, against 64 bits alone)."""
import math

import numpy as np
import pytest
import torch

import cross_ref
import rope_ref as ref
from harness import kvq

pytestmark = pytest.mark.gpu
MODES = ["INT4_TOKEN_HEAD", "INT2_TOKEN_HEAD", "INT4_STEGO", "INT8_TOKEN_HEAD", "FP8_TOKEN_HEAD", "BF16_CACHE"]


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def cu_of(n):
    return i32(np.concatenate([[0], np.cumsum(n)]).tolist())


def make_rope(rot, inter=False, scale=1.0, base=10000.0, factor=1.0):
    f = torch.tensor(ref.frequencies64(rot, base), device="cuda").float() / factor
    return kvq().Rope(f, interleaved=inter, scale=scale)


def rows(seed, *shape, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def check_turn(got, x, pos, rope):
    y = ref.turn64(x, pos, rope.inv_freq, rope.interleaved, rope.scale)
    t = ref.tolerance(x, y, rope.inv_freq, rope.interleaved, rope.scale, x.dtype)
    d = (got.cpu().double() - y).abs()
    assert (d <= t).all(), float((d / t.clamp(min=1e-300)).max())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 16), (64, 48), (64, 64), (128, 32), (128, 80), (128, 128)])
def test_rope_values(D, rot, inter, dtype):
    K = kvq()
    rope = make_rope(rot, inter, scale=1.0 if rot % 32 else 1.2079)
    pos = i32([0, 1, 2, 77, 8191, 131071, 1000003, 2 ** 31 - 1, -1, -4097, -2 ** 31])
    q, k = rows(rot, 11, 5, D, dtype=dtype), rows(rot + 1, 11, 2, D, dtype=dtype)
    qo, ko = K.kvq_rope(rope, q, k, positions=pos)
    check_turn(qo, q, pos, rope)
    check_turn(ko, k, pos, rope)
    assert torch.equal(qo[..., rot:], q[..., rot:])
    only, none = K.kvq_rope(rope, None, k, positions=pos)
    assert only is None and torch.equal(none, ko)


@pytest.mark.parametrize("tokens", [1, 5, 700, 5000])
@pytest.mark.parametrize("heads", [(1, 1), (32, 8), (7, 3)])
def test_rope_sizes(tokens, heads):
    """Every number of tokens per CTA, heads that do not fill its threads."""
    K = kvq()
    rope = make_rope(128, base=500000.0)
    n = [tokens // 3, 0, tokens - tokens // 3]
    past = [1000, 5, 0]
    lens = i32([a + b for a, b in zip(n, past)])
    q, k = rows(tokens, tokens, heads[0], 128, dtype=torch.bfloat16), rows(7, tokens, heads[1], 128, dtype=torch.bfloat16)
    qo, ko = K.kvq_rope(rope, q, k, lens, cu_of(n))
    pos = torch.cat([torch.arange(a, a + b) for a, b in zip(past, n)])
    check_turn(qo, q, pos, rope)
    check_turn(ko, k, pos, rope)


def test_rope_in_place_and_packed_rows():
    """q and k as slices of one packed projection, turned in place and out of it."""
    K = kvq()
    rope = make_rope(64, inter=True)
    T, Hq, Hk, D = 37, 6, 2, 64
    packed = rows(3, T, Hq + 2 * Hk, D, dtype=torch.bfloat16)
    before = packed.clone()
    q, k, v = packed[:, :Hq], packed[:, Hq:Hq + Hk], packed[:, Hq + Hk:]
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 31
    qo, ko = K.kvq_rope(rope, q, k, positions=pos)
    assert qo.is_contiguous() and torch.equal(packed, before)
    check_turn(qo, q, pos, rope)
    K.kvq_rope(rope, q, k, positions=pos, q_out=q, k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(v, before[:, Hq + Hk:])


def test_rope_there_and_back():
    """Keys moved to other positions: turned by the difference, backwards too."""
    K = kvq()
    rope = make_rope(128)
    x = rows(1, 9, 4, 128)
    there, _ = K.kvq_rope(rope, x, None, positions=i32([100] * 9))
    back, _ = K.kvq_rope(rope, there, None, positions=i32([-100] * 9))
    assert (back - x).abs().max() < 2 * 2.0 ** -21 * 2 * x.abs().max()


def test_rope_rows_behind_the_last_sequence_and_bad_lengths():
    K = kvq()
    rope = make_rope(64)
    q = rows(2, 12, 2, 64, dtype=torch.bfloat16)
    out = torch.full_like(q, 7)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    # 3 tokens of 10; 4 of a sequence of 2 (too many); 2 of 5; 3 rows of padding
    K.kvq_rope(rope, q, None, i32([10, 2, 5]), i32([0, 3, 7, 9]), q_out=out, dev_error=err)
    check_turn(out[:3], q[:3], torch.arange(7, 10), rope)
    check_turn(out[7:9], q[7:9], torch.arange(3, 5), rope)
    assert (out[3:7] == 7).all() and (out[9:] == 7).all()
    assert int(err.item()) == K.KVQ_DEVERR_SEQ_LEN


def test_rope_on_another_stream_and_captured():
    K = kvq()
    rope = make_rope(128)
    q, pos = rows(4, 64, 8, 128, dtype=torch.bfloat16), torch.arange(64, dtype=torch.int32, device="cuda")
    want, _ = K.kvq_rope(rope, q, None, positions=pos)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, _ = K.kvq_rope(rope, q, None, positions=pos, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        K.kvq_rope(rope, q, None, positions=pos, q_out=out)
    q.copy_(rows(5, 64, 8, 128, dtype=torch.bfloat16))
    pos.add_(1000)
    g.replay()
    torch.cuda.synchronize()
    check_turn(out, q, pos, rope)


# ---------------------------------------------------------------------------
# the write and the step, against the separate calls

def make_cache(mode, H, D, bs, blocks, seed=0, rht=True):
    K = kvq()
    m = getattr(K, "KVQ_" + mode)
    signs = None
    if rht and mode != "BF16_CACHE":
        signs = (torch.from_numpy(np.random.Generator(np.random.PCG64(seed)).integers(0, 2, D)).to("cuda") * 2 - 1).to(torch.int8)
    c = K.PagedCache(m, blocks, H, bs, D, signs)
    c.k_pages.fill_(0x5A)
    c.v_pages.fill_(0x5A)
    return c


def twin(c):
    K = kvq()
    return K.PagedCache(c.mode, c.num_blocks, c.num_kv_heads, c.block_size, c.head_dim, c.rht_signs,
                        k_pages=c.k_pages.clone(), v_pages=c.v_pages.clone())


def paging(lens, H, bs, headwise, seed=0, holes=False):
    K = kvq()
    r = np.random.Generator(np.random.PCG64(seed))
    width = max(1, max(-(-int(x) // bs) for x in lens))
    spaces, B = (H if headwise else 1), len(lens)
    blocks = B * width + 3
    t = np.stack([r.permutation(blocks)[: B * width].reshape(B, width) for _ in range(spaces)], 1)
    if holes:
        t[0, 0, 0] = -1
        t[-1, -1, -1] = -1
    t = torch.from_numpy(t.reshape(B * spaces, width).astype(np.int32)).to("cuda")
    kw = dict(block_tables_headwise=t) if headwise else dict(block_tables=t)
    return K.Paging(i32([int(x) for x in lens]), **kw), blocks


def turned(rope, x, lens, cu, positions):
    """x turned in fp32, unrounded."""
    y, _ = kvq().kvq_rope(rope, x.float().contiguous(), None, lens, cu, positions=positions)
    return y


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("D,rot,inter,dtype,headwise,explicit", [
    (128, 128, False, torch.bfloat16, False, False), (128, 48, False, torch.float32, True, False),
    (64, 64, True, torch.bfloat16, True, True), (64, 16, False, torch.float32, False, True),
    (128, 80, True, torch.bfloat16, False, False)])
@pytest.mark.parametrize("sizes", [(1, 33, 0, 7), (511,), (300, 1, 400), (1030, 5)])
def test_rope_write_is_rope_then_write(mode, D, rot, inter, dtype, headwise, explicit, sizes):
    """Both kernels (below and from 512 tokens), 16-bit rows, evicted pages, padded rows."""
    K = kvq()
    H = 3
    rope = make_rope(rot, inter, scale=1.1)
    lens = [n + p for n, p in zip(sizes, (5, 0, 17, 40))]
    pag, blocks = paging(lens, H, 16, headwise, holes=True)
    a = make_cache(mode, H, D, 16, blocks)
    b = twin(a)
    T = sum(sizes)
    k, v = rows(1, T + 6, H, D, dtype=dtype), rows(2, T + 6, H, D, dtype=dtype)  # six rows of padding behind
    cu = cu_of(sizes)
    pos = (torch.arange(T + 6, dtype=torch.int32, device="cuda") * 977 % 100003) if explicit else None
    err = torch.zeros(2, dtype=torch.int32, device="cuda")
    K.kvq_rope_write(a, pag, rope, k, v, cu, positions=pos, dev_error=err[:1])
    y = turned(rope, k, pag.seq_lens, cu, pos)
    K.kvq_write(b, pag, y, v.float(), cu, dev_error=err[1:])
    torch.cuda.synchronize()
    assert torch.equal(a.k_pages, b.k_pages) and torch.equal(a.v_pages, b.v_pages)
    assert err.tolist() == [0, 0]


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("D,rot,inter,G,dtype,headwise,explicit", [
    (128, 128, False, 4, torch.bfloat16, False, False), (64, 32, True, 1, torch.float32, True, False),
    (128, 96, False, 5, torch.float32, False, True), (64, 64, False, 8, torch.bfloat16, True, True)])
def test_rope_step_is_rope_then_step(mode, D, rot, inter, G, dtype, headwise, explicit):
    """Sequences with one new token, several and none; lengths from one token."""
    K = kvq()
    H, n, lens = 2, [1, 1, 3, 0, 1], [1, 300, 50, 20, 1000]
    rope = make_rope(rot, inter, scale=0.9)
    pag, blocks = paging(lens, H, 16, headwise)
    a = make_cache(mode, H, D, 16, blocks)
    cu, T = cu_of(n), sum(n)
    fill = cu_of(lens)
    K.kvq_write(a, pag, rows(8, sum(lens), H, D), rows(9, sum(lens), H, D), fill)
    b = twin(a)
    k, v, q = rows(1, T, H, D, dtype=dtype), rows(2, T, H, D, dtype=dtype), rows(3, len(n), H * G, D, dtype=dtype)
    pos = i32([5, 100000, 7, 8, 9, 3]) if explicit else None
    scale = 1 / math.sqrt(D)
    got = K.kvq_rope_write_decode_attn(a, pag, rope, k, v, cu, q, scale, positions=pos)
    at = [x - 1 for x in lens]
    if explicit:
        at = [5, 100000, 9, 19, 3]
    qt, _ = K.kvq_rope(rope, q.float(), None, positions=i32(at))
    want = K.kvq_write_decode_attn(b, pag, turned(rope, k, pag.seq_lens, cu, pos), v.float(), cu, qt, scale)
    torch.cuda.synchronize()
    assert torch.equal(a.k_pages, b.k_pages) and torch.equal(a.v_pages, b.v_pages)
    same = mode.startswith("INT4") or mode == "BF16_CACHE"
    kk, vv = K.kvq_gather(a, pag, fill, sum(lens))
    assert not same or torch.equal(got, want)
    cross_ref.check(got, qt, kk, vv, [1] * len(n), lens, scale)
    # no new tokens at all: the queries alone
    none = torch.zeros((0, H, D), dtype=dtype, device="cuda")
    got = K.kvq_rope_write_decode_attn(a, pag, rope, none, none, i32([0] * 6), q, scale)
    qt, _ = K.kvq_rope(rope, q.float(), None, positions=i32([x - 1 for x in lens]))
    assert not same or torch.equal(got, K.kvq_decode_attn(b, pag, qt, scale))
    cross_ref.check(got, qt, kk, vv, [1] * len(n), lens, scale)


@pytest.mark.parametrize("mode", ["INT8_TOKEN_HEAD", "BF16_CACHE"])
def test_rope_write_flags(mode):
    """A sequence with too many new tokens, a position past the table, an entry past the pool."""
    K = kvq()
    rope = make_rope(64)
    t = i32([[0, 1], [2, 3], [99, 4]])
    c = make_cache(mode, 1, 64, 16, 8)
    before = c.k_pages.clone()
    k = rows(1, 9, 1, 64)
    for lens, n, bit in (([2, 20, 3], [3, 0, 0], K.KVQ_DEVERR_SEQ_LEN), ([5, 40, 3], [0, 2, 0], K.KVQ_DEVERR_TABLE_RANGE),
                         ([5, 20, 3], [0, 0, 2], K.KVQ_DEVERR_BLOCK_RANGE), ([-1, 20, 3], [1, 0, 0], K.KVQ_DEVERR_SEQ_LEN)):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        K.kvq_rope_write(c, K.Paging(i32(lens), block_tables=t), rope, k, k, cu_of(n), dev_error=err)
        assert int(err.item()) == bit
        assert torch.equal(c.k_pages, before)


def test_prompt_then_steps_against_64_bits():
    """As a model uses them: a prompt turned, written and prefilled in two chunks, then steps in a captured graph."""
    K = kvq()
    H, G, D, bs, B = 2, 4, 128, 16, 3
    n0, steps = [40, 7, 90], 4
    rope = make_rope(128, base=500000.0)
    total = [n + steps for n in n0]
    pag, blocks = paging(total, H, bs, False, seed=5)
    cache = make_cache("BF16_CACHE", H, D, bs, blocks)
    cache.k_pages.fill_(0xFF)
    cache.v_pages.fill_(0xFF)
    k, v = (rows(s, sum(total), H, D, dtype=torch.bfloat16) for s in (11, 12))
    q = rows(13, sum(total), H * G, D, dtype=torch.bfloat16)
    base = np.concatenate([[0], np.cumsum(total)])
    first = torch.cat([torch.arange(base[b], base[b] + n0[b]) for b in range(B)]).cuda()
    scale = 1 / math.sqrt(D)
    pag.seq_lens = i32(n0)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = cu_of(n0)
    K.kvq_rope_write(cache, pag, rope, k[first], v[first], cu, dev_error=err)
    qt, _ = K.kvq_rope(rope, q[first], None, pag.seq_lens, cu)
    kd, vd = K.kvq_gather(cache, pag, cu, len(first), torch.bfloat16)
    out = [K.kvq_prefill_dense_attn(kd, vd, cu, pag.seq_lens, qt, cu, max(n0), scale, dev_error=err)]
    kin, vin, qin = (torch.zeros((B, h, D), dtype=torch.bfloat16, device="cuda") for h in (H, H, H * G))
    one = cu_of([1] * B)
    ws = torch.empty(K.kvq_decode_workspace_size(cache, pag, H * G)[0], dtype=torch.uint8, device="cuda")
    res = torch.empty((B, H * G, D), device="cuda")
    K.kvq_rope_write_decode_attn(cache, pag, rope, kin[:0], vin[:0], one * 0, qin, scale, out=res, workspace=ws)  # warm
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pag.seq_lens.add_(1)
        K.kvq_rope_write_decode_attn(cache, pag, rope, kin, vin, one, qin, scale, out=res, workspace=ws, dev_error=err)
    outs = []
    for s in range(steps):
        at = torch.tensor([base[b] + n0[b] + s for b in range(B)], device="cuda")
        kin.copy_(k[at])
        vin.copy_(v[at])
        qin.copy_(q[at])
        g.replay()
        outs.append(res.clone())
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    pos = torch.cat([torch.arange(t) for t in total])
    kt = ref.turn64(k, pos, rope.inv_freq, False).to(torch.bfloat16)  # (a rounding may fall the other way: below)
    qf = ref.turn64(q, pos, rope.inv_freq, False)
    for b in range(B):
        for s in range(steps):
            n = n0[b] + s + 1
            for h in range(H):
                rowsl = slice(base[b], base[b] + n)
                kk, vv = kt[rowsl, h].double().numpy(), v[rowsl, h].cpu().double().numpy()
                for i in range(G):
                    x = kk @ qf[base[b] + n - 1, h * G + i].numpy() * scale
                    p = np.exp(x - x.max())
                    p /= p.sum()
                    want = p @ vv
                    # a key element may round the other way (2^-8 of it, at a tie that the fp32 turn moves): at most
                    # one in 2^13 elements does, so one of them per logit, |q k| 2^-7 at most; the rest is the decode's
                    # own 1e-5, as in its tests
                    A = np.abs(kk * qf[base[b] + n - 1, h * G + i].numpy()).max() * scale
                    tol = 2 * (A * 2.0 ** -7 + 1e-5) * (p @ np.abs(vv))
                    d = np.abs(outs[s][b, h * G + i].cpu().double().numpy() - want)
                    assert (d <= tol).all()
    # the prompt's last queries see the whole prompt
    for b in range(B):
        n = n0[b]
        kk, vv = kt[base[b]:base[b] + n, 0].double().numpy(), v[base[b]:base[b] + n, 0].cpu().double().numpy()
        x = kk @ qf[base[b] + n - 1, 0].to(torch.bfloat16).double().numpy() * scale
        p = np.exp(x - x.max())
        p /= p.sum()
        A = np.abs(kk).max(0) @ np.abs(qf[base[b] + n - 1, 0].numpy()) * scale
        tol = 2 * (A * 2.0 ** -7 + 1e-5) * (p @ np.abs(vv))
        d = np.abs(out[0][sum(n0[:b + 1]) - 1, 0].cpu().double().numpy() - p @ vv)
        assert (d <= tol).all()
