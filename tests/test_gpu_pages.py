"""kvq_copy_pages, kvq_fork and kvq_compact against plain sequential code, bit
for bit: tables, lengths, counts and every byte of every layer's pools."""
import numpy as np
import pytest
import torch

import decode16_ref
import pages_ref as ref
from harness import kvq

pytestmark = pytest.mark.gpu


def caches(blocks, Hkv, bs, modes=("INT4_TOKEN_HEAD", "BF16_CACHE", "INT2_TOKEN_HEAD"), dims=(64, 128, 64), seed=0):
    K = kvq()
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    out = []
    for m, d in zip(modes, dims):
        c = K.PagedCache(getattr(K, "KVQ_" + m), blocks, Hkv, bs, d)
        for p in (c.k_pages, c.v_pages):
            p.copy_(torch.randint(0, 256, p.shape, generator=g, device="cuda", dtype=torch.uint8))
        out.append(c)
    return out


def pools(cs):
    return [p.cpu().numpy().copy() for c in cs for p in (c.k_pages, c.v_pages)]


def apply(before, copies, headwise):
    want = [p.copy() for p in before]
    for w, b in zip(want, before):
        for s, src, dst in copies:
            if headwise:
                w[dst, s] = b[src, s]
            else:
                w[dst] = b[src]
    return want


def same(got, want):
    assert all(np.array_equal(a, b) for a, b in zip(got, want))


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def paging(table, lens, headwise):
    K = kvq()
    t = i32(np.asarray(table).reshape(-1, np.asarray(table).shape[-1]))
    return K.Paging(i32(lens), **({"block_tables_headwise": t} if headwise else {"block_tables": t}))


def rows(r, B, S, width, nb, bs, shared, holes=0.05):
    """Random rows: some share the first pages of the row before, some entries are -1 and some point past the pool."""
    lens = r.integers(0, width * bs + 1, B)
    table = np.full((B, S, width), -1)
    for s in range(S):
        perm, o = r.permutation(nb), 0
        for b in range(B):
            n = -(-int(lens[b]) // bs)
            k = min(n, -(-int(lens[b - 1]) // bs)) if b and r.random() < shared else 0
            k = int(r.integers(0, k + 1))
            table[b, s, :k] = table[b - 1, s, :k]
            m = min(n - k, nb - o)
            table[b, s, k:k + m] = perm[o:o + m]
            o += m
    table[r.random(table.shape) < holes] = -1
    return table, lens


@pytest.mark.parametrize("headwise", [False, True])
@pytest.mark.parametrize("blocks,pairs,Hkv,bs", [(5, 1, 1, 16), (64, 20, 3, 16), (300, 150, 2, 64), (5000, 2400, 1, 32)])
def test_copy_pages(blocks, pairs, Hkv, bs, headwise):
    K = kvq()
    cs = caches(blocks, Hkv, bs)
    units = blocks * (Hkv if headwise else 1)
    r = np.random.default_rng(blocks + pairs)
    order = r.permutation(units)
    src, dst = order[:pairs], order[pairs:2 * pairs]
    before, err = pools(cs), torch.zeros(1, dtype=torch.int32, device="cuda")
    K.kvq_copy_pages(cs, i32(src), i32(dst), headwise=headwise, dev_error=err)
    split = lambda u: (u % Hkv, u // Hkv) if headwise else (0, u)  # noqa: E731
    same(pools(cs), apply(before, [(split(a)[0], split(a)[1], split(b)[1]) for a, b in zip(src, dst)], False)
         if not headwise else _flat(before, list(zip(src, dst))))
    assert int(err.item()) == 0


def _flat(before, pairs):
    want = [p.copy() for p in before]
    for w, b in zip(want, before):
        wf, bf = w.reshape(-1, *w.shape[2:]), b.reshape(-1, *b.shape[2:])
        for s, d in pairs:
            wf[d] = bf[s]
    return want


@pytest.mark.parametrize("seed", range(6))
def test_copy_pages_conflicts(seed):
    """Chains, cycles, a destination named twice, a page onto itself, numbers past the pool and negative ones."""
    K = kvq()
    r = np.random.default_rng(seed)
    blocks = 40
    n = int(r.integers(1, 60))
    src, dst = r.integers(-2, blocks + 3, n), r.integers(-2, blocks + 3, n)
    layers = 1 if seed % 2 else 3   # runs of copy steps that span pairs, or stay within one
    cs = caches(blocks, 2, 16, ("INT4_TOKEN_HEAD", "BF16_CACHE", "INT2_TOKEN_HEAD") * layers, (64, 128, 64) * layers, seed=seed)
    before, err = pools(cs), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.full((K.kvq_copy_workspace_size(cs, n),), 0x5A, dtype=torch.uint8, device="cuda")
    K.kvq_copy_pages(cs, i32(src), i32(dst), workspace=ws, dev_error=err)
    done, bits = ref.copy_pairs(src, dst, blocks)
    same(pools(cs), apply(before, [(0, a, b) for a, b in done], False))
    assert int(err.item()) == bits


FORK = [  # rows, new rows, spaces, width, blocks, bs
    (1, 1, 1, 1, 1, 16), (4, 4, 1, 7, 40, 16), (4, 9, 1, 5, 60, 32), (6, 3, 3, 9, 70, 16), (33, 40, 2, 130, 9000, 64),
    (12, 17, 1, 4, 25, 16), (300, 1100, 1, 3, 5000, 16)]


@pytest.mark.parametrize("shape", FORK)
@pytest.mark.parametrize("seed", range(3))
def test_fork(shape, seed):
    K = kvq()
    B, n, S, width, nb, bs = shape
    r = np.random.default_rng(seed * 100 + B)
    headwise = S > 1
    table, lens = rows(r, B, S, width, nb, bs, 0.5)
    parents = r.integers(-1, B, n)
    new = r.choice([0, 0, 1, 2, bs, 3 * bs], n)
    keep = r.integers(0, width * bs + 1, n) if seed else None
    pins = (r.random((S, nb)) < 0.1).astype(np.int32) * 2 if seed == 2 else None
    if seed == 2:
        parents[0], lens[0] = B + 3, width * bs + 5
        table[-1, 0, 0] = nb + 1
        new[-1] = -4
    cs = caches(nb, S if headwise else 2, bs, seed=seed)
    before, err = pools(cs), torch.zeros(1, dtype=torch.int32, device="cuda")
    opt = lambda x: None if x is None else i32(x)  # noqa: E731
    out, refs = K.kvq_fork(cs, paging(table, lens, headwise), i32(parents), new_tokens=i32(new), keep_tokens=opt(keep),
                           pins=opt(pins), dev_error=err)
    t, L, want, copies, bits = ref.fork(table, lens, parents, nb, bs, width, S, keep, new, pins)
    got = (out.block_tables_headwise if headwise else out.block_tables).cpu().numpy()
    assert np.array_equal(got.reshape(n, S, width), t)
    assert np.array_equal(out.seq_lens.cpu().numpy(), L)
    assert np.array_equal(refs.cpu().numpy(), want)
    same(pools(cs), apply(before, copies, headwise))
    assert int(err.item()) == bits


def test_fork_without_old_rows_and_until_the_pool_is_empty():
    K = kvq()
    cs = caches(10, 2, 16)
    out = paging(np.zeros((3, 1, 6), np.int64), [7, 7, 7], False)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got, refs = K.kvq_fork(cs, None, i32([-1, -1, 0]), new_tokens=i32([40, 17, 5]), out=out, dev_error=err)
    assert got is out and int(err.item()) == K.KVQ_DEVERR_ROW_RANGE   # there is no row 0 yet
    assert out.block_tables.cpu().tolist() == [[0, 1, 2, -1, -1, -1], [3, 4, -1, -1, -1, -1], [-1] * 6]
    assert out.seq_lens.cpu().tolist() == [40, 17, 0] and refs.cpu().tolist() == [[1] * 5 + [0] * 5]
    # four rows continue row 0, one row 1: three copies of page 2 and pages for 17 more tokens each; too few are left
    err.zero_()
    got, refs = K.kvq_fork(cs, out, i32([0, 0, 0, 0, 1]), new_tokens=i32([17, 17, 17, 17, 0]), dev_error=err)
    assert int(err.item()) == K.KVQ_DEVERR_NO_PAGES
    t = got.block_tables.cpu().tolist()
    assert t == [[0, 1, 2, 5, -1, -1], [0, 1, 6, 7, -1, -1], [0, 1, 8, 9, -1, -1], [0, 1, -1, -1, -1, -1], [3, 4, -1, -1, -1, -1]]
    assert refs.cpu().tolist() == [[4, 4] + [1] * 8]
    # every row ends: every page is free again
    _, refs = K.kvq_fork(cs, got, i32([-1, -1]))
    assert not refs.any()


COMPACT = [(1, 1, 1, 1, 16), (3, 1, 6, 40, 16), (5, 3, 8, 60, 32), (40, 1, 100, 9001, 16), (64, 4, 33, 4097, 64), (2, 1, 3, 4, 16)]


@pytest.mark.parametrize("shape", COMPACT)
@pytest.mark.parametrize("seed", range(3))
@pytest.mark.parametrize("inplace", [False, True])
def test_compact(shape, seed, inplace):
    K = kvq()
    B, S, width, nb, bs = shape
    r = np.random.default_rng(seed * 7 + B)
    headwise = S > 1
    table, lens = rows(r, B, S, width, nb, bs, 0.3)
    pins = (r.random((S, nb)) < 0.05).astype(np.int32) * 3 - 1 if seed else None
    if seed == 2:
        lens[0], table[-1, 0, 0] = -3, nb
    cs = caches(nb, S if headwise else 1, bs, seed=seed)
    before, err = pools(cs), torch.zeros(1, dtype=torch.int32, device="cuda")
    p = paging(table, lens, headwise)
    out, page_map, refs, used = K.kvq_compact(cs, p, pins=None if pins is None else i32(pins), out=p if inplace else None,
                                              dev_error=err)
    t, m, want, n, copies, bits = ref.compact(table, lens, nb, bs, S, pins)
    got = (out.block_tables_headwise if headwise else out.block_tables).cpu().numpy()
    assert np.array_equal(got.reshape(t.shape), t)
    assert np.array_equal(page_map.cpu().numpy(), m) and np.array_equal(refs.cpu().numpy(), want)
    assert np.array_equal(used.cpu().numpy(), n)
    same(pools(cs), apply(before, copies, headwise))
    assert int(err.item()) == bits


def test_fork_and_compact_of_a_large_pool():
    """1.2 million pages: past what one cluster plans, every phase is a launch of its own."""
    K = kvq()
    nb, bs, width = 1200000, 16, 500
    cs = [K.PagedCache(K.KVQ_INT2_TOKEN_HEAD, nb, 1, bs, 64)]
    cs[0].k_pages.view(torch.int32).copy_(torch.arange(cs[0].k_pages.numel() // 4, device="cuda").view(cs[0].k_pages.view(torch.int32).shape))
    r = np.random.default_rng(3)
    B = 300
    lens = r.integers(1, width * bs, B)
    lens[::9] = 0
    need = -(-lens // bs)
    order, o = r.permutation(nb), 0
    table = np.full((B, 1, width), -1)
    for b in range(B):
        table[b, 0, :need[b]] = order[o:o + need[b]]
        o += need[b]
    parents = r.integers(0, B, 350)
    before = pools(cs)
    out, refs = K.kvq_fork(cs, paging(table, lens, False), i32(parents), new_tokens=i32(np.full(350, 3)))
    t, L, want, copies, _ = ref.fork(table, lens, parents, nb, bs, width, 1, None, np.full(350, 3))
    assert np.array_equal(out.block_tables.cpu().numpy(), t[:, 0]) and np.array_equal(refs.cpu().numpy(), want)
    mid = apply(before, copies, False)
    same(pools(cs), mid)
    got, page_map, refs, used = K.kvq_compact(cs, out)
    t, m, want, n, copies, _ = ref.compact(t, L, nb, bs, 1)
    assert np.array_equal(got.block_tables.cpu().numpy(), t[:, 0]) and np.array_equal(page_map.cpu().numpy(), m)
    assert np.array_equal(refs.cpu().numpy(), want) and used.cpu().tolist() == n.tolist()
    same(pools(cs), apply(mid, copies, False))


def test_page_calls_captured_and_on_another_stream():
    K = kvq()
    r = np.random.default_rng(1)
    table, lens = rows(r, 6, 1, 9, 80, 16, 0.5, 0)
    parents = i32([0, 0, 2, 5, 5, 5])
    cs = caches(80, 2, 16)
    p = paging(table, lens, False)
    before = pools(cs)
    t, L, want, copies, _ = ref.fork(table, lens, parents.cpu().numpy(), 80, 16, 9, 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, refs = K.kvq_fork(cs, p, parents, stream=side)
    side.synchronize()
    assert np.array_equal(out.block_tables.cpu().numpy(), t[:, 0]) and np.array_equal(refs.cpu().numpy(), want)
    same(pools(cs), apply(before, copies, False))
    # captured: fork, then the compaction of what it made; replayed from the same start
    graph, ws = torch.cuda.CUDAGraph(), torch.empty(K.kvq_fork_workspace_size(cs, p, 6), dtype=torch.uint8, device="cuda")
    with torch.cuda.graph(graph):
        K.kvq_fork(cs, p, parents, out=out, page_refs=refs, workspace=ws)
        got = K.kvq_compact(cs, out)
    for _ in range(2):
        for c, k, v in zip(cs, before[::2], before[1::2]):
            c.k_pages.copy_(torch.from_numpy(k))
            c.v_pages.copy_(torch.from_numpy(v))
        ws.fill_(0xFF)
        out.block_tables.fill_(12345)
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(out.block_tables.cpu().numpy(), t[:, 0])
        t2, m2, w2, n2, c2, _ = ref.compact(t, L, 80, 16, 1)
        assert np.array_equal(got[0].block_tables.cpu().numpy(), t2[:, 0]) and np.array_equal(got[1].cpu().numpy(), m2)
        same(pools(cs), apply(apply(before, copies, False), c2, False))


@pytest.mark.parametrize("headwise", [False, True])
def test_a_search_over_both_kinds_of_layers(headwise):
    """Prompts admitted, written and read; beams forked, advanced token by token, some dropped; the pool compacted: the
    attention over the moved pages stays what the sequences' own rows give."""
    K = kvq()
    Hkv, G, D, bs, nb, width = 2, 4, 128, 16, 64, 8
    r = np.random.Generator(np.random.PCG64(4))
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    full = K.PagedCache(K.KVQ_BF16_CACHE, nb, Hkv, bs, D)
    low = K.PagedCache(K.KVQ_INT8_TOKEN_HEAD, nb, Hkv, bs, D)
    cs = [full, low]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    S = Hkv if headwise else 1
    p = paging(np.full((2, S, width), -1), [0, 0], headwise)
    p, _ = K.kvq_fork(cs, p, i32([-1, -1]), new_tokens=i32([37, 64]), dev_error=err)
    hist = [torch.randn((2, n, Hkv, D), generator=g, device="cuda").bfloat16() for n in (37, 64)]

    def write(new):     # the last new[b] rows of each history
        k = torch.cat([h[0, h.shape[1] - n:] for h, n in zip(hist, new)])
        v = torch.cat([h[1, h.shape[1] - n:] for h, n in zip(hist, new)])
        cu = i32(np.concatenate([[0], np.cumsum(new)]))
        for c in cs:
            K.kvq_write(c, p, k, v, cu, dev_error=err)

    def check():
        q = torch.randn((len(hist), Hkv * G, D), generator=g, device="cuda").bfloat16()
        lens = np.array([h.shape[1] for h in hist])
        assert p.seq_lens.cpu().tolist() == lens.tolist()
        c = dict(k=torch.cat([h[0] for h in hist]), v=torch.cat([h[1] for h in hist]), q=q, lens=lens, D=D, G=G, bs=bs, Hkv=Hkv,
                 window=None, sink=0, scale=D ** -0.5,
                 table=(p.block_tables_headwise if headwise else p.block_tables).cpu().numpy().reshape(len(hist), S, width))
        want = decode16_ref.attention64(c)
        decode16_ref.check(K.kvq_decode_attn(full, p, q, D ** -0.5, dev_error=err), want)
        # 8-bit rows: half a step of amax / 127 per value; the keys' error moves a weight by scale |q|_1 step / 2
        got = K.kvq_decode_attn(low, p, q, D ** -0.5, dev_error=err).double().cpu().numpy()
        step = max(float(h.float().abs().max()) for h in hist) / 127
        dy = D ** -0.5 * float(q.float().abs().sum(2).max()) * step / 2
        vmax = float(torch.cat([h[1].float().abs().amax()[None] for h in hist]).max())
        assert np.abs(got - want[0]).max() <= step / 2 + 2 * np.expm1(2 * dy) * vmax

    write([37, 64])
    check()
    for parents, keep in [([0, 0, 0, 1, 1], None), ([2, 0, 4, 4, 1], None), ([3, 3, 0], [70, 30, 200]), ([2, 1], None)]:
        n = len(parents)
        p, refs = K.kvq_fork(cs, p, i32(parents), new_tokens=i32([1] * n), keep_tokens=None if keep is None else i32(keep),
                             dev_error=err)
        hist = [torch.cat([hist[b][:, :keep[i] if keep else None], torch.randn((2, 1, Hkv, D), generator=g, device="cuda").bfloat16()], 1)
                for i, b in enumerate(parents)]
        write([1] * n)
        check()
        p, _, refs2, used = K.kvq_compact(cs, p, out=p, dev_error=err)
        assert torch.equal(refs2.sort(1).values, refs.sort(1).values)
        assert int((p.block_tables_headwise if headwise else p.block_tables).max()) < int(used.max())
        check()
    assert int(err.item()) == 0


@pytest.mark.parametrize("n", [2048, 2049, 5000])
def test_copy_pages_conflicts_of_long_lists(n):
    """The same answers on both sides of the list length from which pages are claimed in scratch."""
    K = kvq()
    r = np.random.default_rng(n)
    blocks = 6000
    src, dst = r.integers(-1, blocks + 1, n), r.integers(-1, blocks + 1, n)
    src[::3] = r.permutation(blocks)[:len(src[::3])]
    layers = 10 if n == 5000 else 2
    cs = caches(blocks, 1, 16, ("INT2_TOKEN_HEAD", "INT4_TOKEN_HEAD") * (layers // 2), (64, 64) * (layers // 2))
    before, err = pools(cs), torch.zeros(1, dtype=torch.int32, device="cuda")
    K.kvq_copy_pages(cs, i32(src), i32(dst), dev_error=err)
    done, bits = ref.copy_pairs(src, dst, blocks)
    assert len(done) > 100 and bits & ref.CONFLICT
    same(pools(cs), apply(before, [(0, a, b) for a, b in done], False))
    assert int(err.item()) == bits


def test_copy_pages_of_small_and_large_pages_together():
    """Caches whose pages differ in size, small (laid end to end) and large (in pieces), and 128 caches at once."""
    K = kvq()
    r = np.random.default_rng(0)
    for Hkv, bs, modes, dims in [(1, 16, ("INT2_TOKEN_HEAD", "INT8_TOKEN_HEAD", "INT4_TOKEN_HEAD"), (64, 64, 128)),
                                 (3, 64, ("INT2_TOKEN_HEAD", "BF16_CACHE", "INT8_TOKEN_HEAD"), (64, 128, 64)),
                                 (1, 16, ("INT4_TOKEN_HEAD",) * 128, (64,) * 128)]:
        for headwise in (False, True):
            cs = caches(50, Hkv, bs, modes, dims)
            order = r.permutation(50 * (Hkv if headwise else 1))
            src, dst = order[:20], order[20:40]
            before = pools(cs)
            K.kvq_copy_pages(cs, i32(src), i32(dst), headwise=headwise)
            same(pools(cs), _flat(before, list(zip(src, dst))) if headwise else apply(before, [(0, a, b) for a, b in zip(src, dst)], False))


def test_pages_past_four_gigabytes():
    K = kvq()
    blocks, Hkv, bs, D = 150000, 8, 16, 128     # 4.9 GB a pool
    shape = (blocks, Hkv, bs, 2 * D)
    c = K.PagedCache(K.KVQ_BF16_CACHE, blocks, Hkv, bs, D, k_pages=torch.empty(shape, dtype=torch.uint8, device="cuda"),
                     v_pages=torch.empty(shape, dtype=torch.uint8, device="cuda"))
    for n, p in enumerate((c.k_pages, c.v_pages)):
        for i in (3, 149998):
            p[i] = torch.randint(0, 256, p[i].shape, dtype=torch.uint8, device="cuda")
    k, v = c.k_pages[149998].clone(), c.v_pages[3].clone()
    K.kvq_copy_pages(c, i32([149998, 3]), i32([7, 149999]))
    assert torch.equal(c.k_pages[7], k) and torch.equal(c.v_pages[149999], v)
    # two rows that end in page 149998, and their compaction to pages 0 and 1
    p = paging([[[149998]], [[149998]]], [9, 9], False)
    out, _ = K.kvq_fork(c, p, i32([1, 0]))
    assert out.block_tables.cpu().tolist() == [[149998], [0]]
    assert torch.equal(c.k_pages[0], k)
    out, _, _, used = K.kvq_compact(c, out)
    assert out.block_tables.cpu().tolist() == [[1], [0]] and used.item() == 2
    assert torch.equal(c.k_pages[1], k)


@pytest.mark.parametrize("big", [False, True])
def test_decode_right_behind_a_fork_and_a_compaction(big):
    """No wait, no other kernel between: the decode starts from the tables and lengths that the call before writes."""
    K = kvq()
    Hkv, G, D, bs, width = 2, 4, 128, 16, 9
    n = 40 if big else 4
    cs = caches(2000 if big else 60, Hkv, bs, ("BF16_CACHE",) * 3, (D,) * 3)
    full = cs[0]
    lens = np.array([100 + 3 * (i % 9) for i in range(n)])
    k = torch.randn((2, int(lens.sum()), Hkv, D), device="cuda").bfloat16()
    p = paging(np.full((n, 1, width), -1), np.zeros(n), False)
    p, _ = K.kvq_fork(cs, p, i32([-1] * n), new_tokens=i32(lens))
    K.kvq_write(full, p, k[0], k[1], i32(np.concatenate([[0], np.cumsum(lens)])))
    parents = np.arange(n)[::-1] // 2
    start = np.concatenate([[0], np.cumsum(lens)])
    hist = [k[:, start[b]:start[b + 1]] for b in parents]
    q = torch.randn((n, Hkv * G, D), device="cuda").bfloat16()
    par = i32(parents)
    new = paging(np.full((n, 1, width), 7), np.full(n, 5), False)     # wrong until the fork has run
    torch.cuda.synchronize()
    K.kvq_fork(cs, p, par, out=new)
    outs = [K.kvq_decode_attn(full, new, q, D ** -0.5)]
    K.kvq_compact(cs, new, out=new)
    outs.append(K.kvq_decode_attn(full, new, q, D ** -0.5))
    c = dict(k=torch.cat([h[0] for h in hist]), v=torch.cat([h[1] for h in hist]), q=q, lens=lens[parents], D=D, G=G, bs=bs,
             Hkv=Hkv, window=None, sink=0, scale=D ** -0.5, table=new.block_tables.cpu().numpy().reshape(n, 1, width))
    want = decode16_ref.attention64(c)
    for o in outs:
        decode16_ref.check(o, want)


def test_a_call_keeps_no_other_cache_alive():
    import weakref
    K = kvq()
    cs = caches(8, 1, 16)
    K.kvq_copy_pages(cs, i32([1]), i32([2]))
    gone = weakref.ref(cs[1].k_pages)
    del cs[1:]
    assert gone() is None
    # and a changed handle is seen
    new = torch.zeros_like(cs[0].k_pages)
    new[1] = 7
    cs[0].k_pages = new
    K.kvq_copy_pages(cs, i32([1]), i32([2]))
    assert bool((new[2] == 7).all())
