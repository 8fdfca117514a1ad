"""Operator cases of the paged cache: 16-bit pages with the attention that
reads them, and the calls that copy, fork, free and compact pages.

Five operators, each reached through the Python binding's calls:

  decode   kvq_decode_attn over bf16 pages: one query per sequence
  step     kvq_write_decode_attn over bf16 pages: the step's new rows, then
           the same attention
  copy     kvq_copy_pages: (source, destination) pairs over every layer's pools
  fork     kvq_fork: new table rows from parent rows (beam search), shared full
           pages, a private copy of each partly filled last page, pages for the
           coming tokens, and the pages of rows without a child freed
  compact  kvq_compact: the used pages moved to the lowest page numbers, tables
           rewritten

``own`` False computes them with elementary torch operations, True calls the
package.  Lengths and parents follow from a case alone (so that its work is
known), page numbers and values from the seed.
"""
import math

import numpy as np
import torch

own = False

_DEV = "cuda"
_ROW = {"int4": lambda d: d // 2 + 4, "int2": lambda d: d // 4 + 4, "int8": lambda d: d + 4, "bf16": lambda d: 2 * d}


def listed():
    return [
        # one chat turn's first tokens, fp32 activations: nothing but latency
        dict(name="decode: one short sequence", op="decode", batch=1, hq=4, hkv=2, d=64, bs=16, lo=37, hi=37, qtype="f32",
             headwise=False, window=0, sink=0),
        # a serving batch of ragged contexts, grouped heads 4 : 1, 16-token pages
        dict(name="decode: 64 ragged sequences", op="decode", batch=64, hq=32, hkv=8, d=128, bs=16, lo=1024, hi=8192,
             qtype="bf16", headwise=False, window=0, sink=0),
        # half of the heads keep a window and sinks, their other pages evicted
        dict(name="decode: head-wise windows", op="decode", batch=32, hq=40, hkv=8, d=128, bs=64, lo=32768, hi=32768,
             qtype="bf16", headwise=True, window=4096, sink=4),
        # one long document: all of the card for four heads' keys
        dict(name="decode: one long sequence", op="decode", batch=1, hq=20, hkv=4, d=128, bs=64, lo=131071, hi=131071,
             qtype="bf16", headwise=False, window=0, sink=0),
        # a small batch's whole step: the new token's rows written, then read
        dict(name="step: 7 short sequences", op="step", batch=7, hq=32, hkv=8, d=128, bs=16, lo=1, hi=401, qtype="bf16",
             headwise=False, window=0, sink=0),
        # a large batch's step, grouped heads 5 : 1, 64-token pages
        dict(name="step: 96 ragged sequences", op="step", batch=96, hq=20, hkv=4, d=128, bs=64, lo=512, hi=8192,
             qtype="bf16", headwise=False, window=0, sink=0),
        # one sequence's last page duplicated by a host scheduler
        dict(name="copy: 3 pages of 2 layers", op="copy", layers=2, mode="int4", hkv=2, d=64, bs=16, blocks=64, pairs=3,
             headwise=False),
        # pages of many sequences moved at once in every layer of a model
        dict(name="copy: 1200 pages of 32 layers", op="copy", layers=32, mode="int4", hkv=8, d=128, bs=16, blocks=4001,
             pairs=1200, headwise=False),
        # one request's four beams
        dict(name="fork: 4 beams", op="fork", layers=2, mode="int4", hkv=2, d=64, bs=16, groups=1, beams=4, lo=100, hi=100,
             new=1, headwise=False),
        # a batch of beam searches, shared prefixes
        dict(name="fork: 64 searches of 4 beams", op="fork", layers=8, mode="int4", hkv=8, d=128, bs=16, groups=64, beams=4,
             lo=500, hi=4096, new=1, headwise=False),
        # a small cache after a few requests ended
        dict(name="compact: 3 sequences", op="compact", layers=2, mode="int2", hkv=4, d=128, bs=64, batch=3, lo=100, hi=900,
             used=0.4, headwise=False),
        # a fragmented pool of 16-bit pages, half in use
        dict(name="compact: 96 sequences", op="compact", layers=8, mode="bf16", hkv=4, d=128, bs=16, batch=96, lo=300,
             hi=1500, used=0.5, headwise=False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "step", "copy", "fork", "compact"])
    d, bs, hkv = rng.choice([64, 128]), rng.choice([16, 32, 64]), rng.choice([1, 2, 3, 4, 8])
    if op in ("decode", "step"):
        batch, group = _log(rng, 1, 96), rng.randint(1, 8)
        most = min(131072, (3 << 28) // (batch * hkv * d))
        if op == "step":
            most = min(most, (1 << 28) // (batch * hkv * d))
        hi = _log(rng, 1, most)
        lo = rng.choice([1, max(1, hi // 8), hi]) if op == "step" else rng.choice([0, max(1, hi // 8), hi])
        headwise = rng.random() < 0.3
        window = _log(rng, 1, hi) if headwise and rng.random() < 0.7 else 0
        return dict(op=op, batch=batch, hq=hkv * group, hkv=hkv, d=d, bs=bs, lo=lo, hi=hi,
                    qtype=rng.choice(["bf16", "bf16", "f32"]), headwise=headwise, window=window,
                    sink=rng.randint(0, 8) if window else 0)
    mode, layers = rng.choice(["int4", "int2", "int8", "bf16"]), _log(rng, 1, 32)
    unit = hkv * bs * _ROW[mode](d)
    pool_pages = (2 << 30) // (2 * layers * unit)
    headwise = rng.random() < 0.3
    if op == "copy":
        blocks = _log(rng, 8, max(8, min(100000, pool_pages)))
        return dict(op=op, layers=layers, mode=mode, hkv=hkv, d=d, bs=bs, blocks=blocks,
                    pairs=_log(rng, 1, max(1, (blocks * (hkv if headwise else 1)) // 2)), headwise=headwise)
    if op == "fork":
        groups, beams = _log(rng, 1, 64), rng.randint(1, 8)
        hi = _log(rng, 1, max(1, min(8192, pool_pages // (groups * (beams + 1)) * bs)))
        return dict(op=op, layers=layers, mode=mode, hkv=hkv, d=d, bs=bs, groups=groups, beams=beams,
                    lo=rng.choice([1, max(1, hi // 4), hi]), hi=hi, new=rng.choice([0, 1, 1, 5, 40]), headwise=headwise)
    batch = _log(rng, 1, 96)
    hi = _log(rng, 1, max(1, min(16384, pool_pages // (2 * batch) * bs)))
    return dict(op=op, layers=layers, mode=mode, hkv=hkv, d=d, bs=bs, batch=batch, lo=rng.choice([0, max(1, hi // 4), hi]),
                hi=hi, used=rng.choice([0.3, 0.5, 0.8]), headwise=headwise)


# ---------------------------------------------------------------------------
# inputs

def _lens(n, lo, hi):
    """Lengths spread over lo .. hi, odd ones among them: a case's own, whatever the seed."""
    f = np.modf(0.5 + np.arange(n) * 0.6180339887498949)[0]
    return (lo + np.floor((hi - lo + 1) * f)).astype(np.int64)


def _windows(case):
    """Per kv head: the upper half of the heads slide where the case has a window."""
    if not case["window"]:
        return None
    w = np.zeros(case["hkv"], np.int32)
    w[case["hkv"] // 2:] = case["window"]
    return w


def _evicted(case, lens, pages):
    """[batch, hkv, pages]: pages that hold neither sinks nor the window of the last position."""
    w = _windows(case)
    e = np.arange(pages)[None, None, :]
    if w is None:
        return np.zeros((len(lens), case["hkv"], pages), bool)
    first = (lens[:, None] - w[None, :])[:, :, None] // case["bs"]
    last_sink = (case["sink"] - 1) // case["bs"] if case["sink"] else -1
    return (w[None, :, None] > 0) & (e > last_sink) & (e < first)


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(_DEV)


def _spread(gen, counts, width, spaces, blocks):
    """[spaces, rows, width] tables: row r's first counts[r] entries are distinct pages of its space, the others -1."""
    order = torch.rand((spaces, blocks), generator=gen, device=_DEV).argsort(1).to(torch.int32)
    c = torch.from_numpy(counts).to(_DEV)
    at = (c.cumsum(0) - c)[:, None] + torch.arange(width, device=_DEV)[None, :]
    inside = torch.arange(width, device=_DEV)[None, :] < c[:, None]
    return torch.where(inside[None], order[:, at.clamp(max=blocks - 1)], -1)


def _bytes(gen, shape):
    n = math.prod(shape)
    return torch.randint(-2**62, 2**62, (n // 8 + 1,), generator=gen, device=_DEV).view(torch.uint8)[:n].view(shape).clone()


def _attention_state(case, gen):
    B, H, D, bs = case["batch"], case["hkv"], case["d"], case["bs"]
    lens = _lens(B, case["lo"], case["hi"])
    width = max(1, -(-case["hi"] // bs))
    counts = -(-lens // bs)
    blocks = int(counts.sum()) + int(counts.sum()) // 20 + 8
    spaces = H if case["headwise"] else 1
    table = _spread(gen, counts, width, spaces, blocks).permute(1, 0, 2)
    if case["headwise"]:
        table = torch.where(torch.from_numpy(_evicted(case, lens, width)).to(_DEV), -1, table)
    s = dict(table=table.reshape(B * spaces, width).contiguous(), lens=_i32(lens), blocks=blocks)
    for name in ("k", "v"):
        p = torch.randn((blocks, H, bs, D), generator=gen, device=_DEV, dtype=torch.bfloat16)
        hot = torch.randint(0, H * D, (max(1, H * D // 100),), generator=gen, device=_DEV)  # outlier channels
        p[:, hot // D, :, hot % D] *= 10
        s[name] = p
    t = torch.float32 if case["qtype"] == "f32" else torch.bfloat16
    s["q"] = torch.randn((B, case["hq"], D), generator=gen, device=_DEV, dtype=torch.float32).to(t)
    w = _windows(case)
    s["window"] = None if w is None else _i32(w)
    if case["op"] == "step":  # one new token per sequence, at its last position
        s["k_new"] = torch.randn((B, H, D), generator=gen, device=_DEV, dtype=torch.float32).to(t)
        s["v_new"] = torch.randn((B, H, D), generator=gen, device=_DEV, dtype=torch.float32).to(t)
        s["cu"] = _i32(np.arange(B + 1))
    return s


def _parents(case):
    """Beam search: each new row continues one of its group's rows, some twice or more and some not at all."""
    n, k = case["groups"], case["beams"]
    i = np.arange(n * k)
    return ((i // k) * k + (i * i * 3 + i // k) % k % max(1, k - 1)).astype(np.int64)


def _fork_lens(case):
    return np.repeat(_lens(case["groups"], case["lo"], case["hi"]), case["beams"])


def _fork_table(case, gen, spaces):
    """Rows of a group share their first pages (four fifths of the full ones); the rest is each row's own."""
    bs, k = case["bs"], case["beams"]
    lens = _lens(case["groups"], case["lo"], case["hi"])
    counts, shared = -(-lens // bs), (lens // bs) * 4 // 5
    width = max(1, -(-(case["hi"] + case["new"]) // bs))
    need = int((shared + k * (counts - shared)).sum())
    blocks = need + len(lens) * k * (1 + -(-case["new"] // bs)) + 8
    parts = np.concatenate([shared[:, None], np.repeat((counts - shared)[:, None], k, 1)], 1).reshape(-1)
    t = _spread(gen, parts, width, spaces, blocks).view(spaces, len(lens), k + 1, width)
    sh = torch.from_numpy(shared).to(_DEV)[None, :, None, None]
    e = torch.arange(width, device=_DEV).expand(spaces, len(lens), k, width)
    mine = t[:, :, 1:].gather(3, (e - sh).clamp(min=0))
    rows = torch.where(e < sh, t[:, :, :1], mine).reshape(spaces, len(lens) * k, width)
    return rows, blocks, need


def _page_state(case, gen):
    H, bs, R, L = case["hkv"], case["bs"], _ROW[case["mode"]](case["d"]), case["layers"]
    spaces = H if case["headwise"] else 1
    s = {}
    if case["op"] == "copy":
        blocks = case["blocks"]
        order = torch.rand(blocks * spaces, generator=gen, device=_DEV).argsort().to(torch.int32)
        s["src"], s["dst"] = order[:case["pairs"]].contiguous(), order[case["pairs"]:2 * case["pairs"]].contiguous()
    elif case["op"] == "fork":
        rows, blocks, _ = _fork_table(case, gen, spaces)
        n = case["groups"] * case["beams"]
        s["table"] = rows.permute(1, 0, 2).reshape(n * spaces, -1).contiguous()
        s["lens"], s["parents"] = _i32(_fork_lens(case)), _i32(_parents(case))
        s["new"] = _i32(np.full(n, case["new"]))
        s["table_out"], s["lens_out"] = torch.empty_like(s["table"]), torch.empty_like(s["lens"])
    else:
        lens = _lens(case["batch"], case["lo"], case["hi"])
        counts = -(-lens // bs)
        width = max(1, -(-case["hi"] // bs))
        blocks = int(math.ceil(max(1, int(counts.sum())) / case["used"]))
        s["table"] = _spread(gen, counts, width, spaces, blocks).permute(1, 0, 2).reshape(-1, width).contiguous()
        s["lens"], s["table_out"] = _i32(lens), torch.empty_like(s["table"])
    s["blocks"] = blocks
    s["pools"] = _bytes(gen, (L, 2, blocks, H, bs, R))
    return s


def prepare(case, seed):
    gen = torch.Generator(device=_DEV)
    gen.manual_seed(seed)
    attention = case["op"] in ("decode", "step")
    s = _attention_state(case, gen) if attention else _page_state(case, gen)
    s["case"] = case
    if own:  # the handles that a user's program keeps: the cache of each layer, the paging state and scratch
        import sub_byte_quantized_write_gb300 as K
        mode = {"int4": K.KVQ_INT4_TOKEN_HEAD, "int2": K.KVQ_INT2_TOKEN_HEAD, "int8": K.KVQ_INT8_TOKEN_HEAD,
                "bf16": K.KVQ_BF16_CACHE}["bf16" if attention else case["mode"]]
        shape = (s["blocks"], case["hkv"], case["bs"], case["d"])
        if attention:
            pools = [(s["k"].view(torch.uint8), s["v"].view(torch.uint8))]
        else:
            pools = [(s["pools"][i, 0], s["pools"][i, 1]) for i in range(case["layers"])]
        s["caches"] = [K.PagedCache(mode, *shape, k_pages=k, v_pages=v) for k, v in pools]
        tables = "block_tables_headwise" if case["headwise"] else "block_tables"
        if "table" in s:
            s["paging"] = K.Paging(s["lens"], window_per_kv_head=s.get("window"), sink_size=case.get("sink", 0),
                                   **{tables: s["table"]})
        if attention:
            n, _ = K.kvq_decode_workspace_size(s["caches"][0], s["paging"], case["hq"])
        elif case["op"] == "copy":
            n = K.kvq_copy_workspace_size(s["caches"], case["pairs"], case["headwise"])
        elif case["op"] == "fork":
            n = K.kvq_fork_workspace_size(s["caches"], s["paging"], s["parents"].shape[0])
            s["paging_out"] = K.Paging(s["lens_out"], **{tables: s["table_out"]})
        else:
            n = K.kvq_compact_workspace_size(s["caches"], s["paging"])
            s["paging_out"] = K.Paging(s["lens"], **{tables: s["table_out"]})
        s["ws"] = torch.empty(max(n, 256), dtype=torch.uint8, device=_DEV)
    return s


# ---------------------------------------------------------------------------
# the plain forms

def _plain_write(s):
    """The new rows into their pages; the step's token sits at the sequence's last position."""
    c = s["case"]
    H, bs = c["hkv"], c["bs"]
    pos = s["lens"].long() - 1
    b, h = torch.arange(c["batch"], device=_DEV)[:, None], torch.arange(H, device=_DEV)[None, :]
    row = b * H + h if c["headwise"] else b + 0 * h
    blk = s["table"][row, (pos // bs)[:, None]].long()
    b, h, blk = b.expand_as(blk)[blk >= 0], h.expand_as(blk)[blk >= 0], blk[blk >= 0]
    s["k"][blk, h, pos[b] % bs] = s["k_new"][b, h].to(torch.bfloat16)
    s["v"][blk, h, pos[b] % bs] = s["v_new"][b, h].to(torch.bfloat16)


def _plain_attention(s):
    c = s["case"]
    B, H, D, bs = c["batch"], c["hkv"], c["d"], c["bs"]
    M = s["table"].shape[1]
    table = s["table"].view(B, -1, M).expand(B, H, M).long()
    heads = torch.arange(H, device=_DEV)[None, :, None]
    k = s["k"][table.clamp(min=0), heads].view(B, H, M * bs, D)
    v = s["v"][table.clamp(min=0), heads].view(B, H, M * bs, D)
    j = torch.arange(M * bs, device=_DEV)[None, None, :]
    last = (s["lens"].long() - 1)[:, None, None]
    seen = (j <= last) & (table >= 0).repeat_interleave(bs, 2)
    if s["window"] is not None:
        w = s["window"].long()[None, :, None]
        seen = seen & ((w == 0) | (j < c["sink"]) | (j > last - w))
    q = s["q"].float().view(B, H, -1, D) / math.sqrt(D)
    x = torch.matmul(q, k.float().transpose(2, 3))
    x = torch.where(seen[:, :, None], x, -math.inf)
    p = torch.exp(x - x.amax(3, keepdim=True).clamp(min=-1e30))
    v = torch.where(seen[:, :, :, None], v, torch.zeros((), dtype=v.dtype, device=_DEV))
    out = torch.matmul(p, v.float()) / p.sum(3, keepdim=True).clamp(min=1e-30)
    return out.view(B, -1, D)


def _plain_copy(s):
    p, src, dst = s["pools"], s["src"].long(), s["dst"].long()
    if s["case"]["headwise"]:  # page numbers count the heads' pages as they lie
        p = p.view(*p.shape[:2], -1, *p.shape[4:])
    p[:, :, dst] = p[:, :, src]
    return s["pools"]


def _move(pools, headwise, head, src, dst):
    if headwise:
        pools[:, :, dst, head] = pools[:, :, src, head]
    else:
        pools[:, :, dst] = pools[:, :, src]


def _count(units, ids):
    return torch.zeros(units, dtype=torch.int64, device=_DEV).scatter_add_(0, ids, torch.ones_like(ids))


def _plain_fork(s):
    c = s["case"]
    H, bs, nb = (c["hkv"] if c["headwise"] else 1), c["bs"], s["blocks"]
    M = s["table"].shape[1]
    parents, lens, add = s["parents"].long(), s["lens"].long(), s["new"].long()
    n = parents.shape[0]
    kept = lens[parents]
    total = kept + add
    e, head = torch.arange(M, device=_DEV)[None, None, :], torch.arange(H, device=_DEV)[None, :, None]
    row = torch.arange(n, device=_DEV)[:, None, None].expand(n, H, M)
    have = (-(-kept // bs))[:, None, None]
    page = torch.where(e < have, s["table"].view(-1, H, M)[parents].long(), -1)
    unit = head * nb + page
    tail = (e == (kept // bs)[:, None, None]) & (page >= 0)
    whole = (page >= 0) & ~tail
    uses = _count(H * nb, unit[whole])
    owner = torch.full((H * nb,), n, dtype=torch.int64, device=_DEV).scatter_reduce_(0, unit[tail], row[tail], "amin")
    held = (uses > 0) | (owner < n)
    u = unit.clamp(min=0)
    split = tail & ((uses[u] > 0) | (owner[u] != row))
    ask = split | ((e >= have) & (e < (-(-total // bs))[:, None, None]))
    rank = ask.transpose(0, 1).reshape(H, -1).long().cumsum(1).view(H, n, M).transpose(0, 1) - 1
    free = torch.sort(held.view(H, nb).to(torch.uint8), dim=1, stable=True).indices
    left = nb - held.view(H, nb).sum(1)
    given = torch.where(rank < left[None, :, None], free[head, rank.clamp(0, nb - 1)], -1)
    table = torch.where(ask, given, page)
    copied = split & (table >= 0)
    _move(s["pools"], c["headwise"], head.expand(n, H, M)[copied], page[copied], table[copied])
    refs = _count(H * nb, (head * nb + table)[table >= 0])
    s["table_out"].copy_(table.view(-1, M))
    s["lens_out"].copy_(total)
    return dict(table=s["table_out"], lens=s["lens_out"], refs=refs.view(H, nb).to(torch.int32), pools=s["pools"])


def _plain_compact(s):
    c = s["case"]
    H, bs, nb = (c["hkv"] if c["headwise"] else 1), c["bs"], s["blocks"]
    M = s["table"].shape[1]
    t = s["table"].view(-1, H, M).long()
    head = torch.arange(H, device=_DEV)[None, :, None]
    live = (t >= 0) & (torch.arange(M, device=_DEV)[None, None, :] < (-(-s["lens"].long() // bs))[:, None, None])
    unit = (head * nb + t).clamp(min=0)
    refs = _count(H * nb, unit[live]).view(H, nb)
    used = refs > 0
    n_used = used.sum(1)
    ids = torch.arange(nb, device=_DEV)[None, :].expand(H, nb)
    mover, hole = used & (ids >= n_used[:, None]), ~used & (ids < n_used[:, None])
    at = torch.sort((~hole).to(torch.uint8), dim=1, stable=True).indices  # the holes first, in order
    to = at.gather(1, (mover.long().cumsum(1) - 1).clamp(min=0))
    page_map = torch.where(used, torch.where(mover, to, ids), -1)
    _move(s["pools"], c["headwise"], torch.arange(H, device=_DEV)[:, None].expand(H, nb)[mover], ids[mover], to[mover])
    s["table_out"].copy_(torch.where(live, page_map.view(-1)[unit], -1).view(-1, M))
    moved = torch.zeros_like(refs)
    moved[torch.arange(H, device=_DEV)[:, None].expand(H, nb)[used], page_map[used]] = refs[used]
    return dict(table=s["table_out"], map=page_map.to(torch.int32), refs=moved.to(torch.int32), used=n_used.to(torch.int32),
                pools=s["pools"])


def run(state):
    s = state
    c = s["case"]
    if own:
        import sub_byte_quantized_write_gb300 as K
        if c["op"] == "decode":
            return K.kvq_decode_attn(s["caches"][0], s["paging"], s["q"], 1 / math.sqrt(c["d"]), workspace=s["ws"])
        if c["op"] == "step":
            out = K.kvq_write_decode_attn(s["caches"][0], s["paging"], s["k_new"], s["v_new"], s["cu"], s["q"],
                                          1 / math.sqrt(c["d"]), workspace=s["ws"])
            return dict(out=out, k=s["k"], v=s["v"])
        if c["op"] == "copy":
            K.kvq_copy_pages(s["caches"], s["src"], s["dst"], headwise=c["headwise"], workspace=s["ws"])
            return s["pools"]
        if c["op"] == "fork":
            _, refs = K.kvq_fork(s["caches"], s["paging"], s["parents"], new_tokens=s["new"], out=s["paging_out"],
                                 workspace=s["ws"])
            return dict(table=s["table_out"], lens=s["lens_out"], refs=refs, pools=s["pools"])
        _, page_map, refs, used = K.kvq_compact(s["caches"], s["paging"], out=s["paging_out"], workspace=s["ws"])
        return dict(table=s["table_out"], map=page_map, refs=refs, used=used, pools=s["pools"])
    if c["op"] == "decode":
        return _plain_attention(s)
    if c["op"] == "step":
        _plain_write(s)
        return dict(out=_plain_attention(s), k=s["k"], v=s["v"])
    return {"copy": _plain_copy, "fork": _plain_fork, "compact": _plain_compact}[c["op"]](s)


# ---------------------------------------------------------------------------
# work and the definition in 64 bits

def work(case):
    c = case
    if c["op"] in ("decode", "step"):
        lens = _lens(c["batch"], c["lo"], c["hi"])
        w = _windows(c)
        w = np.zeros(c["hkv"], np.int64) if w is None else w.astype(np.int64)
        n = lens[:, None]
        keys = np.where(w[None, :] == 0, n, np.minimum(n, np.minimum(w[None, :], n) + np.minimum(c["sink"], np.maximum(0, n - w[None, :]))))
        pages = -(-keys // c["bs"])
        size = 4 if c["qtype"] == "f32" else 2
        io = c["batch"] * c["hq"] * c["d"] * (size + 4) + 4 * c["batch"]
        rows = int(keys.sum()) * 2 * 2 * c["d"] + 4 * int(pages.sum() if c["headwise"] else pages.max(1).sum())
        new = c["batch"] * c["hkv"] * c["d"] * 2 * (size + 2) if c["op"] == "step" else 0
        return {"bytes": rows + io + new, "flops": 4 * c["d"] * (c["hq"] // c["hkv"]) * int(keys.sum())}
    unit = c["bs"] * _ROW[c["mode"]](c["d"]) * (1 if c["headwise"] else c["hkv"])
    spaces = c["hkv"] if c["headwise"] else 1
    if c["op"] == "copy":
        return {"bytes": c["pairs"] * (8 + 4 * c["layers"] * unit), "flops": 0}
    if c["op"] == "fork":
        lens, p = _fork_lens(c), _parents(c)
        kept, first = lens[p], np.zeros(len(p), bool)
        first[np.unique(p, return_index=True)[1]] = True
        copies = int(((kept % c["bs"] != 0) & ~first).sum())
        entries = int((-(-kept // c["bs"])).sum()) * spaces
        width = max(1, -(-(c["hi"] + c["new"]) // c["bs"]))
        return {"bytes": 4 * entries + 4 * len(p) * spaces * width + 16 * len(p) + copies * spaces * 4 * c["layers"] * unit, "flops": 0}
    pages = int((-(-_lens(c["batch"], c["lo"], c["hi"]) // c["bs"])).sum())
    blocks = int(math.ceil(max(1, pages) / c["used"]))
    moves = pages * (1 - pages / blocks)
    width = max(1, -(-c["hi"] // c["bs"]))
    return {"bytes": spaces * (4 * pages + 4 * c["batch"] * width + 8 * blocks + moves * 4 * c["layers"] * unit), "flops": 0}


def exact(case, seed):
    if case["op"] not in ("decode", "step"):
        return None  # whole numbers and bytes only
    s = prepare(case, seed)
    H, G, bs = case["hkv"], case["hq"] // case["hkv"], case["bs"]
    lens, table = s["lens"].tolist(), s["table"].long()
    w = _windows(case)
    out = torch.zeros((case["batch"], case["hq"], case["d"]), dtype=torch.float64, device=_DEV)
    for b, n in enumerate(lens):
        for h in range(H):
            at = torch.arange(n, device=_DEV)
            page = table[b * H + h if case["headwise"] else b][at // bs]
            if case["op"] == "step" and n > 0 and int(page[-1]) >= 0:
                for name in ("k", "v"):
                    s[name][page[-1], h, (n - 1) % bs] = s[name + "_new"][b, h].to(torch.bfloat16)
            keep = page >= 0
            if w is not None and w[h]:
                keep &= (at < case["sink"]) | (at > n - 1 - int(w[h]))
            at, page = at[keep], page[keep]
            if at.numel() == 0:
                continue
            k, v = s["k"][page, h, at % bs].double(), s["v"][page, h, at % bs].double()
            x = (s["q"][b, h * G:(h + 1) * G].double() @ k.T) / math.sqrt(case["d"])
            out[b, h * G:(h + 1) * G] = torch.softmax(x, 1) @ v
    if case["op"] == "decode":
        return out
    return dict(out=out, k=s["k"].double(), v=s["v"].double())
