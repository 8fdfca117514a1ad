"""Operator cases of the paged cache: rotary positions where rows enter the
cache, and cross attention to an encoder's states.

Five operators, each reached through the Python binding's calls:

  rope    kvq_rope: the queries and keys of a prompt turned to their positions
  write   kvq_rope_write: new K rows turned, then both K and V rows quantised
          (or kept in 16 bits) into the pages; read back with kvq_gather
  step    kvq_rope_write_decode_attn: a decode step's query and new key
          turned, the new rows written, the attention over the pages
  cross   kvq_cross_attn: some queries per sequence attend to every cached row
          of an encoder's states, whose length is another
  dense   kvq_cross_dense_attn: the same over dense 16-bit rows

``own`` False computes them with elementary torch operations, True calls the
package.  Lengths follow from a case alone (so that its work is known), page
numbers and values from the seed.
"""
import math

import numpy as np
import torch

own = False

_DEV = "cuda"
_ROW = {"int4": lambda d: d // 2 + 4, "int2": lambda d: d // 4 + 4, "int8": lambda d: d + 4, "fp8": lambda d: d + 4,
        "bf16": lambda d: 2 * d}


def listed():
    return [
        # one chat turn's next token, fp32 activations: nothing but latency
        dict(name="rope: one token", op="rope", batch=1, lo=1, hi=1, past=36, hq=4, hkv=2, d=64, rot=64, inter=True,
             dtype="f32", scaling="none", factor=1.0),
        # a serving batch's chunk of 8192 tokens far into long contexts
        dict(name="rope: chunk of 8192 tokens", op="rope", batch=8, lo=1024, hi=1024, past=120000, hq=32, hkv=8, d=128,
             rot=128, inter=False, dtype="bf16", scaling="parts", factor=8.0),
        # ragged small prompts, half of each head turned, 8-bit rows
        dict(name="write: 7 short prompts", op="write", batch=7, lo=1, hi=401, past=0, hkv=4, d=64, rot=32, inter=True,
             dtype="f32", scaling="none", factor=1.0, mode="int8", bs=16, headwise=True),
        # the prompt chunk of a 4-bit cache
        dict(name="write: chunk of 8192 tokens", op="write", batch=4, lo=2048, hi=2048, past=8192, hkv=8, d=128, rot=128,
             inter=False, dtype="bf16", scaling="linear", factor=4.0, mode="int4", bs=16, headwise=False),
        # a small batch's whole step over 16-bit pages
        dict(name="step: 7 short sequences", op="step", batch=7, lo=1, hi=401, hq=32, hkv=8, d=128, rot=128, inter=False,
             dtype="bf16", scaling="none", factor=1.0, mode="bf16", bs=16, headwise=False),
        # a serving batch of ragged contexts, grouped heads 4 : 1, 4-bit rows
        dict(name="step: 64 ragged sequences", op="step", batch=64, lo=1024, hi=8192, hq=32, hkv=8, d=128, rot=128,
             inter=False, dtype="bf16", scaling="none", factor=1.0, mode="int4", bs=16, headwise=False),
        # a large batch over long contexts, grouped heads 5 : 1, 2-bit rows, part of each head turned
        dict(name="step: 96 long sequences", op="step", batch=96, lo=8192, hi=24576, hq=20, hkv=4, d=128, rot=64,
             inter=True, dtype="bf16", scaling="parts", factor=4.0, mode="int2", bs=64, headwise=False),
        # four beams of one short source
        dict(name="cross: 4 beams of one source", op="cross", batch=1, qlo=4, qhi=4, lo=37, hi=37, hq=4, hkv=2, d=64,
             dtype="f32", mode="int8", bs=16, headwise=False),
        # the decode steps of a batch of searches: few queries, the sources' pages are what is read
        dict(name="cross: 64 sources, 2 queries", op="cross", batch=64, qlo=2, qhi=2, lo=1024, hi=8192, hq=32, hkv=8, d=128,
             dtype="bf16", mode="fp8", bs=16, headwise=False),
        # prompts of the decoder over 4-bit pages, ragged on both sides
        dict(name="cross: 16 ragged prompts", op="cross", batch=16, qlo=101, qhi=700, lo=500, hi=4000, hq=32, hkv=8, d=128,
             dtype="bf16", mode="int4", bs=16, headwise=False),
        # five queries over one long document: all of the card for four heads' rows
        dict(name="dense: 5 queries, long source", op="dense", batch=1, qlo=5, qhi=5, lo=131071, hi=131071, hq=20, hkv=4,
             d=128, dtype="bf16"),
        # prompts over long sources in 16 bits
        dict(name="dense: 8 prompts", op="dense", batch=8, qlo=1024, qhi=1024, lo=2048, hi=8192, hq=32, hkv=8, d=128,
             dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "write", "write", "step", "step", "cross", "cross", "dense"])
    d, bs, hkv = rng.choice([64, 128]), rng.choice([16, 32, 64]), rng.choice([1, 2, 3, 4, 8])
    group, dtype = rng.randint(1, 8), rng.choice(["bf16", "bf16", "f32"])
    c = dict(op=op, batch=_log(rng, 1, 64), hkv=hkv, d=d, dtype=dtype)
    if op != "write":
        c["hq"] = hkv * group
    if op in ("rope", "write", "step"):
        scaling = rng.choice(["none", "linear", "parts"])
        c.update(rot=rng.choice([16, 32, 48, d // 2, d, d, d]), inter=rng.random() < 0.4, scaling=scaling,
                 factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0]))
    if op in ("write", "step"):
        c.update(mode=rng.choice(["int4", "int2", "int8", "fp8", "bf16"]), bs=bs, headwise=rng.random() < 0.3)
    if op in ("rope", "write"):
        hi = _log(rng, 1, max(1, 8192 // c["batch"]))
        c.update(lo=rng.choice([0, max(1, hi // 8), hi]), hi=hi, past=rng.choice([0, rng.randint(1, 1000), _log(rng, 1000, 1000000)]))
        if op == "write":
            c["past"] = min(c["past"], 131072)
    elif op == "step":
        hi = _log(rng, 1, min(32768, (1 << 28) // (c["batch"] * hkv * d)))
        c.update(lo=rng.choice([1, max(1, hi // 8), hi]), hi=hi)
    else:
        hi = _log(rng, 1, min(32768, (1 << 28) // (c["batch"] * hkv * d)))
        qhi = rng.choice([_log(rng, 1, 8), _log(rng, 1, 1024)])
        # no more products than the largest listed case
        qhi = max(1, min(qhi, (1 << 40) // (4 * c["batch"] * hkv * group * d * hi)))
        c.update(qlo=rng.choice([0, max(1, qhi // 4), qhi]), qhi=qhi, lo=rng.choice([0, max(1, hi // 8), hi]), hi=hi)
        if op == "cross":
            c.update(mode=rng.choice(["int4", "int2", "int8", "fp8", "bf16"]), bs=bs, headwise=rng.random() < 0.3)
    return c


# ---------------------------------------------------------------------------
# inputs

def _lens(n, lo, hi):
    """Lengths spread over lo .. hi, odd ones among them: a case's own, whatever the seed."""
    f = np.modf(0.5 + np.arange(n) * 0.6180339887498949)[0]
    return (lo + np.floor((hi - lo + 1) * f)).astype(np.int64)


def _shapes(case):
    """(new tokens or queries, keys) of each sequence."""
    c = case
    if c["op"] in ("rope", "write"):
        n = _lens(c["batch"], c["lo"], c["hi"])
        n[0] = max(n[0], 1)  # never nothing at all
        return n, n + c["past"] + (np.arange(c["batch"]) * 37 % 101 if c["past"] else 0)
    if c["op"] == "step":
        return np.ones(c["batch"], np.int64), _lens(c["batch"], c["lo"], c["hi"])
    n = _lens(c["batch"], c["qlo"], c["qhi"])
    n[0] = max(n[0], 1)
    return n, _lens(c["batch"], c["lo"], c["hi"])[::-1].copy()


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(_DEV)


def _cu(n):
    return _i32(np.concatenate([[0], np.cumsum(n)]))


def _spread(gen, counts, width, spaces, blocks):
    """[spaces, rows, width] tables: row r's first counts[r] entries are distinct pages of its space, the others -1."""
    order = torch.rand((spaces, blocks), generator=gen, device=_DEV).argsort(1).to(torch.int32)
    c = torch.from_numpy(counts).to(_DEV)
    at = (c.cumsum(0) - c)[:, None] + torch.arange(width, device=_DEV)[None, :]
    inside = torch.arange(width, device=_DEV)[None, :] < c[:, None]
    return torch.where(inside[None], order[:, at.clamp(max=blocks - 1)], -1)


def _frequencies(case):
    """Radians per position of each pair, and the factor on cosine and sine, for a context `factor` times the first."""
    rot, base, first = case["rot"], 500000.0, 8192
    f = base ** -(np.arange(0, rot, 2) / rot)
    if case["scaling"] == "linear":
        return f / case["factor"], 1.0
    if case["scaling"] == "parts":  # slow pairs interpolated, fast ones as they were, a ramp between
        def pair(turns):
            return rot * math.log(first / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), rot - 1)
        ramp = np.clip((np.arange(rot // 2) - lo) / max(hi - lo, 0.001), 0, 1)
        return f * (1 - ramp) + f / case["factor"] * ramp, 0.1 * math.log(case["factor"]) + 1.0
    return f, 1.0


def _values_like(gen, rows, heads, d, dtype):
    """Projected rows: normal values, a few channels ten times as large."""
    x = torch.randn((rows, heads, d), generator=gen, device=_DEV)
    hot = torch.randint(0, heads * d, (max(1, heads * d // 100),), generator=gen, device=_DEV)
    x[:, hot // d, hot % d] *= 10
    return x if dtype == "f32" else x.to(torch.bfloat16)


def _hadamard(d):
    h = torch.ones((1, 1), device=_DEV)
    while h.shape[0] < d:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h


def _pages(case, s, gen, counts, first=0):
    """Tables (entries before page `first[b]` are -1) and pools of filled pages."""
    H, d, bs, mode = case["hkv"], case["d"], case["bs"], case["mode"]
    width = max(1, int(np.max(counts + first)))
    spaces = H if case["headwise"] else 1
    blocks = int(counts.sum()) + int(counts.sum()) // 20 + 8
    t = _spread(gen, counts, width, spaces, blocks)
    if np.any(first):  # move each row's pages behind the `first` evicted ones
        at = torch.arange(width, device=_DEV)[None, :] - torch.from_numpy(first).to(_DEV)[:, None]
        t = torch.where((at >= 0)[None], t.gather(2, at.clamp(min=0)[None].expand(spaces, -1, -1)), -1)
    s["table"] = t.permute(1, 0, 2).reshape(-1, width).contiguous()
    s["signs"] = None
    if mode in ("int4", "int2"):
        s["signs"] = (torch.randint(0, 2, (d,), generator=gen, device=_DEV, dtype=torch.int32) * 2 - 1).to(torch.int8)
    s["had"] = _hadamard(d)
    for name in ("k", "v"):
        x = _values_like(gen, blocks * bs, H, d, "bf16").float()
        s[name] = _rows(x, mode, s).view(blocks, bs, H, -1).transpose(1, 2).contiguous()
    s["blocks"] = blocks


def prepare(case, seed):
    gen = torch.Generator(device=_DEV)
    gen.manual_seed(seed)
    c, op = case, case["op"]
    n, lens = _shapes(c)
    T = int(n.sum())
    s = dict(case=c, lens=_i32(lens), cu=_cu(n), tokens=T, most=int(n.max()))
    if "rot" in c:
        f, s["amp"] = _frequencies(c)
        s["freq"] = torch.from_numpy(f).to(_DEV).float()
    if "hq" in c:
        s["q"] = _values_like(gen, T, c["hq"], c["d"], c["dtype"])
    if op in ("rope", "write", "step"):
        s["k_new"] = _values_like(gen, T, c["hkv"], c["d"], c["dtype"])
    if op in ("write", "step"):
        s["v_new"] = _values_like(gen, T, c["hkv"], c["d"], c["dtype"])
    if op == "dense":
        s["cu_kv"] = _cu(lens)
        rows = max(1, int(lens.sum()))
        s["k"], s["v"] = (_values_like(gen, rows, c["hkv"], c["d"], "bf16") for _ in range(2))
    elif op != "rope":
        first = (lens - n) // c["bs"] if op == "write" else np.zeros_like(lens)
        _pages(c, s, gen, -(-lens // c["bs"]) - first, first)
    if own:  # the handles that a user's program keeps: the cache, the paging state, frequencies, outputs and scratch
        import sub_byte_quantized_write_gb300 as K
        mode = {"int4": K.KVQ_INT4_TOKEN_HEAD, "int2": K.KVQ_INT2_TOKEN_HEAD, "int8": K.KVQ_INT8_TOKEN_HEAD,
                "fp8": K.KVQ_FP8_TOKEN_HEAD, "bf16": K.KVQ_BF16_CACHE}
        nbytes = 0
        if "rot" in c:
            s["rope"] = K.Rope(s["freq"], interleaved=c["inter"], scale=s["amp"])
        if "table" in s:
            s["cache"] = K.PagedCache(mode[c["mode"]], s["blocks"], c["hkv"], c["bs"], c["d"], rht_signs=s["signs"],
                                      k_pages=s["k"], v_pages=s["v"])
            s["paging"] = K.Paging(s["lens"], **{"block_tables_headwise" if c["headwise"] else "block_tables": s["table"]})
        if op in ("write", "step"):
            s["k_out"], s["v_out"] = (torch.empty((T, c["hkv"], c["d"]), dtype=torch.bfloat16, device=_DEV) for _ in range(2))
        if op == "step":
            nbytes, _ = K.kvq_decode_workspace_size(s["cache"], s["paging"], c["hq"])
        elif op == "cross":
            nbytes = K.kvq_cross_workspace_size(s["cache"], s["paging"], c["hq"], s["most"])
        elif op == "dense":
            nbytes = K.kvq_cross_dense_workspace_size(s["k"], s["lens"], c["hq"], s["most"])
        if op == "rope":
            s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k_new"])
        elif op != "write":
            s["out"] = torch.empty(s["q"].shape, dtype=torch.float32, device=_DEV)
        s["ws"] = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=_DEV)
    return s


# ---------------------------------------------------------------------------
# the plain forms

def _rows(x, mode, s):
    """The cache rows (bytes) of x [..., d] in fp32."""
    d = x.shape[-1]
    if mode == "bf16":
        return x.to(torch.bfloat16).view(torch.uint8)
    if s["signs"] is not None:
        x = (x * s["signs"].float()) @ s["had"]
    if mode in ("int8", "fp8"):
        scale = x.abs().amax(-1, keepdim=True) / (127.0 if mode == "int8" else 448.0)
        y = torch.where(scale > 0, x / scale, 0.0)
        code = y.round().clamp(-127, 127).to(torch.int8) if mode == "int8" else y.clamp(-448, 448).to(torch.float8_e4m3fn)
        return torch.cat([code.view(torch.uint8), scale.view(torch.uint8)], -1)
    bits = 4 if mode == "int4" else 2
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    scale = ((hi - lo) / (2 ** bits - 1)).clamp(-65504, 65504).to(torch.float16)
    zero = lo.clamp(-65504, 65504).to(torch.float16)
    u = torch.where(scale > 0, (x - zero.float()) / scale.float(), 0.0).round().clamp(0, 2 ** bits - 1).to(torch.int32)
    per = 8 // bits
    shift = torch.arange(per, device=x.device, dtype=torch.int32) * bits
    code = (u.view(*u.shape[:-1], d // per, per) << shift).sum(-1).to(torch.uint8)
    return torch.cat([code, scale.view(torch.uint8), zero.view(torch.uint8)], -1)


def _read(rows, mode, s):
    """The values in fp32 that cache rows (bytes) [..., row] stand for."""
    if mode == "bf16":
        return rows.view(torch.bfloat16).float()
    d = s["case"]["d"]
    if mode in ("int8", "fp8"):
        code = rows[..., :d].contiguous().view(torch.int8 if mode == "int8" else torch.float8_e4m3fn).float()
        y = code * rows[..., d:].contiguous().view(torch.float32)
    else:
        bits = 4 if mode == "int4" else 2
        per = 8 // bits
        shift = torch.arange(per, device=rows.device, dtype=torch.int32) * bits
        u = ((rows[..., : d // per, None].to(torch.int32) >> shift) & (2 ** bits - 1)).flatten(-2).float()
        pad = rows[..., d // per:].contiguous().view(torch.float16).float()
        y = u * pad[..., :1] + pad[..., 1:]
    if s["signs"] is not None:
        y = (y @ s["had"]) * s["signs"].float() / d
    return y


def _positions(s):
    """(sequence, position) of each token."""
    cu, lens = s["cu"].long(), s["lens"].long()
    t = torch.arange(s["tokens"], device=_DEV)
    b = torch.searchsorted(cu, t, right=True) - 1
    return b, lens[b] - cu[b + 1] + t


def _turn(x, pos, s):
    """x [tokens, heads, d] turned to its positions, in fp32; angles in 64 bits."""
    c = s["case"]
    angle = pos.double()[:, None] * s["freq"].double()
    co, si = (angle.cos() * s["amp"]).float()[:, None], (angle.sin() * s["amp"]).float()[:, None]
    x = x.float()
    head, tail = x[..., : c["rot"]], x[..., c["rot"]:]
    if c["inter"]:
        a, b = head[..., 0::2], head[..., 1::2]
        y = torch.stack([a * co - b * si, b * co + a * si], -1).flatten(-2)
    else:
        a, b = head.chunk(2, -1)
        y = torch.cat([a * co - b * si, b * co + a * si], -1)
    return torch.cat([y, tail], -1)


def _plain_write(s, k, v):
    """The rows into their pages; the values that the pages then hold."""
    c = s["case"]
    b, pos = _positions(s)
    h = torch.arange(c["hkv"], device=_DEV)[None, :]
    row = b[:, None] * c["hkv"] + h if c["headwise"] else b[:, None] + 0 * h
    blk = s["table"][row, (pos // c["bs"])[:, None]].long()
    slot = (pos % c["bs"])[:, None].expand_as(blk)
    for name, x in (("k", k), ("v", v)):
        s[name][blk, h.expand_as(blk), slot] = _rows(x.float(), c["mode"], s)
    return [_read(s[name][blk, h.expand_as(blk), slot], c["mode"], s).to(torch.bfloat16) for name in ("k", "v")]


def _dense_rows(s, name, b, j):
    """Rows of `name` at keys j [keys] of each sequence [batch, hkv, keys, d], and whether there is such a key."""
    c = s["case"]
    H, lens = c["hkv"], s["lens"].long()[b]
    seen = j[None, None, :] < lens[:, None, None]
    h = torch.arange(H, device=_DEV)[None, :, None]
    if c["op"] == "dense":
        at = (s["cu_kv"].long()[b][:, None] + j[None, :]).clamp(max=s[name].shape[0] - 1)
        return s[name][at].float().transpose(1, 2), seen.expand(-1, H, -1)
    entry = (j // c["bs"]).clamp(max=s["table"].shape[1] - 1)
    row = (b[:, None] * H + h[:, :, 0] if c["headwise"] else b[:, None].expand(-1, H))[:, :, None]
    blk = s["table"][row, entry[None, None, :]].long()
    return _read(s[name][blk.clamp(min=0), h, (j % c["bs"])[None, None, :]], c["mode"], s), seen & (blk >= 0)


def _plain_attention(s, q):
    """Every query of a sequence attends to all of its rows; q [tokens, hq, d].  Sequences in equal parts, so that
    what is held at once stays in bounds."""
    c = s["case"]
    B, H, D, most = c["batch"], c["hkv"], c["d"], s["most"]
    G = c["hq"] // H
    keys = max(1, c["hi"])
    out = torch.zeros((s["tokens"], c["hq"], D), device=_DEV)
    part = max(1, min(B, int(6e9 // (H * keys * (G * most * 8 + 24 * D)))))
    i, j = torch.arange(most, device=_DEV), torch.arange(keys, device=_DEV)
    for b0 in range(0, B, part):
        b = torch.arange(b0, min(B, b0 + part), device=_DEV)
        cu = s["cu"].long()
        at = cu[b][:, None] + i[None, :]
        real = at < cu[b + 1][:, None]
        x = q[at.clamp(max=s["tokens"] - 1)].float().view(len(b), most, H, G, D).permute(0, 2, 3, 1, 4)
        x = x.reshape(len(b), H, G * most, D) / math.sqrt(D)
        k, seen = _dense_rows(s, "k", b, j)
        w = torch.where(seen[:, :, None], torch.matmul(x, k.transpose(2, 3)), -math.inf)
        w = torch.exp(w - w.amax(3, keepdim=True).clamp(min=-1e30))
        v, _ = _dense_rows(s, "v", b, j)
        v = torch.where(seen[..., None], v, 0.0)
        o = torch.matmul(w, v) / w.sum(3, keepdim=True).clamp(min=1e-30)
        o = o.view(len(b), H, G, most, D).permute(0, 3, 1, 2, 4).reshape(len(b), most, c["hq"], D)
        out[at[real]] = o[real]
    return out


def run(state):
    s = state
    c = s["case"]
    scale = 1 / math.sqrt(c["d"])
    if own:
        import sub_byte_quantized_write_gb300 as K
        if c["op"] == "rope":
            q, k = K.kvq_rope(s["rope"], s["q"], s["k_new"], s["lens"], s["cu"], q_out=s["q_out"], k_out=s["k_out"])
            return dict(q=q, k=k)
        if c["op"] == "write":
            K.kvq_rope_write(s["cache"], s["paging"], s["rope"], s["k_new"], s["v_new"], s["cu"])
            k, v = K.kvq_gather(s["cache"], s["paging"], s["cu"], s["tokens"], k_out=s["k_out"], v_out=s["v_out"])
            return dict(k=k, v=v)
        if c["op"] == "step":
            out = K.kvq_rope_write_decode_attn(s["cache"], s["paging"], s["rope"], s["k_new"], s["v_new"], s["cu"], s["q"],
                                               scale, out=s["out"], workspace=s["ws"])
            k, v = K.kvq_gather(s["cache"], s["paging"], s["cu"], s["tokens"], k_out=s["k_out"], v_out=s["v_out"])
            return dict(out=out, k=k, v=v)
        if c["op"] == "cross":
            return K.kvq_cross_attn(s["cache"], s["paging"], s["q"], s["cu"], s["most"], scale, out=s["out"],
                                    workspace=s["ws"])
        return K.kvq_cross_dense_attn(s["k"], s["v"], s["cu_kv"], s["lens"], s["q"], s["cu"], s["most"], scale,
                                      out=s["out"], workspace=s["ws"])
    if c["op"] in ("cross", "dense"):
        return _plain_attention(s, s["q"])
    _, pos = _positions(s)
    if c["op"] == "rope":
        return dict(q=_turn(s["q"], pos, s).to(s["q"].dtype), k=_turn(s["k_new"], pos, s).to(s["k_new"].dtype))
    k, v = _plain_write(s, _turn(s["k_new"], pos, s), s["v_new"])
    if c["op"] == "write":
        return dict(k=k, v=v)
    return dict(out=_plain_attention(s, _turn(s["q"], pos, s)), k=k, v=v)


# ---------------------------------------------------------------------------
# work and the definition in 64 bits

def work(case):
    c = case
    n, lens = _shapes(c)
    T, size, d = int(n.sum()), 4 if c["dtype"] == "f32" else 2, c["d"]
    new = T * c["hkv"] * d
    if c["op"] == "rope":
        return {"bytes": 2 * size * d * T * (c["hq"] + c["hkv"]), "flops": 3 * c["rot"] * T * (c["hq"] + c["hkv"])}
    row = 2 * d if c["op"] == "dense" else _ROW[c["mode"]](d)
    if c["op"] == "write":  # in, into the pages, and back out in 16 bits
        return {"bytes": 2 * size * new + 2 * T * c["hkv"] * 2 * row + 2 * 2 * new, "flops": 3 * c["rot"] * T * c["hkv"]}
    keys = int(lens.sum()) * c["hkv"]
    pairs = int((n * lens).sum()) * c["hq"]
    table = 0 if c["op"] == "dense" else 4 * int((-(-lens // c["bs"])).sum()) * (c["hkv"] if c["headwise"] else 1)
    io = T * c["hq"] * d * (size + 4)
    more = 2 * size * new + 2 * T * c["hkv"] * 2 * row + 4 * new if c["op"] == "step" else 0
    return {"bytes": keys * 2 * row + table + io + more, "flops": 4 * d * pairs}


def _exact_row_values(x, case, signs):
    """What the cache rows of x [heads, d] (64 bits) stand for."""
    mode, d = case["mode"], case["d"]
    if mode == "bf16":
        return x.to(torch.bfloat16).double()
    if signs is not None:
        i = torch.arange(d, device=x.device)
        bits = i[:, None] & i[None, :]
        odd = sum((bits >> k) & 1 for k in range(7)) % 2
        turn = (1.0 - 2.0 * odd.double()) * signs.double()[None, :]
        x = x @ turn.T
    if mode in ("int8", "fp8"):
        scale = (x.abs().amax(1, keepdim=True) / (127 if mode == "int8" else 448)).float().double()
        y = x / torch.where(scale > 0, scale, 1.0)
        if mode == "int8":
            y = y.round().clamp(-127, 127)
        else:  # the nearest of 4 significant bits, 2^-9 the smallest step
            step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
            y = (torch.round(y / step) * step).clamp(-448, 448)
        y = y * scale
    else:
        top = 15 if mode == "int4" else 3
        lo, hi = x.amin(1, keepdim=True), x.amax(1, keepdim=True)
        scale, zero = ((hi - lo) / top).half().double(), lo.half().double()
        u = ((x - zero) / torch.where(scale > 0, scale, 1.0)).round().clamp(0, top)
        y = torch.where(scale > 0, u, 0.0) * scale + zero
    return y if signs is None else (y @ turn) / d


def _exact_turn(x, pos, s):
    """Pairs as complex numbers, multiplied by amp * exp(i * angle)."""
    c = s["case"]
    x, r = x.double().clone(), c["rot"]
    angle = pos.double().view(-1, 1, 1) * s["freq"].double()
    z = torch.polar(torch.full_like(angle, s["amp"]), angle)
    i = torch.arange(r // 2, device=_DEV)
    first, second = (2 * i, 2 * i + 1) if c["inter"] else (i, i + r // 2)
    w = torch.complex(x[..., first], x[..., second]) * z
    x[..., first], x[..., second] = w.real, w.imag
    return x


def exact(case, seed):
    n, lens = _shapes(case)
    if "hq" in case and case["op"] != "rope" and 4e-12 * case["d"] * case["hq"] * float((n * lens).sum()) > 8:
        return None
    s = prepare(case, seed)
    c, H, d = case, case["hkv"], case["d"]
    start = np.concatenate([[0], np.cumsum(n)])
    pos = torch.from_numpy(np.concatenate([np.arange(L - m, L) for m, L in zip(n, lens)])).to(_DEV)
    if c["op"] == "rope":
        return dict(q=_exact_turn(s["q"], pos, s), k=_exact_turn(s["k_new"], pos, s))
    new = {}
    if c["op"] in ("write", "step"):
        signs = s["signs"]
        new = {"k": _exact_turn(s["k_new"], pos, s), "v": s["v_new"].double()}
        new = {name: _exact_row_values(x.reshape(-1, d), c, signs).view(x.shape) for name, x in new.items()}
        if c["op"] == "write":
            return new
    q = s["q"].double() if c["op"] != "step" else _exact_turn(s["q"], pos, s)
    G = c["hq"] // H
    out = torch.zeros((int(n.sum()), c["hq"], d), dtype=torch.float64, device=_DEV)
    at_kv = np.concatenate([[0], np.cumsum(lens)])
    for b, (m, L) in enumerate(zip(n, lens)):
        if m == 0 or L == 0:
            continue
        for h in range(H):
            if c["op"] == "dense":
                k, v = (s[x][at_kv[b]:at_kv[b + 1], h].double() for x in ("k", "v"))
            else:
                j = torch.arange(int(L), device=_DEV)
                page = s["table"][b * H + h if c["headwise"] else b][j // c["bs"]].long()
                k, v = (_stored(s[x][page, h, j % c["bs"]], s) for x in ("k", "v"))
            if c["op"] == "step":
                k[-1], v[-1] = new["k"][b, h], new["v"][b, h]
            x = q[start[b]:start[b + 1], h * G:(h + 1) * G].reshape(-1, d) @ k.T / math.sqrt(d)
            out[start[b]:start[b + 1], h * G:(h + 1) * G] = (torch.softmax(x, 1) @ v).view(int(m), G, d)
    return out if c["op"] != "step" else dict(out=out, **new)


def _stored(rows, s):
    """The values (64 bits) of cache rows [keys, bytes], element by element of the row layout."""
    c = s["case"]
    d, mode = c["d"], c["mode"]
    if mode == "bf16":
        return rows.view(torch.bfloat16).double()
    e = torch.arange(d, device=rows.device)
    if mode in ("int4", "int2"):
        b = 4 if mode == "int4" else 2
        u = (rows[:, e * b // 8].long() >> (e * b % 8)) % 2 ** b
        pad = rows[:, d * b // 8:].clone().view(torch.float16).double()
        y = u * pad[:, :1] + pad[:, 1:]
    else:
        u = rows[:, :d].long()
        if mode == "int8":
            y = (u - 256 * (u > 127)).double()
        else:  # sign, 4 bits of exponent (7 is 0), 3 of the fraction
            ex, fr = (u >> 3) % 16, u % 8
            y = torch.where(ex > 0, (8 + fr) * torch.exp2(ex.double() - 10), fr * 2.0 ** -9) * torch.where(u > 127, -1.0, 1.0)
        y = y * rows[:, d:].clone().view(torch.float32).double()
    if s["signs"] is None:
        return y
    bits = e[:, None] & e[None, :]
    odd = sum((bits >> k) & 1 for k in range(7)) % 2
    return y @ (1.0 - 2.0 * odd.double()) * s["signs"].double() / d
