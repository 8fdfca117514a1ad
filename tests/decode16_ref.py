"""Plain 64-bit attention over 16-bit pages and small caches to run it on."""
import math

import numpy as np
import torch


def make(B, Hkv, G, D, bs, lens, dtype=torch.bfloat16, headwise=False, window=None, sink=0, seed=0, outliers=True,
         device="cuda", spare=7, max_blocks=None, write=True):
    """A bf16 cache whose every byte starts as 0xFF (NaN rows), with the rows of `lens` tokens per sequence written
    through kvq_write, and q.  Returns a dict with the handles and the written K and V (fp32 of the bf16 rows)."""
    import sub_byte_quantized_write_gb300 as K
    r = np.random.Generator(np.random.PCG64([seed, 77]))
    lens = np.asarray(lens, np.int32)
    need = -(-lens // bs)
    width = max_blocks or max(1, int(need.max()) if len(need) else 1)
    blocks = int(need.sum()) + spare
    spaces = Hkv if headwise else 1
    table = np.full((B, spaces, width), -1, np.int32)
    for s in range(spaces):
        perm, o = r.permutation(blocks), 0
        for b in range(B):
            table[b, s, :need[b]] = perm[o:o + need[b]]
            o += need[b]
    cache = K.PagedCache(K.KVQ_BF16_CACHE, blocks, Hkv, bs, D, None, device)
    cache.k_pages.fill_(0xFF)
    cache.v_pages.fill_(0xFF)
    n = int(lens.sum())
    x = torch.from_numpy(r.standard_normal((2, n, Hkv, D), dtype=np.float32)).to(device)
    if outliers:
        x[0, :, :, D // 3] *= 10
    x = x.to(dtype)
    tbl = torch.from_numpy(table.reshape(B * spaces, width)).to(device)
    lt = torch.from_numpy(lens).to(device)
    win = None if window is None else torch.tensor(window, dtype=torch.int32, device=device)
    kw = dict(block_tables_headwise=tbl) if headwise else dict(block_tables=tbl)
    pag = K.Paging(lt, window_per_kv_head=win, sink_size=sink, **kw)
    err = torch.zeros(1, dtype=torch.int32, device=device)
    cu = torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)).to(device)
    if n and write:
        K.kvq_write(cache, pag, x[0], x[1], cu, dev_error=err)
    q = torch.from_numpy(r.standard_normal((B, Hkv * G, D), dtype=np.float32)).to(device).to(dtype)
    return dict(cache=cache, pag=pag, q=q, k=x[0], v=x[1], cu=cu, lens=lens, table=table, window=window, sink=sink, err=err,
                G=G, D=D, bs=bs, Hkv=Hkv, scale=1 / math.sqrt(D))


def attention64(c, table=None, lens=None):
    """(out, tolerance) in float64 from the rows given to the write.

    The tolerance counts the fp32 roundings: a logit is a sum of D products in D / 16 matrix instructions and a few
    joins, each off by at most 2^-22 of the sum of magnitudes A; a weight is off by that, relatively, and by the
    exponent's 2^-21; the output sums n / 16 chunks of three terms, each rounding at most 2^-22 of sum p |v|.  Weight
    errors enter the numerator and the normalisation, hence the factor 2."""
    table = c["table"] if table is None else table
    lens = c["lens"] if lens is None else lens
    D, G, bs = c["D"], c["G"], c["bs"]
    B = len(lens)
    out = np.zeros((B, c["Hkv"] * G, D))
    tol = np.zeros((B, c["Hkv"] * G, 1))
    k = c["k"].to(torch.bfloat16).float().cpu().numpy().astype(np.float64)
    v = c["v"].to(torch.bfloat16).float().cpu().numpy().astype(np.float64)
    q = c["q"].float().cpu().numpy().astype(np.float64)
    start = np.concatenate([[0], np.cumsum(c["lens"])])
    for b in range(B):
        n = max(0, min(int(lens[b]), table.shape[2] * bs))
        for h in range(c["Hkv"]):
            j = np.arange(n)
            keep = table[b, h if table.shape[1] > 1 else 0][j // bs] >= 0
            if c["window"] is not None and c["window"][h] > 0:
                keep &= (j < c["sink"]) | (j > int(lens[b]) - 1 - c["window"][h])
            j = j[keep]
            if len(j) == 0:
                continue
            kk, vv = k[start[b] + j, h], v[start[b] + j, h]
            for g in range(G):
                x = kk @ q[b, h * G + g] * c["scale"]
                p = np.exp(x - x.max())
                p /= p.sum()
                out[b, h * G + g] = p @ vv
                A = (np.abs(kk) @ np.abs(q[b, h * G + g])).max() * c["scale"]
                dy = (D / 16 + 4) * 2.0 ** -22 * A + 2.0 ** -21
                tol[b, h * G + g] = (2 * dy + (3 * len(j) / 16 + 8) * 2.0 ** -22) * (p @ np.abs(vv)).max()
    return out, tol


def check(got, want):
    out, tol = want
    d = np.abs(got.double().cpu().numpy() - out)
    assert np.isfinite(got.cpu().numpy()).all()
    assert (d <= tol).all(), "off by %.3g of the tolerance" % float((d / np.maximum(tol, 1e-300)).max())
