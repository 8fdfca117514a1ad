"""Plain 64-bit cross attention and what the kernels' fp32 arithmetic may be off by."""
import numpy as np
import torch


def attention64(q, k, v, seen, scale):
    """(out, tolerance) of queries q [n, hq, d] over rows k, v [keys, hkv, d] (numpy, 64 bits), `seen` [hkv, keys].

    The tolerance counts fp32 roundings, each at most 2^-22 of the magnitudes summed (the tensor cores truncate, so
    twice half a step): a logit sums D products in D / 16 steps, of up to three terms each, times codes that a zero
    point or fold offsets, A = |q| |k| summed bounds it and 16 A the folded form (codes -8..7 about 72: the constants are
    at most nine times the codes' range); the exponent adds 2^-21; weights of two 8-bit terms or of fp16 pairs 2^-17;
    the output sums keys / 16 steps of two terms.  Weight errors enter the numerator and the normalisation: twice."""
    n, hq, d = q.shape
    keys, hkv = k.shape[:2]
    g = hq // hkv
    out, tol = np.zeros((n, hq, d)), np.zeros((n, hq, 1))
    for h in range(hkv):
        j = np.flatnonzero(seen[h])
        if len(j) == 0:
            continue
        kk, vv = k[j, h], v[j, h]
        for i in range(g):
            x = q[:, h * g + i] @ kk.T * scale
            p = np.exp(x - x.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            out[:, h * g + i] = p @ vv
            a = (np.abs(q[:, h * g + i]) @ np.abs(kk).T).max(1, keepdims=True) * abs(scale)
            dy = (3 * d / 16 + 4) * 2.0 ** -22 * 16 * a + 2.0 ** -21
            most = (p @ np.abs(vv)).max(1, keepdims=True)
            tol[:, h * g + i] = (2 * dy + 2.0 ** -17 + (2 * len(j) / 16 + 8) * 2.0 ** -22) * most
    return out, tol


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def check(got, q, k, v, n, lens, scale, seen=None, start=None):
    """got [tokens, hq, d] against 64 bits for each sequence: n queries, lens rows (of k, v [rows, hkv, d], sequence b's
    from start[b] on); seen(b) [hkv, keys] or None (all)."""
    qh, kh, vh, o = host(q), host(k), host(v), host(got)
    cu = np.concatenate([[0], np.cumsum(n)])
    start = np.concatenate([[0], np.cumsum(lens)]) if start is None else start
    assert np.isfinite(o[: cu[-1]]).all()
    for b in range(len(n)):
        if n[b] == 0:
            continue
        rows = slice(int(start[b]), int(start[b]) + int(lens[b]))
        vis = np.ones((kh.shape[1], int(lens[b])), bool) if seen is None else seen(b)
        want, tol = attention64(qh[cu[b]:cu[b + 1]], kh[rows], vh[rows], vis, scale)
        d = np.abs(o[cu[b]:cu[b + 1]] - want)
        assert (d <= tol).all(), (b, float((d / np.maximum(tol, 1e-300)).max()), float(d.max()))
