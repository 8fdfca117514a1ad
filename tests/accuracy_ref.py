"""Attention in 64 bits on the GPU, and how far an output is from it as a whole."""
import torch


def attention64(q, k, v, n, lens, scale):
    """(outputs [sum(n), hq, d], largest logit in size, in powers of two) of n[b] queries over lens[b] rows each; q, k, v
    [rows, heads, d] one sequence after another."""
    hkv, g = k.shape[1], q.shape[1] // k.shape[1]
    out, most, iq, ik = torch.zeros(q.shape, dtype=torch.float64, device=q.device), 0.0, 0, 0
    for m, L in zip(n, lens):
        for h in range(hkv):
            if m == 0 or L == 0:
                continue
            x = q[iq:iq + m, h * g:(h + 1) * g].double() * scale
            x = torch.einsum("mgd,kd->mgk", x, k[ik:ik + L, h].double())
            most = max(most, float(x.abs().max()) / 0.6931471805599453)
            out[iq:iq + m, h * g:(h + 1) * g] = torch.softmax(x, -1) @ v[ik:ik + L, h].double()
        iq, ik = iq + m, ik + L
    return out, most


def off(got, want):
    """2-norm of the difference over 2-norm of `want`."""
    return float((got.double() - want).norm() / want.norm())
