"""What the cross-attention kernels' operand terms leave of an output: attention in 64 bits whose queries and weights are
cut to terms of bf16 or fp16 as the kernels cut theirs, with any of the terms left out."""
import numpy as np
import torch


def terms(x, dtype, count):
    """The sum of `count` terms of `dtype`: each the rounding of what the ones before it leave."""
    x = torch.from_numpy(np.ascontiguousarray(x))
    total = torch.zeros_like(x)
    for _ in range(count):
        total = total + (x - total).float().to(dtype).double()
    return total.numpy()


def attention(q, k, v, scale, q_terms=None, weight_terms=None):
    """Outputs [n, d] of q [n, d] over k, v [keys, d] (float64); the terms as (dtype, count), None: exact."""
    if q_terms:
        q = terms(q, *q_terms)
    x = q @ k.T * scale
    p = np.exp(x - x.max(1, keepdims=True))
    w = terms(p, *weight_terms) if weight_terms else p
    return w @ v / p.sum(1, keepdims=True)


def inputs(seed, n, keys, d, q_bf16=False, size=1.0):
    """Queries of `size`, bf16 rows with an outlier channel among the keys, values whose mean is not zero."""
    g = torch.Generator().manual_seed(seed)
    q, k, v = (torch.randn((m, d), generator=g) for m in (n, keys, keys))
    q = q * size
    k[:, d // 3] *= 6
    v[:, 5] += 0.5
    k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    return (q.to(torch.bfloat16) if q_bf16 else q), k, v


def off(got, want):
    return float(np.linalg.norm(got - want) / np.linalg.norm(want))
