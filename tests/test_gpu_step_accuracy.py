"""The calls with rope and cross attention that the decode kernels serve, as a whole against 64 bits: queries that lie
in one element.

The bound, 3e-6 of the outputs' 2-norm.  Outputs are averages of values, so errors of single weights, which differ from
key to key, move the outputs by their root mean square at most.  A logit below 2^4 in powers of two (asserted) is made by
three fp32 operations whose terms are below 2^5, each off by 2^-24 of its size at most, so by 2^-24 2^5 / sqrt(3) as a
root mean square, and by 2^-24 2^5 together: 1.9e-6 of a weight, counting every term as large as the largest.  A query's
two terms leave 2^-12 of elements up to 2^10 .. 2^11, again of every dim another error: 2^-22 of a logit's size at most,
2^-18 ln 2 / sqrt(12) of a weight: 0.8e-6.  Weights and sums, 2^-22 and 2^-23: 0.3e-6."""
import math

import pytest
import torch

import accuracy_ref as ref
from harness import kvq
from test_gpu_rope import cu_of, i32, make_cache, make_rope, paging, rows

pytestmark = pytest.mark.gpu
BOUND = 3e-6


def filled(mode, lens, H, D, seed=0):
    """A cache of `lens` tokens, an outlier channel among the keys, values whose mean is not zero; its rows; the paging."""
    K = kvq()
    pag, blocks = paging(lens, H, 16, False, seed=seed)
    c = make_cache(mode, H, D, 16, blocks, seed, mode != "INT8_CHANNEL")
    k, v = rows(seed + 1, sum(lens), H, D), rows(seed + 2, sum(lens), H, D)
    k[:, :, D // 3] *= 6
    v[:, :, 5] += 0.5
    K.kvq_write(c, pag, k, v, cu_of(lens))
    return c, pag, *K.kvq_gather(c, pag, cu_of(lens), sum(lens))


@pytest.mark.parametrize("mode", ["INT4_TOKEN_HEAD", "INT4_STEGO", "INT2_TOKEN_HEAD"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 4, 5, 8])
@pytest.mark.parametrize("dim", [0, 7])
def test_query_in_one_element(mode, D, G, dim):
    """After the turn (at position 0: none) nearly all of a query is one element: its transform is D times it."""
    K = kvq()
    H, lens = 2, [1500, 700, 33, 1]
    c, pag, _, _ = filled(mode, lens, H, D)
    B = len(lens)
    q = rows(3, B, H * G, D) * 0.05
    q[:, :, dim] = 2 * math.sqrt(D)
    zero = i32([0] * B)
    new = rows(4, B, H, D), rows(5, B, H, D)
    out = K.kvq_rope_write_decode_attn(c, pag, make_rope(D), *new, cu_of([1] * B), q, D ** -0.5, positions=zero)
    k, v = K.kvq_gather(c, pag, cu_of(lens), sum(lens))
    want, most = ref.attention64(q, k, v, [1] * B, lens, D ** -0.5)
    assert most < 16 and ref.off(out, want) < BOUND
    out = K.kvq_cross_attn(c, pag, q, cu_of([1] * B), 1, D ** -0.5)
    assert ref.off(out, want) < BOUND


@pytest.mark.parametrize("mode", ["INT4_TOKEN_HEAD", "INT4_STEGO", "INT2_TOKEN_HEAD"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 4, 5, 8])
def test_query_in_eight_elements(mode, D, G):
    """One of the eight is the element whose transform is the same in every dim.  The bound, for logits below 24: no part of
    one is above 28 here (a row's middle adds gamma, below 1.5, times less than 3), so the three operations' errors, as root
    mean squares and squares added, are 2^-24 28 = 1.7e-6, the query's 24 / 16 of 0.8e-6, the rest 0.3e-6: 2.1e-6."""
    K = kvq()
    H, lens = 2, [1500, 700, 33, 1]
    c, pag, _, _ = filled(mode, lens, H, D)
    B = len(lens)
    q = rows(3, B, H * G, D)
    q[:, :, [0, 9, 17, 30, 33, 41, 50, 58]] = 0.7 * math.sqrt(D)
    out = K.kvq_rope_write_decode_attn(c, pag, make_rope(D), rows(4, B, H, D), rows(5, B, H, D), cu_of([1] * B), q, D ** -0.5,
                                       positions=i32([0] * B))
    k, v = K.kvq_gather(c, pag, cu_of(lens), sum(lens))
    want, most = ref.attention64(q, k, v, [1] * B, lens, D ** -0.5)
    assert most < 24 and ref.off(out, want) < BOUND
