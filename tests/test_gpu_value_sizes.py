"""Quantised rows whose values are of very different sizes, the small ones looked at: a call's weights times a row's scale
have to keep their bits whatever the largest scale is.  As a whole against 64 bits.

The bound, 6e-6 of a sequence's outputs: as test_gpu_step_accuracy's, of logits below 2^5 (asserted) whose parts, a row's
codes and its zero point, are below 2^6 and cancel: 2^-24 2^6 = 3.8e-6 of a weight, the query's terms 2^-17 ln 2 / sqrt(12)
= 1.6e-6, weights and sums 0.3e-6."""
import math

import pytest
import torch

import accuracy_ref as ref
from harness import kvq
from test_gpu_rope import cu_of, make_cache, paging, rows

pytestmark = pytest.mark.gpu
BOUND = 6e-6


def check(mode, D, n, lens, k, v, unseen=()):
    """Queries with 4 in element 3 beside normal values; the logits of rows that have no weight are not bounded."""
    K = kvq()
    H, G = k.shape[1], 4
    pag, blocks = paging(lens, H, 16, False)
    c = make_cache(mode, H, D, 16, blocks, 0, False)
    K.kvq_write(c, pag, k, v, cu_of(lens))
    k, v = K.kvq_gather(c, pag, cu_of(lens), sum(lens))
    q = rows(3, sum(n), H * G, D)
    q[:, :, 3] = 4
    out = K.kvq_cross_attn(c, pag, q, cu_of(n), max(n), D ** -0.5)
    want, _ = ref.attention64(q, k, v, n, lens, D ** -0.5)
    k[list(unseen)] = 0
    most = ref.attention64(q, k, v, n, lens, D ** -0.5)[1]
    assert most < 2 ** 5 and float(want.abs().max()) < 20
    at = 0
    for m in n:  # (sequence by sequence: their outputs may be of other sizes)
        assert ref.off(out[at:at + m], want[at:at + m]) < BOUND
        at += m


@pytest.mark.parametrize("mode", ["INT8_TOKEN_HEAD", "FP8_TOKEN_HEAD", "INT4_TOKEN_HEAD", "INT4_STEGO", "INT2_TOKEN_HEAD"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [(2, 1), (40, 5)])
@pytest.mark.parametrize("at", [0, 60, 300])
def test_a_large_row_that_no_query_looks_at(mode, D, n, at):
    """Its scale is a million times the others' (fp16 scales: 2^14 times), its weight 2^-40 or less."""
    H, lens = 1, [400, 333]
    k, v = rows(1, sum(lens), H, D), rows(2, sum(lens), H, D)
    for b in (at, lens[0] + at):
        v[b] *= 1e6 if "8" in mode or "STEGO" in mode else 2.0 ** 14
        k[b, :, 3] = -8 * math.sqrt(D)
    check(mode, D, n, lens, k, v, unseen=(at, lens[0] + at))


@pytest.mark.parametrize("mode,decades", [("INT8_TOKEN_HEAD", 8), ("FP8_TOKEN_HEAD", 8), ("INT4_STEGO", 8), ("INT4_TOKEN_HEAD", 4), ("INT2_TOKEN_HEAD", 4)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [(2, 1), (40, 5)])
def test_values_that_shrink_along_the_sequence(mode, decades, D, n):
    """Weights grow as values shrink, so that each row's part of an output is of one size."""
    H, lens = 1, [700, 97]
    k, v = rows(1, sum(lens), H, D) * 0.5, rows(2, sum(lens), H, D)
    at = 0
    for L in lens:
        down = torch.linspace(0, decades * math.log(10), L, device="cuda")
        v[at:at + L] *= torch.exp(-down)[:, None, None] * 10.0 ** (decades // 2)
        k[at:at + L, :, 3] = (down * math.sqrt(D) / 4)[:, None]
        at += L
    check(mode, D, n, lens, k, v)
