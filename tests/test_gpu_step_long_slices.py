"""The fused step over slices of many tiles, values whose mean is not zero, as a whole against 64 bits: what a sum of
products loses at each step would add up.  The bound is test_gpu_step_accuracy's; the sums of 16 keys' products join in
fp32, which over n keys in one slice leaves sqrt(n / 16) 2^-24 of the largest sum as a root mean square, 43 * 2^-24 of it
for 30011 keys if that were the output's own all along: its half, counted as it grows, is 1.3e-6, within what the bound
leaves beside test_gpu_step_accuracy's roundings of logits of 16 (these are below 12)."""
import math

import pytest

import accuracy_ref as ref
from harness import kvq
from test_gpu_rope import cu_of, i32, make_rope, rows
from test_gpu_step_accuracy import BOUND, filled

pytestmark = pytest.mark.gpu
MODES = ["INT4_TOKEN_HEAD", "INT4_STEGO", "INT2_TOKEN_HEAD", "INT8_TOKEN_HEAD", "FP8_TOKEN_HEAD"]


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("D,G", [(64, 4), (128, 1), (128, 8)])
@pytest.mark.parametrize("splits", [1, 6])
def test_long_slices(mode, D, G, splits):
    """A warp's slice of many tiles: what a sum of its products loses at each step would add up."""
    K = kvq()
    H, lens = 1, [30011]
    c, pag, _, _ = filled(mode, lens, H, D, seed=6)
    q = rows(3, 1, H * G, D)
    new = rows(4, 1, H, D), rows(5, 1, H, D)
    out = K.kvq_rope_write_decode_attn(c, pag, make_rope(D), *new, cu_of([1]), q, D ** -0.5, positions=i32([0]), num_splits=splits)
    k, v = K.kvq_gather(c, pag, cu_of(lens), sum(lens))
    want, most = ref.attention64(q, k, v, [1], lens, D ** -0.5)
    assert most < 12 and ref.off(out, want) < BOUND


@pytest.mark.parametrize("mode", MODES[:3])
@pytest.mark.parametrize("D,G", [(64, 4), (128, 4), (128, 8)])
def test_query_in_one_element(mode, D, G):
    """All of a batch's tiles in one slice, the queries in the element that the transform spreads evenly."""
    K = kvq()
    H, lens = 2, [1500, 700, 33, 1]
    c, pag, _, _ = filled(mode, lens, H, D)
    B = len(lens)
    q = rows(3, B, H * G, D) * 0.05
    q[:, :, 0] = 2 * math.sqrt(D)
    out = K.kvq_rope_write_decode_attn(c, pag, make_rope(D), rows(4, B, H, D), rows(5, B, H, D), cu_of([1] * B), q, D ** -0.5,
                                       positions=i32([0] * B), num_splits=1)
    k, v = K.kvq_gather(c, pag, cu_of(lens), sum(lens))
    want, most = ref.attention64(q, k, v, [1] * B, lens, D ** -0.5)
    assert most < 16 and ref.off(out, want) < BOUND
