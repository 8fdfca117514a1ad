"""The fused step over 4-bit rows whose keys have an element ten times the others', so that one key has most of a query's
weight: nothing averages what its logit is off by.  test_gpu_step_accuracy's bound, for logits below 36: their parts are
below 36 as well (a row's middle adds less than 1), the operations' errors, squares added, 2^-24 36 = 2.1e-6 for the largest
logit, the query's terms 36 / 16 of 0.8e-6, the rest 0.3e-6: squares added 2.8e-6."""
import pytest

import accuracy_ref as ref
from harness import kvq
from test_gpu_rope import cu_of, i32, make_cache, make_rope, paging, rows
from test_gpu_step_accuracy import BOUND

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mode", ["INT4_TOKEN_HEAD", "INT4_STEGO", "INT2_TOKEN_HEAD"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 3, 8])
def test_hot_keys(mode, D, G):
    K = kvq()
    H, B = 2, 20
    lens = [1500 + 37 * b for b in range(B)]
    pag, blocks = paging(lens, H, 32, False)
    c = make_cache(mode, H, D, 32, blocks)
    k, v = rows(1, sum(lens), H, D), rows(2, sum(lens), H, D)
    k[:, :, D // 2] *= 10
    K.kvq_write(c, pag, k, v, cu_of(lens))
    q = rows(3, B, H * G, D)
    q[:, :, D // 2] = 3
    out = K.kvq_rope_write_decode_attn(c, pag, make_rope(16), rows(4, B, H, D), rows(5, B, H, D), cu_of([1] * B), q, D ** -0.5,
                                       positions=i32([0] * B))
    k, v = K.kvq_gather(c, pag, cu_of(lens), sum(lens))
    want, most = ref.attention64(q, k, v, [1] * B, lens, D ** -0.5)
    assert most < 36 and ref.off(out, want) < BOUND
