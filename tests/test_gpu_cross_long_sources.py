"""Many queries over long sources whose values' mean is not zero, as a whole against 64 bits.

The bound, 1e-5 of the outputs' 2-norm: the tensor cores' accumulators are cut at 2^-23 at most at each step of 16 keys and
two terms, and are added up every 16 tiles of 128 keys, 256 steps.  A sum that grows evenly loses half a cut of half its
end at each, 256 / 4 * 2^-23 = 7.6e-6 of it, if all of the output comes from the values' mean; beside that the 2.9e-6 of
test_gpu_cross_accuracy.  A sum of something else than the output, which is then taken off again, loses as much of that."""
import pytest
import torch

import accuracy_ref as ref
from harness import kvq
from test_gpu_cross_accuracy import MODES
from test_gpu_rope import cu_of, make_cache, paging, rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,n", [(4, (300, 260, 300, 130)), (1, (40, 33, 50, 21))])
def test_long_sources(mode, D, G, n):
    """As many CTAs as the card has SMs, and few whose keys are cut into parts."""
    K = kvq()
    H, lens = 4, [8192, 8200, 6000, 4111]
    pag, blocks = paging(lens, H, 64, False)
    c = make_cache(mode, H, D, 64, blocks, 0, mode != "INT8_CHANNEL")
    k, v = rows(1, sum(lens), H, D), rows(2, sum(lens), H, D)
    k[:, :, D // 3] *= 6
    v[:, :, 5] += 0.5
    K.kvq_write(c, pag, k, v, cu_of(lens))
    k, v = K.kvq_gather(c, pag, cu_of(lens), sum(lens))
    q = rows(3, sum(n), H * G, D)
    out = K.kvq_cross_attn(c, pag, q, cu_of(n), max(n), D ** -0.5)
    want, most = ref.attention64(q, k, v, n, lens, D ** -0.5)
    assert most < 2 ** 6 and ref.off(out, want) < 1e-5
