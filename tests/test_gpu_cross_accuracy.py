"""Cross attention over short sources as a whole against 64 bits, closely enough that a term left out shows
(test_cross_model_host.py).

The bound, 3.5e-6 of the outputs' 2-norm, errors of single weights counted by their root mean square (outputs are averages
of values).  Weights of two bf16 terms: 2^-18 of them at most, 2^-18 / sqrt(3) = 2.2e-6 as a root mean square.  Logits below
2^6 in powers of two (asserted), summed from D / 16 steps of up to three terms, the low ones first, each step cut at 2^-24
of a sum that grows to the logit: on average a quarter of the steps' worth, ln 2 * 2^6 * 2 * 2^-24 = 5.3e-6 for the largest
logit, of which a typical weight's is a third, 1.8e-6.  Outputs are cut at 2^-23 at each of up to 256 steps while they grow,
but for weights as uneven as these most of an output comes in a few steps.  As squares these come to 2.9e-6."""
import pytest
import torch

import accuracy_ref as ref
import cross_model as model
from harness import kvq
from test_gpu_rope import cu_of, i32, make_cache, paging, rows

pytestmark = pytest.mark.gpu
BOUND = 3.5e-6
SIZES = [(2, 130, 3.0), (40, 130, 3.0), (40, 700, 3.0), (300, 1900, 3.0)]  # queries, keys, size of the queries
MODES = ["INT4_TOKEN_HEAD", "INT4_STEGO", "INT2_TOKEN_HEAD", "INT8_TOKEN_HEAD", "FP8_TOKEN_HEAD", "BF16_CACHE", "INT8_CHANNEL"]


def source(keys, H, D):
    """The rows of a source, [keys, H, D] in bf16."""
    kv = [model.inputs(keys + h, 1, keys, D)[1:] for h in range(H)]
    return tuple(torch.stack([x[i] for x in kv], 1).cuda() for i in (0, 1))


@pytest.mark.parametrize("D,G", [(64, 4), (128, 3), (128, 8)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,keys,size", SIZES)
def test_dense(D, G, dtype, n, keys, size):
    k, v = source(keys, 2, D)
    q = (rows(1, n, 2 * G, D) * size).to(dtype)
    out = kvq().kvq_cross_dense_attn(k, v, i32([0, keys]), i32([keys]), q, i32([0, n]), n, D ** -0.5)
    want, most = ref.attention64(q, k, v, [n], [keys], D ** -0.5)
    assert most < 2 ** 6 and ref.off(out, want) < BOUND


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("D,G", [(64, 4), (128, 3), (128, 8)])
@pytest.mark.parametrize("n,keys,size", SIZES)
def test_pages(mode, D, G, n, keys, size):
    K = kvq()
    H, lens = 2, [keys, 37]
    pag, blocks = paging(lens, H, 16, True)
    c = make_cache(mode, H, D, 16, blocks, 0, mode != "INT8_CHANNEL")
    k, v = (torch.cat([a, b]) for a, b in zip(source(keys, H, D), source(37, H, D)))
    K.kvq_write(c, pag, k, v, cu_of(lens))
    k, v = K.kvq_gather(c, pag, cu_of(lens), sum(lens))
    q = rows(1, n + 1, H * G, D) * size
    out = K.kvq_cross_attn(c, pag, q, cu_of([n, 1]), n, D ** -0.5)
    want, most = ref.attention64(q, k, v, [n, 1], lens, D ** -0.5)
    assert most < 2 ** 6 and ref.off(out, want) < BOUND
