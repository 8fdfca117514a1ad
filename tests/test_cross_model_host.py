"""The bound of test_gpu_cross_accuracy.py against a model of the kernels' operand terms: with every term the model stays
well inside it, with the last of a weight's or of a query's terms left out it does not, at any size."""
import pytest
import torch

import cross_model as model
from test_gpu_cross_accuracy import BOUND, SIZES

BF16, FP16 = torch.bfloat16, torch.float16


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,keys,size", SIZES)
def test_terms_left_out(D, n, keys, size):
    q, k, v = (t.double().numpy() for t in model.inputs(keys, 6 * n, keys, D, size=size))  # (heads of a group and of the cache: as many queries)
    want = model.attention(q, k, v, D ** -0.5)

    def off(q_terms, weight_terms):
        return model.off(model.attention(q, k, v, D ** -0.5, q_terms, weight_terms), want)
    # 16-bit rows: three bf16 terms of a query, two of a weight; quantised ones: two fp16 terms of each
    assert off((BF16, 3), (BF16, 2)) < 0.7 * BOUND and off((FP16, 2), (FP16, 2)) < 0.7 * BOUND
    assert off((BF16, 3), (BF16, 1)) > BOUND and off((FP16, 2), (FP16, 1)) > BOUND
    assert off((FP16, 1), (FP16, 2)) > BOUND
    # (of two queries over 130 rows, three quarters of it: 2.8e-6)
    assert off((BF16, 2), (BF16, 2)) > (BOUND if n > 2 else 0.75 * BOUND)
