"""A NaN among the values of 8-bit floating rows reaches the outputs of the queries that see it, by the kernels for few
queries and for many alike; one in a row that they do not see (behind the last, in a page that is not theirs) does not."""
import pytest
import torch

from harness import kvq
from test_gpu_rope import cu_of, make_cache, make_rope, paging, rows


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 4, 8])
@pytest.mark.parametrize("row", [0, 70, 191, 192, 199])  # in full tiles of 32 and 128 keys, in the last and behind its page's first half
def test_visible_nan(D, G, row):
    K = kvq()
    H, lens = 2, [200, 90]
    pag, blocks = paging(lens, H, 16, False)
    c = make_cache("FP8_TOKEN_HEAD", H, D, 16, blocks, 0, False)
    c.k_pages.fill_(0xFF)  # (a NaN in E4M3: rows behind a sequence's last hold nothing else)
    c.v_pages.fill_(0xFF)
    k, v = rows(1, sum(lens), H, D), rows(2, sum(lens), H, D)
    v[row, 1, 5] = float("nan")
    K.kvq_write(c, pag, k, v, cu_of(lens))
    _, back = K.kvq_gather(c, pag, cu_of(lens), sum(lens))
    assert int(torch.isnan(back).sum()) == 1 and bool(torch.isnan(back[row, 1, 5]))
    for n in ((2, 1), (40, 3), (1, 1)):
        q = rows(3, sum(n), H * G, D)
        out = K.kvq_cross_attn(c, pag, q, cu_of(n), max(n), D ** -0.5)
        want = torch.zeros(out.shape, dtype=torch.bool, device="cuda")
        want[:n[0], G:, 5] = True
        assert torch.equal(torch.isnan(out), want), n
        assert bool(torch.isfinite(out[~want]).all())
    # a step's values: the new row holds it
    new = rows(4, 2, H, D), rows(5, 2, H, D)
    new[1][0, 0, 7] = float("nan")
    q = rows(6, 2, H * G, D)
    out = K.kvq_rope_write_decode_attn(c, pag, make_rope(D), *new, cu_of((1, 1)), q, D ** -0.5)
    want = torch.zeros(out.shape, dtype=torch.bool, device="cuda")
    want[0, :G, 7] = True
    want[0, G:, 5] = row != 199  # (the new row takes the last one's place)
    assert torch.equal(torch.isnan(out), want)
