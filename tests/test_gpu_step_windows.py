"""The fused step with windows and sinks per kv head, over every mode, against 64 bits on the rows that are seen; a NaN in
a row outside the window stays outside.  test_gpu_step_accuracy's bound."""
import math

import pytest
import torch

import accuracy_ref as ref
from harness import kvq
from test_gpu_rope import MODES, cu_of, i32, make_cache, make_rope, paging, rows
from test_gpu_step_accuracy import BOUND

pytestmark = pytest.mark.gpu


def seen_rows(L, window, sink):
    j = torch.arange(L, device="cuda")
    return (j < sink) | (j > L - 1 - window) if window > 0 else j >= 0


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("D,G", [(64, 4), (128, 5), (128, 1)])
@pytest.mark.parametrize("wide", [0, 4096])
def test_windows(mode, D, G, wide):
    """`wide`: pages of room behind each sequence's own, so that the call is not a small one."""
    K = kvq()
    lens, sink, wins = [1, 33, 300, 777], 5, [0, 40, 129]
    H, B = len(wins), len(lens)
    pag, blocks = paging(lens, H, 16, False)
    t = torch.nn.functional.pad(pag.block_tables, (0, wide), value=-1).contiguous()
    pag = K.Paging(pag.seq_lens, block_tables=t, window_per_kv_head=i32(wins), sink_size=sink)
    c = make_cache(mode, H, D, 16, blocks)
    K.kvq_write(c, pag, rows(8, sum(lens), H, D), rows(9, sum(lens), H, D), cu_of(lens))
    q, new = rows(3, B, H * G, D), (rows(4, B, H, D), rows(5, B, H, D))
    rope = make_rope(D)
    out = K.kvq_rope_write_decode_attn(c, pag, rope, *new, cu_of([1] * B), q, D ** -0.5)
    qt, _ = K.kvq_rope(rope, q, None, positions=pag.seq_lens - 1)
    k, v = K.kvq_gather(c, pag, cu_of(lens), sum(lens))
    want, at = torch.zeros_like(out, dtype=torch.float64), 0
    for b, L in enumerate(lens):
        for h, w in enumerate(wins):
            s = seen_rows(L, w, sink)
            got, most = ref.attention64(qt[b:b + 1, h * G:(h + 1) * G], k[at:at + L][s][:, h:h + 1], v[at:at + L][s][:, h:h + 1], [1],
                                        [int(s.sum())], D ** -0.5)
            want[b:b + 1, h * G:(h + 1) * G] = got
            assert most < 16
        at += L
    assert ref.off(out, want) < BOUND


@pytest.mark.parametrize("at,reaches", [(2, True), (7, False), (500, False), (700, True), (776, True)])
def test_nan_outside_a_window(at, reaches):
    K = kvq()
    H, G, D, L, sink, win = 1, 4, 128, 778, 5, 129
    pag, blocks = paging([L], H, 16, False)
    pag = K.Paging(pag.seq_lens, block_tables=pag.block_tables, window_per_kv_head=i32([win]), sink_size=sink)
    c = make_cache("FP8_TOKEN_HEAD", H, D, 16, blocks, 0, False)
    k, v = rows(1, L, H, D), rows(2, L, H, D)
    v[at, 0, 9] = math.nan
    K.kvq_write(c, pag, k, v, cu_of([L]))
    out = K.kvq_rope_write_decode_attn(c, pag, make_rope(D), rows(4, 1, H, D), rows(5, 1, H, D), cu_of([1]), rows(3, 1, G, D), D ** -0.5)
    bad = torch.isnan(out)
    assert bool(bad[:, :, 9].all()) is reaches and int(bad.sum()) == (G if reaches else 0)
