"""Windows and sinks of 16-bit pages under a uniform table: some heads slide, some see everything, over the same pages."""
import numpy as np
import pytest
import torch

import decode16_ref as ref
from harness import kvq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("window", [[0, 1, 16], [40, 0, 300], [17, 17, 17], [5000, 64, 33]])
@pytest.mark.parametrize("sink,bs,D", [(0, 16, 128), (3, 32, 64), (20, 64, 128), (70, 16, 64)])
def test_windows_under_a_uniform_table(window, sink, bs, D, dtype):
    lens = [900, 75, 17, 300, 1, 0]
    c = ref.make(6, 3, 5, D, bs, lens, dtype, window=window, sink=sink, seed=sink + window[0])
    t = c["pag"].block_tables
    t[0, 1] = -1                # a hole inside a sequence, for every head
    t[2] = -1                   # a sequence that leaves nothing
    c["table"] = t.view(6, 1, -1).cpu().numpy().copy()
    out = kvq().kvq_decode_attn(c["cache"], c["pag"], c["q"], c["scale"], dev_error=c["err"])
    want = ref.attention64(c)
    ref.check(out, want)
    assert not out[2].any() and not out[5].any() and int(c["err"].item()) == 0
    for splits in (1, 7, 500):
        ref.check(kvq().kvq_decode_attn(c["cache"], c["pag"], c["q"], c["scale"], num_splits=splits), want)


def test_short_calls_with_windows_under_a_uniform_table():
    """A narrow table: the form of one launch."""
    c = ref.make(3, 2, 4, 128, 16, [48, 20, 33], window=[7, 0], sink=2, seed=4)
    ref.check(kvq().kvq_decode_attn(c["cache"], c["pag"], c["q"], c["scale"]), ref.attention64(c))


def test_a_window_that_starts_past_the_table():
    K = kvq()
    c = ref.make(3, 2, 4, 128, 16, [90, 208, 40], window=[16, 0], sink=20, seed=12, max_blocks=13)
    c["pag"].seq_lens.copy_(torch.tensor([90, 5000, 40]))
    out = K.kvq_decode_attn(c["cache"], c["pag"], c["q"], c["scale"], dev_error=c["err"])
    ref.check(out, ref.attention64(c, lens=np.array([90, 5000, 40])))
    assert int(c["err"].item()) == K.KVQ_DEVERR_TABLE_RANGE
