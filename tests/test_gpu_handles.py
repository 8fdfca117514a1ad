"""Handles that change after their first call, on the GPU."""
import numpy as np
import pytest
import torch

import decode16_ref as ref
from harness import kvq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("headwise", [False, True])
def test_tables_of_other_widths_on_a_used_handle(headwise):
    """A wider table, then a narrower one: what a call reads and writes goes by the width of the table that is set."""
    K = kvq()
    B, Hkv, bs = 3, 2, 16
    c = ref.make(B, Hkv, 4, 128, bs, [100, 33, 60], headwise=headwise, seed=7)
    kind = "block_tables_headwise" if headwise else "block_tables"
    pag, spaces = c["pag"], Hkv if headwise else 1
    want = ref.attention64(c)
    ref.check(K.kvq_decode_attn(c["cache"], pag, c["q"], c["scale"]), want)
    held = getattr(pag, kind)
    wide = torch.full((B * spaces, 11), 10 ** 6, dtype=torch.int32, device="cuda")
    wide[:, :7] = held
    setattr(pag, kind, wide)
    ref.check(K.kvq_decode_attn(c["cache"], pag, c["q"], c["scale"], dev_error=c["err"]), want)
    assert int(c["err"].item()) == 0
    # the narrower one stands between guards; a fork into it and an in-place compaction leave them alone
    buf = torch.full((B * spaces * 5 + 200,), 77, dtype=torch.int32, device="cuda")
    narrow = buf[100:100 + B * spaces * 5].view(B * spaces, 5)
    out = K.Paging(torch.zeros(B, dtype=torch.int32, device="cuda"), **{kind: torch.empty_like(wide)})
    out.struct()
    setattr(out, kind, narrow)
    old = K.Paging(torch.tensor([64, 33, 60], dtype=torch.int32, device="cuda"), **{kind: held[:, :5].contiguous()})
    K.kvq_fork(c["cache"], old, torch.arange(B, dtype=torch.int32, device="cuda"), out=out, dev_error=c["err"])
    K.kvq_compact(c["cache"], out, out=out, dev_error=c["err"])
    got = K.kvq_decode_attn(c["cache"], out, c["q"], c["scale"], dev_error=c["err"])
    ref.check(got, ref.attention64(c, lens=np.array([64, 33, 60])))
    assert int(c["err"].item()) == 0
    assert bool((buf[:100] == 77).all()) and bool((buf[-100:] == 77).all())
    used = (torch.tensor([64, 33, 60]) + bs - 1) // bs
    assert ((narrow >= 0).sum(1).view(B, spaces).cpu() == used[:, None]).all()


@pytest.mark.parametrize("side", [False, True])
def test_compaction_into_a_state_with_lengths_of_its_own(side):
    K = kvq()
    c = ref.make(3, 2, 4, 128, 16, [100, 33, 60], seed=8)
    want = ref.attention64(c)
    pag = c["pag"]
    out = K.Paging(torch.full((3,), 10 ** 6, dtype=torch.int32, device="cuda"), block_tables=torch.empty_like(pag.block_tables))
    stream = torch.cuda.Stream() if side else None
    if side:
        stream.wait_stream(torch.cuda.current_stream())
    got, _, _, used = K.kvq_compact(c["cache"], pag, out=out, stream=stream)
    o = K.kvq_decode_attn(c["cache"], got, c["q"], c["scale"], dev_error=c["err"], stream=stream)
    torch.cuda.synchronize()
    assert got is out and out.seq_lens.tolist() == [100, 33, 60] and int(c["err"].item()) == 0
    assert int(out.block_tables.max()) == int(used) - 1
    ref.check(o, want)
    with pytest.raises(ValueError):     # lengths of another number of rows
        K.kvq_compact(c["cache"], pag, out=K.Paging(out.seq_lens[:2], block_tables=out.block_tables))
    # captured: the lengths follow at each replay
    graph, ws = torch.cuda.CUDAGraph(), torch.empty(K.kvq_compact_workspace_size(c["cache"], pag), dtype=torch.uint8, device="cuda")
    with torch.cuda.graph(graph):
        K.kvq_compact(c["cache"], got, out=pag, workspace=ws)
    pag.seq_lens.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert pag.seq_lens.tolist() == [100, 33, 60]


def test_compaction_into_a_table_without_lengths():
    K = kvq()
    c = ref.make(3, 2, 4, 128, 16, [100, 33, 60], seed=8)
    out, _, _, used = K.kvq_compact(c["cache"], c["pag"], out=K.Paging(None, block_tables=torch.empty_like(c["pag"].block_tables)))
    assert out.seq_lens is None and int(out.block_tables.max()) == int(used) - 1
