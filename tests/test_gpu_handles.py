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
