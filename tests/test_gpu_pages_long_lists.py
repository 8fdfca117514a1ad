"""kvq_copy_pages over lists long enough to be checked in scratch: every kind of conflict, in both forms of the copies."""
import numpy as np
import pytest
import torch

import pages_ref as ref
from harness import kvq
from test_gpu_pages import apply, caches, i32, pools, same

pytestmark = pytest.mark.gpu


def pairs(r, blocks, fill):
    """Chains, cycles, destinations named twice, pages onto themselves (some of them written by another pair, some read),
    pairs past the pool and negative ones, and `fill` pairs that conflict with nothing, in random order."""
    order = r.permutation(blocks)
    at = 0

    def take(n):
        nonlocal at
        at += n
        return list(order[at - n:at])

    out = []
    for n in (2, 3, 40):
        c = take(n)
        out += list(zip(c, c[1:]))                      # a chain
        c = take(n)
        out += list(zip(c, c[1:] + c[:1]))              # a cycle
    for _ in range(30):
        a, b, c, d = take(4)
        out += [(a, d), (b, d), (c, d)]                 # one destination, three sources
        a, b, c = take(3)
        out += [(a, a), (b, a), (a, c)]                 # onto itself, written by another pair and read by a third
        a, b = take(2)
        out += [(a, b), (a, b)]                         # the same pair twice
        a, b = take(2)
        out += [(a, blocks), (blocks + 7, b), (-1, b), (a, -3)]
    out += [(a, b) for a, b in zip(take(fill), take(fill))]
    out = np.array(out)[r.permutation(len(out))]
    return out[:, 0], out[:, 1]


# pools of one piece a page: one layer (runs over several pairs, eight steps), three with more pairs (32 steps), sixteen
# (runs within a pair)
@pytest.mark.parametrize("layers,fill", [(1, 2000), (3, 3500), (16, 2000)])
@pytest.mark.parametrize("headwise", [False, True])
def test_conflicts(layers, fill, headwise):
    K = kvq()
    r = np.random.default_rng(layers)
    Hkv, blocks = (2, 5000) if headwise else (1, 10000)
    modes, dims = ("INT2_TOKEN_HEAD", "INT4_TOKEN_HEAD", "INT8_TOKEN_HEAD"), (64, 64, 128)
    cs = caches(blocks, Hkv, 16, [modes[i % 3] for i in range(layers)], [dims[i % 3] for i in range(layers)], seed=layers)
    src, dst = pairs(r, blocks * Hkv if headwise else blocks, fill)
    assert len(src) > 2048
    need = K.kvq_copy_workspace_size(cs, len(src), headwise)
    assert need >= 4 * blocks * (Hkv if headwise else 1)
    ws = torch.full((need,), 0x5A, dtype=torch.uint8, device="cuda")
    before, err = pools(cs), torch.zeros(1, dtype=torch.int32, device="cuda")
    done, bits = ref.copy_pairs(src, dst, blocks * (Hkv if headwise else 1))
    assert len(done) >= fill + 30 and bits == ref.CONFLICT | K.KVQ_DEVERR_BLOCK_RANGE
    flat = [p.reshape(-1, *p.shape[2:]) for p in before] if headwise else before
    want = apply(flat, [(0, a, b) for a, b in done], False)
    for fill_byte in (0x5A, 0xFF, 0x00):        # what the scratch holds does not matter
        ws.fill_(fill_byte)
        for c, k, v in zip(cs, before[::2], before[1::2]):
            c.k_pages.copy_(torch.from_numpy(k))
            c.v_pages.copy_(torch.from_numpy(v))
        err.zero_()
        K.kvq_copy_pages(cs, i32(src), i32(dst), headwise=headwise, workspace=ws, dev_error=err)
        got = pools(cs)
        same([p.reshape(w.shape) for p, w in zip(got, want)], want)
        assert int(err.item()) == bits
