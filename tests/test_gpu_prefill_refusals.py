"""The prefill calls of the binding refuse what would pass the end of a tensor, and take larger buffers."""
import pytest
import torch

import kvq_inputs as gen
from harness import build_case, kvq, q_host, to_dev_input, write_step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def case():
    wl = gen.custom(gen.MODE_INT4, 8, 2, 128, 16, "bf16", seq_lens=[70, 33], n_new=[20, 33], step="prefill",
                    seed=6)
    c = build_case(wl)
    write_step(c)
    q = to_dev_input(q_host(wl), wl.dtype)
    cu = torch.from_numpy(wl.cu(wl.n_new)).cuda()
    return c, q, cu


def test_paged_prefill(case):
    K = kvq()
    c, q, cu = case
    T = q.shape[0]
    call = lambda q=q, cu=cu, **kw: K.kvq_prefill_attn(c.gcache, c.gpag, q, cu, 33, 0.1, **kw)  # noqa: E731
    want = call()
    f = lambda *s: torch.full(s, -3.0, device="cuda")  # noqa: E731
    for kw in (dict(q=q[:, :, :64].contiguous()), dict(cu=cu[:2].contiguous()), dict(out=f(T - 1, 8, 128)),
               dict(out=f(T, 8, 64)), dict(q=q.cpu()), dict(cu=cu.cpu()), dict(out=torch.empty((T, 8, 128)))):
        with pytest.raises(ValueError):
            call(**kw)
    out = f(T + 2, 8, 128)
    wide = torch.cat([cu, cu[-1:], cu[-1:]])
    assert call(cu=wide, out=out) is out
    assert torch.equal(out[:T], want) and bool((out[T:] == -3).all())


def test_dense_prefill(case):
    K = kvq()
    c, q, cu = case
    T = q.shape[0]
    lens = c.gpag.seq_lens
    cu_kv = torch.tensor([0, 70, 103], dtype=torch.int32, device="cuda")
    k, v = K.kvq_gather(c.gcache, c.gpag, cu_kv, 103, out_dtype=torch.bfloat16)
    ok = dict(k=k, v=v, cu_kv=cu_kv, seq_lens=lens, q=q, cu_q=cu)
    call = lambda **kw: K.kvq_prefill_dense_attn(max_q_per_seq=33, softmax_scale=0.1, **{**ok, **kw})  # noqa: E731
    want = call()
    f = lambda *s: torch.full(s, -3.0, device="cuda")  # noqa: E731
    win = torch.zeros(1, dtype=torch.int32, device="cuda")
    for kw in (dict(q=q[:, :, :64].contiguous()), dict(cu_q=cu[:2].contiguous()), dict(cu_kv=cu_kv[:2].contiguous()),
               dict(out=f(T - 1, 8, 128)), dict(window_per_kv_head=win), dict(k=k.view(103, 256), v=v.view(103, 256)),
               *({n: t.cpu()} for n, t in ok.items() if n != "k"), dict(out=torch.empty((T, 8, 128)))):
        with pytest.raises(ValueError):
            call(**kw)
    out = f(T + 2, 8, 128)
    assert torch.equal(call(out=out, cu_q=torch.cat([cu, cu[-1:]]), cu_kv=torch.cat([cu_kv, cu_kv[-1:]]))[:T], want)
    assert bool((out[T:] == -3).all())
