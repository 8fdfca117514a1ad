"""Decode calls behind a kernel that lets them start while it still runs: what that kernel writes is read after it has,
and what it reads is written after it has."""
import ctypes
import importlib.util
import os
import subprocess

import numpy as np
import pytest
import torch

from harness import kvq

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
WAIT_NS = 300000    # longer than any of the calls below takes
MODES = ["BF16_CACHE", "INT4_TOKEN_HEAD", "INT2_TOKEN_HEAD", "INT4_STEGO", "INT8_TOKEN_HEAD", "FP8_TOKEN_HEAD", "INT8_CHANNEL"]


@pytest.fixture(scope="module")
def late(tmp_path_factory):
    """late(dst, src): dst = src, some time after the next kernel may have started."""
    spec = importlib.util.spec_from_file_location(
        "kvq_build_lib", os.path.join(os.path.dirname(HERE), "sub_byte_quantized_write_gb300", "build_lib.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    so = str(tmp_path_factory.mktemp("early") / "libearly_release.so")
    subprocess.run([b._nvcc(), *b.ARCH, "-O2", "-std=c++17", "-Xcompiler", "-fPIC", "-shared", "-o", so,
                    os.path.join(HERE, "early_release.cu")], check=True)
    f = ctypes.CDLL(so).late_copy
    f.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_longlong, ctypes.c_ulonglong, ctypes.c_void_p]

    def copy(dst, src):
        assert dst.is_contiguous() and src.is_contiguous() and dst.nbytes == src.nbytes and dst.nbytes % 4 == 0
        assert f(dst.data_ptr(), src.data_ptr(), dst.nbytes // 4, WAIT_NS, torch.cuda.current_stream().cuda_stream) == 0
    return copy


def state(mode, D, short):
    """A cache of four sequences with two tables, lengths and queries to choose from, all of them in range."""
    K = kvq()
    H, G, bs = 2, 4, 16
    lens = np.array([20, 31, 7, 16] if short else [900, 40, 333, 1200])
    width = 2 if short else 80
    r = np.random.default_rng(D + short)
    n = -(-lens // bs)
    blocks = int(n.sum()) + 9
    cache = K.PagedCache(getattr(K, "KVQ_" + mode), blocks, H, bs, D)
    tables = np.zeros((2, 4, width), np.int32)
    for t in tables:
        perm, o = r.permutation(blocks), 0
        for b in range(4):
            t[b, :n[b]] = perm[o:o + n[b]]
            o += n[b]
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    T = int(lens.sum())
    k = torch.from_numpy(r.standard_normal((2, T, H, D), dtype=np.float32)).cuda().bfloat16()
    cu = i32(np.concatenate([[0], np.cumsum(lens)]))
    for t in tables[::-1]:      # (pages of both hold rows; the first table's win)
        K.kvq_write(cache, K.Paging(i32(lens), block_tables=i32(t)), k[0], k[1], cu)
    q = torch.from_numpy(r.standard_normal((2, 4, H * G, D), dtype=np.float32)).cuda().bfloat16()
    new = torch.from_numpy(r.standard_normal((2, 2, 4, H, D), dtype=np.float32)).cuda().bfloat16()
    return dict(cache=cache, scale=D ** -0.5, window=i32([0, 24]),
                block_tables=(i32(tables[0]), i32(tables[1])), seq_lens=(i32(lens), i32(np.maximum(1, lens // 2))),
                q=(q[0], q[1]), k=(new[0, 0], new[1, 0]), v=(new[0, 1], new[1, 1]), cu=(i32([0, 1, 2, 3, 4]), i32([0, 1, 2, 2, 2])))


def caller(s, kind, x, ws, out):
    """The call over the tensors x, with the cache as it was before it."""
    K = kvq()
    pag = K.Paging(x["seq_lens"], block_tables=x["block_tables"], window_per_kv_head=s["window"], sink_size=3)
    if kind == "noalloc":
        return lambda: K.kvq_decode_attn_noalloc(s["cache"], pag, x["q"], s["scale"], out=out)
    if kind == "step":
        return lambda: K.kvq_write_decode_attn(s["cache"], pag, x["k"], x["v"], x["cu"], x["q"], s["scale"], out=out, workspace=ws)
    return lambda: K.kvq_decode_attn(s["cache"], pag, x["q"], s["scale"], out=out, workspace=ws)


NAMES = ("block_tables", "seq_lens", "q", "k", "v", "cu")
CASES = [(m, d, short, kind) for m in MODES for d in (64, 128) for short in (False, True) for kind in ("decode", "noalloc", "step")
         if not (m == "INT8_CHANNEL" and kind == "step") and not (d == 64 and kind == "noalloc") and not (short and m not in MODES[:2])]


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("mode,D,short,kind", CASES)
def test_inputs_and_buffers_of_a_kernel_that_still_runs(mode, D, short, kind, captured, late):
    K = kvq()
    s = state(mode, D, short)
    pools = s["cache"].k_pages.clone(), s["cache"].v_pages.clone()

    def reset():
        s["cache"].k_pages.copy_(pools[0])
        s["cache"].v_pages.copy_(pools[1])

    x = {n: s[n][0].clone() for n in NAMES}
    need, _ = K.kvq_decode_workspace_size(s["cache"], K.Paging(x["seq_lens"], block_tables=x["block_tables"]), 8)
    ws, out = torch.empty(need, dtype=torch.uint8, device="cuda"), torch.empty((4, 8, D), device="cuda")
    call = caller(s, kind, x, ws, out)
    call()                      # (the first call sets kernel attributes)
    reset()
    call()
    want = out.clone()
    after = s["cache"].k_pages.clone(), s["cache"].v_pages.clone()

    def run(before):
        if not captured:
            before()
            call()
        else:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                before()
                call()
            graph.replay()
        torch.cuda.synchronize()

    for n in NAMES if kind == "step" else NAMES[:3]:    # other values, until the kernel before has written these
        reset()
        x[n].copy_(s[n][1])
        out.fill_(-3)
        torch.cuda.synchronize()
        run(lambda: late(x[n], s[n][0]))
        assert torch.equal(out, want), n
        assert torch.equal(s["cache"].k_pages, after[0]) and torch.equal(s["cache"].v_pages, after[1]), n
    for buf in ([] if kind == "noalloc" else [ws[:need // 4 * 4]]) + [out]:     # what the kernel before still reads
        reset()
        held = torch.empty_like(buf)
        buf.view(torch.int32).fill_(0x12345678)
        torch.cuda.synchronize()
        run(lambda: late(held, buf))
        assert bool((held.view(torch.int32) == 0x12345678).all())
        assert torch.equal(out, want)
