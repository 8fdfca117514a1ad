"""Rotary positions without a GPU: the frequencies of every kind of scaling, the refusals of the calls, and the
fixed-point angles against exact integers."""
import ctypes

import numpy as np
import pytest
import torch

import rope_ref as ref
from test_abi import K, _cache, _paging  # noqa: F401  (K: the fixture)


@pytest.mark.parametrize("rot", [16, 48, 64, 128])
@pytest.mark.parametrize("base", [10000.0, 500000.0])
def test_frequencies(K, rot, base):  # noqa: F811
    cases = [(K.KVQ_ROPE_PLAIN, {}, (ref.frequencies64(rot, base), 1.0)),
             (K.KVQ_ROPE_LINEAR, dict(factor=4.0), ([f / 4 for f in ref.frequencies64(rot, base)], 1.0)),
             (K.KVQ_ROPE_BASE, dict(factor=8.0), (ref.frequencies64(rot, base * 8.0 ** (rot / (rot - 2))), 1.0)),
             (K.KVQ_ROPE_TURNS, dict(factor=16.0, context=4096, fast=32, slow=1),
              ref.by_turns(rot, base, 16.0, 4096, 32, 1)),
             (K.KVQ_ROPE_WAVELENGTH, dict(factor=8.0, context=8192, fast=4, slow=1),
              ref.by_wavelength(rot, base, 8.0, 8192, 4, 1))]
    for kind, kw, (want, scale) in cases:
        got, s = K.kvq_rope_frequencies(rot, base, kind, device="cpu", **kw)
        # fp32 of a value worked out in 64 bits: half a step, 2^-24, and a few roundings of 2^-53
        assert np.allclose(got.double().numpy(), want, rtol=2.0 ** -24 * 1.001, atol=0), kind
        assert abs(s - scale) <= 2.0 ** -24 * scale


def test_frequency_refusals(K):  # noqa: F811
    for a, kw in (((0,), {}), ((15,), {}), ((64, 1.0), {}), ((64, float("inf")), {}), ((64, 1e4, 9), {}),
                  ((64, 1e4, K.KVQ_ROPE_LINEAR), dict(factor=0.5)), ((2, 1e4, K.KVQ_ROPE_BASE), dict(factor=2.0)),
                  ((64, 1e4, K.KVQ_ROPE_TURNS), dict(factor=2.0)),
                  ((64, 1e4, K.KVQ_ROPE_WAVELENGTH), dict(factor=2.0, context=4096, fast=1, slow=1))):
        with pytest.raises(K.KvqError):
            K.kvq_rope_frequencies(*a, device="cpu", **kw)


def test_angles_in_fixed_point():
    """The integer steps of the kernels' angles (a restatement), against exact integers: below 2^-31 of a turn off."""
    from fractions import Fraction
    inv_two_pi = Fraction(0x28BE60DB9391054A7F09D5F47D4D377036D8A5664F10E410, 1 << 192)  # 1 / (2 pi)
    C, M64 = 0xA2F9836E4E44152A, (1 << 64) - 1
    r = np.random.Generator(np.random.PCG64(3))
    f = np.concatenate([np.float32([1.0, 0.5, 1e-4, 1e-6, 0.99999994, 3.0, 200.0, 1e-38, 0.0]),
                        (10.0 ** r.uniform(-6, 0, 200)).astype(np.float32)])
    pos = [0, 1, -1, 8191, 131071, 1000003, 2 ** 31 - 1, -2 ** 31]
    for x in f:
        for sign in (1, -1):
            bits = int(np.float32(x).view(np.uint32))
            ex, m = bits >> 23 & 255, (bits & 0x7FFFFF) | (0x800000 if bits >> 23 & 255 else 0)
            sh = 2 - ((ex or 1) - 150)
            u = ((m * C >> sh) if sh >= 0 else m * C << -sh) & M64
            u = -u & M64 if sign < 0 else u
            for p in pos:
                ul, uh, up = u & 0xFFFFFFFF, u >> 32, p & 0xFFFFFFFF
                top = ((ul * up >> 32) + uh * up - (ul if p < 0 else 0)) & 0xFFFFFFFF
                turn = Fraction(top, 1 << 32) - sign * Fraction(float(x)) * p * inv_two_pi
                off = abs(turn - round(turn))
                assert off < Fraction(1, 1 << 31), (x, p, float(off))


def _rotary(K, **kw):
    base = dict(inv_freq=4096, rot_dim=128, interleaved=0, scale=1.0)
    base.update(kw)
    return K.KvqRotary(**base)


def test_rope_refusals(K):  # noqa: F811
    L, ref_ = K.lib(), ctypes.byref
    pg = _paging(K)

    def rope(r, pos=None, paging=pg, cu=4096, q=4096, qo=1 << 20, hq=2, qs=0, qos=0, k=None, ko=None, hk=0, ks=0, kos=0,
             d=128, dtype=1, n=4):
        return L.kvq_rope(None if r is None else ref_(r), pos, None if paging is None else ref_(paging), cu, q, qo, hq, qs,
                          qos, k, ko, hk, ks, kos, d, dtype, n, None, None)
    bad, no = K.KVQ_ERR_INVALID_ARG, K.KVQ_ERR_UNSUPPORTED
    r = _rotary(K)
    assert rope(None) == bad and rope(_rotary(K, inv_freq=None)) == bad and rope(_rotary(K, inv_freq=4097)) == bad
    for rot in (0, -16, 8, 24, 144):
        assert rope(_rotary(K, rot_dim=rot)) == no
    assert rope(_rotary(K, rot_dim=128), d=64) == no and rope(r, d=96) == no and rope(r, dtype=2) == no
    assert rope(_rotary(K, interleaved=2)) == bad
    assert rope(_rotary(K, scale=float("nan"))) == bad and rope(_rotary(K, scale=float("inf"))) == bad
    assert rope(r, n=-1) == bad and rope(r, paging=None) == bad and rope(r, cu=None) == bad
    assert rope(r, paging=_paging(K, seq_lens=None)) == bad and rope(r, paging=_paging(K, batch=-1)) == bad
    assert rope(r, q=None) == bad and rope(r, qo=None) == bad and rope(r, hq=0) == bad
    assert rope(r, q=4104) == bad and rope(r, qo=(1 << 20) + 8) == bad
    assert rope(r, qs=128) == bad and rope(r, qs=260) == bad and rope(r, qos=-256) == bad
    assert rope(r, qs=1 << 62) == no and rope(r, hq=1 << 22) == no
    # outputs over inputs that are not themselves
    assert rope(r, qo=4096 + 256) == bad                               # half a row on
    assert rope(r, qo=4096, qs=256, qos=512) == bad                    # itself at another stride
    assert rope(r, k=8192, ko=1 << 20, hk=2) == bad                    # both outputs in one place
    assert rope(r, k=8192, ko=4096, hk=2) == bad                       # k's output over q
    assert rope(r, qs=512, qos=512, qo=4096 + 256, k=8192, ko=1 << 21, hk=1) == bad
    assert rope(r, n=0) == K.KVQ_OK and rope(r, pos=4096, paging=None, cu=None, n=0) == K.KVQ_OK
    assert rope(r, paging=_paging(K, batch=0)) == K.KVQ_OK


def test_rope_write_refusals(K):  # noqa: F811
    L, ref_ = K.lib(), ctypes.byref
    int8 = _cache(K, mode=K.KVQ_INT8_CHANNEL, ch_amax=4096, ch_amax_ready=4096)

    def write(c, r, k=4096, dtype=1, n=2):
        return L.kvq_rope_write(ref_(c), ref_(_paging(K)), None if r is None else ref_(r), None, k, 4096, dtype, 4096, n,
                                None, None)

    def step(c, r, k=4096, dtype=1, ws=1 << 20):
        return L.kvq_rope_write_decode_attn(ref_(c), ref_(_paging(K)), None if r is None else ref_(r), None, k, 4096, dtype,
                                            4096, 2, 256, 1, 8, 0.1, 256, 256, ws, 0, None, None)
    bad, no = K.KVQ_ERR_INVALID_ARG, K.KVQ_ERR_UNSUPPORTED
    r, c64 = _rotary(K), _cache(K, head_dim=64)
    for f in (write, step):
        assert f(int8, r) == no and f(_cache(K), None) == bad and f(_cache(K), r, k=None) == bad
        assert f(c64, r) == no and f(_cache(K), _rotary(K, rot_dim=40)) == no and f(_cache(K), r, dtype=7) == no
        assert f(_cache(K), _rotary(K, inv_freq=None)) == bad
    assert step(_cache(K), r, ws=16) == K.KVQ_ERR_WORKSPACE
    assert write(_cache(K), r, n=0) == K.KVQ_OK and write(_cache(K), r, n=-1) == bad


def test_binding_refusals(K):  # noqa: F811
    rope = K.Rope(torch.zeros(32))
    q = torch.zeros((3, 2, 64))
    with pytest.raises(ValueError, match="CUDA|device"):
        K.kvq_rope(rope, q, None, positions=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="neither"):
        K.kvq_rope(rope, None, None)
    assert rope.rot_dim == 64 and rope.scale == 1.0 and not rope.interleaved
