"""Rotary positions in 64 bits, and what the fp32 arithmetic may be off by."""
import math

import torch


def turn64(x, pos, freq, inter, scale=1.0):
    """x [tokens, heads, d] at positions pos [tokens], in float64 on the CPU; freq [rot / 2] (the fp32 values)."""
    x = x.detach().cpu().double()
    f = freq.detach().cpu().double()
    r = 2 * f.numel()
    a = pos.detach().cpu().double()[:, None, None] * f
    c, s = torch.cos(a) * scale, torch.sin(a) * scale
    y = x.clone()
    i = torch.arange(r // 2)
    p, q = (2 * i, 2 * i + 1) if inter else (i, i + r // 2)
    y[..., p] = x[..., p] * c - x[..., q] * s
    y[..., q] = x[..., q] * c + x[..., p] * s
    return y


def tolerance(x, y, freq, inter, scale, dtype):
    """How far turned rows may be from y = turn64(x).

    The angle: what is left of a quadrant is at most pi / 4 radians, rounded to fp32 and multiplied by a rounded
    constant with one more rounding, 3 * 2^-24 of it; the fixed point drops 2^-32 + 2^-33 of a turn.  Together
    pi / 4 * 3 * 2^-24 + 2 pi * 1.5 * 2^-32 < 1.45e-7.  Sine and cosine: the series' rest (2e-9) and its last two
    roundings, 2 * 2^-24, the others being damped by z <= 0.62 and its coefficients: < 1.3e-7; the scale's product
    2^-24.  So each is off by less than 3.4e-7 of `scale`; the row's product and sum add 2 * 2^-24 of |a| + |b|.
    4.7e-7 < 2^-21 in all.  A bf16 result is off by half a step more, 2^-8 of its size."""
    x = x.detach().cpu().double()
    r = 2 * freq.numel()
    i = torch.arange(r // 2)
    p, q = (2 * i, 2 * i + 1) if inter else (i, i + r // 2)
    t = torch.zeros_like(x)
    both = (x[..., p].abs() + x[..., q].abs()) * abs(scale) * 2.0 ** -21
    t[..., p] = both
    t[..., q] = both
    if dtype == torch.bfloat16:
        t = t + (y.abs() + t) * 2.0 ** -8
        if r < x.shape[-1]:
            t[..., r:] = 0  # dims that do not turn come back as they were
    return t


def frequencies64(rot, base=10000.0):
    return [base ** (-2 * i / rot) for i in range(rot // 2)]


def by_turns(rot, base, factor, context, fast, slow):
    """(frequencies, scale) of the ramp over the pairs' numbers, element by element."""
    def pair(turns):
        return rot * math.log(context / (turns * 2 * math.pi)) / (2 * math.log(base))
    lo, hi = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), rot - 1)
    out = []
    for i, f in enumerate(frequencies64(rot, base)):
        ramp = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
        out.append(f * (1 - ramp) + f / factor * ramp)
    return out, 0.1 * math.log(factor) + 1


def by_wavelength(rot, base, factor, context, fast, slow):
    out = []
    for f in frequencies64(rot, base):
        wave = 2 * math.pi / f
        if wave < context / fast:
            out.append(f)
        elif wave > context / slow:
            out.append(f / factor)
        else:
            s = (context / wave - slow) / (fast - slow)
            out.append((1 - s) * f / factor + s * f)
    return out, 1.0
