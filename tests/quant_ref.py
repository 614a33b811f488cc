"""Plain 64-bit references of the quantised cache's operators (lora_quant.h) on the CPU, and the tolerances their
tests use.  Test infrastructure only.

  quantise  exact: a block's exponent and codes by their definition, from inputs of 32 bits or fewer.
  append    v is quantised from 16-bit values, exactly.  k is turned in 64 bits (products and sums off by 2^-50 of
            |a| + |b|, the reference's own angle by 2^-53 of itself) and rounded to 32 (2^-24 of its value), so the
            quantised value lies between those of y - d and y + d (rounding to a grid is monotone), with
            d = 2^-24 |y| + (|a| + |b|) (2^-48 + 2^-52 angle).
  q_out     as step_ref: half_step |y| + 2^-21 (|a| + |b|).
  attention the cells' values are 16-bit values, so step_ref's bounds of the 16-bit attention hold; weights here are
            cut off below 2^-38 of the row's largest (fp16), which adds n 2^-37 max|v| to a row of n tokens.
"""
import math

import torch

from tests import step_ref as R

F64 = torch.float64
E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=F64)
E4M3 = torch.tensor([m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1],
                    dtype=F64)


def blocks(D):
    return -(-D // 32)


def grid(bits):
    return E2M1 if bits == 4 else E4M3


def exponent_range(dtype, bits):
    """Of e - 127 as written, straight from the table in lora_quant.h."""
    return {(torch.float16, 4): (-23, 13), (torch.float16, 8): (-15, 7), (torch.bfloat16, 4): (-125, 125),
            (torch.bfloat16, 8): (-117, 119)}[dtype, bits]


def exponents(x, bits, dtype):
    """Exponent bytes [..., blocks] of x [..., D] (64-bit): the smallest power that fits, one by one."""
    D = x.shape[-1]
    x = torch.nn.functional.pad(x, (0, 32 * blocks(D) - D)).reshape(*x.shape[:-1], -1, 32)
    most = x.abs().amax(-1)
    lo, hi = exponent_range(dtype, bits)
    edge = 7.0 if bits == 4 else 464.0
    e = torch.full_like(most, lo)
    for i in range(lo, hi):
        e += (most >= edge * 2.0 ** i).to(F64)
    e = e + 127
    return torch.where(torch.isfinite(x).all(-1), e, torch.full_like(e, 255.0))


def nearest(x, exps, bits):
    """x [..., D] on the grid of its block's exponent: nearest, ties to the even code, too large ones to the largest."""
    D = x.shape[-1]
    unit = torch.exp2(exps - 127).repeat_interleave(32, -1)[..., :D]
    g = grid(bits)
    a = (x.abs() / unit).clamp(max=float(g[-1])).nan_to_num(0.0)
    hi = torch.searchsorted(g, a.contiguous()).clamp(1, g.numel() - 1)
    down, up = a - g[hi - 1], g[hi] - a
    pick = torch.where((down < up) | ((down == up) & (hi % 2 == 1)), hi - 1, hi)
    y = torch.copysign(g[pick] * unit, x)
    return torch.where(exps.repeat_interleave(32, -1)[..., :D] == 255, torch.full_like(y, math.nan), y)


def quantise(x, bits, dtype):
    """(values, exponent bytes) of x [..., D] in 64 bits."""
    e = exponents(x, bits, dtype)
    return nearest(x, e, bits), e


def values(code, exp, bits, D):
    """What codes and exponents stand for (uint8, CPU), bit by bit."""
    code = code.long()
    if bits == 4:
        code = torch.stack([code % 16, code // 16], -1).flatten(-2)
        sign, mag = code // 8, code % 8
    else:
        sign, mag = code // 128, code % 128
    g = torch.cat([grid(bits), torch.tensor([math.nan], dtype=F64)])
    x = g[mag] * (1 - 2 * sign)
    e = exp.to(F64).repeat_interleave(32, -1)
    return torch.where(e == 255, torch.full_like(x, math.nan), x * torch.exp2(e - 127))[..., :D]


def pack(x, exps, bits):
    """Codes uint8 of values x [..., D] that lie on their blocks' grids (padded with 0)."""
    D = x.shape[-1]
    unit = torch.exp2(exps.to(F64) - 127).repeat_interleave(32, -1)
    x = torch.nn.functional.pad(x, (0, unit.shape[-1] - D))
    g = grid(bits)
    mag = torch.searchsorted(g, (x.abs() / unit).nan_to_num(0.0).contiguous()).clamp(max=g.numel() - 1)
    code = (mag + (8 if bits == 4 else 128) * torch.signbit(x).long()).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4) if bits == 4 else code


def rotated_bounds(x, pos, inv_freq, axis, n_axes, interleaved):
    """(y, d) of k [n, heads, D]: the turned values and how far the kernel's may be off before they are quantised."""
    y, _ = R.rotate(x, pos, inv_freq, axis, n_axes, interleaved)
    d = torch.zeros_like(y)
    for i in range(len(inv_freq)):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, len(inv_freq) + i)
        ax = 0 if axis is None else int(axis[i])
        if not 0 <= ax < n_axes:
            continue
        ang = (pos[ax].to(F64) * float(inv_freq[i])).abs()[:, None]
        mag = x[:, :, a].to(F64).abs() + x[:, :, b].to(F64).abs()
        d[:, :, a] = d[:, :, b] = mag * (2.0 ** -48 + ang * 2.0 ** -52)
    return y, d + 2.0 ** -24 * y.abs()


def check_quantised(got, exps, y, d, bits, dtype, what):
    """got [..., D] (64-bit) with exponent bytes exps: what some value within d of y quantises to, block by block."""
    lo, hi = exponents(y.abs() - d.clamp(max=y.abs()), bits, dtype), exponents(y.abs() + d, bits, dtype)
    e = exps.to(F64)
    assert bool(((e >= lo) & (e <= hi)).all()), f"{what}: exponents {e[(e < lo) | (e > hi)][:4].tolist()}"
    least, most = nearest(y - d, e, bits), nearest(y + d, e, bits)
    bad = ~((got >= least) & (got <= most)) & ~(got.isnan() & least.isnan())
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, first {got[bad][0]} for {y[bad][0]}"


def attention(q, k, v, table, kv_len, req, scale, window, heads):
    """step_ref.attention over values k, v [pages, page, kv_heads, D] of q's type, with the bound above."""
    res = R.attention(q, k, v, table, kv_len, req, scale, window, heads)
    top = v.to(F64).abs().nan_to_num(0.0).max() if v.numel() else 0.0
    cut = 2.0 ** -37 if q.dtype == torch.float16 else 0.0
    return [None if r is None else (r[0], r[1], r[2] + cut * max(int(kv_len[i]), 0) * top, r[3]) for i, r in enumerate(res)]
