"""Plain reference of sampling (lora_sample.h) on the CPU, row by row by its definition.  Test infrastructure only.

Weights are floor(2^40 exp(z)) of a 64-bit exponential here and of one right to 2^-37 in the kernel, so that they differ
by 2^-37 of a weight and a unit; the masses up to a token then by 2^-37 of themselves and a unit a token, and a draw whose
u M lies that near a border between two of n tokens takes the other one: a chance below n (2^-37 + n 2^-40) a row,
5 10^-3 at 70,000 tokens of equal weight and far less where few hold the mass; the inputs here are fixed and were drawn
once.  logprob: z and the logarithm in 64 bits, rounded to 32: 2^-24 (|z| + |log|) and half a step of the result; the
mass M by 2^-37 of itself, within half of the bound from 8 tokens on (one token's weight is exact), and a unit in 2^40 a token.
"""
import math

import torch

F64 = torch.float64
UNIT = 2.0 ** 40


def sample(logits, t, k, p, m, u):
    """(token, logprob, bound of logprob) of one row (any float type, CPU); None where its settings are out of range."""
    if not (t >= 0 and t < math.inf and k >= 0 and 0 <= p <= 1 and 0 <= m <= 1 and 0 <= u < 1):
        return None
    x = logits.to(F64).nan_to_num(nan=-math.inf, posinf=math.inf, neginf=-math.inf)
    V = x.numel()
    top = float(x.max())
    if top == -math.inf:
        return -1, -math.inf, 0.0
    x, order = torch.sort(x, descending=True, stable=True)     # -0 equals 0
    if t == 0:
        return int(order[0]), 0.0, 0.0
    if top == math.inf:
        z = torch.where(x == math.inf, 0.0, -math.inf).to(F64)
    else:
        z = (x - top) / t
    w = (torch.exp(z) * UNIT).floor().to(torch.int64)
    k = V if k == 0 else min(k, V)
    w[k:] = 0
    before = w.cumsum(0) - w
    total = int(w.sum())
    keep = before.to(F64) < p * float(total)
    keep[0] = True
    keep &= w.to(F64) >= m * UNIT
    w = torch.where(keep, w, 0)
    line = torch.zeros_like(w)
    line[order] = w
    line = line.cumsum(0)
    total = int(line[-1])
    at = min(int(u * float(total)), total - 1)
    token = int((line <= at).sum())
    zt = float(z[(order == token).nonzero()[0, 0]])
    mass = math.log(total / UNIT)
    lp = zt - mass
    return token, lp, 2.0 ** -23 * (abs(zt) + abs(mass)) + V * 2.0 ** -40
