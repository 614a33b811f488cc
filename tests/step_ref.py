"""Plain 64-bit references of the decode-step operators (lora_step.h) on the CPU, and the
tolerances their tests use.  Test infrastructure only.

Roundings counted by the tolerances, with u = 2^-24 (half a step of fp32, relative) and
half_step(t) = finfo(t).eps / 2 for the output type t:
  rotary   cos and sin are off by at most pi 2^-25 (the reduced angle rounded to fp32) plus
           4 u (two fp32 units of the sine), under 2^-22; a product and a fused
           multiply-add round twice more: |err| <= half_step |y| + 2^-21 (|a| + |b|).  The
           reference's own angle is a 64-bit product, off by 2^-53 of itself: where that is
           more than 2^-23 (positions beyond 10^9), it is counted too, in (|a| + |b|).
  attention  a score is a sum of D products in fp32, scaled and moved to base 2:
           ds = (D + 8) u |scale| max_t sum_d |q_d k_td|, both for the score and for the
           maximum it is compared with; exp2, the split of p into two 16-bit parts and the
           rescaling: 2^-15 for bf16 (two parts of 8 bits), 2^-20 for fp16; sums over
           tokens run in chains of at most n/16 + 64 terms: (n/16 + 64) u.  With
           rel = 2 ds + that + the chain, the numerator is off by rel sum p|v| and the
           denominator by rel: |err| <= half_step |o| + 2 rel sum_t p_t |v_t|;
           lse: rel + 4 u (|lse| + ds).
  norm     the mean of squares is a chain of at most hidden/64 + 32 terms of one sign, a
           division, a square root and a reciprocal: inv is off by r = (hidden/64 + 40) u
           relative; h by 4 u (|res| + |alpha g p|) plus r |alpha g p| with a post norm.
"""
import math

import torch

U = 2.0 ** -24
F64 = torch.float64


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Half of the smallest step (outputs below the normal range)."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


# ------------------------------------------------------------------ step plan
def plan(kv_len, new_len, table, free, top, page, max_tokens, req_slot=None):
    """The plan by its definition, one request after another, on Python lists."""
    n, num_pages, max_blocks = len(kv_len), len(free), len(table[0]) if table else 1
    blocks = lambda t: -(-t // page)
    bits = 0
    tokens = taken = given = 0
    for c, m in zip(kv_len, new_len):
        if c < 0 or m < -1:
            bits |= 8
            continue
        if c + max(m, 0) > max_blocks * page:
            bits |= 2
        tokens += max(m, 0)
        if m < 0:
            given += blocks(c)
        else:
            taken += blocks(c + m) - blocks(c)
    if not 0 <= top <= num_pages or top + given > num_pages:
        bits |= 8
    if taken > top + given:
        bits |= 1
    if tokens > max_tokens:
        bits |= 4
    status = [bits] + [min(v, 2 ** 31 - 1) for v in (tokens, taken, given)]
    if bits:
        none = [-1] * max_tokens
        return dict(status=status, kv_end=list(kv_len), free_top=top, q_ptr=[0] * (n + 1), tok_req=none, tok_pos=none,
                    slots=none, idx=none, table=table, free=free)
    table, free = [list(r) for r in table], list(free)
    for r in range(n):
        if new_len[r] < 0:
            for b in range(blocks(kv_len[r])):
                free[top] = table[r][b]
                top += 1
    q_ptr, tok_req, tok_pos, slots, idx, kv_end = [0], [], [], [], [], []
    for r in range(n):
        m = max(new_len[r], 0)
        end = 0 if new_len[r] < 0 else kv_len[r] + m
        if new_len[r] >= 0:
            for b in range(blocks(kv_len[r]), blocks(end)):
                top -= 1
                table[r][b] = free[top]
        for i in range(m):
            pos = kv_len[r] + i
            pg = table[r][pos // page]
            tok_req.append(r)
            tok_pos.append(pos)
            slots.append(pg * page + pos % page if 0 <= pg < num_pages else -1)
            idx.append(-1 if req_slot is None else req_slot[r])
        q_ptr.append(q_ptr[-1] + m)
        kv_end.append(end)
    pad = [-1] * (max_tokens - len(tok_req))
    return dict(status=status, kv_end=kv_end, free_top=top, q_ptr=q_ptr, tok_req=tok_req + pad, tok_pos=tok_pos + pad,
                slots=slots + pad, idx=idx + pad, table=table, free=free)


# ------------------------------------------------------------------ rotary positions
def rotate(x, pos, inv_freq, axis, n_axes, interleaved):
    """x [n, heads, D] (16-bit) -> (rotated in 64 bits, |a| + |b| of each element's pair)."""
    y = x.to(F64).clone()
    mag = torch.zeros_like(y)
    for i in range(len(inv_freq)):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, len(inv_freq) + i)
        ax = 0 if axis is None else int(axis[i])
        ang = pos[ax].to(F64) * float(inv_freq[i]) if 0 <= ax < n_axes else torch.zeros(x.shape[0], dtype=F64)
        c, s = ang.cos()[:, None], ang.sin()[:, None]
        xa, xb = x[:, :, a].to(F64), x[:, :, b].to(F64)
        y[:, :, a], y[:, :, b] = xa * c - xb * s, xa * s + xb * c
        mag[:, :, a] = mag[:, :, b] = (xa.abs() + xb.abs()) * (1 + ang.abs()[:, None] * 2.0 ** (21 - 53))
    return y, mag


# ------------------------------------------------------------------ attention
def attention(q, k, v, table, kv_len, req, scale, window, heads):
    """q [n, heads, D]; k, v [pages, page, kv_heads, D] (all CPU).  (out, lse, bound of out,
    bound of lse) in 64 bits; rows that are not active give None."""
    pages, P, K, D = k.shape
    G = heads // K
    bf = q.dtype == torch.bfloat16
    res = []
    for i in range(q.shape[0]):
        r = i if req is None else int(req[i])
        n = int(kv_len[i])
        if n < 0 or n > table.shape[1] * P or not 0 <= r < table.shape[0]:
            res.append(None)
            continue
        t = torch.arange(max(0, n - window) if window else 0, n)
        pg = table[r].long()[t // P]
        ok = (pg >= 0) & (pg < pages)
        t, pg = t[ok], pg[ok]
        kk, vv = k[pg, t % P].to(F64), v[pg, t % P].to(F64)     # [T, K, D]
        qq = q[i].to(F64).reshape(K, G, D)
        s = torch.stack([qq[g] @ kk[:, g].T for g in range(K)]) * scale   # [K, G, T]
        ab = torch.stack([qq[g].abs() @ kk[:, g].abs().T for g in range(K)]) * abs(scale)
        if t.numel() == 0 or bool((s == -math.inf).all()):
            none = torch.zeros(heads, D, dtype=F64)
            res.append((none, torch.full((heads,), -math.inf, dtype=F64), none, torch.zeros(heads, dtype=F64)))
            continue
        m = s.amax(-1, keepdim=True)
        m = torch.where(m == -math.inf, torch.zeros_like(m), m)
        p = torch.exp(s - m)
        l = p.sum(-1, keepdim=True)
        w = torch.where(l == 0, torch.zeros_like(p), p / l)      # a NaN score makes its row NaN
        o = torch.stack([w[g] @ vv[:, g] for g in range(K)])
        av = torch.stack([w[g] @ vv[:, g].abs() for g in range(K)])
        ds = (D + 8) * U * ab.amax(-1, keepdim=True)
        rel = 2 * ds + (2.0 ** -15 if bf else 2.0 ** -20) + (t.numel() / 16 + 64) * U
        lse = torch.where(l == 0, torch.full_like(l, -math.inf), m + l.log())
        bo = half_step(q.dtype) * o.abs() + 2 * rel * av + tiny(q.dtype)
        bl = rel + 4 * U * (lse.abs() + ds)
        res.append(tuple(x.reshape(heads, -1) if x.dim() == 3 and x.shape[-1] == D else x.reshape(heads)
                         for x in (o, lse, bo, bl)))
    return res


# ------------------------------------------------------------------ norms
def residual_norm(res, x, w, post_w, gate, gate_idx, alpha, eps, w_offset):
    """(h, y, bound of h, bound of y) in 64 bits, before rounding (all inputs 16-bit, CPU)."""
    hid = res.shape[1]
    r = (hid / 64 + 40) * U
    rms = lambda z: 1.0 / torch.sqrt((z * z).mean(-1, keepdim=True) + eps)
    res = res.to(F64)
    add = torch.zeros_like(res)
    e_add = torch.zeros_like(res)
    if x is not None:
        p = x.to(F64)
        if post_w is not None:
            p = p * rms(p) * (post_w.to(F64) + w_offset)
        if gate is not None:
            g = torch.ones_like(res) if gate_idx is not None else gate[:1].to(F64).expand_as(res).clone()
            if gate_idx is not None:
                on = gate_idx >= 0
                g[on] = gate.to(F64)[gate_idx[on].long().clamp(max=gate.shape[0] - 1)]
            p = p * g
        add = alpha * p
        e_add = (r if post_w is not None else 0.0) * add.abs()
    h = res + add
    e_h = 4 * U * (res.abs() + add.abs()) + e_add
    inv = rms(h)
    y = e_y = None
    if w is not None:
        ww = w.to(F64) + w_offset
        y = h * inv * ww
        # inv from h's own error: d inv / inv <= rms-relative error of h
        e_inv = r + torch.sqrt((e_h * e_h).mean(-1, keepdim=True)) * inv
        e_y = (e_inv + 4 * U) * y.abs() + e_h * inv * ww.abs()
    return h, y, e_h, e_y
