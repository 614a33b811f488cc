"""The key/value cache in 4 or 8 bits: the ctypes binding of ``include/lora_quant.h``.

* ``lora_quant_append``: rotary positions of q and k, and the append of k and v to the cache,
  quantised as they are written;
* ``lora_quant_read``: cells as 16-bit rows;
* ``lora_quant_attention``: one query token per row over the cache.

The calls are those of ``step`` over a ``QuantKV`` in the place of its ``PagedKV``: the same
plans, tables, slots, ropes and workspaces, the same checks, torch's current stream.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import binding as B
from . import step as S

BLOCK = 32
EXPORTS = ["lora_quant_append", "lora_quant_read", "lora_quant_attention_bytes", "lora_quant_attention"]

_P, _I32, _I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


class CQuantCache(ctypes.Structure):
    _fields_ = [("type", _I32), ("bits", _I32), ("page_size", _I32), ("num_pages", _I32), ("kv_heads", _I32),
                ("head_dim", _I32), ("page_stride", _I64), ("token_stride", _I64), ("head_stride", _I64),
                ("exp_page_stride", _I64), ("exp_token_stride", _I64), ("exp_head_stride", _I64), ("k", _P), ("v", _P),
                ("k_exp", _P), ("v_exp", _P)]


def _cells(t, what, shape):
    """t: uint8 [num_pages, page_size, kv_heads, cell], unit stride along a cell, entries apart; the bytes from
    its first entry to its last."""
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.uint8:
        raise ValueError(f"{what} must have dtype uint8 (got {getattr(t, 'dtype', type(t).__name__)})")
    if t.layout is not torch.strided or t.is_nested:
        raise ValueError(f"{what} must be a plain strided tensor")
    if tuple(t.shape) != shape:
        raise ValueError(f"{what} is {tuple(t.shape)}, must be {shape}")
    if t.stride(3) != 1 and shape[3] > 1:
        raise ValueError(f"{what} needs unit stride along a cell (stride {t.stride(3)})")
    reach = shape[3]
    for s, n in sorted((s, n) for n, s in zip(shape[:3], t.stride()[:3]) if n > 1):
        if s < reach:
            raise ValueError(f"{what} has overlapping entries (shape {shape}, strides {t.stride()})")
        reach = s * (n - 1) + reach
    return reach


def _apart(x, y, whole_x, whole_y):
    """x and y (of that many bytes from first to last) share no entry: they lie apart, or were cut from records that
    repeat along some dimension and all those outside it: pages with both, or tokens or heads with both."""
    off = y.data_ptr() - x.data_ptr()
    if off < 0:
        x, y, whole_x, whole_y, off = y, x, whole_y, whole_x, -off
    if off >= whole_x:
        return True
    dims = sorted(((s, t, n) for n, s, t in zip(x.shape[:3], x.stride(), y.stride()) if n > 1), reverse=True)
    for i, (s, t, n) in enumerate(dims):
        if s != t:
            return False
        # records of s bytes hold an entry of each, in the same place wherever one begins: at multiples of s, or where
        # the outer dimensions keep them apart
        in_x = x.shape[3] + sum((m - 1) * a for a, _, m in dims[i + 1:])
        in_y = y.shape[3] + sum((m - 1) * b for _, b, m in dims[i + 1:])
        at, reach, clear = off, s * n, True
        if all(a % s == 0 for a, _, _ in dims[:i]):
            at = off % s
        else:
            for a, _, m in reversed(dims[:i]):
                clear = clear and a >= reach
                reach = a * (m - 1) + reach
        if clear and in_x <= at and at + in_y <= s:
            return True
    return False


class QuantKV:
    """lora_quant_cache: k and v uint8 [num_pages, page_size, kv_heads, bytes of codes], k_exp and v_exp uint8
    [num_pages, page_size, kv_heads, blocks], of heads of head_dim columns whose values have dtype (f16 or bf16).
    bits (4 or 8) goes by the bytes of a cell.  Views of another memory order are fine (equal strides for k and v,
    and for k_exp and v_exp), and views of one tensor, cut from pages, tokens or heads that hold several of the four;
    ``zeros`` has heads before tokens in memory, which the attention reads fastest."""

    def __init__(self, k, v, k_exp, v_exp, head_dim, dtype):
        ty = S._TYPES.get(dtype)
        if ty is None:
            raise ValueError(f"dtype must be f16 or bf16 (got {dtype})")
        if not isinstance(k, torch.Tensor) or k.dim() != 4:
            raise ValueError("k must be uint8 [num_pages, page_size, kv_heads, bytes]")
        D = int(head_dim)
        if D < 8 or D > S.MAX_HEAD_DIM or D % 8:
            raise ValueError(f"head_dim = {head_dim} is not a multiple of 8 in 8..{S.MAX_HEAD_DIM}")
        blocks = -(-D // BLOCK)
        bits = {16 * blocks: 4, 32 * blocks: 8}.get(k.shape[3])
        if bits is None:
            raise ValueError(f"cells of {k.shape[3]} bytes: {blocks} blocks of {BLOCK} columns take {16 * blocks} (4 bits) "
                             f"or {32 * blocks} (8 bits)")
        if not k.numel():
            raise ValueError(f"k and v are empty ({tuple(k.shape)})")
        for n, what in zip(k.shape, ("num_pages", "page_size", "kv_heads")):
            S._count(n, what)
        shape, exps = tuple(k.shape), (*k.shape[:3], blocks)
        names = ("k", "v", "k_exp", "v_exp")
        all_ = (k, v, k_exp, v_exp)
        sizes = [_cells(t, what, sh) for t, what, sh in zip(all_, names, (shape, shape, exps, exps))]
        for (t, w), (u, x) in (((k, "k"), (v, "v")), ((k_exp, "k_exp"), (v_exp, "v_exp"))):
            if any(a != b for a, b, n in zip(t.stride(), u.stride(), t.shape) if n > 1):
                raise ValueError(f"{w} and {x} need equal strides (got {t.stride()}, {u.stride()})")
        for t, what in zip(all_[1:], names[1:]):
            if t.device != k.device:
                raise ValueError(f"k is on {k.device}, {what} on {t.device}")
        for i in range(4):
            for j in range(i + 1, 4):
                if not _apart(all_[i], all_[j], sizes[i], sizes[j]):
                    raise ValueError(f"{names[i]} and {names[j]} overlap")
        # a dimension of one entry may have any stride; give the library a valid one
        st = [s if n > 1 else shape[3] for n, s in zip(shape[:3], k.stride()[:3])]
        es = [s if n > 1 else blocks for n, s in zip(shape[:3], k_exp.stride()[:3])]
        self.k, self.v, self.k_exp, self.v_exp, self.bits, self.dtype = k, v, k_exp, v_exp, bits, dtype
        self.num_pages, self.page_size, self.kv_heads, self.head_dim = *shape[:3], D
        self.c = CQuantCache(ty, bits, self.page_size, self.num_pages, self.kv_heads, D, *st, *es, *(S._ptr(t) for t in all_))
        self.ref, self.address = ctypes.byref(self.c), ctypes.addressof(self.c)

    @classmethod
    def zeros(cls, num_pages, page_size, kv_heads, head_dim, dtype=torch.float16, bits=4, device="cuda"):
        """A cache of zeros, heads before tokens in memory."""
        if bits not in (4, 8):
            raise ValueError(f"bits = {bits} is not 4 or 8")
        blocks = -(-int(head_dim) // BLOCK)

        def new(n):
            return torch.zeros((num_pages, kv_heads, page_size, n), dtype=torch.uint8, device=device).transpose(1, 2)

        return cls(new(4 * bits * blocks), new(4 * bits * blocks), new(blocks), new(blocks), head_dim, dtype)


def workspace(n_rows, heads, kv_heads, head_dim, device="cuda"):
    """A zeroed workspace for lora_quant_attention calls of up to n_rows rows and this head layout (the library
    leaves its counters zero after every call)."""
    n = int(B.lib().lora_quant_attention_bytes(S._count(int(n_rows), "n_rows"), S._count(int(heads), "heads"),
                                               S._count(int(kv_heads), "kv_heads"), S._count(int(head_dim), "head_dim")))
    if n == 0:
        raise ValueError(f"{heads} query heads over {kv_heads} key/value heads of {head_dim}, {n_rows} rows")
    return torch.zeros(n // 4, dtype=torch.int32, device=device)


def attention_workspace(n_rows, heads, cache: QuantKV, device=None):
    """workspace for calls over `cache`."""
    return workspace(n_rows, heads, cache.kv_heads, cache.head_dim, cache.k.device if device is None else device)


def _quantised(cache):
    """The library reads a descriptor by its address, so another cache's must not get there."""
    if not isinstance(cache, QuantKV):
        raise ValueError(f"cache must be a QuantKV (got {type(cache).__name__})")


def lora_quant_append(q_out, q, k, v, cache: QuantKV, slots, rope: S.Rope | None = None, positions=None, stream=None):
    """Rotate q into q_out and k into the cache at `slots`, and append v; k and v are quantised.  Arguments as for
    step.lora_rope_append."""
    _quantised(cache)
    rope = S._NoRope if rope is None else rope
    if S._fast:
        dev = S._device(slots)
        if dev >= 0 and S._done(S._fast.quant_append(S._address("lora_quant_append"), S._raw(stream, dev), dev, q_out, q, k,
                                                     v, cache.address, cache.k, slots, rope.address, rope.inv_freq,
                                                     rope.axis, positions)):
            return
    S._append_checked("lora_quant_append", q_out, q, k, v, cache, slots, rope, positions, stream)


def lora_quant_read(k_out, v_out, cache: QuantKV, slots, stream=None):
    """k_out and v_out [n_rows, kv_heads * head_dim] take the values of the cells at `slots` int32 [n_rows]; rows of
    another slot than one of the cache's (-1: none) stay as they were.  Either output may be None."""
    _quantised(cache)
    if S._fast:
        dev = S._device(slots)
        if dev >= 0 and S._done(S._fast.quant_read(S._address("lora_quant_read"), S._raw(stream, dev), dev, k_out, v_out,
                                                   slots, cache.address, cache.k)):
            return
    S._vector(slots, "slots", torch.int32, 0)
    n, cols = S._count(slots.numel(), "n_rows"), cache.kv_heads * cache.head_dim
    ldk = 0 if k_out is None else S._matrix(k_out, "k_out", cache.dtype, n, cols)
    ldv = 0 if v_out is None else S._matrix(v_out, "v_out", cache.dtype, n, cols)
    dev = S._here("slots k_out v_out cache.k", slots, k_out, v_out, cache.k)
    S._call("lora_quant_read", S._raw(stream, dev), n, S._ptr(k_out), ldk, S._ptr(v_out), ldv, slots.data_ptr(), cache.ref)


def lora_quant_attention(out, q, cache: QuantKV, block_table, kv_len, work, req=None, scale=None, window=0, lse=None,
                         stream=None):
    """Attention of one query token per row over the values of the cells; arguments as for
    step.lora_paged_attention, work from attention_workspace."""
    _quantised(cache)
    scale = 1.0 / math.sqrt(cache.head_dim) if scale is None else scale
    if S._fast:
        dev = S._device(q)
        if dev >= 0 and S._done(S._fast.quant_attention(S._address("lora_quant_attention"), S._raw(stream, dev), dev, out, q,
                                                        cache.address, cache.k, block_table, kv_len, work, req, scale,
                                                        window, lse)):
            return
    S._attention_checked("lora_quant_attention", out, q, cache, block_table, kv_len, work, req, scale, window, lse, stream)
