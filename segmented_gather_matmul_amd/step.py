"""Decode-step operators beside the LoRA add-on: the ctypes binding of ``include/lora_step.h``.

* ``lora_kv_plan``: pages, slots and token maps of a step from the requests' lengths;
* ``lora_rope_append``: rotary positions (one or several axes) of q and k, and the append
  of k and v to the paged cache;
* ``lora_paged_attention``: one query token per row over the paged cache;
* ``lora_residual_norm``: the residual add with an optional norm, gate and scale, and the
  next norm.

As in ``binding``, functions carry the C names, tensors are torch tensors on the current
GPU (fp16 or bf16 data, int32 metadata), every tensor is checked before the call, work
runs on torch's current stream, and there is no fallback path.
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch

from . import binding as B

TYPE_F16, TYPE_BF16 = 0, 1
MAX_PAGE, MAX_HEAD_DIM, MAX_AXES, MAX_HIDDEN = 1024, 256, 4, 65536
KV_NO_PAGES, KV_TOO_LONG, KV_TOO_MANY, KV_INVALID = 1, 2, 4, 8
EXPORTS = ["lora_kv_plan", "lora_rope_append", "lora_paged_attention_bytes", "lora_paged_attention",
           "lora_residual_norm"]

_TYPES = {torch.float16: TYPE_F16, torch.bfloat16: TYPE_BF16}
_P, _I32, _I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


class CKVCache(ctypes.Structure):
    _fields_ = [("type", _I32), ("page_size", _I32), ("num_pages", _I32), ("kv_heads", _I32), ("head_dim", _I32),
                ("reserved", _I32), ("page_stride", _I64), ("token_stride", _I64), ("head_stride", _I64), ("k", _P),
                ("v", _P)]


class CKVPages(ctypes.Structure):
    _fields_ = [("n_req", _I32), ("page_size", _I32), ("num_pages", _I32), ("max_blocks", _I32), ("ld_table", _I64),
                ("block_table", _P), ("free_pages", _P), ("free_top", _P)]


class CKVPlanOut(ctypes.Structure):
    _fields_ = [("max_tokens", _I32), ("reserved", _I32), ("status", _P), ("kv_end", _P), ("free_top", _P),
                ("q_ptr", _P), ("tok_req", _P), ("tok_pos", _P), ("slots", _P), ("idx", _P)]


class CRope(ctypes.Structure):
    _fields_ = [("rot_dim", _I32), ("n_axes", _I32), ("interleaved", _I32), ("reserved", _I32), ("inv_freq", _P),
                ("axis", _P)]


class CNormArgs(ctypes.Structure):
    _fields_ = [("type", _I32), ("n_rows", _I32), ("hidden", _I32), ("n_gates", _I32), ("y", _P), ("ldy", _I64),
                ("res_out", _P), ("ldro", _I64), ("res", _P), ("ldr", _I64), ("x", _P), ("ldx", _I64), ("w", _P),
                ("post_w", _P), ("gate", _P), ("ldg", _I64), ("gate_idx", _P), ("alpha", ctypes.c_float),
                ("eps", ctypes.c_float), ("w_offset", ctypes.c_float), ("reserved", _I32)]


_pack_norm = struct.Struct("4i13q3fi").pack   # the bytes of a CNormArgs, in a fifth of the time
assert struct.calcsize("4i13q3fi") == ctypes.sizeof(CNormArgs)


# ------------------------------------------------------------------ argument checks
_NAMES = {torch.float16: "f16", torch.bfloat16: "bf16", torch.float32: "f32", torch.int32: "i32"}


def _type(t, what):
    ty = _TYPES.get(getattr(t, "dtype", None))
    if ty is None:
        raise ValueError(f"{what} must have dtype f16 or bf16 (got {getattr(t, 'dtype', type(t).__name__)})")
    return ty


def _count(n, what):
    """n, which the library takes as 32 bits (ctypes would cut a larger one off)."""
    if not -2 ** 31 <= n < 2 ** 31:
        raise ValueError(f"{what} = {n} does not fit 32 bits")
    return n


# Every call checks every tensor.  A small compiled module makes the checks and the call
# together (2 to 3 microseconds less than Python takes); where it has not been built, or a
# check does not hold, the same rules are gone through below, which say what is wrong.
try:
    from . import _step_args as _fast
except ImportError:
    _fast = None
_CODES = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2, torch.int32: 3}


def _matrix(t, what, dtype, rows, cols):
    """t: 2-D, of `dtype`, unit column stride, >= rows rows and >= cols columns; its row stride."""
    ld = _fast.matrix(t, _CODES[dtype], rows, cols) if _fast else -1
    return ld if ld >= 0 else _matrix_checked(t, what, dtype, rows, cols)


def _matrix_checked(t, what, dtype, rows, cols):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{what} must be a tensor (got {type(t).__name__})")
    if t.dtype is not dtype:
        raise ValueError(f"{what} must have dtype {_NAMES[dtype]} (got {t.dtype})")
    if t.layout is not torch.strided or t.is_nested:
        raise ValueError(f"{what} must be a plain strided tensor")
    if t.dim() != 2:
        raise ValueError(f"{what} must be 2-D (got {t.dim()}-D)")
    n, c = t.shape
    ld, sc = t.stride()
    if c > 1 and sc != 1:
        raise ValueError(f"{what} needs unit stride along its columns (stride {sc})")
    if n < rows or c < cols:
        raise ValueError(f"{what} is {tuple(t.shape)}, needs at least ({rows}, {cols})")
    if n <= 1:  # the stride of a single row has no meaning
        return -(-max(ld, cols) // 8) * 8
    if ld < cols:
        raise ValueError(f"{what} has row stride {ld} < {cols} columns")
    return ld


def _vector(t, what, dtype, n):
    """t: contiguous, of `dtype`, at least n elements."""
    if _fast and _fast.vector(t, _CODES[dtype], n):
        return
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{what} must be a tensor (got {type(t).__name__})")
    if t.dtype is not dtype:
        raise ValueError(f"{what} must have dtype {_NAMES[dtype]} (got {t.dtype})")
    if t.layout is not torch.strided or t.is_nested:
        raise ValueError(f"{what} must be a plain strided tensor")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if t.numel() < n:
        raise ValueError(f"{what} has {t.numel()} elements, needs at least {n}")


def _here(names, *tensors):
    """Every tensor (None: not given) is on the current GPU; its index."""
    dev = _fast.here(*tensors) if _fast else -1
    if dev >= 0 and dev == torch.cuda.current_device():
        return dev
    for what, t in zip(names.split(), tensors):
        if t is not None and not t.is_cuda:
            raise ValueError(f"{what} must be a GPU tensor (got device {t.device})")
    dev = torch.cuda.current_device()
    for what, t in zip(names.split(), tensors):
        if t is not None and t.get_device() != dev:
            raise ValueError(f"{what} is on {t.device}, the current device is cuda:{dev}")
    return dev


def _call(name, *args):
    code = getattr(B._lib or B.lib(), name)(*args)
    if code:
        B._check(code)


_addresses = {}


def _address(name):
    """The library function's address, for the compiled module."""
    a = _addresses.get(name)
    if a is None:
        a = _addresses[name] = ctypes.cast(getattr(B.lib(), name), ctypes.c_void_p).value
    return a


def _done(code):
    """A call by the compiled module: whether it was made (None: a check does not hold)."""
    if code:
        B._check(code)
    return code is not None


def _device(t):
    """The current GPU's index if t is on it, else -1."""
    dev = t.get_device() if isinstance(t, torch.Tensor) else -1
    return dev if dev >= 0 and dev == torch.cuda.current_device() else -1


def _raw(stream, dev):
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else getattr(stream, "cuda_stream", stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


# ------------------------------------------------------------------ descriptors
class PagedKV:
    """lora_kv_cache over k and v tensors [num_pages, page_size, kv_heads, head_dim] (views of
    another memory order, such as head before token, are fine: equal strides for both, unit
    stride along head_dim)."""

    def __init__(self, k, v):
        ty = _type(k, "k")
        if not isinstance(v, torch.Tensor) or v.dtype is not k.dtype:
            raise ValueError(f"v must have k's dtype (got {getattr(v, 'dtype', type(v).__name__)})")
        if k.dim() != 4 or v.shape != k.shape:
            raise ValueError(f"k and v must be [num_pages, page_size, kv_heads, head_dim] (got {tuple(k.shape)}, "
                             f"{tuple(v.shape)})")
        if v.stride() != k.stride() or k.stride(3) != 1:
            raise ValueError(f"k and v need equal strides and unit stride along head_dim (got {k.stride()}, {v.stride()})")
        if k.device != v.device:
            raise ValueError(f"k is on {k.device}, v on {v.device}")
        pages, P, K, D = k.shape
        if not k.numel():
            raise ValueError(f"k and v are empty ({tuple(k.shape)})")
        for n, what in zip(k.shape, ("num_pages", "page_size", "kv_heads", "head_dim")):
            _count(n, what)
        # a dimension of one entry may have any stride; give the library a valid one
        st = [s if n > 1 else max(D, 8) for n, s in zip(k.shape[:3], k.stride()[:3])]
        cells = sorted((s, n) for n, s in zip(k.shape[:3], k.stride()[:3]) if n > 1)
        reach = D
        for s, n in cells:
            if s < reach:
                raise ValueError(f"k has overlapping entries (shape {tuple(k.shape)}, strides {k.stride()})")
            reach = s * (n - 1) + reach
        if not _apart(k, v, reach):
            raise ValueError("k and v overlap")
        self.k, self.v = k, v
        self.dtype, self.num_pages, self.page_size, self.kv_heads, self.head_dim = k.dtype, pages, P, K, D
        self.c = CKVCache(ty, P, pages, K, D, 0, st[0], st[1], st[2], _ptr(k), _ptr(v))
        self.ref, self.address = ctypes.byref(self.c), ctypes.addressof(self.c)


def _apart(k, v, reach):
    """k and v (`reach` elements each) do not overlap, or are taken from one tensor along a
    dimension between theirs (e.g. [pages, 2, ...])."""
    off = abs(v.data_ptr() - k.data_ptr()) // k.element_size()
    if off >= reach:
        return True
    dims = sorted(((s, n) for n, s in zip(k.shape, k.stride()) if n > 1), reverse=True)
    for i, (s, n) in enumerate(dims):
        inner = sum((m - 1) * t for t, m in dims[i + 1:]) + 1
        if inner <= off and off + inner <= s:
            return True
    return False


class KVPages:
    """lora_kv_pages: block_table int32 [n_req, max_blocks], free_pages int32 [num_pages] (a
    stack, last id taken first) and free_top int32 [1], all on the GPU."""

    def __init__(self, block_table, free_pages, free_top, page_size):
        if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2 or block_table.shape[1] < 1:
            raise ValueError("block_table must be int32 [n_req, max_blocks >= 1]")
        n, blocks = _count(block_table.shape[0], "n_req"), _count(block_table.shape[1], "max_blocks")
        _matrix(block_table, "block_table", torch.int32, n, blocks)
        _vector(free_pages, "free_pages", torch.int32, 1)
        _vector(free_top, "free_top", torch.int32, 1)
        if page_size < 1 or page_size > MAX_PAGE or page_size & (page_size - 1):
            raise ValueError(f"page_size = {page_size} is not a power of two in 1..{MAX_PAGE}")
        self.block_table, self.free_pages, self.free_top = block_table, free_pages, free_top
        self.n_req, self.max_blocks, self.page_size = n, blocks, int(page_size)
        ld = block_table.stride(0) if n > 1 else max(block_table.stride(0), blocks)
        self.c = CKVPages(n, self.page_size, _count(free_pages.numel(), "num_pages"), blocks, ld, _ptr(block_table), _ptr(free_pages),
                          _ptr(free_top))
        self.ref, self.address = ctypes.byref(self.c), ctypes.addressof(self.c)

    @classmethod
    def fresh(cls, n_req, max_blocks, num_pages, page_size, device="cuda"):
        """Empty tables over num_pages free pages (handed out 0, 1, 2, ...)."""
        free = torch.arange(num_pages - 1, -1, -1, dtype=torch.int32, device=device)
        return cls(torch.full((n_req, max_blocks), -1, dtype=torch.int32, device=device), free,
                   torch.full((1,), num_pages, dtype=torch.int32, device=device), page_size)


class KVPlan:
    """The output arrays of lora_kv_plan for up to n_req requests and max_tokens token rows.
    kv_end and free_top may be given (e.g. the very tensors the plan reads, to update them
    in place)."""

    def __init__(self, n_req, max_tokens, device="cuda", kv_end=None, free_top=None):
        def new(n):
            return torch.zeros(max(int(n), 1), dtype=torch.int32, device=device)

        self.n_req, self.max_tokens = _count(int(n_req), "n_req"), _count(int(max_tokens), "max_tokens")
        if self.n_req < 0 or self.max_tokens < 0:
            raise ValueError(f"n_req = {n_req}, max_tokens = {max_tokens}")
        if kv_end is not None:
            _vector(kv_end, "kv_end", torch.int32, self.n_req)
        if free_top is not None:
            _vector(free_top, "free_top", torch.int32, 1)
        self.status = new(4)
        self.kv_end = new(self.n_req) if kv_end is None else kv_end
        self.free_top = new(1) if free_top is None else free_top
        self.q_ptr = new(self.n_req + 1)
        self.tok_req, self.tok_pos, self.slots, self.idx = (new(max_tokens)[:self.max_tokens] for _ in range(4))
        self.c = CKVPlanOut(self.max_tokens, 0, _ptr(self.status), _ptr(self.kv_end), _ptr(self.free_top),
                            _ptr(self.q_ptr), _ptr(self.tok_req), _ptr(self.tok_pos), _ptr(self.slots), _ptr(self.idx))
        self.ref, self.address = ctypes.byref(self.c), ctypes.addressof(self.c)


class Rope:
    """lora_rope: inv_freq fp32 [rot_dim / 2]; axis int32 [rot_dim / 2] or None (all on axis 0);
    axes position axes; interleaved pairs (x[2i], x[2i + 1]) or halves (x[i], x[i + rot_dim/2])."""

    def __init__(self, inv_freq, axis=None, axes=1, interleaved=False):
        _vector(inv_freq, "inv_freq", torch.float32, 0)
        half = inv_freq.numel()
        _count(2 * half, "rot_dim")
        if axis is not None:
            _vector(axis, "axis", torch.int32, half)
        if half % 8 or not 1 <= axes <= MAX_AXES:
            raise ValueError(f"{half} frequencies (a multiple of 8), {axes} axes (1..{MAX_AXES})")
        self.inv_freq, self.axis, self.axes, self.rot_dim = inv_freq, axis, int(axes), 2 * half
        self.c = CRope(2 * half, self.axes, 1 if interleaved else 0, 0, _ptr(inv_freq) if half else None, _ptr(axis))
        self.ref, self.address = ctypes.byref(self.c), ctypes.addressof(self.c)

    @classmethod
    def base(cls, rot_dim, theta=10000.0, axis=None, axes=1, interleaved=False, device="cuda"):
        """inv_freq[i] = theta^(-2i / rot_dim)."""
        f = torch.tensor([theta ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)], dtype=torch.float32, device=device)
        return cls(f, axis, axes, interleaved)


class _NoRope:
    rot_dim, inv_freq, axis = 0, None, None
    c = CRope(0, 1, 0, 0, None, None)
    ref, address = ctypes.byref(c), ctypes.addressof(c)


def workspace(n_rows, heads, kv_heads, head_dim, device="cuda"):
    """A zeroed workspace for lora_paged_attention calls of up to n_rows rows and this head
    layout (the library leaves its counters zero after every call)."""
    n = int(B.lib().lora_paged_attention_bytes(_count(int(n_rows), "n_rows"), _count(int(heads), "heads"),
                                               _count(int(kv_heads), "kv_heads"), _count(int(head_dim), "head_dim")))
    if n == 0:
        raise ValueError(f"{heads} query heads over {kv_heads} key/value heads of {head_dim}, {n_rows} rows")
    return torch.zeros(n // 4, dtype=torch.int32, device=device)


def attention_workspace(n_rows, heads, cache: PagedKV, device=None):
    """workspace for calls over `cache`."""
    return workspace(n_rows, heads, cache.kv_heads, cache.head_dim, cache.k.device if device is None else device)


# ------------------------------------------------------------------ launches
def lora_kv_plan(plan: KVPlan, pages: KVPages, kv_len, new_len, req_slot=None, stream=None):
    """Plan one step: new_len tokens (-1: ended) for each request of kv_len cached tokens; pages
    move between pages.free_pages and pages.block_table, and `plan` receives the maps."""
    n = pages.n_req
    if n > plan.n_req:
        raise ValueError(f"a plan for {plan.n_req} requests, tables of {n}")
    if _fast:
        dev = _device(kv_len)
        if dev >= 0 and _done(_fast.plan(_address("lora_kv_plan"), _raw(stream, dev), dev, plan.address, pages.address,
                                         kv_len, new_len, req_slot, pages.block_table, pages.free_pages, pages.free_top,
                                         plan.status, plan.kv_end, plan.free_top)):
            return
    _vector(kv_len, "kv_len", torch.int32, n)
    _vector(new_len, "new_len", torch.int32, n)
    if req_slot is not None:
        _vector(req_slot, "req_slot", torch.int32, n)
    dev = _here("kv_len new_len req_slot block_table free_pages free_top status kv_end plan.free_top", kv_len, new_len,
                req_slot, pages.block_table, pages.free_pages, pages.free_top, plan.status, plan.kv_end, plan.free_top)
    _call("lora_kv_plan", _raw(stream, dev), pages.ref, kv_len.data_ptr(), new_len.data_ptr(),
                                  _ptr(req_slot), plan.ref)


def _paged(cache):
    """The library reads a descriptor by its address, so another cache's must not get there."""
    if not isinstance(cache, PagedKV):
        raise ValueError(f"cache must be a PagedKV (got {type(cache).__name__})")


def lora_rope_append(q_out, q, k, v, cache: PagedKV, slots, rope: Rope | None = None, positions=None, stream=None):
    """Rotate q into q_out and k into the cache at `slots`, and append v.  positions int32
    [axes, n_rows] (1-D for one axis); rope None appends without rotation.  q and q_out may
    both be None (k and v only); q_out may be q."""
    _paged(cache)
    rope = _NoRope if rope is None else rope
    if _fast:
        dev = _device(slots)
        if dev >= 0 and _done(_fast.append(_address("lora_rope_append"), _raw(stream, dev), dev, q_out, q, k, v,
                                           cache.address, cache.k, slots, rope.address, rope.inv_freq, rope.axis,
                                           positions)):
            return
    _append_checked("lora_rope_append", q_out, q, k, v, cache, slots, rope, positions, stream)


def _append_checked(entry, q_out, q, k, v, cache, slots, rope, positions, stream):
    dt, D = cache.dtype, cache.head_dim
    _vector(slots, "slots", torch.int32, 0)
    n = _count(slots.numel(), "n_rows")
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out go together")
    heads = ldq = ldqo = 0
    if q is not None:
        if q.dim() != 2 or q.shape[1] % D:
            raise ValueError(f"q is {tuple(q.shape)}, its columns must be heads of {D}")
        heads = _count(q.shape[1] // D, "heads")
        ldq = _matrix(q, "q", dt, n, heads * D)
        ldqo = _matrix(q_out, "q_out", dt, n, heads * D)
    ldk = _matrix(k, "k", dt, n, cache.kv_heads * D)
    ldv = _matrix(v, "v", dt, n, cache.kv_heads * D)
    ldp = n
    if not rope.rot_dim:
        positions = None
    else:
        if not isinstance(positions, torch.Tensor):
            raise ValueError("positions must be a tensor")
        if positions.dim() not in (1, 2):
            raise ValueError(f"positions must be [axes, n_rows] or, for one axis, [n_rows] (got {positions.dim()}-D)")
        p2 = positions if positions.dim() == 2 else positions[None]
        ldp = _matrix(p2, "positions", torch.int32, rope.axes, n)
        ldp = p2.stride(0) if p2.shape[0] > 1 else max(n, 1)
    dev = _here("slots k v q q_out positions cache.k inv_freq axis", slots, k, v, q, q_out, positions, cache.k,
                rope.inv_freq, rope.axis)
    _call(entry, _raw(stream, dev), n, heads, _ptr(q_out), ldqo, _ptr(q), ldq, k.data_ptr(), ldk,
                                      v.data_ptr(), ldv, rope.ref, _ptr(positions), ldp, slots.data_ptr(), cache.ref)


def lora_paged_attention(out, q, cache: PagedKV, block_table, kv_len, work, req=None, scale=None, window=0, lse=None,
                         stream=None):
    """Attention of one query token per row: q and out [n_rows, heads * head_dim], block_table
    int32 [n_req, max_blocks], kv_len int32 [n_rows], req int32 [n_rows] or None (row i reads
    table row i), lse fp32 [n_rows, heads] or None, work from attention_workspace."""
    _paged(cache)
    scale = 1.0 / math.sqrt(cache.head_dim) if scale is None else scale
    if _fast:
        dev = _device(q)
        if dev >= 0 and _done(_fast.attention(_address("lora_paged_attention"), _raw(stream, dev), dev, out, q,
                                              cache.address, cache.k, block_table, kv_len, work, req, scale, window, lse)):
            return
    _attention_checked("lora_paged_attention", out, q, cache, block_table, kv_len, work, req, scale, window, lse, stream)


def _attention_checked(entry, out, q, cache, block_table, kv_len, work, req, scale, window, lse, stream):
    dt, D = cache.dtype, cache.head_dim
    if not isinstance(q, torch.Tensor) or q.dim() != 2 or q.shape[1] % D:
        raise ValueError(f"q must be [n_rows, heads * {D}]")
    n, cols = q.shape
    heads = _count(cols // D, "heads")
    _count(n, "n_rows")
    window = _count(int(window), "window")
    ldq = _matrix(q, "q", dt, n, cols)
    ldo = _matrix(out, "out", dt, n, cols)
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be int32 [n_req, max_blocks]")
    n_req, blocks = _count(block_table.shape[0], "n_req"), _count(block_table.shape[1], "max_blocks")
    _matrix(block_table, "block_table", torch.int32, n_req, blocks)
    ldt = block_table.stride(0) if n_req > 1 else max(blocks, 1)
    _vector(kv_len, "kv_len", torch.int32, n)
    if req is not None:
        _vector(req, "req", torch.int32, n)
    if lse is not None:
        _vector(lse, "lse", torch.float32, n * heads)
        if n > 1 and lse.dim() > 1 and lse.numel() != lse.shape[0] * heads:
            raise ValueError(f"lse is {tuple(lse.shape)}, its rows must be of {heads} heads")
    _vector(work, "work", torch.int32, 1)
    dev = _here("q out block_table kv_len req lse work cache.k", q, out, block_table, kv_len, req, lse, work, cache.k)
    _call(entry, _raw(stream, dev), n, heads, out.data_ptr(), ldo, q.data_ptr(), ldq,
                                          cache.ref, n_req, block_table.data_ptr(), ldt, blocks, kv_len.data_ptr(),
                                          _ptr(req), float(scale), window,
                                          _ptr(lse), work.data_ptr(), 4 * work.numel())


def lora_residual_norm(y, res, w=None, x=None, res_out=None, post_w=None, gate=None, gate_idx=None, alpha=1.0, eps=1e-5,
                       w_offset=0.0, stream=None):
    """h = res + alpha * gate * (norm of x with post_w, or x); res_out <- h, y <- norm of h with
    w.  y or res_out may be None; res_out may be res, y may be x; x None adds nothing."""
    if _fast:
        dev = _device(res)
        if dev >= 0 and _done(_fast.norm(_address("lora_residual_norm"), _raw(stream, dev), dev, y, res, w, x, res_out,
                                         post_w, gate, gate_idx, alpha, eps, w_offset)):
            return
    ty = _type(res, "res")
    if res.dim() != 2:
        raise ValueError(f"res must be 2-D (got {res.dim()}-D)")
    n, h = _count(res.shape[0], "n_rows"), _count(res.shape[1], "hidden")
    dt = res.dtype
    ldr = _matrix(res, "res", dt, n, h)
    yp = ldy = wp = rp = ldro = xp = ldx = pp = gp = ldg = ip = n_gates = 0
    if y is not None:
        ldy, yp = _matrix(y, "y", dt, n, h), y.data_ptr()
        _vector(w, "w", dt, h)
        wp = w.data_ptr()
    else:
        w = None
    if res_out is not None:
        ldro, rp = _matrix(res_out, "res_out", dt, n, h), res_out.data_ptr()
    if x is not None:
        ldx, xp = _matrix(x, "x", dt, n, h), x.data_ptr()
    if post_w is not None:
        _vector(post_w, "post_w", dt, h)
        pp = post_w.data_ptr()
    if gate is not None:
        ldg, gp, n_gates = _matrix(gate, "gate", dt, 1, h), gate.data_ptr(), _count(gate.shape[0], "n_gates")
    if gate_idx is not None:
        _vector(gate_idx, "gate_idx", torch.int32, n)
        ip = gate_idx.data_ptr()
    dev = _here("res y res_out x w post_w gate gate_idx", res, y, res_out, x, w, post_w, gate, gate_idx)
    _call("lora_residual_norm", _raw(stream, dev),
          _pack_norm(ty, n, h, n_gates, yp, ldy, rp, ldro, res.data_ptr(), ldr, xp, ldx, wp, pp, gp, ldg, ip, alpha, eps,
                     w_offset, 0))
