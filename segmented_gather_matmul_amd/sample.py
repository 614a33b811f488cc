"""The end of a serving step, from logits to tokens: the ctypes binding of ``include/lora_sample.h``.

* ``lora_sample``: temperature, top-k, top-p and min-p, each row with settings of its own, and the draw
  from given random numbers.

As in ``step``: the C name, torch tensors on the current GPU, every tensor checked before the call, torch's
current stream, no fallback path.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import binding as B
from . import step as S

TYPE_F32 = 2
MAX_VOCAB = 1 << 22
EXPORTS = ["lora_sample_bytes", "lora_sample"]

_TYPES = {torch.float16: S.TYPE_F16, torch.bfloat16: S.TYPE_BF16, torch.float32: TYPE_F32}
_P, _I32, _I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


class CSampleArgs(ctypes.Structure):
    _fields_ = [("type", _I32), ("n_rows", _I32), ("vocab", _I32), ("n_logits", _I32), ("logits", _P), ("ld", _I64),
                ("rows", _P), ("temperature", _P), ("top_k", _P), ("top_p", _P), ("min_p", _P), ("u", _P), ("token", _P),
                ("logprob", _P), ("work", _P), ("work_bytes", ctypes.c_size_t)]


_pack = struct.Struct("4i12q").pack   # the bytes of a CSampleArgs
assert struct.calcsize("4i12q") == ctypes.sizeof(CSampleArgs)


def sample_workspace(n_rows, vocab, device="cuda"):
    """A workspace for lora_sample calls of up to n_rows rows of up to vocab logits."""
    n = int(B.lib().lora_sample_bytes(S._count(int(n_rows), "n_rows"), S._count(int(vocab), "vocab")))
    if n == 0:
        raise ValueError(f"{n_rows} rows of {vocab} logits (1..{MAX_VOCAB})")
    return torch.empty(n // 4, dtype=torch.int32, device=device)


def lora_sample(token, logits, u, work, temperature=None, top_k=None, top_p=None, min_p=None, rows=None, logprob=None,
                stream=None):
    """Draw a token for each entry of `token` int32 [n_rows] from logits [n_logits, vocab] (f16, bf16 or f32; row
    rows[i], or row i) with u fp32 [n_rows] in [0, 1).  temperature (1; 0: the largest logit), top_p (1), min_p (0)
    fp32 and top_k (0: all) int32 [n_rows], or None for the value in brackets; logprob fp32 [n_rows] or None
    takes the drawn token's log-probability among what the filters left."""
    if S._fast:
        dev = S._device(logits)
        if dev >= 0 and S._done(S._fast.sample(S._address("lora_sample"), S._raw(stream, dev), dev, token, logits, u, work,
                                               temperature, top_k, top_p, min_p, rows, logprob)):
            return
    if not isinstance(logits, torch.Tensor) or logits.dtype not in _TYPES:
        raise ValueError(f"logits must have dtype f16, bf16 or f32 (got {getattr(logits, 'dtype', type(logits).__name__)})")
    if logits.layout is not torch.strided or logits.is_nested or logits.dim() != 2:
        raise ValueError("logits must be a plain 2-D tensor")
    m, vocab = S._count(logits.shape[0], "n_logits"), S._count(logits.shape[1], "vocab")
    S._matrix(logits, "logits", logits.dtype, m, vocab)
    ld = logits.stride(0) if m > 1 else vocab
    S._vector(token, "token", torch.int32, 0)
    n = S._count(token.numel(), "n_rows")
    S._vector(u, "u", torch.float32, n)
    S._vector(work, "work", torch.int32, 1)
    for t, what, dtype in ((temperature, "temperature", torch.float32), (top_k, "top_k", torch.int32),
                           (top_p, "top_p", torch.float32), (min_p, "min_p", torch.float32), (rows, "rows", torch.int32),
                           (logprob, "logprob", torch.float32)):
        if t is not None:
            S._vector(t, what, dtype, n)
    dev = S._here("token logits u work temperature top_k top_p min_p rows logprob", token, logits, u, work, temperature,
                  top_k, top_p, min_p, rows, logprob)
    at = lambda t: 0 if t is None else t.data_ptr()
    S._call("lora_sample", S._raw(stream, dev),
            _pack(_TYPES[logits.dtype], n, vocab, m, at(logits), ld, at(rows), at(temperature), at(top_k), at(top_p), at(min_p),
                  at(u), at(token), at(logprob), at(work), 4 * work.numel()))
