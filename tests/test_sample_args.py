"""CPU: sampling's C ABI and binding -- exports, every refusal that the host checks make before a launch, and the
reference the GPU tests compare against.  No test here launches a kernel."""
import ctypes
import importlib
import math
import os
import re
import subprocess

import pytest
import torch

from segmented_gather_matmul_amd import binding as B
from segmented_gather_matmul_amd import build as build_mod
from segmented_gather_matmul_amd import sample as SA
from segmented_gather_matmul_amd import step as S
from tests import sample_ref as SR

PTR = 0x10000   # an aligned address that is never followed: every call here is refused


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if build_mod.stale():
        build_mod.build()
    if S._fast is None:
        importlib.invalidate_caches()
        S._fast = importlib.import_module("segmented_gather_matmul_amd._step_args")
    return B.lib()


def test_exports():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(build_mod.INCLUDE, "lora_sample.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(lora_[a-z0-9_]+)\s*\(", text))
    assert names == set(SA.EXPORTS)
    out = subprocess.run(["nm", "-D", "--defined-only", build_mod.LIB], capture_output=True, text=True, check=True).stdout
    assert names <= set(re.findall(r"\bT (lora_\w+)", out))


def test_the_arguments_are_laid_out_as_in_the_header(tmp_path):
    fields = [f[0] for f in SA.CSampleArgs._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "lora_sample.h"\nint main(void) {\n'
                   + "".join(f'printf("%zu ", offsetof(lora_sample_args, {f}));\n' for f in fields)
                   + 'printf("%zu %d\\n", sizeof(lora_sample_args), LORA_SAMPLE_MAX_VOCAB); return 0; }\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", f"-I{build_mod.INCLUDE}", str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [getattr(SA.CSampleArgs, f).offset for f in fields] + [ctypes.sizeof(SA.CSampleArgs), SA.MAX_VOCAB]


def _sample(**kw):
    d = dict(type=0, n_rows=2, vocab=100, n_logits=2, logits=PTR, ld=100, rows=None, temperature=None, top_k=None,
             top_p=None, min_p=None, u=PTR, token=PTR, logprob=None, work=PTR, work_bytes=1 << 30)
    d.update(kw)
    a = SA.CSampleArgs(*[d[f[0]] for f in SA.CSampleArgs._fields_])
    return B.lib().lora_sample(None, ctypes.byref(a))


@pytest.mark.parametrize("kw,code", [
    (dict(type=3), B.LORA_E_UNSUPPORTED), (dict(type=-1), B.LORA_E_UNSUPPORTED), (dict(n_rows=-1), B.LORA_E_SHAPE),
    (dict(n_logits=-1), B.LORA_E_SHAPE), (dict(n_logits=1), B.LORA_E_SHAPE), (dict(vocab=0), B.LORA_E_SHAPE),
    (dict(vocab=(1 << 22) + 1, ld=1 << 23), B.LORA_E_SHAPE), (dict(ld=99), B.LORA_E_SHAPE), (dict(ld=1 << 62), B.LORA_E_SHAPE),
    (dict(logits=None), B.LORA_E_NULL), (dict(u=None), B.LORA_E_NULL), (dict(token=None), B.LORA_E_NULL),
    (dict(logits=PTR + 1), B.LORA_E_ALIGN), (dict(type=2, logits=PTR + 2), B.LORA_E_ALIGN), (dict(rows=PTR + 1), B.LORA_E_ALIGN),
    (dict(top_k=PTR + 2), B.LORA_E_ALIGN), (dict(logprob=PTR + 2), B.LORA_E_ALIGN), (dict(work=None), B.LORA_E_NULL),
    (dict(work=PTR + 128), B.LORA_E_ALIGN), (dict(work_bytes=8), B.LORA_E_SHAPE),
    (dict(n_rows=1 << 22, n_logits=1 << 22), B.LORA_E_UNSUPPORTED)], ids=lambda x: str(x))
def test_refusals(kw, code):
    assert _sample(**kw) == code and B.last_error()


def test_calls_of_no_rows_are_nothing_and_null_arguments_refused():
    assert _sample(n_rows=0, logits=None, u=None, token=None, work=None) == B.LORA_OK
    assert B.lib().lora_sample(None, None) == B.LORA_E_NULL
    assert B.lib().lora_sample_bytes(-1, 5) == 0 and B.lib().lora_sample_bytes(1, 0) == 0
    assert B.lib().lora_sample_bytes(1, (1 << 22) + 1) == 0 and B.lib().lora_sample_bytes(1, 1 << 22) > 0


def test_binding_rejects_wrong_tensors(monkeypatch):
    x, u, tok, w = torch.zeros(3, 50), torch.zeros(3), torch.zeros(3, dtype=torch.int32), torch.zeros(64, dtype=torch.int32)
    call = lambda **k: SA.lora_sample(**{**dict(token=tok, logits=x, u=u, work=w), **k})
    for fast in (S._fast, None):
        monkeypatch.setattr(S, "_fast", fast)
        for k, msg in ((dict(logits=x.double()), "dtype"), (dict(logits=x[0]), "2-D"), (dict(logits=x.t()), "stride"),
                       (dict(logits=None), "dtype"), (dict(token=tok.long()), "dtype"), (dict(token=None), "tensor"),
                       (dict(u=u[:2]), "elements"), (dict(u=u.half()), "dtype"), (dict(u=None), "tensor"), (dict(work=None), "tensor"),
                       (dict(temperature=u[:1]), "elements"), (dict(temperature=0.7), "tensor"), (dict(top_k=u), "dtype"),
                       (dict(top_p=tok), "dtype"), (dict(min_p=u[::2]), "contiguous"), (dict(rows=tok.long()), "dtype"),
                       (dict(logprob=u[:2]), "elements"), (dict(), "GPU tensor")):
            with pytest.raises(ValueError, match=msg):
                call(**k)
    with pytest.raises(ValueError, match="logits"):
        SA.sample_workspace(1, 0, device="cpu")
    with pytest.raises(ValueError, match="32 bits"):
        SA.sample_workspace(2 ** 32, 5, device="cpu")


def test_counts_that_pass_32_bits_are_refused(monkeypatch):
    far = 2 ** 32 + 8
    monkeypatch.setattr(S, "_here", lambda *a: 0)
    monkeypatch.setattr(S, "_raw", lambda *a: None)
    calls = []
    monkeypatch.setattr(S, "_call", lambda *a: calls.append(a))
    e = lambda *s, dt=torch.float32: torch.empty(s, dtype=dt, device="meta")
    i = torch.int32
    for kw, what in ((dict(token=e(far, dt=i), logits=e(2, 50), u=e(far)), "n_rows"), (dict(token=e(2, dt=i), logits=e(far, 50), u=e(2)), "n_logits"),
                     (dict(token=e(2, dt=i), logits=e(2, far), u=e(2)), "vocab")):
        with pytest.raises(ValueError, match=what):
            SA.lora_sample(work=e(64, dt=i), **kw)
    assert not calls


def test_reference_on_worked_rows():
    x = torch.tensor([1.0, 3.0, 3.0, -math.inf, math.nan, 2.0])
    assert SR.sample(x, 0.0, 0, 1.0, 0.0, 0.9)[:2] == (1, 0.0)
    assert SR.sample(x, 1.0, 1, 1.0, 0.0, 0.9)[:2] == (1, 0.0)
    assert SR.sample(x, 1.0, 2, 1.0, 0.0, 0.6)[0] == 2 and SR.sample(x, 1.0, 2, 1.0, 0.0, 0.4)[0] == 1
    assert SR.sample(x, 1.0, 2, 0.5, 0.0, 0.99)[0] == 1          # before the second lies half of the mass
    assert SR.sample(x, 1.0, 0, 1.0, 0.0, 0.0)[0] == 0           # index order
    assert SR.sample(x, 1.0, 0, 1.0, 1.0, 0.0)[0] == 1
    assert SR.sample(x, 1.0, 0, 1.0, 0.0, 0.9999)[0] == 5
    assert abs(SR.sample(x, 1.0, 2, 1.0, 0.0, 0.6)[1] + math.log(2)) < 1e-12
    assert SR.sample(torch.full((4,), -math.inf), 1.0, 0, 1.0, 0.0, 0.5)[0] == -1
    assert SR.sample(torch.tensor([1.0, math.inf, 5.0, math.inf]), 1.0, 0, 1.0, 0.0, 0.7)[0] == 3
    assert SR.sample(x, -1.0, 0, 1.0, 0.0, 0.5) is None and SR.sample(x, 1.0, 0, 1.0, 0.0, 1.0) is None
