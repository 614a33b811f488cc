"""CPU: the decode-step operators' C ABI and binding -- exports, every refusal that the host
checks make before a launch, and the references the GPU tests compare against.  No test
here launches a kernel."""
import ctypes
import importlib
import os
import re
import subprocess

import pytest
import torch

from segmented_gather_matmul_amd import binding as B
from segmented_gather_matmul_amd import build as build_mod
from segmented_gather_matmul_amd import step as S
from tests import step_ref as R

PTR = 0x10000   # an aligned address that is never followed: every call here is refused


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if build_mod.stale():
        build_mod.build()
    if S._fast is None:      # built only just now, after the binding was imported
        importlib.invalidate_caches()
        S._fast = importlib.import_module("segmented_gather_matmul_amd._step_args")
    return B.lib()


def test_exports():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(build_mod.INCLUDE, "lora_step.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(lora_[a-z0-9_]+)\s*\(", text))
    assert names == set(S.EXPORTS)
    out = subprocess.run(["nm", "-D", "--defined-only", build_mod.LIB], capture_output=True, text=True, check=True).stdout
    assert names <= set(re.findall(r"\bT (lora_\w+)", out))


def _cache(**kw):
    d = dict(type=0, page_size=16, num_pages=8, kv_heads=2, head_dim=64, reserved=0, page_stride=2048, token_stride=128,
             head_stride=64, k=PTR, v=PTR)
    d.update(kw)
    return S.CKVCache(*[d[f[0]] for f in S.CKVCache._fields_])


def _code(fn, *args):
    return getattr(B.lib(), fn)(*args)


CACHE_FAULTS = [(dict(type=2), B.LORA_E_UNSUPPORTED), (dict(page_size=0), B.LORA_E_SHAPE),
                (dict(page_size=12), B.LORA_E_SHAPE), (dict(page_size=2048), B.LORA_E_SHAPE),
                (dict(num_pages=0), B.LORA_E_SHAPE), (dict(num_pages=1 << 28), B.LORA_E_SHAPE),
                (dict(kv_heads=0), B.LORA_E_SHAPE), (dict(head_dim=0), B.LORA_E_SHAPE),
                (dict(head_dim=60), B.LORA_E_SHAPE), (dict(head_dim=264), B.LORA_E_SHAPE),
                (dict(reserved=1), B.LORA_E_SHAPE), (dict(k=None), B.LORA_E_NULL), (dict(v=None), B.LORA_E_NULL),
                (dict(k=PTR + 8), B.LORA_E_ALIGN), (dict(token_stride=32), B.LORA_E_SHAPE),
                (dict(head_stride=68), B.LORA_E_ALIGN), (dict(page_stride=-2048), B.LORA_E_SHAPE),
                (dict(page_stride=1 << 62), B.LORA_E_SHAPE), (dict(token_stride=(1 << 63) - 8), B.LORA_E_SHAPE)]


@pytest.mark.parametrize("kw,code", CACHE_FAULTS, ids=lambda x: str(x))
def test_bad_caches_are_refused(kw, code):
    c = _cache(**kw)
    rope = S.CRope(0, 1, 0, 0, None, None)
    assert _code("lora_rope_append", None, 1, 0, None, 0, None, 0, PTR, 128, PTR, 128, ctypes.byref(rope), None, 0, PTR,
                 ctypes.byref(c)) == code
    assert _code("lora_paged_attention", None, 1, 2, PTR, 128, PTR + 4096, 128, ctypes.byref(c), 1, PTR, 4, 4, PTR, None,
                 1.0, 0, None, PTR, 1 << 30) == code
    assert B.last_error()


def _attn(**kw):
    d = dict(n_rows=2, heads=4, out=PTR, ldo=256, q=PTR + 4096, ldq=256, cache=_cache(), n_req=2, table=PTR, ldt=4,
             blocks=4, kv_len=PTR, req=None, scale=1.0, window=0, lse=None, work=PTR, work_bytes=1 << 30)
    d.update(kw)
    c = d["cache"]
    return _code("lora_paged_attention", None, d["n_rows"], d["heads"], d["out"], d["ldo"], d["q"], d["ldq"],
                 ctypes.byref(c) if c else None, d["n_req"], d["table"], d["ldt"], d["blocks"], d["kv_len"], d["req"],
                 d["scale"], d["window"], d["lse"], d["work"], d["work_bytes"])


@pytest.mark.parametrize("kw,code", [
    (dict(n_rows=-1), B.LORA_E_SHAPE), (dict(n_req=-1), B.LORA_E_SHAPE), (dict(heads=3), B.LORA_E_SHAPE),
    (dict(heads=0), B.LORA_E_SHAPE), (dict(cache=None), B.LORA_E_NULL), (dict(out=None), B.LORA_E_NULL),
    (dict(q=None), B.LORA_E_NULL), (dict(q=PTR + 4098), B.LORA_E_ALIGN), (dict(ldq=255), B.LORA_E_SHAPE),
    (dict(ldo=260), B.LORA_E_ALIGN), (dict(blocks=0), B.LORA_E_SHAPE), (dict(ldt=3), B.LORA_E_SHAPE),
    (dict(blocks=1 << 28, ldt=1 << 28), B.LORA_E_SHAPE), (dict(blocks=(1 << 26) + 1, ldt=1 << 27), B.LORA_E_SHAPE),
    (dict(n_rows=65536, blocks=1 << 26, ldt=1 << 26, out=PTR + (1 << 40)), B.LORA_E_UNSUPPORTED), (dict(kv_len=None), B.LORA_E_NULL),
    (dict(table=None), B.LORA_E_NULL), (dict(window=-1), B.LORA_E_SHAPE), (dict(scale=float("inf")), B.LORA_E_SHAPE),
    (dict(scale=float("nan")), B.LORA_E_SHAPE), (dict(lse=PTR + 2), B.LORA_E_ALIGN), (dict(work=None), B.LORA_E_NULL),
    (dict(work=PTR + 128), B.LORA_E_ALIGN), (dict(work_bytes=0), B.LORA_E_SHAPE),
    (dict(q=PTR + 16), B.LORA_E_SHAPE), (dict(q=PTR), B.LORA_E_SHAPE),
    (dict(n_rows=1 << 29), B.LORA_E_SHAPE)], ids=lambda x: str(x))
def test_attention_refusals(kw, code):
    assert _attn(**kw) == code


def test_attention_lines_that_pass_32_bits_are_refused():
    """The rows' tiles and four more each lie on one line of 32-bit positions, and its length is
    rounded up to whole shares of it: there is room for that too."""
    for rows, tiles in ((66, 32537627), (66, 32537628), (64, 1 << 25), (66, 32537627 - 3)):   # 2^31 - 2, past it; 200 short of it with 256 shares
        code = _attn(n_rows=rows, cache=_cache(page_size=1), blocks=32 * tiles, ldt=32 * tiles, out=PTR + (1 << 40))
        assert code == B.LORA_E_UNSUPPORTED, (rows, tiles, code, B.last_error())


def test_attention_of_no_rows_is_nothing():
    assert _attn(n_rows=0, q=None, out=None, kv_len=None, work=None) == B.LORA_OK


def _append(**kw):
    d = dict(n=2, heads=4, qo=PTR, ldqo=256, q=PTR + 4096, ldq=256, k=PTR + 8192, ldk=128, v=PTR + 16384, ldv=128,
             rope=S.CRope(64, 1, 0, 0, PTR, None), pos=PTR, ldp=2, slots=PTR, cache=_cache())
    d.update(kw)
    r, c = d["rope"], d["cache"]
    return _code("lora_rope_append", None, d["n"], d["heads"], d["qo"], d["ldqo"], d["q"], d["ldq"], d["k"], d["ldk"],
                 d["v"], d["ldv"], ctypes.byref(r) if r else None, d["pos"], d["ldp"], d["slots"], ctypes.byref(c))


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), B.LORA_E_SHAPE), (dict(heads=-1), B.LORA_E_SHAPE), (dict(rope=None), B.LORA_E_NULL),
    (dict(rope=S.CRope(72, 1, 0, 0, PTR, None)), B.LORA_E_SHAPE), (dict(rope=S.CRope(80, 1, 0, 0, PTR, None)), B.LORA_E_SHAPE),
    (dict(rope=S.CRope(-16, 1, 0, 0, PTR, None)), B.LORA_E_SHAPE), (dict(rope=S.CRope(64, 0, 0, 0, PTR, None)), B.LORA_E_SHAPE),
    (dict(rope=S.CRope(64, 5, 0, 0, PTR, None)), B.LORA_E_SHAPE), (dict(rope=S.CRope(64, 1, 2, 0, PTR, None)), B.LORA_E_SHAPE),
    (dict(rope=S.CRope(64, 1, 0, 0, None, None)), B.LORA_E_NULL), (dict(pos=None), B.LORA_E_NULL),
    (dict(ldp=1), B.LORA_E_SHAPE), (dict(slots=None), B.LORA_E_NULL), (dict(q=None), B.LORA_E_NULL),
    (dict(qo=None), B.LORA_E_NULL), (dict(k=None), B.LORA_E_NULL), (dict(v=PTR + 4), B.LORA_E_ALIGN),
    (dict(ldk=120), B.LORA_E_SHAPE), (dict(ldv=132), B.LORA_E_ALIGN), (dict(qo=PTR + 4096, ldqo=264), B.LORA_E_SHAPE),
    (dict(qo=PTR + 8192 - 16), B.LORA_E_SHAPE), (dict(qo=PTR + 16384), B.LORA_E_SHAPE)], ids=lambda x: str(x))
def test_append_refusals(kw, code):
    assert _append(**kw) == code


def _plan(pages=None, out=None, kv=PTR, new=PTR):
    p = dict(n_req=3, page_size=16, num_pages=8, max_blocks=4, ld_table=4, block_table=PTR, free_pages=PTR, free_top=PTR)
    o = dict(max_tokens=4, reserved=0, status=PTR, kv_end=PTR, free_top=PTR, q_ptr=PTR, tok_req=PTR, tok_pos=PTR,
             slots=PTR, idx=None)
    p.update(pages or {})
    o.update(out or {})
    cp = S.CKVPages(*[p[f[0]] for f in S.CKVPages._fields_])
    co = S.CKVPlanOut(*[o[f[0]] for f in S.CKVPlanOut._fields_])
    return _code("lora_kv_plan", None, ctypes.byref(cp), kv, new, None, ctypes.byref(co))


@pytest.mark.parametrize("pages,out,code", [
    (dict(page_size=3), {}, B.LORA_E_SHAPE), (dict(n_req=-1), {}, B.LORA_E_SHAPE), (dict(num_pages=0), {}, B.LORA_E_SHAPE),
    (dict(num_pages=1 << 30), {}, B.LORA_E_SHAPE), (dict(max_blocks=0), {}, B.LORA_E_SHAPE),
    (dict(ld_table=3), {}, B.LORA_E_SHAPE), (dict(block_table=None), {}, B.LORA_E_NULL),
    (dict(free_pages=None), {}, B.LORA_E_NULL), (dict(free_top=None), {}, B.LORA_E_NULL),
    ({}, dict(max_tokens=-1), B.LORA_E_SHAPE), ({}, dict(reserved=1), B.LORA_E_SHAPE),
    ({}, dict(status=None), B.LORA_E_NULL), ({}, dict(kv_end=None), B.LORA_E_NULL),
    ({}, dict(q_ptr=None), B.LORA_E_NULL), ({}, dict(slots=None), B.LORA_E_NULL)], ids=lambda x: str(x))
def test_plan_refusals(pages, out, code):
    assert _plan(pages, out) == code


def test_plan_arrays_must_be_apart():
    """Only kv_end over kv_len and the free top over itself, entry for entry, are taken."""
    names = ["status", "kv_end", "free_top", "q_ptr", "tok_req", "tok_pos", "slots", "idx"]
    at = {x: PTR + 4096 * i for i, x in enumerate(names + ["kv", "new", "old_top", "free_pages", "table"])}

    def plan(**kw):
        a = {**at, **kw}
        return _plan(dict(free_pages=a["free_pages"], free_top=a["old_top"], block_table=a["table"]),
                     {x: a[x] for x in names}, a["kv"], a["new"])

    for kw, what in ((dict(kv_end=at["new"]), "kv_end and new_len"), (dict(kv_end=at["kv"] + 4), "kv_end and kv_len"),
                     (dict(kv_end=at["kv"] - 8), "kv_end and kv_len"), (dict(q_ptr=at["kv"]), "q_ptr and kv_len"),
                     (dict(free_top=at["kv_end"]), "kv_end and out free_top"), (dict(free_top=at["free_pages"] + 28), "free_pages"),
                     (dict(old_top=at["status"] + 12), "status and free_top"), (dict(idx=at["slots"] + 12), "slots and idx"),
                     (dict(tok_pos=at["new"] + 8), "tok_pos and new_len"), (dict(new=at["free_pages"] + 8), "free_pages and new_len")):
        assert plan(**kw) == B.LORA_E_SHAPE and what in B.last_error(), (kw, B.last_error())


def _apart_plan(pages=None, **kw):
    """A plan over arrays that lie apart; kw moves some of them."""
    names = ["status", "kv_end", "free_top", "q_ptr", "tok_req", "tok_pos", "slots", "idx"]
    at = {x: PTR + (i << 16) for i, x in enumerate(names + ["kv", "new", "old_top", "free_pages", "table"])}
    at.update(kw)
    return _plan(dict(free_pages=at["free_pages"], free_top=at["old_top"], block_table=at["table"], **(pages or {})),
                 {x: at[x] for x in names}, at["kv"], at["new"])


def test_plan_tables_wider_than_a_position_are_refused():
    """A position is 32 bits: a table row of 2^31 tokens or more would plan requests that end
    behind it, whose positions wrap to negative ones and read the table far before its row."""
    for page, blocks in ((1024, 1 << 21), (1024, (1 << 21) + 1), (2, 1 << 30), (16, 2 ** 31 - 1)):
        code = _apart_plan(dict(page_size=page, max_blocks=blocks, ld_table=blocks, n_req=1, num_pages=1))
        assert code == B.LORA_E_SHAPE and "max_blocks" in B.last_error(), (page, blocks, code, B.last_error())


def test_plan_tables_lie_apart_from_the_other_arrays():
    """The table is written too: no other array may hold one of its entries.  What lies between
    its rows, behind max_blocks, is no entry."""
    table = PTR + (64 << 16)
    sizes = dict(status=4, kv_end=3, free_top=1, q_ptr=4, tok_req=4, tok_pos=4, slots=4, idx=4, kv=3, new=3, old_top=1,
                 free_pages=8)
    named = dict(kv="kv_len", new="new_len", old_top="free_top")

    def meets(at, what, ld):
        """Whether an array `at` entries from the table's first is refused for it.  (Two other
        arrays overlap in every call, so that none of them goes on to a launch.)"""
        pair = ("slots", "idx") if what not in ("slots", "idx") else ("tok_req", "tok_pos")
        kw = {x: PTR + (65 << 16) for x in pair}
        assert _apart_plan(dict(ld_table=ld), **{**kw, "table": table, what: table + 4 * at}) == B.LORA_E_SHAPE
        if "block_table" in B.last_error():
            assert named.get(what, what) in B.last_error()
            return True
        assert B.last_error() == f"{pair[0]} and {pair[1]} overlap"
        return False

    for what, n in sizes.items():
        for ld in (4, 7, 8):          # three rows of four entries
            entries = {ld * r + c for r in range(3) for c in range(4)}
            for at in range(-9, 3 * ld + 2):
                assert meets(at, what, ld) == bool(entries & set(range(at, at + n))), (what, ld, at, B.last_error())


def test_plans_of_more_requests_than_an_index_can_halve_are_refused():
    """The search of q_ptr adds two request numbers, and the walk of the requests steps past the last
    one: both are 32 bits."""
    far = {x: PTR + ((i + 1) << 40) for i, x in enumerate(["status", "kv_end", "free_top", "q_ptr", "tok_req", "tok_pos", "slots",
                                                            "idx", "kv", "new", "old_top", "free_pages", "table"])}
    for n in ((1 << 30) + 1, 2 ** 31 - 1025, 2 ** 31 - 1):
        assert _apart_plan(dict(n_req=n), **far) == B.LORA_E_SHAPE and "n_req" in B.last_error(), (n, B.last_error())


def test_plan_needs_its_lengths():
    assert _plan(kv=None) == B.LORA_E_NULL and _plan(new=None) == B.LORA_E_NULL


def _norm(**kw):
    d = dict(type=0, n_rows=2, hidden=64, n_gates=0, y=PTR, ldy=64, res_out=PTR + 4096, ldro=64, res=PTR + 8192, ldr=64,
             x=PTR + 16384, ldx=64, w=PTR, post_w=None, gate=None, ldg=64, gate_idx=None, alpha=1.0, eps=1e-5,
             w_offset=0.0, reserved=0)
    d.update(kw)
    a = S.CNormArgs(*[d[f[0]] for f in S.CNormArgs._fields_])
    return _code("lora_residual_norm", None, ctypes.byref(a))


@pytest.mark.parametrize("kw,code", [
    (dict(type=3), B.LORA_E_UNSUPPORTED), (dict(n_rows=-1), B.LORA_E_SHAPE), (dict(hidden=60), B.LORA_E_SHAPE),
    (dict(hidden=0), B.LORA_E_SHAPE), (dict(hidden=65544), B.LORA_E_SHAPE), (dict(eps=-1.0), B.LORA_E_SHAPE),
    (dict(eps=float("nan")), B.LORA_E_SHAPE), (dict(alpha=float("inf")), B.LORA_E_SHAPE),
    (dict(y=None, res_out=None), B.LORA_E_NULL), (dict(x=None, post_w=PTR), B.LORA_E_NULL),
    (dict(x=None, gate=PTR, n_gates=1), B.LORA_E_NULL), (dict(gate_idx=PTR), B.LORA_E_NULL), (dict(res=None), B.LORA_E_NULL),
    (dict(w=None), B.LORA_E_NULL), (dict(ldr=56), B.LORA_E_SHAPE), (dict(ldx=68), B.LORA_E_ALIGN),
    (dict(post_w=PTR + 2), B.LORA_E_ALIGN), (dict(gate=PTR, n_gates=2), B.LORA_E_SHAPE),
    (dict(gate=PTR, n_gates=0, gate_idx=PTR), B.LORA_E_SHAPE), (dict(y=PTR + 8192), B.LORA_E_SHAPE),
    (dict(y=PTR + 4096), B.LORA_E_SHAPE), (dict(res_out=PTR + 16384), B.LORA_E_SHAPE),
    (dict(res_out=PTR + 8192 + 16), B.LORA_E_SHAPE), (dict(reserved=1), B.LORA_E_SHAPE)], ids=lambda x: str(x))
def test_norm_refusals(kw, code):
    assert _norm(**kw) == code
    assert _norm(n_rows=0) == B.LORA_OK


def test_launches_of_more_threads_than_a_grid_holds_are_refused():
    """A launch has at most 2^32 - 1 threads along its rows."""
    far, n = PTR + (1 << 45), 1 << 22      # rows of more than 8192 columns take 1024 threads each
    for rows, hidden in ((n, 8200), (n, 65536), (1 << 23, 4104), (2 ** 31 - 1, 4096), (1 << 26, 8)):
        ld = hidden
        assert _norm(n_rows=rows, hidden=hidden, y=None, res_out=far, x=None, ldro=ld, ldr=ld) == B.LORA_E_UNSUPPORTED
        assert str(rows) in B.last_error()
    cache = _cache(num_pages=1, kv_heads=32, head_dim=128, token_stride=4096, head_stride=128, page_stride=65536)
    for rows, heads in ((1 << 24, 0), (2 ** 31 - 1, 0), (1 << 24, 32)):
        assert _append(n=rows, heads=heads, qo=far, ldqo=4096, q=PTR, ldq=4096, k=2 * far, ldk=4096, v=3 * far, ldv=4096,
                       cache=cache, rope=S.CRope(0, 1, 0, 0, None, None)) == B.LORA_E_UNSUPPORTED
        assert str(rows) in B.last_error()


def test_null_descriptors():
    assert _code("lora_residual_norm", None, None) == B.LORA_E_NULL
    assert _code("lora_kv_plan", None, None, PTR, PTR, None, None) == B.LORA_E_NULL
    assert B.lib().lora_paged_attention_bytes(-1, 4, 2, 64) == 0
    assert B.lib().lora_paged_attention_bytes(2, 3, 2, 64) == 0


# ------------------------------------------------------------------ the binding
def test_binding_rejects_wrong_tensors():
    h = torch.float16
    kc = torch.zeros(4, 16, 2, 64, dtype=h)
    cache = S.PagedKV(kc, torch.zeros_like(kc))
    assert (cache.num_pages, cache.page_size, cache.kv_heads, cache.head_dim) == (4, 16, 2, 64)
    q = torch.zeros(2, 256, dtype=h)
    tab, n, w = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(64, dtype=torch.int32)
    call = lambda **k: S.lora_paged_attention(**{**dict(out=q.clone(), q=q, cache=cache, block_table=tab, kv_len=n, work=w), **k})
    for k, msg in ((dict(q=q.float()), "dtype"), (dict(q=q[:, :200]), "heads"), (dict(out=q[:1]), "at least"),
                   (dict(kv_len=n.long()), "dtype"), (dict(kv_len=n[:1]), "elements"), (dict(block_table=tab.long()), "dtype"),
                   (dict(lse=torch.zeros(3)), "elements"), (dict(lse=torch.zeros(8, dtype=h)), "dtype"),
                   (dict(req=n.float()), "dtype"), (dict(), "GPU tensor")):
        with pytest.raises(ValueError, match=msg):
            call(**k)
    k2 = torch.zeros(2, 128, dtype=h)
    rope = S.Rope(torch.ones(32))
    app = lambda **k: S.lora_rope_append(**{**dict(q_out=q.clone(), q=q, k=k2, v=k2.clone(), cache=cache, slots=n, rope=rope,
                                                    positions=torch.zeros(1, 2, dtype=torch.int32)), **k})
    for k, msg in ((dict(q_out=None), "together"), (dict(k=k2.bfloat16()), "dtype"), (dict(positions=None), "tensor"),
                   (dict(positions=torch.zeros(1, 1, dtype=torch.int32)), "at least"), (dict(v=k2[:, :64]), "at least"),
                   (dict(slots=n.long()), "dtype"), (dict(), "GPU tensor"),
                   (dict(positions=torch.zeros(2, 3, 2, dtype=torch.int32)[:, :1]), "3-D"),   # not a view of one row
                   (dict(positions=torch.zeros(4, dtype=torch.int32)[::2]), "stride")):
        with pytest.raises(ValueError, match=msg):
            app(**k)
    r = torch.zeros(2, 64, dtype=h)
    nrm = lambda **k: S.lora_residual_norm(**{**dict(y=r.clone(), res=r, w=torch.ones(64, dtype=h)), **k})
    for k, msg in ((dict(w=None), "tensor"), (dict(w=torch.ones(64)), "dtype"), (dict(x=r.t()), "stride|at least"),
                   (dict(res=r.float()), "dtype"), (dict(gate=r, x=r.clone(), gate_idx=n[:1]), "elements"), (dict(), "GPU tensor")):
        with pytest.raises(ValueError, match=msg):
            nrm(**k)


def test_compiled_checks_agree_with_the_python_ones():
    """What the compiled module accepts, the rules in Python accept with the same answer; what
    they refuse, it refuses (it may leave odd cases to them)."""
    assert S._fast is not None, "the module is built with the library"
    base = torch.zeros(6, 40, dtype=torch.float16)
    tensors = [base, base[:, :24], base[:, 8:32], base[1:2], base[:1, :17], base[:0], base[:, :0], base.t(), base[::2],
               base[:, ::2], base[0], base.view(2, 3, 40), base.float(), base.bfloat16(), base.int(), base.expand(6, 40),
               base[:1].expand(6, 40), torch.zeros(40, dtype=torch.float16)[None], torch.zeros(3, 1, dtype=torch.float16),
               None, 5, "q", [1.0]]
    agreed = 0
    for t in tensors:
        for dt in S._CODES:
            for rows, cols in ((0, 0), (1, 17), (2, 24), (6, 40), (7, 40), (6, 41), (1, 1)):
                ld = S._fast.matrix(t, S._CODES[dt], rows, cols)
                try:
                    want = S._matrix_checked(t, "t", dt, rows, cols)
                except ValueError:
                    want = None
                if ld >= 0:
                    assert want == ld, (getattr(t, "shape", t), dt, rows, cols)
                    agreed += 1
                elif want is not None:
                    assert t.shape[0] < 2 or t.numel() == 0, "only rows without a meaningful stride are left to Python"
            for n in (0, 1, 40, 240, 241):
                fast, held = S._fast.vector(t, S._CODES[dt], n), S._fast
                try:
                    S._fast = None
                    S._vector(t, "t", dt, n)
                    ok = True
                except ValueError:
                    ok = False
                finally:
                    S._fast = held
                assert fast == ok, (getattr(t, "shape", t), dt, n)
    assert agreed > 20
    assert S._fast.here(base, None, base) == -1 and S._fast.here(base, 5) == -1


@pytest.mark.parametrize("kind", ["nested", "sparse"])
def test_tensors_without_plain_memory_are_refused(kind):
    """They throw from their accessors; the process goes on and the check says what is wrong."""
    def make(dt):
        if kind == "sparse":
            return torch.eye(16, dtype=dt).to_sparse()
        return torch.nested.nested_tensor([torch.zeros(8, dtype=dt), torch.zeros(16, dtype=dt)])

    for dt in S._CODES:
        t = make(dt)
        assert S._fast.matrix(t, S._CODES[dt], 1, 4) == -1
        assert not S._fast.vector(t, S._CODES[dt], 1)
        assert S._fast.here(t) == -1
        with pytest.raises(ValueError, match="strided"):
            S._matrix(t, "t", dt, 1, 4)
    with pytest.raises(ValueError, match="strided"):
        S._vector(make(torch.int32), "t", torch.int32, 1)


def test_descriptors_reject_wrong_layouts():
    h = torch.float16
    k = torch.zeros(4, 16, 2, 64, dtype=h)
    S.PagedKV(k.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3), k.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3))
    both = torch.zeros(4, 2, 16, 2, 64, dtype=h)
    S.PagedKV(both[:, 0], both[:, 1])
    for args, msg in (((k, k), "overlap"), ((k, k.bfloat16()), "dtype"), ((k.float(), k.float()), "dtype"),
                      ((k[0], k[0]), "must be"), ((k, k.permute(0, 2, 1, 3)), "must be|strides"),
                      ((k.expand(4, 16, 2, 64)[:1].expand(4, 16, 2, 64), torch.zeros_like(k)), "strides|overlapping")):
        with pytest.raises(ValueError, match=msg):
            S.PagedKV(*args)
    for shape in ((0, 16, 2, 64), (4, 0, 2, 64), (4, 16, 0, 64), (4, 16, 2, 0)):  # (heads of 0 columns: a division by 0)
        with pytest.raises(ValueError, match="empty"):
            S.PagedKV(torch.zeros(shape, dtype=h), torch.zeros(shape, dtype=h))
    t, f, top = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    S.KVPages(t, f, top, 16)
    for args, msg in (((t, f, top, 12), "power"), ((t.long(), f, top, 16), "dtype"), ((t[0], f, top, 16), "block_table"),
                      ((t, f[::2], top, 16), "contiguous")):
        with pytest.raises(ValueError, match=msg):
            S.KVPages(*args)
    with pytest.raises(ValueError, match="frequencies"):
        S.Rope(torch.ones(12))
    with pytest.raises(ValueError, match="axes"):
        S.Rope(torch.ones(16), axes=5)


def test_an_lse_of_other_columns_is_refused():
    """It is written as [n_rows, heads]: in a wider array the rows would not be where they are read."""
    h = torch.float16
    cache = S.PagedKV(torch.zeros(4, 16, 2, 64, dtype=h), torch.zeros(4, 16, 2, 64, dtype=h))
    q, tab, n, w = torch.zeros(2, 256, dtype=h), torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(64, dtype=torch.int32)
    call = lambda lse: S.lora_paged_attention(q.clone(), q, cache, tab, n, w, lse=lse)
    for shape in ((2, 8), (4, 2), (2, 5), (1, 8), (2, 2, 4)):
        with pytest.raises(ValueError, match="lse is"):
            call(torch.zeros(shape))
    for shape in ((2, 4), (3, 4), (8,), (9,), (2, 2, 2), (2, 4, 1)):     # rows of one head after another
        with pytest.raises(ValueError, match="GPU tensor"):
            call(torch.zeros(shape))
    with pytest.raises(ValueError, match="GPU tensor"):                   # (one row begins where the array does)
        S.lora_paged_attention(q[:1].clone(), q[:1], cache, tab, n, w, lse=torch.zeros(1, 9))


def test_counts_that_pass_32_bits_are_refused(monkeypatch):
    """The library's counts are 32 bits, and ctypes would cut a larger one off: 2^32 + 8 rows would
    be a call on 8 of them.  (Tensors without memory; nothing is called.)"""
    far, h, i32 = 2 ** 32 + 8, torch.float16, torch.int32
    monkeypatch.setattr(S, "_here", lambda *a: 0)
    monkeypatch.setattr(S, "_raw", lambda *a: None)
    calls = []
    monkeypatch.setattr(S, "_call", lambda *a: calls.append(a))
    e = lambda *shape, dt=i32: torch.empty(shape, dtype=dt, device="meta")
    cache = S.PagedKV(torch.zeros(4, 16, 2, 64, dtype=h), torch.zeros(4, 16, 2, 64, dtype=h))
    for make, what in ((lambda: S.PagedKV(e(far, 1, 1, 8, dt=h), e(far, 1, 1, 8, dt=h)), "num_pages"),
                       (lambda: S.PagedKV(e(1, 1, far, 8, dt=h), e(1, 1, far, 8, dt=h)), "kv_heads"),
                       (lambda: S.KVPages(e(2, 4), e(far), e(1), 16), "num_pages"),
                       (lambda: S.KVPages(e(far, 4), e(8), e(1), 16), "n_req"),
                       (lambda: S.KVPages(e(2, far), e(8), e(1), 16), "max_blocks"),
                       (lambda: S.KVPlan(4, far, device="meta"), "max_tokens"),
                       (lambda: S.KVPlan(far, 4, device="meta"), "n_req"),
                       (lambda: S.Rope(e(far, dt=torch.float32)), "rot_dim"),
                       (lambda: S.workspace(far, 4, 2, 64, device="meta"), "n_rows"),
                       (lambda: S.workspace(4, 4, 2, far, device="meta"), "head_dim")):
        with pytest.raises(ValueError, match=what):
            make()
    attn = dict(out=e(far, 256, dt=h), q=e(far, 256, dt=h), cache=cache, block_table=e(far, 4), kv_len=e(far), work=e(64))
    for kw, what in ((attn, "n_rows"), ({**attn, "q": e(2, 256, dt=h)}, "n_req"),
                     ({**attn, "q": e(2, 256, dt=h), "block_table": e(2, far)}, "max_blocks"),
                     ({**attn, "q": e(2, 256, dt=h), "block_table": e(2, 4), "window": far}, "window"),
                     ({**attn, "q": e(2, 64 * far, dt=h), "out": e(2, 64 * far, dt=h), "block_table": e(2, 4)}, "heads")):
        with pytest.raises(ValueError, match=what):
            S.lora_paged_attention(**kw)
    kv = dict(k=e(far, 128, dt=h), v=e(far, 128, dt=h), cache=cache, slots=e(far))
    for kw, what in (({**kv, "q_out": None, "q": None}, "n_rows"),
                     ({**kv, "slots": e(2), "q_out": e(2, 64 * far, dt=h), "q": e(2, 64 * far, dt=h)}, "heads")):
        with pytest.raises(ValueError, match=what):
            S.lora_rope_append(**kw)
    for res, what in ((e(far, 64, dt=h), "n_rows"), (e(2, far, dt=h), "hidden")):
        with pytest.raises(ValueError, match=what):
            S.lora_residual_norm(res, res, w=e(res.shape[1], dt=h))
    with pytest.raises(ValueError, match="n_gates"):
        S.lora_residual_norm(e(2, 64, dt=h), e(2, 64, dt=h), w=e(64, dt=h), x=e(2, 64, dt=h), gate=e(far, 64, dt=h), gate_idx=e(2))
    assert not calls


# ------------------------------------------------------------------ the references
def test_plan_reference_on_a_worked_example():
    # pages of 4 tokens; request 0 grows from 3 to 5, request 1 (6 tokens) ends, request 2 starts with 2
    got = R.plan([3, 6, 0], [2, -1, 2], [[7, -1], [1, 4], [-1, -1]], [2, 9, -1, -1, -1, -1, -1, -1, -1, -1], 2, 4, 6, [5, 6, 7])
    assert got["status"] == [0, 4, 2, 2] and got["kv_end"] == [5, 0, 2] and got["q_ptr"] == [0, 2, 2, 4]
    # 1 and 4 go on the list (2 9 1 4); request 0 takes 4, request 2 takes 1
    assert got["table"] == [[7, 4], [1, 4], [1, -1]] and got["free_top"] == 2 and got["free"][:4] == [2, 9, 1, 4]
    assert got["tok_req"] == [0, 0, 2, 2, -1, -1] and got["tok_pos"] == [3, 4, 0, 1, -1, -1]
    assert got["slots"] == [31, 16, 4, 5, -1, -1] and got["idx"] == [5, 5, 7, 7, -1, -1]
    assert R.plan([3], [2], [[7, -1]], [2], 0, 4, 6)["status"][0] == 1


def test_attention_reference_on_one_token_and_on_none():
    q = torch.ones(3, 2, 8, dtype=torch.float16)
    k, v = torch.full((2, 4, 1, 8), float("nan"), dtype=torch.float16), torch.full((2, 4, 1, 8), float("nan"), dtype=torch.float16)
    k[1, 0], v[1, 0] = 0.5, 3.0
    o = R.attention(q, k, v, torch.tensor([[1], [0], [5]], dtype=torch.int32), [1, 0, 2], None, 1.0, 0, 2)
    assert torch.equal(o[0][0], torch.full((2, 8), 3.0, dtype=torch.float64)) and o[0][1].tolist() == [4.0, 4.0]
    assert not o[1][0].any() and not o[2][0].any() and o[2][1].tolist() == [float("-inf")] * 2
