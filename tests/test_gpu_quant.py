"""GPU: the quantised key/value cache (lora_quant.h) against its 64-bit references, at the sizes, layouts, masks and
values where it can go wrong.  Tolerances are derived in quant_ref."""
import math
import random

import pytest
import torch

from segmented_gather_matmul_amd import binding as B
from segmented_gather_matmul_amd import quant as Q
from segmented_gather_matmul_amd import step as S
from tests import quant_ref as QR
from tests import step_ref as R
from tests.gpu_cases import say
from tests.test_gpu_step import close, ints

pytestmark = pytest.mark.gpu
F16, BF16, F64 = torch.float16, torch.bfloat16, torch.float64


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()
    yield


def new_cache(pages, P, K, D, dt, bits, layout="heads", seed=0):
    """A cache full of random bytes.  layout: memory order, or all four arrays inside one buffer of records."""
    g = torch.Generator().manual_seed(seed)
    cb, eb = 4 * bits * QR.blocks(D), QR.blocks(D)
    rnd = lambda *s: torch.randint(0, 256, s, generator=g, dtype=torch.uint8).cuda()
    if layout == "heads":
        t = [rnd(pages, K, P, n).transpose(1, 2) for n in (cb, cb, eb, eb)]
    elif layout == "tokens":
        t = [rnd(pages, P, K, n) for n in (cb, cb, eb, eb)]
    elif layout == "gaps":      # wider cells than needed, an odd offset for the exponents
        t = [rnd(pages, P, K, cb + 48)[..., 16:16 + cb] for _ in range(2)] + [rnd(pages, P, K, eb + 3)[..., 1:1 + eb] for _ in range(2)]
    else:                       # one record a page: k, v, their exponents
        one = rnd(pages, -(-(2 * P * K * (cb + eb)) // 16) * 16)
        cut = lambda at, n: one[:, at:at + P * K * n].view(pages, K, P, n).transpose(1, 2)
        t = [cut(0, cb), cut(P * K * cb, cb), cut(2 * P * K * cb, eb), cut(2 * P * K * cb + P * K * eb, eb)]
    return Q.QuantKV(*t, D, dt)


def cells(c, what):
    code, exp = (c.k, c.k_exp) if what == "k" else (c.v, c.v_exp)
    return QR.values(code.cpu(), exp.cpu(), c.bits, c.head_dim)


def bytes_of(c):
    return [t.clone() for t in (c.k, c.v, c.k_exp, c.v_exp)]


# ------------------------------------------------------------------ append
# heads, kv_heads, D, rot, axes, interleaved, page, rows, pad, layout
APPEND = [(4, 2, 128, 128, 1, False, 16, 33, 3, "heads"), (4, 4, 128, 128, 2, True, 8, 7, 0, "tokens"),
          (8, 1, 64, 64, 1, False, 1, 1, 0, "record"), (6, 3, 80, 80, 3, False, 16, 19, 2, "gaps"),
          (2, 2, 80, 48, 1, True, 4, 65, 1, "heads"), (3, 3, 8, 0, 1, False, 2, 9, 0, "heads"),
          (5, 1, 40, 16, 1, False, 64, 130, 5, "tokens"), (2, 1, 256, 256, 4, False, 32, 12, 1, "record"),
          (2, 1, 96, 64, 1, False, 16, 1100, 7, "heads"), (0, 2, 160, 32, 2, True, 16, 21, 0, "heads"),
          (40, 40, 128, 128, 1, False, 16, 5, 0, "heads"), (64, 8, 128, 128, 3, True, 32, 40, 8, "tokens")]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dt", [F16, BF16], ids=["f16", "bf16"])
def test_append_matches_the_formula(case, bits, dt):
    H, K, D, rot, axes, inter, P, n, pad, layout = case
    say(f"case quant-append {case} bits={bits} {dt}")
    g = torch.Generator().manual_seed(n + D)
    pages = -(-n // P) + 3
    c = new_cache(pages, P, K, D, dt, bits, layout, seed=n)
    x = torch.randn(n + pad, (H + 2 * K) * D + 24, generator=g)
    x[:, H * D:(H + K) * D] *= torch.where(torch.rand(K * D, generator=g) < 0.1, 30.0, 1.0)
    x = x.to(dt).cuda()
    q, k, v = x[:, :H * D], x[:, H * D:(H + K) * D], x[:, (H + K) * D:(H + 2 * K) * D]
    slots = torch.randperm(pages * P, generator=g)[:n + pad].int()
    slots[n:] = torch.tensor([-1, pages * P, 2 ** 31 - 1, -(2 ** 31), -7, -1, -1, -1][:pad], dtype=torch.int32)
    slots = slots[torch.randperm(n + pad, generator=g)]
    pos = torch.randint(0, 100000, (axes, n + pad), generator=g, dtype=torch.int32)
    pos[:, 0] = 0
    half = rot // 2
    axis = torch.randint(0, axes + 1, (half,), generator=g, dtype=torch.int32) if axes > 1 else None
    inv = torch.tensor([10000.0 ** (-2.0 * i / max(rot, 1)) for i in range(half)], dtype=torch.float32)
    rope = S.Rope(inv.cuda(), None if axis is None else axis.cuda(), axes, inter) if rot else None
    before = bytes_of(c)
    qo = torch.full((n + pad, H * D + 8), 7.0, dtype=dt, device="cuda")
    out = qo[:, :H * D] if H else None
    Q.lora_quant_append(out, q if H else None, k, v, c, slots.cuda(), rope=rope, positions=pos.cuda() if rot else None)
    torch.cuda.synchronize()
    live = (slots >= 0) & (slots < pages * P)
    at = slots[live].long()
    kc, vc = k.cpu().reshape(-1, K, D)[live], v.cpu().reshape(-1, K, D)[live]
    lp = pos[:, live]
    y, d = QR.rotated_bounds(kc, lp, inv, axis, axes, inter)
    QR.check_quantised(cells(c, "k")[at // P, at % P], c.k_exp.cpu()[at // P, at % P], y, d, bits, dt, "k")
    want, exps = QR.quantise(vc.to(F64), bits, dt)
    assert torch.equal(c.v_exp.cpu()[at // P, at % P].to(F64), exps)
    assert torch.equal(cells(c, "v")[at // P, at % P], want)
    if H:
        qy, mag = R.rotate(q.cpu().reshape(-1, H, D)[live], lp, inv, axis, axes, inter)
        close(out.cpu()[live].reshape(-1, H, D), qy, R.half_step(dt) * qy.abs() + 2.0 ** -21 * mag + R.tiny(dt), "q_out")
        assert bool((out.cpu()[~live] == 7.0).all()) and bool((qo[:, H * D:] == 7.0).all())
    # nothing else moved, and columns behind head_dim are zeros
    touched = torch.zeros(pages * P, dtype=torch.bool)
    touched[at] = True
    for b, a in zip(before, bytes_of(c)):
        assert torch.equal(a.cpu().reshape(pages * P, K, -1)[~touched], b.cpu().reshape(pages * P, K, -1)[~touched])
    tail = (32 * QR.blocks(D) - D) * bits // 8
    if tail:
        for t in (c.k, c.v):
            assert not bool(t.cpu()[at // P, at % P][..., -tail:].any())


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dt", [F16, BF16], ids=["f16", "bf16"])
def test_append_of_ties_limits_zeros_and_what_is_not_finite(dt, bits):
    say(f"case quant-append-special bits={bits} {dt}")
    D, K = 64, 2
    big = torch.finfo(dt).max
    tiny = torch.finfo(dt).smallest_normal
    step = tiny * torch.finfo(dt).eps
    # every midpoint of the grid and its neighbours, at several powers; block maxima around their edges
    gr = QR.grid(bits)
    mid = ((gr[1:] + gr[:-1]) / 2).tolist()
    rows = []
    for p in (-6, 0, 3):
        for i in range(0, len(mid), 20):
            vals = [m * 2.0 ** p for m in mid[i:i + 20]]
            rows.append(vals + [-x for x in vals[:10]] + [float(gr[-1]) * 2.0 ** p])
    edge = 7.0 if bits == 4 else 464.0
    for s in (edge, edge * (1 - torch.finfo(dt).eps), edge * (1 + torch.finfo(dt).eps), 6.0, 448.0, 480.0, 1.0):
        for p in (-10, -2, 5):
            rows.append([s * 2.0 ** p, -s * 2.0 ** p / 3, 0.1, -0.0])
    rows += [[0.0] * 4, [-0.0] * 3, [big, -big, 1.0, big / 3], [tiny, -tiny / 2], [step, -step, 3 * step], [big / 2, step],
             [math.inf, 1.0], [1.0, -math.inf], [math.nan, 2.0], [math.nan, math.inf], [big, big / 7, big / 8]]
    x = torch.zeros(len(rows), K * D, dtype=F64)
    for i, r in enumerate(rows):
        x[i, 5:5 + len(r[:27])] = torch.tensor(r[:27], dtype=F64)     # within the first block of the first head
        x[i, 32:32 + len(r[27:])] = torch.tensor(r[27:], dtype=F64)
        x[i, D + 40] = r[0]
    x = x.to(dt)
    n = len(rows)
    c = new_cache(-(-n // 16), 16, K, D, dt, bits)
    Q.lora_quant_append(None, None, x.cuda(), x.cuda(), c, ints(list(range(n))))
    want, exps = QR.quantise(x.reshape(n, K, D).to(F64), bits, dt)
    for what in "kv":
        got = cells(c, what).reshape(-1, K, D)[:n]
        exp = (c.k_exp if what == "k" else c.v_exp).cpu().reshape(-1, K, D // 32)[:n]
        assert torch.equal(exp.to(F64), exps), what
        assert bool(((got == want) | (got.isnan() & want.isnan())).all()), what
        assert torch.equal(torch.signbit(got)[~got.isnan()], torch.signbit(want)[~want.isnan()])
    # what is read back is those values, and finite where they are
    ko, vo = (torch.empty(n, K * D, dtype=dt, device="cuda") for _ in range(2))
    Q.lora_quant_read(ko, vo, c, ints(list(range(n))))
    for o in (ko, vo):
        got = o.cpu().to(F64).reshape(n, K, D)
        assert bool(((got == want) | (got.isnan() & want.isnan())).all())


def test_append_in_place_and_without_rotation():
    n, H, K, D = 37, 4, 2, 128
    x = torch.randn(n, (H + 2 * K) * D, dtype=F16, device="cuda")
    q, k, v = x[:, :H * D], x[:, H * D:(H + K) * D], x[:, (H + K) * D:]
    rope, pos = S.Rope.base(D), torch.arange(n, dtype=torch.int32, device="cuda") * 100
    slots = ints(list(range(n)))
    a, b = Q.QuantKV.zeros(3, 16, K, D), Q.QuantKV.zeros(3, 16, K, D)
    out = torch.empty_like(q)
    Q.lora_quant_append(out, q, k, v, a, slots, rope=rope, positions=pos)
    Q.lora_quant_append(q, q, k, v, b, slots, rope=rope, positions=pos)
    assert torch.equal(out, q) and all(torch.equal(s, t) for s, t in zip(bytes_of(a), bytes_of(b)))
    plain = torch.empty_like(out)
    Q.lora_quant_append(plain, out, k, v, a, slots)
    assert torch.equal(plain, out) and torch.equal(a.v, b.v)
    want, exps = QR.quantise(k.cpu().reshape(n, K, D).to(F64), 4, F16)
    assert torch.equal(cells(a, "k").reshape(-1, K, D)[:n], want)


# ------------------------------------------------------------------ read
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dt", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("K,D,P,layout", [(2, 128, 16, "heads"), (3, 80, 8, "tokens"), (1, 8, 1, "heads"), (5, 40, 4, "gaps"),
                                          (2, 256, 32, "record"), (4, 64, 64, "heads")])
def test_read_gives_every_code_at_every_exponent(K, D, P, layout, bits, dt):
    """Any bytes: each value is the code times the power, rounded to the type where it does not hold it."""
    say(f"case quant-read K={K} D={D} bits={bits} {dt}")
    pages = 40
    c = new_cache(pages, P, K, D, dt, bits, layout, seed=D)
    n = 1500
    g = torch.Generator().manual_seed(1)
    slots = torch.randint(-3, pages * P + 3, (n,), generator=g).int()
    slots[7], slots[8] = -(2 ** 31), 2 ** 31 - 1
    wide = torch.full((n, K * D + 16), 5.0, dtype=dt, device="cuda")
    ko, vo = wide[:, :K * D], torch.full((n, K * D), 5.0, dtype=dt, device="cuda")
    Q.lora_quant_read(ko, vo, c, slots.cuda())
    torch.cuda.synchronize()
    live = (slots >= 0) & (slots < pages * P)
    at = slots[live].long()
    lo, hi = QR.exponent_range(dt, bits)
    for out, what in ((ko, "k"), (vo, "v")):
        want = cells(c, what)[at // P, at % P].reshape(-1, K * D)
        exp = (c.k_exp if what == "k" else c.v_exp).cpu()[at // P, at % P].long() - 127
        held = ((exp >= lo) & (exp <= hi)).repeat_interleave(32, -1)[..., :D].reshape(-1, K * D)
        got = out.cpu()[live].to(F64)
        same = (got == want) | (got.isnan() & want.isnan())
        assert bool(same[held].all())
        nan = (exp == 128).repeat_interleave(32, -1)[..., :D].reshape(-1, K * D)
        assert bool(got[nan].isnan().all())
        assert bool((out.cpu()[~live] == 5.0).all())
    assert bool((wide[:, K * D:] == 5.0).all())
    only = torch.full((n, K * D), 5.0, dtype=dt, device="cuda")
    Q.lora_quant_read(None, only, c, slots.cuda())
    assert torch.equal(only.view(torch.int16), vo.view(torch.int16))
    only.fill_(5.0)
    Q.lora_quant_read(only, None, c, slots.cuda())
    assert torch.equal(only.view(torch.int16), ko.contiguous().view(torch.int16))


def every_code_at_every_exponent(dt, bits, least=0, most=255):
    """256 tokens: block b of token t has exponent byte t (kept to least..most); with 8 bits a token's first 256 columns
    have all codes, with 4 bits the 16 of them over and over."""
    D, P = 256, 16
    c = Q.QuantKV.zeros(16, P, 1, D, dt, bits)
    codes = torch.arange(256) if bits == 8 else (torch.arange(128) * 2 % 16) | ((torch.arange(128) * 2 + 1) % 16) << 4
    exps = torch.arange(256).clamp(least, most).to(torch.uint8).view(16, P, 1, 1).cuda()
    for code, exp in ((c.k, c.k_exp), (c.v, c.v_exp)):
        code.copy_(codes.to(torch.uint8).cuda().expand_as(code))
        exp.copy_(exps.expand_as(exp))
    return c


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dt", [F16, BF16], ids=["f16", "bf16"])
def test_read_rounds_what_the_type_does_not_hold(dt, bits):
    """Every exponent byte, 0 and those that an append never writes too: to nearest even, down to 0, up to infinity.  (The
    values have four significant bits, so one rounding to 32 bits on the way to dt changes none.)"""
    say(f"case quant-read-foreign bits={bits} {dt}")
    c = every_code_at_every_exponent(dt, bits)
    outs = [torch.empty(256, 256, dtype=dt, device="cuda") for _ in range(2)]
    Q.lora_quant_read(*outs, c, torch.arange(256, dtype=torch.int32, device="cuda"))
    for o, what in zip(outs, "kv"):
        want, got = cells(c, what).reshape(256, 256).to(dt), o.cpu()
        assert bool(((got == want) | (got.isnan() & want.isnan())).all())
        assert torch.equal(torch.signbit(got)[~want.isnan()], torch.signbit(want)[~want.isnan()])
        assert bool(want.isinf().any()) and bool((want[1:128] == 0).any()) and bool(got[255].isnan().all())


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dt", [F16, BF16], ids=["f16", "bf16"])
def test_attention_over_cells_that_the_type_does_not_hold(dt, bits):
    """Exponents below those that an append writes: the products are those of the values as they are read back."""
    say(f"case quant-attention-foreign bits={bits} {dt}")
    c = every_code_at_every_exponent(dt, bits, most=127)
    if bits == 8:       # no NaN codes
        for code in (c.k, c.v):
            code[code % 128 == 127] = 0
    H, n = 3, 256
    val = [cells(c, what).to(dt) for what in "kv"]
    g = torch.Generator().manual_seed(bits)
    q = torch.randn(1, H * 256, generator=g).to(dt)
    out, lse = torch.empty(1, H * 256, dtype=dt, device="cuda"), torch.empty(1, H, device="cuda")
    table = torch.arange(16, dtype=torch.int32)[None]
    Q.lora_quant_attention(out, q.cuda(), c, table.cuda(), ints([n]), Q.attention_workspace(1, H, c), scale=0.01, lse=lse)
    w = QR.attention(q.reshape(1, H, 256), *val, table, [n], None, 0.01, 0, H)[0]
    close(out.reshape(H, 256), w[0], w[2], "out")
    close(lse[0], w[1], w[3], "lse")


@pytest.mark.parametrize("what", ["k", "v", "kv"])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("K,D,n", [(1, 8, 1100000), (1, 16, 600001), (3, 40, 140003), (2, 256, 17001), (70, 128, 1021)])
def test_reads_of_many_rows_are_those_of_few(K, D, n, bits, what):
    """Rows of one unit and of many, several to a workgroup, outputs beside which the cache does not stay in L2: the
    same bits as one row of each slot at a time."""
    say(f"case quant-read-many K={K} D={D} n={n} bits={bits} {what}")
    pages, P = 9, 8
    c = new_cache(pages, P, K, D, BF16, bits, seed=n)
    each = [torch.full((pages * P, K * D), 5.0, dtype=BF16, device="cuda") for _ in range(2)]
    Q.lora_quant_read(*each, c, torch.arange(pages * P, dtype=torch.int32, device="cuda"))
    g = torch.Generator(device="cuda").manual_seed(n)
    slots = torch.randint(-4, pages * P + 4, (n,), generator=g, device="cuda").int()
    outs = [torch.full((n + 1, K * D), 5.0, dtype=BF16, device="cuda") if w in what else None for w in "kv"]
    Q.lora_quant_read(*[None if o is None else o[:n] for o in outs], c, slots)
    torch.cuda.synchronize()
    live = (slots >= 0) & (slots < pages * P)
    for o, e in zip(outs, each):
        if o is not None:
            want = torch.where(live[:, None], e.view(torch.int16)[slots.clamp(0, pages * P - 1).long()],
                               torch.full((1,), 5.0, dtype=BF16, device="cuda").view(torch.int16))
            assert torch.equal(o[:n].view(torch.int16), want) and bool((o[n:] == 5.0).all())


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("H,K,D,n", [(130, 2, 128, 1031), (2, 1, 64, 5001), (0, 3, 40, 1153), (300, 1, 80, 1025)])
def test_appends_of_many_rows_are_those_of_few(H, K, D, n, bits, inter):
    """A workgroup to a row, in groups, and q_out beyond what the L2s hold: the same bits as the rows a hundred at a
    time, with rows between them that name no slot."""
    say(f"case quant-append-many H={H} K={K} D={D} n={n} bits={bits} inter={inter}")
    g = torch.Generator(device="cuda").manual_seed(n)
    P = 16
    pages = -(-n // P)
    x = torch.randn(n, (H + 2 * K) * D, generator=g, device="cuda").to(BF16)
    q, k, v = x[:, :H * D], x[:, H * D:(H + K) * D], x[:, (H + K) * D:]
    slots = torch.randperm(pages * P, generator=g, device="cuda")[:n].int()
    slots[torch.rand(n, generator=g, device="cuda") < 0.1] = -1
    pos = torch.randint(0, 100000, (1, n), generator=g, device="cuda", dtype=torch.int32)
    rope = S.Rope(S.Rope.base(D if D != 40 else 32).inv_freq, None, 1, inter)
    got = []
    for step in (n, 100):
        c = new_cache(pages, P, K, D, BF16, bits, seed=3)
        out = torch.full((n + 1, max(H, 1) * D), 5.0, dtype=BF16, device="cuda")
        for a in range(0, n, step):
            b = min(a + step, n)
            Q.lora_quant_append(out[a:b] if H else None, q[a:b] if H else None, k[a:b], v[a:b], c, slots[a:b], rope=rope,
                                positions=pos[:, a:b].contiguous())
        torch.cuda.synchronize()
        got.append(bytes_of(c) + [out])
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert bool((got[0][-1][n:] == 5.0).all()) and bool((got[0][-1][:n][slots < 0] == 5.0).all())


# ------------------------------------------------------------------ attention
class Attn:
    """A batch of requests of those lengths over a cache of normal values."""

    def __init__(self, lens, H, K, D, P, dt, bits, layout="heads", seed=0, gain=1.0):
        g = torch.Generator().manual_seed(seed)
        blocks = [-(-max(n, 0) // P) for n in lens]
        pages = sum(blocks) + 2
        self.c = new_cache(pages, P, K, D, dt, bits, layout, seed)
        # unused cells hold NaN blocks: they must not matter
        x = torch.randn(2, pages, P, K, D, generator=g).to(dt).to(F64)
        x[0] *= torch.where(torch.rand(K, D, generator=g) < 0.05, 8.0, 1.0).to(F64)
        self.val = []
        for i, (code, exp) in enumerate(((self.c.k, self.c.k_exp), (self.c.v, self.c.v_exp))):
            y, e = QR.quantise(x[i], bits, dt)
            code.copy_(QR.pack(y, e, bits))
            exp.copy_(e.to(torch.uint8))
            self.val.append(y.to(dt))
            assert torch.equal(self.val[i].to(F64), y)
        ids = torch.randperm(pages, generator=g).int()
        self.used = ids[:sum(blocks)]
        self.table = torch.full((max(len(lens), 1), max(blocks + [0]) + 1), -1, dtype=torch.int32)
        at = 0
        for r, b in enumerate(blocks):
            self.table[r, :b] = ids[at:at + b]
            at += b
        self.lens, self.H, self.dt = list(lens), H, dt
        self.q = (gain * torch.randn(len(lens), H * D, generator=g)).to(dt)
        self.D = D

    def poison(self):
        """NaN blocks wherever no request's token lies."""
        seen = torch.zeros(self.c.num_pages, self.c.page_size, dtype=torch.bool)
        for r, n in enumerate(self.lens):
            t = torch.arange(max(n, 0))
            pg = self.table[r].long()[t // self.c.page_size]
            ok = (pg >= 0) & (pg < self.c.num_pages)
            seen[pg[ok], (t % self.c.page_size)[ok]] = True
        for e in (self.c.k_exp, self.c.v_exp):
            m = e.cpu().clone()
            m[~seen] = 255
            e.copy_(m)

    def run(self, req=None, scale=None, window=0, work=None, lse=True, q=None, kv_len=None, table=None, stride=8):
        q = self.q.cuda() if q is None else q
        n = q.shape[0]
        wide = torch.full((n, q.shape[1] + stride), 9.0, dtype=self.dt, device="cuda")
        self.out = wide[:, :q.shape[1]]
        self.wide = wide
        self.lse = torch.full((n, self.H), 9.0, device="cuda") if lse else None
        work = Q.attention_workspace(n, self.H, self.c) if work is None else work
        Q.lora_quant_attention(self.out, q, self.c, self.table.cuda() if table is None else table,
                               ints(self.lens) if kv_len is None else kv_len, work, req=req, scale=scale, window=window,
                               lse=self.lse)
        return self

    def check(self, req=None, scale=None, window=0, what="", q=None, kv_len=None):
        torch.cuda.synchronize()
        q = self.q if q is None else q
        lens = self.lens if kv_len is None else kv_len
        want = QR.attention(q.reshape(q.shape[0], self.H, self.D), *self.val, self.table, lens, req,
                            1.0 / math.sqrt(self.D) if scale is None else scale, window, self.H)
        out = self.out.cpu().reshape(q.shape[0], self.H, self.D)
        for i, w in enumerate(want):
            if w is None:
                assert bool((out[i] == 9.0).all()) and bool((self.lse[i] == 9.0).all()), f"{what}: row {i} is not active"
                continue
            close(out[i], w[0], w[2], f"{what} row {i} out")
            if self.lse is not None:
                close(self.lse[i], w[1], w[3], f"{what} row {i} lse")
        assert bool((self.wide[:, q.shape[1]:] == 9.0).all())


LENS = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, -1, 511, 700, 1025]
ATTN = [([1], 1, 1, 8, 1), ([17], 32, 32, 128, 16), (LENS, 4, 4, 128, 16), (LENS, 8, 2, 64, 8), (LENS, 8, 1, 128, 64),
        (LENS, 6, 2, 80, 1), (LENS, 5, 1, 96, 32), (LENS, 10, 2, 32, 16), (LENS, 16, 1, 128, 16), (LENS, 34, 2, 40, 4),
        (LENS, 4, 2, 256, 16), (LENS, 18, 2, 160, 8), (LENS, 7, 1, 48, 1024), ([3000, 5, 9000], 8, 2, 128, 16),
        ([20011], 8, 1, 128, 64), ([40000], 3, 1, 64, 32), ([9001, 1], 17, 1, 256, 16)]


@pytest.mark.parametrize("case", ATTN, ids=lambda c: f"{len(c[0])}x{max(c[0])}-" + "-".join(map(str, c[1:])))
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dt", [F16, BF16], ids=["f16", "bf16"])
def test_attention_matches_the_formula(case, bits, dt):
    lens, H, K, D, P = case
    say(f"case quant-attention {case} bits={bits} {dt}")
    layout = ("heads", "tokens", "gaps", "record")[(H + D + bits) % 4]
    a = Attn(lens, H, K, D, P, dt, bits, layout, seed=H + D)
    a.poison()
    a.run().check(what="call")


@pytest.mark.parametrize("window", [1, 5, 16, 63, 64, 65, 100, 4000])
@pytest.mark.parametrize("bits", [4, 8])
def test_attention_window(window, bits):
    say(f"case quant-attention-window {window} bits={bits}")
    Attn(LENS, 8, 2, 128, 16, F16, bits, seed=window).run(window=window).check(window=window, what="window")


def test_attention_pages_that_are_none():
    say("case quant-attention-pages")
    a = Attn([300, 64, 33, 200], 8, 2, 128, 16, F16, 4, seed=3)
    a.table[0, 3], a.table[0, 7], a.table[0, 18] = -1, a.c.num_pages, 2 ** 31 - 1
    a.table[1, :4] = torch.tensor([-5, -1, a.c.num_pages + 9, -(2 ** 31)], dtype=torch.int32)   # nothing left
    a.table[2, 0] = -1
    a.poison()
    a.run().check(what="pages")
    assert not bool(a.out[1].any()) and bool((a.lse[1] == -math.inf).all())


def test_attention_rows_that_are_not_active():
    say("case quant-attention-inactive")
    a = Attn([40, 100, 64, 7, 30], 4, 1, 64, 8, BF16, 4, seed=4)
    req = [0, 5, -1, 3, 2 ** 31 - 1]
    a.run(req=ints(req)).check(req=req, what="req")
    lens = [-1, 2 ** 31 - 1, a.table.shape[1] * 8 + 1, -(2 ** 31), 30]
    a.run(kv_len=ints(lens)).check(kv_len=lens, what="lengths")


@pytest.mark.parametrize("n,every", [(64, 1), (300, 1), (700, 3), (5000, 1111)])
def test_attention_of_many_rows_few_of_them_active(n, every):
    say(f"case quant-attention-many {n} {every}")
    lens = [(37 * i) % 150 if i % every == 0 else -1 for i in range(n)]
    Attn(lens, 4, 1, 64, 16, F16, 4, seed=n).run().check(what="many")


def test_attention_rows_that_share_a_request():
    say("case quant-attention-shared")
    a = Attn([500, 90], 8, 2, 128, 16, F16, 4, seed=6)
    req, lens = [0, 0, 1, 0, 1, 0], [500, 499, 90, 64, 1, 65]
    q = torch.randn(6, 8 * 128).to(F16)
    a.run(req=ints(req), kv_len=ints(lens), q=q.cuda()).check(req=req, kv_len=lens, q=q, what="shared")


@pytest.mark.parametrize("scale", [-0.3, 0.0, 2.0])
def test_attention_scales_and_large_scores(scale):
    say(f"case quant-attention-scale {scale}")
    Attn([70, 300, 1], 4, 2, 128, 16, F16, 4, seed=7, gain=3.0).run(scale=scale).check(scale=scale, what="scale")


@pytest.mark.parametrize("dt", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("bits", [4, 8])
def test_attention_visible_nan_blocks(dt, bits):
    """A NaN block of k makes its head's row NaN; one of v the columns of that block; other heads and rows are as
    they were."""
    say(f"case quant-attention-nan {dt} bits={bits}")
    a = Attn([200, 200, 70], 8, 2, 128, 16, dt, bits, seed=8)
    P = 16
    for r, t, h, blk, which in ((0, 150, 1, 2, 0), (1, 30, 0, 3, 1)):
        pg = int(a.table[r, t // P])
        (a.c.k_exp if which == 0 else a.c.v_exp)[pg, t % P, h, blk] = 255
        a.val[which][pg, t % P, h, 32 * blk:32 * blk + 32] = math.nan
    a.run()
    torch.cuda.synchronize()
    out = a.out.cpu().reshape(3, 8, 128)
    assert bool(out[0, 4:].isnan().all()) and not bool(out[0, :4].isnan().any())
    assert bool(out[1, :4, 96:].isnan().all()) and not bool(out[1, :4, :96].isnan().any()) and not bool(out[1, 4:].isnan().any())
    assert not bool(out[2].isnan().any())
    assert bool(a.lse[0, 4:].isnan().all()) and not bool(a.lse[1:].isnan().any())


def test_attention_small_weights_and_subnormal_values():
    say("case quant-attention-small")
    # one token far ahead of 4000 others whose weights are near the cut
    a = Attn([4001], 1, 1, 32, 16, F16, 4, seed=9)
    k, v = torch.zeros(1, 1, 1, 32, dtype=F64), torch.ones(1, 1, 1, 32, dtype=F64)
    k = k.expand(a.c.num_pages, 16, 1, 32).clone()
    pg = int(a.table[0, 0])
    k[pg, 0, 0, 0] = 6.0
    for i, x in enumerate((k, v.expand_as(k) * 2.0 ** -20)):
        y, e = QR.quantise(x, 4, F16)
        (a.c.k if i == 0 else a.c.v).copy_(QR.pack(y, e, 4))
        (a.c.k_exp if i == 0 else a.c.v_exp).copy_(e.to(torch.uint8))
        a.val[i] = y.to(F16)
    a.q.zero_()
    for s in (1.0, 2.5, 4.3):
        a.q[0, 0] = s
        a.run(scale=1.0).check(scale=1.0, what=f"scale {s}")


def test_attention_equals_the_16_bit_attention_over_the_values():
    """The same numbers in a 16-bit cache: out within both bounds, so within twice one."""
    say("case quant-attention-16")
    lens = [5, 64, 700, 0, 2000, 33]
    for H, K in ((8, 8), (8, 2), (32, 2)):
        a = Attn(lens, H, K, 128, 16, F16, 4, seed=10)
        a.run()
        paged = S.PagedKV(a.val[0].cuda(), a.val[1].cuda())
        out, lse = torch.empty(len(lens), H * 128, dtype=F16, device="cuda"), torch.empty(len(lens), H, device="cuda")
        S.lora_paged_attention(out, a.q.cuda(), paged, a.table.cuda(), ints(lens), S.attention_workspace(len(lens), H, paged), lse=lse)
        want = QR.attention(a.q.reshape(len(lens), H, 128), *a.val, a.table, lens, None, 1 / math.sqrt(128), 0, H)
        for i, w in enumerate(want):
            close(out[i].reshape(H, 128), a.out[i].double().cpu().reshape(H, 128), 2 * w[2], f"row {i}")
            close(lse[i], a.lse[i].double().cpu(), 2 * w[3], f"row {i} lse")


# ------------------------------------------------------------------ calls
def test_results_are_the_same_every_time_and_the_workspace_is_left_clean():
    say("case quant-repeat")
    a = Attn([9000, 3, 700, 64] * 8, 8, 2, 128, 16, F16, 4, seed=11)
    work = Q.attention_workspace(64, 8, a.c)
    a.run(work=work)
    first, lse = a.out.clone(), a.lse.clone()
    counters = work[:2 * (4 * 256 + 4096)]
    for _ in range(3):
        a.run(work=work)
        assert torch.equal(a.out, first) and torch.equal(a.lse, lse)
        assert not bool(counters.any())


def test_the_workspace_is_shared_with_the_16_bit_attention():
    say("case quant-workspace")
    a = Attn([5000, 30], 8, 2, 128, 16, F16, 4, seed=12)
    paged = S.PagedKV(a.val[0].cuda(), a.val[1].cuda())
    work = torch.zeros(max(Q.attention_workspace(2, 8, a.c).numel(), S.attention_workspace(2, 8, paged).numel()),
                       dtype=torch.int32, device="cuda")
    out = torch.empty(2, 8 * 128, dtype=F16, device="cuda")
    for _ in range(2):
        a.run(work=work).check(what="quantised")
        S.lora_paged_attention(out, a.q.cuda(), paged, a.table.cuda(), ints(a.lens), work)
    a.run(work=work).check(what="after")


def test_calls_on_no_rows():
    c = Q.QuantKV.zeros(2, 16, 2, 64)
    e = lambda n: torch.empty(0, n, dtype=F16, device="cuda")
    none = ints([])
    Q.lora_quant_append(e(256), e(256), e(128), e(128), c, none, rope=S.Rope.base(64), positions=torch.empty(1, 0, dtype=torch.int32, device="cuda"))
    Q.lora_quant_read(e(128), e(128), c, none)
    Q.lora_quant_attention(e(256), e(256), c, torch.zeros(1, 2, dtype=torch.int32, device="cuda"), none, Q.attention_workspace(1, 4, c))
    torch.cuda.synchronize()


def test_two_streams_with_workspaces_of_their_own():
    say("case quant-streams")
    cases = [Attn([4000 + i, 200], 8, 2, 128, 16, F16, 4, seed=20 + i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in cases]
    works = [Q.attention_workspace(2, 8, a.c) for a in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for a, st, w in zip(cases, streams, works):
            with torch.cuda.stream(st):
                a.run(work=w)
    torch.cuda.synchronize()
    for a in cases:
        a.check(what="stream")


def test_a_step_captured_and_replayed_with_other_tokens():
    """Append, read and attention as one graph: new slots, positions and lengths in the same arrays before
    every replay, and eager work between them."""
    say("case quant-graph")
    n, H, K, D, P = 6, 8, 2, 128, 16
    c, eager = Q.QuantKV.zeros(64, P, K, D), Q.QuantKV.zeros(64, P, K, D)
    table = torch.arange(n * 8, dtype=torch.int32, device="cuda").view(n, 8)
    rope, work, work2 = S.Rope.base(D), Q.attention_workspace(n, H, c), Q.attention_workspace(n, H, c)
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(n, (H + 2 * K) * D, generator=g, dtype=F16, device="cuda")
    lens, slots, pos = ints([0] * n), ints([0] * n), ints([0] * n)
    q, k, v = x[:, :H * D], x[:, H * D:(H + K) * D], x[:, (H + K) * D:]
    bufs = [[torch.zeros(n, w, dtype=F16, device="cuda") for w in (H * D, K * D, K * D, H * D)] for _ in range(2)]

    def step(cache, work, qo, ko, vo, out):
        Q.lora_quant_append(qo, q, k, v, cache, slots, rope=rope, positions=pos)
        Q.lora_quant_read(ko, vo, cache, slots)
        Q.lora_quant_attention(out, qo, cache, table, lens, work)

    have = [0] * n

    def tokens(i):
        x.copy_(torch.randn(n, (H + 2 * K) * D, generator=g, dtype=F16, device="cuda"))
        for r in range(n):
            have[r] = min(have[r] + 1 + (i + r) % 3 * 0, 128)
        p = [h - 1 for h in have]
        lens.copy_(ints(have))
        pos.copy_(ints(p))
        slots.copy_(ints([int(table[r, p[r] // P]) * P + p[r] % P for r in range(n)]))

    tokens(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(c, work, *bufs[0])
    torch.cuda.current_stream().wait_stream(side)
    step(eager, work2, *bufs[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(c, work, *bufs[0])
    for i in range(1, 20):
        tokens(i)
        graph.replay()
        step(eager, work2, *bufs[1])
        torch.cuda.synchronize()
        for a, b in zip(*bufs):
            assert torch.equal(a, b), i
        assert all(torch.equal(s, t) for s, t in zip(bytes_of(c), bytes_of(eager)))


def test_the_python_and_the_compiled_calls_are_the_same(monkeypatch):
    say("case quant-python")
    a = Attn([100, 40], 4, 2, 64, 16, F16, 8, seed=13)
    n, K, D = 2, 2, 64
    x = torch.randn(n, 4 * D + 2 * K * D, dtype=F16, device="cuda")
    q, k, v = x[:, :4 * D], x[:, 4 * D:4 * D + K * D], x[:, 4 * D + K * D:]
    rope, slots = S.Rope.base(D), ints([3, 17])
    got = []
    for fast in (S._fast, None):
        monkeypatch.setattr(S, "_fast", fast)
        c = Q.QuantKV.zeros(3, 16, K, D, bits=8)
        outs = [torch.zeros(n, w, dtype=F16, device="cuda") for w in (4 * D, K * D, K * D)]
        Q.lora_quant_append(outs[0], q, k, v, c, slots, rope=rope, positions=ints([5, 9]))
        Q.lora_quant_read(outs[1], outs[2], c, slots)
        a.run()
        got.append(outs + bytes_of(c) + [a.out.clone(), a.lse.clone()])
    assert all(torch.equal(x, y) for x, y in zip(*got))
    assert bool(got[0][1].any())


def test_cells_beyond_32_bit_offsets():
    """Pages more than 2^32 bytes apart, codes and exponents."""
    say("case quant-offsets")
    K, D, P = 1, 128, 16
    far = (1 << 32) + 4096
    buf = torch.zeros(2 * far + 65536, dtype=torch.uint8, device="cuda")
    mk = lambda at, n: buf.as_strided((3, P, K, n), (far, n, n, 1), at)
    c = Q.QuantKV(mk(0, 64), mk(4096, 64), mk(8192, 4), mk(12288, 4), D, F16)
    n = 3 * P
    x = torch.randn(n, K * D, dtype=F16, device="cuda")
    Q.lora_quant_append(None, None, x, -x, c, ints(list(range(n))))
    ko, vo = torch.empty_like(x), torch.empty_like(x)
    Q.lora_quant_read(ko, vo, c, ints(list(range(n))))
    want, _ = QR.quantise(x.cpu().reshape(n, K, D).to(F64), 4, F16)
    assert torch.equal(ko.cpu().to(F64), want.reshape(n, -1)) and torch.equal(vo, -ko)
    q = torch.randn(1, D, dtype=F16)
    out, lse = torch.empty(1, D, dtype=F16, device="cuda"), torch.empty(1, 1, device="cuda")
    table = ints([[2, 0, 1]])
    Q.lora_quant_attention(out, q.cuda(), c, table, ints([45]), Q.attention_workspace(1, 1, c), lse=lse)
    kk = ko.cpu().reshape(3, P, K, D)
    w = QR.attention(q.reshape(1, 1, D), kk, -kk, table.cpu(), [45], None, 1 / math.sqrt(D), 0, 1)[0]
    close(out.reshape(1, D), w[0], w[2], "out")
    close(lse[0], w[1], w[3], "lse")


@pytest.mark.parametrize("bits", [4, 8])
def test_cells_in_records_of_one_tensor(bits):
    """Codes of k and v and their exponents side by side, token by token and head by head: the bits of a cache of
    separate tensors."""
    say(f"case quant-records bits={bits}")
    pages, P, H, K, D, n = 9, 16, 8, 2, 64, 130
    cb, eb = 8 * bits, 2
    one = torch.zeros(pages, P, K, -(-2 * (cb + eb) // 16) * 16, dtype=torch.uint8, device="cuda")
    rec = Q.QuantKV(one[..., :cb], one[..., cb:2 * cb], one[..., 2 * cb:2 * cb + eb], one[..., 2 * cb + eb:2 * (cb + eb)], D, F16)
    g = torch.Generator(device="cuda").manual_seed(bits)
    x = torch.randn(n, 2 * K * D, generator=g, device="cuda").to(F16)
    q = torch.randn(1, H * D, generator=g, device="cuda").to(F16)
    slots, table = torch.arange(n, dtype=torch.int32, device="cuda"), torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    got = []
    for c in (rec, Q.QuantKV.zeros(pages, P, K, D, F16, bits)):
        Q.lora_quant_append(None, None, x[:, :K * D], x[:, K * D:], c, slots, rope=S.Rope.base(D), positions=slots)
        outs = [torch.zeros(n, K * D, dtype=F16, device="cuda") for _ in range(2)]
        Q.lora_quant_read(*outs, c, slots)
        out = torch.zeros_like(q)
        Q.lora_quant_attention(out, q, c, table, ints([n]), Q.attention_workspace(1, H, c))
        torch.cuda.synchronize()
        got.append(bytes_of(c) + outs + [out])
    assert all(torch.equal(a, b) for a, b in zip(*got)) and bool(got[0][-1].any())
