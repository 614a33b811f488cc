"""GPU: the decode-step operators (lora_step.h) against their 64-bit references, at the sizes,
layouts and masks where they can go wrong.  Tolerances are derived in step_ref."""
import math
import random

import pytest
import torch

from segmented_gather_matmul_amd import binding as B
from segmented_gather_matmul_amd import step as S
from tests import step_ref as R
from tests.gpu_cases import say

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()
    yield


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def close(got, want, bound, what):
    got, want = got.double().cpu(), want
    bad = ~((got - want).abs() <= bound) & ~((got == want) | (got.isnan() & want.isnan()))
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                           f"{float((got - want).abs()[bad].max())} at {bad.nonzero()[0].tolist()}")


# ------------------------------------------------------------------ step plan
class PlanCase:
    def __init__(self, kv, new, page, max_blocks, spare, max_tokens=None, seed=0, slots=True, pages_short=0):
        rng = random.Random(seed)
        n = len(kv)
        blocks = [min(-(-max(c, 0) // page), max_blocks) for c in kv]
        need = sum(max(0, min(-(-(c + m) // page), max_blocks) - -(-c // page)) for c, m in zip(kv, new) if m > 0 and c >= 0)
        total = max(1, sum(blocks) + max(need - pages_short, 0) + spare)
        ids = list(range(total))
        rng.shuffle(ids)
        self.table = [[ids.pop() for _ in range(b)] + [-7] * (max_blocks - b) for b in blocks]
        self.top = len(ids)
        self.free = ids + [-9] * (total - len(ids))
        self.kv, self.new, self.page = list(kv), list(new), page
        self.req_slot = [rng.randrange(-1, 9) for _ in kv] if slots else None
        self.max_tokens = sum(max(m, 0) for m in new) + 3 if max_tokens is None else max_tokens
        # a wider allocation than the table: the columns behind it are not the plan's
        self.wide = torch.full((max(n, 1), max_blocks + 5), -3, dtype=torch.int32, device="cuda")
        if n:
            self.wide[:, :max_blocks] = ints(self.table)
        self.dev_free, self.dev_top = ints(self.free), ints([self.top])
        self.pages = S.KVPages(self.wide[:n, :max_blocks], self.dev_free, self.dev_top, page)
        self.dev_kv, self.dev_new = ints(self.kv) if n else ints([]), ints(self.new) if n else ints([])
        self.dev_slot = ints(self.req_slot) if slots and n else None

    def want(self):
        return R.plan(self.kv, self.new, self.table, self.free, self.top, self.page, self.max_tokens, self.req_slot)

    def check(self, plan, want, what):
        torch.cuda.synchronize()
        n, mb = len(self.kv), self.pages.max_blocks
        got = dict(status=plan.status, kv_end=plan.kv_end[:n], free_top=plan.free_top[0], q_ptr=plan.q_ptr[:n + 1],
                   tok_req=plan.tok_req[:self.max_tokens], tok_pos=plan.tok_pos[:self.max_tokens],
                   slots=plan.slots[:self.max_tokens], idx=plan.idx[:self.max_tokens], table=self.wide[:n, :mb],
                   free=self.dev_free)
        for k, t in got.items():
            assert t.tolist() == want[k], f"{what}: {k}"
        assert (self.wide[:, mb:] == -3).all(), f"{what}: behind the table"


def _mixed(n, seed, page, most=300, prefill=0.2, ended=0.1):
    rng = random.Random(seed)
    kv = [rng.choice([0, 1, page, page - 1, page + 1, rng.randrange(most)]) for _ in range(n)]
    new = [-1 if rng.random() < ended else rng.randrange(most) if rng.random() < prefill else rng.choice([0, 1, 1, 1])
           for _ in range(n)]
    return kv, new


@pytest.mark.parametrize("n,page,seed", [(1, 16, 0), (3, 1, 1), (32, 16, 2), (61, 1, 3), (64, 1024, 4), (509, 32, 5),
                                         (1023, 8, 6), (1024, 16, 7), (1025, 16, 8), (2500, 4, 9), (4097, 64, 10)])
def test_plan_equals_its_definition(n, page, seed):
    say(f"case plan n={n} page={page}")
    kv, new = _mixed(n, seed, page)
    c = PlanCase(kv, new, page, max_blocks=-(-600 // page) + 1, spare=5, seed=seed)
    plan = S.KVPlan(n, c.max_tokens)
    S.lora_kv_plan(plan, c.pages, c.dev_kv, c.dev_new, req_slot=c.dev_slot)
    want = c.want()
    assert want["status"][0] == 0
    c.check(plan, want, "first call")
    S.lora_kv_plan(plan, c.pages, c.dev_kv, c.dev_new, req_slot=c.dev_slot)   # same lengths: the same step again
    c.check(plan, want, "second call")


@pytest.mark.parametrize("n,page,cap", [(61, 1, 6000), (300, 16, 40000), (700, 8, 60000), (1500, 4, 90000), (40, 16, 900)])
@pytest.mark.parametrize("fits", [True, False])
def test_plan_in_place_equals_its_definition(n, page, cap, fits):
    """kv_end is kv_len and the free top is updated where it is read, in steps of every size."""
    say(f"case plan-in-place n={n} page={page} cap={cap} fits={fits}")
    kv, new = _mixed(n, n, page, most=100)
    c = PlanCase(kv, new, page, max_blocks=-(-300 // page), spare=3, seed=n, max_tokens=cap if fits else 30)
    plan = S.KVPlan(n, c.max_tokens, kv_end=c.dev_kv, free_top=c.dev_top)
    want = c.want()
    assert (want["status"][0] == 0) == fits
    S.lora_kv_plan(plan, c.pages, c.dev_kv, c.dev_new, req_slot=c.dev_slot)
    c.check(plan, want, "in place")
    kv2 = [k if k < 150 else 5 for k in want["kv_end"]]          # and a second step from there
    if fits and kv2 == want["kv_end"]:
        new2 = [1 if i % 3 else 0 for i in range(n)]
        want2 = R.plan(kv2, new2, want["table"], want["free"], want["free_top"], page, cap, c.req_slot)
        c.dev_new.copy_(ints(new2))
        S.lora_kv_plan(plan, c.pages, c.dev_kv, c.dev_new, req_slot=c.dev_slot)
        c.check(plan, want2, "second step")


@pytest.mark.parametrize("n,page,cap", [(40, 16, 900), (300, 16, 40000), (700, 8, 60000), (1024, 8, 500), (1500, 4, 90000)])
def test_plan_in_place_in_chained_steps(n, page, cap):
    """Step after step over the same arrays in place, whatever the lengths have become: each from
    what the one before left, with requests that end and ones that start in their rows again."""
    say(f"case plan-in-place-chained n={n} page={page} cap={cap}")
    rng = random.Random(n)
    kv, new = _mixed(n, n, page, most=min(100, cap // 40))
    mb = -(-300 // page)
    c = PlanCase(kv, new, page, max_blocks=mb, spare=6 * n, seed=n, max_tokens=cap)
    plan = S.KVPlan(n, cap, kv_end=c.dev_kv, free_top=c.dev_top)
    for it in range(4):
        want = R.plan(c.kv, c.new, c.table, c.free, c.top, page, cap, c.req_slot)
        assert want["status"][0] in ((0, 4) if it == 0 else (0,)), (it, want["status"])   # (1024 requests: the first has too many rows)
        S.lora_kv_plan(plan, c.pages, c.dev_kv, c.dev_new, req_slot=c.dev_slot)
        c.check(plan, want, f"step {it}")
        c.kv, c.table, c.free, c.top = want["kv_end"], want["table"], want["free"], want["free_top"]
        left, room = c.top, cap
        c.new = []
        for have in c.kv:          # what the table, the free pages and the rows still hold
            m = rng.choice([-1, 0, 1, 1, 1, 5, 2 * page])
            grow = -(-(have + max(m, 0)) // page) - -(-have // page)
            if m > 0 and (have + m > mb * page or grow > left or m > room):
                m = 0
            if m > 0:
                left, room = left - grow, room - m
            c.new.append(m)
        c.dev_new.copy_(ints(c.new))


@pytest.mark.parametrize("kv,new,page,max_tokens", [
    ([], [], 16, 5), ([0], [0], 16, 0), ([0], [0], 16, 4), ([0, 0], [1, 0], 1, 1), ([5], [-1], 4, 2),
    ([0] * 7, [-1] * 7, 8, 3), ([16], [16], 16, 16), ([4095], [1], 16, 4096), ([0, 3], [5000, 1], 16, 5100),
    ([0, 3], [5000, 1], 1, 5001)])
def test_plan_of_small_and_odd_steps(kv, new, page, max_tokens):
    say(f"case plan-odd {kv} {new} page={page} cap={max_tokens}")
    c = PlanCase(kv, new, page, max_blocks=-(-5100 // page), spare=0, max_tokens=max_tokens, slots=False)
    plan = S.KVPlan(len(kv), max_tokens)
    S.lora_kv_plan(plan, c.pages, c.dev_kv, c.dev_new)
    want = c.want()
    assert want["status"][0] == 0
    c.check(plan, want, "odd")


@pytest.mark.parametrize("kind,kw,bit", [
    ("pages", dict(kv=[3, 20, 7], new=[30, -1, 40], page=4, max_blocks=40, spare=0, pages_short=9), 1),
    ("table", dict(kv=[3, 20], new=[1, 45], page=4, max_blocks=16, spare=9), 2),
    ("held", dict(kv=[3, 70], new=[1, 0], page=4, max_blocks=16, spare=99), 2),
    ("rows", dict(kv=[3, 20], new=[6, 5], page=4, max_blocks=16, spare=9, max_tokens=10), 4),
    ("negative", dict(kv=[3, -2], new=[1, 1], page=4, max_blocks=16, spare=9), 8),
    ("code", dict(kv=[3, 2], new=[1, -2], page=4, max_blocks=16, spare=9), 8),
    ("huge", dict(kv=[2 ** 31 - 1, 2], new=[2 ** 31 - 1, 2 ** 31 - 1], page=4, max_blocks=16, spare=9, max_tokens=10), 6),
    ("many", dict(kv=[0] * 1500, new=[1] * 1499 + [5000], page=4, max_blocks=16, spare=9, max_tokens=7000), 2)])
def test_plan_that_does_not_fit_changes_nothing(kind, kw, bit):
    say(f"case plan-{kind}")
    c = PlanCase(**kw)
    plan = S.KVPlan(len(c.kv), c.max_tokens)
    S.lora_kv_plan(plan, c.pages, c.dev_kv, c.dev_new, req_slot=c.dev_slot)
    want = c.want()
    assert want["status"][0] & bit
    c.check(plan, want, kind)


def test_plan_with_a_bad_free_list_changes_nothing():
    for top in (-1, 10 ** 6):
        c = PlanCase([3, 9], [1, -1], 4, 16, 9)
        c.top = top
        c.dev_top.fill_(top)
        plan = S.KVPlan(2, c.max_tokens)
        S.lora_kv_plan(plan, c.pages, c.dev_kv, c.dev_new, req_slot=c.dev_slot)
        assert c.want()["status"][0] & 8
        c.check(plan, c.want(), f"top {top}")
    c = PlanCase([9, 9], [-1, -1], 4, 16, 0)      # more returned than the list holds
    c.top = len(c.free)
    c.dev_top.fill_(c.top)
    plan = S.KVPlan(2, c.max_tokens)
    S.lora_kv_plan(plan, c.pages, c.dev_kv, c.dev_new, req_slot=c.dev_slot)
    assert c.want()["status"][0] & 8
    c.check(plan, c.want(), "full list")


def test_plan_gives_no_slot_for_a_table_entry_that_is_no_page():
    for page, cap in ((4, 64), (4, 5000)):       # both places that write the maps
        c = PlanCase([6, 9], [1, 2], page, 16, 4, max_tokens=cap)
        bad = [[-5] * 16, [10 ** 6] * 16]
        c.table = bad
        c.wide[:, :16] = ints(bad)
        plan = S.KVPlan(2, cap)
        S.lora_kv_plan(plan, c.pages, c.dev_kv, c.dev_new, req_slot=c.dev_slot)
        assert c.want()["slots"][:2] == [-1, -1]
        c.check(plan, c.want(), f"cap {cap}")


def test_plan_in_place_over_many_captured_steps():
    """kv_len and the free top updated in place by a captured plan, replayed over steps whose
    new_len is written into the same array; requests end and their pages are used again."""
    say("case plan-graph")
    rng = random.Random(5)
    n, page, mb = 37, 8, 12
    pages = S.KVPages.fresh(n, mb, 150, page)
    kv, new, slot = ints([0] * n), ints([0] * n), ints([rng.randrange(-1, 5) for _ in range(n)])
    plan = S.KVPlan(n, 256, kv_end=kv, free_top=pages.free_top)
    S.lora_kv_plan(plan, pages, kv, new, req_slot=slot)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        S.lora_kv_plan(plan, pages, kv, new, req_slot=slot)
    refused = 0
    for it in range(40):
        state = (kv.tolist(), pages.block_table.tolist(), pages.free_pages.tolist(), pages.free_top.item())
        step = [-1 if state[0][r] > 60 or rng.random() < 0.05 else rng.choice([0, 1, 1, 7, 20]) for r in range(n)]
        if sum(max(s, 0) for s in step) > 256:
            step = [min(s, 1) for s in step]
        new.copy_(ints(step))
        want = R.plan(state[0], step, state[1], state[2], state[3], page, 256, slot.tolist())
        g.replay()
        torch.cuda.synchronize()
        got = dict(status=plan.status, kv_end=kv, free_top=pages.free_top[0], q_ptr=plan.q_ptr, tok_req=plan.tok_req,
                   tok_pos=plan.tok_pos, slots=plan.slots, idx=plan.idx, table=pages.block_table, free=pages.free_pages)
        for k, t in got.items():
            assert t.tolist() == want[k], f"step {it}: {k}"
        refused += want["status"][0] != 0
        if want["status"][0] == 0:     # no page is held twice
            held = [p for r in range(n) for p in want["table"][r][:-(-want["kv_end"][r] // page)]]
            held += want["free"][:want["free_top"]]
            assert len(held) == len(set(held)) == 150
    assert 0 < refused < 40
    del g


# ------------------------------------------------------------------ rotary positions and append
def _cache(pages, P, K, D, dt, layout, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(dt)
    if layout == "token":
        k, v = rnd(pages, P, K, D), rnd(pages, P, K, D)
    elif layout == "head":
        k, v = rnd(pages, K, P, D).permute(0, 2, 1, 3), rnd(pages, K, P, D).permute(0, 2, 1, 3)
    elif layout == "pair":
        kv = rnd(pages, 2, P, K, D)
        k, v = kv[:, 0], kv[:, 1]
    else:  # padded rows
        k, v = rnd(pages, P, K, D + 8)[..., :D], rnd(pages, P, K, D + 8)[..., :D]
    return S.PagedKV(k, v)


APPEND = [
    # tokens, heads, kv heads, D, rot, axes, interleaved, page, layout, dtype, far, sections
    (1, 32, 32, 128, 128, 1, False, 16, "token", F16, 4096, None),
    (33, 8, 2, 64, 64, 3, False, 1, "head", BF16, 100000, (3, 1, 2)),
    (70, 12, 4, 80, 80, 2, True, 8, "pair", F16, 1000, (1, 1)),
    (17, 4, 4, 256, 64, 1, False, 32, "pad", BF16, 2 ** 31 - 1, None),
    (17, 4, 4, 256, 256, 4, True, 1024, "pad", F16, 2 ** 31 - 1, (1, 2, 3, 4)),
    (5, 3, 3, 8, 0, 1, False, 16, "token", F16, 10, None),
    (129, 64, 8, 128, 32, 3, True, 16, "head", BF16, 131072, (1, 1, 2)),
    (40, 0, 8, 128, 128, 1, False, 16, "token", F16, 4096, None),
    (2, 1, 1, 24, 16, 2, False, 2, "pair", BF16, 50, (1, 1)),
    (1000, 8, 1, 96, 48, 1, False, 64, "token", F16, 4096, None),
]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("in_place", [False, True])
def test_append_matches_the_formula(case, in_place):
    T, H, K, D, rot, axes, inter, P, layout, dt, far, sections = case
    say(f"case append {case} in_place={in_place}")
    g = torch.Generator().manual_seed(T + D)
    pages = -(-T // P) + 3
    cache = _cache(pages, P, K, D, dt, layout, 3)
    k0, v0 = cache.k.cpu().clone(), cache.v.cpu().clone()
    width = (H + 2 * K) * D + 16
    qkv = torch.randn(T + 4, width, generator=g).to(dt).cuda()      # columns of one product, guard columns and rows
    q, k, v = (qkv[2:2 + T, a:b] for a, b in ((0, H * D), (H * D, (H + K) * D), ((H + K) * D, (H + 2 * K) * D)))
    before = qkv.cpu().clone()
    qo_full = torch.randn(T + 4, H * D + 8, generator=g).to(dt).cuda()
    qo_before = qo_full.cpu().clone()
    q_out = q if in_place else qo_full[2:2 + T, :H * D]
    slots = torch.randperm(pages * P, generator=g)[:T].int()
    off = torch.rand(T, generator=g) < 0.15                        # rows that are no token
    slots[off] = torch.tensor([-1, pages * P, 2 ** 31 - 1, -2 ** 31])[torch.randint(0, 4, (int(off.sum()),), generator=g)].int()
    pos = torch.randint(-far if far < 2 ** 30 else 0, far, (axes, T), generator=g).int()
    inv = torch.tensor([10000.0 ** (-2.0 * i / max(rot, 1)) for i in range(rot // 2)], dtype=torch.float32)
    axis = None
    if sections:
        axis = torch.repeat_interleave(torch.arange(len(sections)), torch.tensor(sections) * (rot // 2))[::sum(sections)].int()
        axis[-1] = 7 if rot > 16 else axis[-1]                     # a frequency on no axis
    rope = S.Rope(inv.cuda(), axis=None if axis is None else axis.cuda(), axes=axes, interleaved=inter) if rot else None
    ldpos = torch.full((axes, T + 3), 5, dtype=torch.int32, device="cuda")
    ldpos[:, :T] = pos.cuda()
    S.lora_rope_append(q_out if H else None, q if H else None, k, v, cache, slots.cuda(), rope=rope, positions=ldpos[:, :T])
    torch.cuda.synchronize()
    live = (slots >= 0) & (slots < pages * P)
    kx = before[2:2 + T, H * D:(H + K) * D].reshape(T, K, D)
    wk, mk = R.rotate(kx, pos, inv, axis, axes, inter)
    want_k, want_v = k0.double().reshape(pages * P, K, D), v0.reshape(pages * P, K, D).clone()
    bound = torch.zeros_like(want_k)
    at = slots[live].long()
    want_k[at], want_v[at] = wk[live], before[2:2 + T, (H + K) * D:(H + 2 * K) * D].reshape(T, K, D)[live]
    bound[at] = (R.half_step(dt) * wk.abs() + 2.0 ** -21 * mk + R.tiny(dt))[live]
    close(cache.k.reshape(pages * P, K, D), want_k, bound, "k")
    assert torch.equal(cache.v.cpu().reshape(pages * P, K, D), want_v), "v"
    if H:
        qx = before[2:2 + T, :H * D].reshape(T, H, D)
        wq, mq = R.rotate(qx, pos, inv, axis, axes, inter)
        old = qx if in_place else qo_before[2:2 + T, :H * D].reshape(T, H, D)
        wq = torch.where(live[:, None, None], wq, old.double())
        bq = torch.where(live[:, None, None], R.half_step(dt) * wq.abs() + 2.0 ** -21 * mq + R.tiny(dt), torch.zeros(()).double())
        close(q_out.reshape(T, H, D), wq, bq, "q")
    keep = qkv.cpu().clone()
    keep[2:2 + T, :H * D] = before[2:2 + T, :H * D]
    assert torch.equal(keep, before), "inputs or guards changed"
    keep = qo_full.cpu().clone()
    keep[2:2 + T, :H * D] = qo_before[2:2 + T, :H * D]
    assert torch.equal(keep, qo_before), "guards of q_out changed"


def test_append_beyond_32_bit_offsets():
    """Cells whose byte and element offsets pass 32 bits (a cache of one wide page stride)."""
    say("case append-far-cells")
    P, K, D, pages = 16, 2, 64, 5
    stride = (1 << 31) // 4 + 8 * 131      # elements between pages: the last page starts past 2^31 elements
    flat = torch.empty(4 * stride + P * K * D, dtype=F16, device="cuda")
    cells = [flat[p * stride:p * stride + P * K * D].view(P, K, D) for p in range(pages)]
    for c in cells:
        c.zero_()
    k = flat.as_strided((pages, P, K, D), (stride, K * D, D, 1))
    vflat = torch.zeros_like(flat)
    v = vflat.as_strided((pages, P, K, D), (stride, K * D, D, 1))
    cache = S.PagedKV(k, v)
    x = torch.randn(3, K * D, device="cuda").half()
    slots = ints([4 * P + 15, 3 * P, 0])
    S.lora_rope_append(None, None, x, (-x).contiguous(), cache, slots)
    q = torch.randn(1, 4 * D, device="cuda").half()
    out = torch.empty_like(q)
    # and read back: one request whose pages are 4 and 3
    S.lora_paged_attention(out, q, cache, ints([[4, 3]]), ints([17]), S.attention_workspace(1, 4, cache))
    torch.cuda.synchronize()
    assert torch.equal(cells[4][15].reshape(-1), x[0]) and torch.equal(cells[3][0].reshape(-1), x[1])
    assert torch.equal(cells[0][0].reshape(-1), x[2])
    kk = torch.stack([cells[4].cpu(), cells[3].cpu()])
    vv = torch.stack([v[4].cpu(), v[3].cpu()])
    w = R.attention(q.cpu().view(1, 4, D), kk, vv, torch.tensor([[0, 1]], dtype=torch.int32), [17], None, 1 / math.sqrt(D), 0, 4)
    close(out.view(4, D), w[0][0], w[0][2], "out")


# ------------------------------------------------------------------ attention
class AttnCase:
    def __init__(self, lens, H, K, D, P, dt, layout="token", seed=0, req=None, garbage=True, qscale=2.0, extra_rows=0):
        g = torch.Generator().manual_seed(seed)
        n_req = len(lens) if req is None else max(r for r in req) + 1
        need = [0] * n_req
        for i, n in enumerate(lens):
            r = i if req is None else req[i]
            if 0 <= r < n_req:
                need[r] = max(need[r], n)
        blocks = [-(-max(n, 0) // P) for n in need]
        pages = sum(blocks) + 2
        self.cache = _cache(pages, P, K, D, dt, layout, seed + 1)
        ids = torch.randperm(pages, generator=g).int()
        self.table = torch.full((n_req, max(blocks + [1]) + 1), -1, dtype=torch.int32)
        used = 0
        seen = torch.zeros(pages, P, dtype=torch.bool)
        for r, b in enumerate(blocks):
            self.table[r, :b] = ids[used:used + b]
            used += b
            for t in range(need[r]):
                seen[self.table[r, t // P], t % P] = True
        if garbage:      # what lies behind the last token is stale
            bad = ~seen.cuda()
            self.cache.k[bad], self.cache.v[bad] = float("nan"), float("inf")
        self.n, self.H, self.D, self.lens, self.req = len(lens), H, D, list(lens), req
        self.q = (qscale * torch.randn(self.n, H * D, generator=g)).to(dt)
        self.dt = dt

    def run(self, window=0, scale=None, lse=True, work=None, out=None):
        n, H, D = self.n, self.H, self.D
        full = torch.full((n + 4, H * D + 8), 7.0, dtype=self.dt, device="cuda")
        self.full, self.lse_full = full, torch.full((n + 2, H), 9.0, device="cuda")
        out = full[2:2 + n, :H * D] if out is None else out
        qd = torch.zeros(n + 1, H * D + 16, dtype=self.dt, device="cuda")[:n, 8:8 + H * D]
        qd.copy_(self.q)
        work = S.attention_workspace(n, H, self.cache) if work is None else work
        S.lora_paged_attention(out, qd, self.cache, self.table.cuda(), ints(self.lens), work,
                               req=None if self.req is None else ints(self.req), scale=scale, window=window,
                               lse=self.lse_full[1:1 + n] if lse else None)
        torch.cuda.synchronize()
        return out, self.lse_full[1:1 + n]

    def want(self, window=0, scale=None):
        return R.attention(self.q.view(self.n, self.H, self.D), self.cache.k.cpu(), self.cache.v.cpu(), self.table,
                           self.lens, self.req, 1.0 / math.sqrt(self.D) if scale is None else scale, window, self.H)

    def check(self, out, lse, want, what, with_lse=True):
        for i, w in enumerate(want):
            o, l = out[i].view(self.H, self.D), lse[i]
            if w is None:
                assert (o == 7.0).all() and (l == 9.0).all(), f"{what} row {i}: an inactive row was written"
                continue
            close(o, w[0], w[2], f"{what} row {i} out")
            if with_lse:
                close(l, w[1], w[3], f"{what} row {i} lse")
        keep = self.full.clone()
        keep[2:2 + self.n, :self.H * self.D] = 7.0
        assert (keep == 7.0).all(), f"{what}: guards"
        assert (self.lse_full[0] == 9.0).all() and (self.lse_full[-1] == 9.0).all(), f"{what}: lse guards"


SHORT = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129, 255, 257, -1]
ATTN = [
    (SHORT, 4, 4, 128, 16, F16, "token"), (SHORT, 16, 2, 128, 16, BF16, "head"), (SHORT, 8, 1, 64, 1, F16, "pair"),
    (SHORT, 12, 4, 80, 8, BF16, "token"), (SHORT, 6, 2, 256, 32, F16, "pad"), (SHORT, 3, 1, 8, 64, F16, "token"),
    (SHORT, 5, 5, 96, 2, BF16, "head"), (SHORT, 40, 2, 128, 16, F16, "token"), (SHORT, 34, 1, 192, 4, BF16, "pair"),
    ([1], 32, 32, 128, 16, F16, "token"), ([17], 32, 32, 128, 16, BF16, "token"), ([4096], 8, 1, 128, 64, F16, "token"),
    ([5000, 1, 0, 777, 33], 8, 2, 128, 16, BF16, "token"), ([2049] * 3 + [3] * 40, 8, 8, 64, 32, F16, "token"),
    ([20011], 16, 1, 128, 1024, BF16, "head"), ([9001, 8], 4, 2, 24, 16, F16, "token"),
    ([300] * 130, 2, 1, 32, 16, F16, "token"),
]


@pytest.mark.parametrize("case", ATTN, ids=lambda c: f"{len(c[0])}x{max(c[0])}-" + "-".join(map(str, c[1:])))
def test_attention_matches_the_formula(case):
    lens, H, K, D, P, dt, layout = case
    say(f"case attention {case}")
    c = AttnCase(lens, H, K, D, P, dt, layout, seed=len(lens) + D)
    out, lse = c.run()
    c.check(out, lse, c.want(), "plain")
    first = (out.clone(), lse.clone())
    out, lse = c.run()                                # the same bits again, whatever the order of workgroups
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    out, lse = c.run(lse=False)
    assert torch.equal(out, first[0])


@pytest.mark.parametrize("window", [1, 5, 16, 100, 4000])
def test_attention_window(window):
    say(f"case attention-window {window}")
    c = AttnCase([0, 1, 4, 5, 6, 99, 100, 101, 700, 3000], 8, 2, 128, 16, F16, seed=window)
    out, lse = c.run(window=window)
    c.check(out, lse, c.want(window=window), f"window {window}")


def test_attention_pages_that_are_none():
    """Table entries outside the cache leave their tokens out; a row of nothing else is empty."""
    say("case attention-bad-pages")
    c = AttnCase([50, 50, 50, 3, 2000], 8, 4, 64, 16, BF16)
    c.table[0, 1], c.table[1, :] = -1, 10 ** 6
    c.table[2, 3] = c.cache.num_pages
    c.table[4, 5:90] = -7
    out, lse = c.run()
    want = c.want()
    assert want[1][1][0] == -math.inf and not want[1][0].any()
    c.check(out, lse, want, "bad pages")


def test_attention_rows_that_are_not_active():
    say("case attention-inactive")
    c = AttnCase([5, 40, 7, 9, 0], 4, 2, 128, 16, F16, req=[0, 1, 1, 0, 1])
    c.lens = [5, c.table.shape[1] * 16 + 1, -3, 9, 0]     # one token more than a table row can hold
    c.req = [0, 1, 1, -1, 2]
    out, lse = c.run()
    want = c.want()
    assert [w is None for w in want] == [False, True, True, True, True]
    c.check(out, lse, want, "inactive")


@pytest.mark.parametrize("n,every", [(64, 1), (65, 64), (300, 1), (700, 3), (5000, 1111), (5000, 5000)])
def test_attention_of_many_rows_few_of_them_active(n, every):
    """A batch padded far beyond its tokens, and rows in more chunks than one wavefront holds."""
    say(f"case attention-rows {n} every {every}")
    lens = [(1 + 37 * i % 200) if i % every == every - 1 else -1 for i in range(n)]
    c = AttnCase(lens, 2, 1, 32, 16, F16, seed=n)
    out, lse = c.run()
    for i, w in enumerate(c.want()):
        if w is not None:
            close(out[i].view(2, 32), w[0], w[2], f"row {i}")
            close(lse[i], w[1], w[3], f"row {i} lse")
    off = torch.tensor([v < 0 for v in lens], device="cuda")
    assert (out[off] == 7.0).all() and (lse[off] == 9.0).all()
    want = torch.zeros(n, dtype=torch.bool)
    want[~off.cpu()] = True
    assert want.any()


def test_attention_rows_that_share_a_request():
    say("case attention-shared")
    req = [0, 0, 0, 2, 2, 1, 0]
    c = AttnCase([100, 101, 102, 1, 33, 0, 7], 8, 2, 128, 16, F16, req=req, seed=4)
    out, lse = c.run()
    c.check(out, lse, c.want(), "shared")


def test_attention_scale_signs_and_zero():
    say("case attention-scale")
    c = AttnCase([100, 3], 8, 2, 64, 16, BF16, seed=4)
    for scale in (0.0, -0.3, 0.02, 3.0):
        out, lse = c.run(scale=scale)
        c.check(out, lse, c.want(scale=scale), f"scale {scale}")


@pytest.mark.parametrize("dt", [F16, BF16])
def test_attention_infinities_and_nan_inside_and_outside_the_mask(dt):
    say(f"case attention-special {dt}")
    D, P = 64, 16
    c = AttnCase([40, 40, 40, 40, 40], 4, 2, D, P, dt, seed=9)
    cell = lambda r, t: (int(c.table[r, t // P]), t % P)
    inf = float("inf")
    c.q = c.q.abs() + 0.5                               # positive queries: the sign of a score is its key's
    c.cache.k[cell(0, 7)] = -inf                        # one score of -inf: weight 0 ...
    c.cache.v[cell(0, 7)] = 1.0
    c.cache.v[cell(1, 3)][:, 5] = inf                   # an infinite value with a weight
    c.cache.v[cell(2, 39)][1, 6] = float("nan")
    c.cache.k[cell(3, 0)][0] = float("nan")             # a NaN score: its head's row is NaN
    for t in range(40):
        c.cache.k[cell(4, t)] = -inf                    # every score -inf: empty
    out, lse = c.run()
    want = c.want()
    assert want[4][1][0] == -inf
    w3 = want[3]
    assert w3[0][:2].isnan().all() and not w3[0][2:].isnan().any()
    c.check(out, lse, want, "special")


def test_attention_large_scores():
    """Scores of both signs up to 1e4: the running maximum carries the sums."""
    say("case attention-large-scores")
    for dt in (F16, BF16):
        c = AttnCase([700, 64, 1], 4, 1, 128, 16, dt, seed=2, qscale=100.0)
        out, lse = c.run()
        c.check(out, lse, c.want(), str(dt))


def test_attention_small_weights_add_up():
    """A long tail of weights near 2^-20 of the largest one still counts."""
    say("case attention-tail")
    n, D = 8192, 64
    for dt in (F16, BF16):
        c = AttnCase([n], 2, 1, D, 64, dt, seed=3)
        c.q = torch.ones_like(c.q)
        c.cache.k.zero_()
        page = c.table[0].long()
        c.cache.k[int(page[0]), 0] = 14.0 / 8.0         # one score of 14, the rest 0
        c.cache.v.copy_(torch.randn(c.cache.v.shape).to(dt).abs())
        out, lse = c.run()
        c.check(out, lse, c.want(), str(dt))


def test_attention_subnormal_keys_and_values():
    """fp16 keys and values below 2^-14 (its subnormals) count like any others."""
    say("case attention-subnormal")
    c = AttnCase([300, 5], 4, 2, 64, 16, F16, seed=12)
    c.cache.v.mul_(2.0 ** -16)
    c.cache.k.mul_(2.0 ** -17)
    c.q = (c.q.float() * 2000).to(F16)          # scores of a few units from subnormal keys
    c.cache.k[c.cache.k.isnan()] = 0.0
    c.cache.v[c.cache.v.isnan()] = 0.0
    out, lse = c.run(scale=2.0)
    want = c.want(scale=2.0)
    assert float(want[0][0].abs().max()) < 2.0 ** -14 and float(want[0][1].abs().max()) > 0.5
    c.check(out, lse, want, "subnormal")


def test_attention_reads_a_table_of_wider_rows():
    say("case attention-wide-table")
    c = AttnCase([100, 37, 64], 4, 2, 64, 16, F16, seed=13)
    n, wide = 3, torch.full((3, c.table.shape[1] + 9), 10 ** 9, dtype=torch.int32, device="cuda")
    wide[:, 4:4 + c.table.shape[1]] = c.table.cuda()
    view = wide[:, 4:4 + c.table.shape[1]]
    out, lse = torch.empty(n, 4 * 64, dtype=F16, device="cuda"), torch.empty(n, 4, device="cuda")
    S.lora_paged_attention(out, c.q.cuda(), c.cache, view, ints(c.lens), S.attention_workspace(n, 4, c.cache), lse=lse)
    torch.cuda.synchronize()
    for i, w in enumerate(c.want()):
        close(out[i].view(4, 64), w[0], w[2], f"row {i}")


def test_two_streams_with_workspaces_of_their_own():
    """Calls that run at the same time, each split over many workgroups."""
    say("case attention-two-streams")
    cases = [AttnCase([20000, 3, 900], 8, 1, 128, 16, F16, seed=20 + i) for i in range(2)]
    alone = [tuple(t.clone() for t in c.run()) for c in cases]
    streams, args, outs = [torch.cuda.Stream() for _ in cases], [], []
    for c in cases:
        outs.append((torch.zeros(3, 8 * 128, dtype=F16, device="cuda"), torch.zeros(3, 8, device="cuda")))
        args.append((c.q.cuda(), c.cache, c.table.cuda(), ints(c.lens), S.attention_workspace(3, 8, c.cache)))
    torch.cuda.synchronize()
    for _ in range(20):
        for st, (o, l), a in zip(streams, outs, args):
            with torch.cuda.stream(st):
                S.lora_paged_attention(o, *a, lse=l)
    torch.cuda.synchronize()
    for (o, l), (wo, wl), a in zip(outs, alone, args):
        assert torch.equal(o, wo) and torch.equal(l, wl)
        assert not a[4][:2 * (4 * 256 + 4096)].any(), "counters are zero again"


def test_calls_on_no_rows():
    say("case no-rows")
    cache = _cache(2, 16, 2, 64, F16, "token", 1)
    k0, v0 = cache.k.clone(), cache.v.clone()
    e = lambda c: torch.empty(0, c, dtype=F16, device="cuda")
    S.lora_paged_attention(e(256), e(256), cache, ints([[0]]), ints([]), S.attention_workspace(0, 4, cache))
    S.lora_rope_append(e(256), e(256), e(128), e(128), cache, ints([]), rope=S.Rope.base(64),
                       positions=torch.empty(1, 0, dtype=torch.int32, device="cuda"))
    S.lora_residual_norm(e(64), e(64), torch.ones(64, dtype=F16, device="cuda"), x=e(64), res_out=e(64))
    torch.cuda.synchronize()
    assert torch.equal(cache.k, k0) and torch.equal(cache.v, v0)


def test_attention_workspace_is_left_clean_and_may_be_shared():
    say("case attention-workspace")
    big = AttnCase([9000, 3, 0, 512], 8, 1, 128, 16, F16, seed=1)
    small = AttnCase([700, 70], 8, 1, 128, 16, F16, seed=2)
    work = S.attention_workspace(4, 8, big.cache)
    wb, ws = big.want(), small.want()
    for _ in range(3):
        out, lse = big.run(work=work)
        big.check(out, lse, wb, "big")
        out, lse = small.run(work=work)
        small.check(out, lse, ws, "small")


@pytest.mark.parametrize("n", [2047, 2048, 2049, 4096, 4097, 8193])
def test_attention_joins_of_every_depth(n):
    """One row cut into 16, 17, 32 and more parts: one join or two, whole and broken groups."""
    say(f"case attention-parts n={n}")
    for H, D, dt in ((8, 128, F16), (3, 24, BF16), (20, 80, F16)):
        c = AttnCase([n], H, 1, D, 64, dt, seed=n % 97)
        out, lse = c.run()
        c.check(out, lse, c.want(), f"{H} heads of {D}")


def test_calls_of_different_shapes_share_a_workspace():
    """The counters lie where every shape looks for them: sums of one call never become another's."""
    say("case attention-shapes-share")
    cases = [AttnCase([9000, 40], 8, 1, 128, 16, F16, seed=1), AttnCase([700, 3, 2500], 32, 32, 64, 16, BF16, seed=2),
             AttnCase([5000], 40, 2, 128, 16, F16, seed=3), AttnCase([3000, 1, 0], 6, 3, 256, 16, BF16, seed=4)]
    work = torch.zeros(max(S.attention_workspace(c.n, c.H, c.cache).numel() for c in cases), dtype=torch.int32, device="cuda")
    wants = [c.want() for c in cases]
    for _ in range(3):
        for c, w in zip(cases, wants):
            out, lse = c.run(work=work)
            c.check(out, lse, w, f"{c.H} heads of {c.D}")


def test_attention_captured_with_lengths_that_change():
    say("case attention-graph")
    lens = [600, 0, 33, 2500, 1, 17]
    c = AttnCase(lens, 8, 2, 128, 16, F16, seed=8)
    n, H, D = c.n, c.H, c.D
    q, table, ln = c.q.cuda(), c.table.cuda(), ints(lens)
    work = S.attention_workspace(n, H, c.cache)
    out, lse = torch.zeros(n, H * D, dtype=F16, device="cuda"), torch.zeros(n, H, device="cuda")
    call = lambda: S.lora_paged_attention(out, q, c.cache, table, ln, work, lse=lse)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    g2 = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g2):      # a second graph over the same workspace
        call()
    for it, new in enumerate(([600, 0, 33, 2500, 1, 17], [1, 0, 0, 2499, 0, -1], [599, 0, 2, 64, 1, 16], [0] * 6, lens)):
        ln.copy_(ints(new))
        out.zero_()
        lse.zero_()
        (g if it % 2 == 0 else g2).replay()
        torch.cuda.synchronize()
        got = (out.clone(), lse.clone())
        out.zero_()
        lse.zero_()
        call()
        torch.cuda.synchronize()
        assert torch.equal(got[0], out) and torch.equal(got[1], lse), f"replay {it}"
        c.lens = new
        for i, w in enumerate(c.want()):
            if w is not None:
                close(got[0][i].view(H, D), w[0], w[2], f"replay {it} row {i}")
    del g, g2


# ------------------------------------------------------------------ residual add and norms
NORM = [
    # rows, hidden, dtype, post, gates (0 none, 1 broadcast, n indexed), alpha, w_offset
    (1, 8, F16, False, 0, 1.0, 0.0), (32, 4096, F16, False, 0, 1.0, 0.0), (7, 5120, BF16, True, 0, 1.0, 1.0),
    (3, 8192, BF16, True, 5, 0.75, 0.0), (130, 1000, F16, True, 1, -0.5, 1.0), (2, 65536, F16, True, 2, 1.0, 0.0),
    (5, 16392, BF16, False, 3, 0.22, 0.0), (4, 504, F16, False, 1, 0.0, 0.0), (513, 64, BF16, True, 40, 2.0, 1.0),
    (3, 28672, F16, False, 0, 1.0, 0.0),
]


@pytest.mark.parametrize("case", NORM, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("form", ["apart", "in_place", "no_y", "no_res_out", "no_x"])
def test_norm_matches_the_formula(case, form):
    n, h, dt, post, gates, alpha, off = case
    say(f"case norm {case} {form}")
    g = torch.Generator().manual_seed(n + h)
    rnd = lambda *s: torch.randn(s, generator=g).to(dt)

    def dev(t, guard):
        full = torch.full((t.shape[0] + 2, t.shape[1] + 8), guard, dtype=dt, device="cuda")
        full[1:1 + t.shape[0], :t.shape[1]] = t.cuda()
        return full, full[1:1 + t.shape[0], :t.shape[1]]

    x, res = rnd(n, h), (3 * rnd(n, h)).to(dt)
    w, pw = (1 + rnd(h) / 8).to(dt), (1 + rnd(h) / 8).to(dt) if post else None
    gate = rnd(gates, h) if gates else None
    gi = torch.randint(-1, gates, (n,), generator=g).int() if gates > 1 else None
    dead = torch.zeros(n, dtype=torch.bool)
    if gi is not None:
        gi[n // 2] = gates          # outside: the row is left as it was
        dead[n // 2] = True
    if form == "no_x":
        x = pw = gate = gi = None
        dead[:] = False
    xf, xd = dev(x, 5.0) if x is not None else (None, None)
    rf, rd = dev(res, 5.0)
    yf, yd = dev(torch.full((n, h), 7.0, dtype=dt), 5.0)
    of, od = dev(torch.full((n, h), 7.0, dtype=dt), 5.0)
    y, ro = yd, od
    if form == "in_place":
        y, ro = xd, rd
    y = None if form == "no_y" else y
    ro = None if form == "no_res_out" else ro
    S.lora_residual_norm(y, rd, None if form == "no_y" else w.cuda(), x=xd, res_out=ro,
                         post_w=None if pw is None else pw.cuda(), gate=None if gate is None else gate.cuda(),
                         gate_idx=None if gi is None else gi.cuda(), alpha=alpha, eps=1e-5, w_offset=off)
    torch.cuda.synchronize()
    wh, wy, bh, by = R.residual_norm(res, x, w, pw, gate, gi, alpha, 1e-5, off)
    for got, want, bound, old, what in ((y, wy, by, x if form == "in_place" else None, "y"),
                                        (ro, wh, bh, res if form == "in_place" else None, "res_out")):
        if got is None:
            continue
        bound = bound + R.half_step(dt) * want.abs() + R.tiny(dt)
        o = torch.full((n, h), 7.0, dtype=torch.float64) if old is None else old.double()
        want, bound = torch.where(dead[:, None], o, want), torch.where(dead[:, None], torch.zeros((), dtype=torch.float64), bound)
        close(got, want, bound, what)
    for full in (xf, rf, yf, of):
        if full is not None:
            assert (full[0] == 5.0).all() and (full[-1] == 5.0).all() and (full[:, h:] == 5.0).all(), "guards"
    if form != "in_place":
        assert torch.equal(rd.cpu(), res) and (x is None or torch.equal(xd.cpu(), x)), "inputs changed"


def test_norm_of_zeros_and_large_rows():
    say("case norm-zeros")
    for dt in (F16, BF16):
        h = 4096
        res = torch.zeros(3, h, dtype=dt)
        res[1] = 60000.0                # squares far beyond fp16
        res[2, 5] = 2.0 ** -14
        y = torch.empty(3, h, dtype=dt, device="cuda")
        w = torch.ones(h, dtype=dt)
        S.lora_residual_norm(y, res.cuda(), w.cuda())
        _, wy, _, by = R.residual_norm(res, None, w, None, None, None, 1.0, 1e-5, 0.0)
        close(y, wy, by + R.half_step(dt) * wy.abs() + R.tiny(dt), str(dt))


def test_norm_beyond_32_bit_offsets():
    say("case norm-far-rows")
    h, ld = 64, (1 << 30) + 72
    flat = [torch.empty(2 * ld + h, dtype=F16, device="cuda") for _ in range(2)]
    res, y = (f.as_strided((3, h), (ld, 1)) for f in flat)
    vals = torch.randn(3, h).half()
    res.copy_(vals)
    y.zero_()
    w = torch.ones(h, dtype=F16)
    S.lora_residual_norm(y, res, w.cuda())
    torch.cuda.synchronize()
    _, wy, _, by = R.residual_norm(vals, None, w, None, None, None, 1.0, 1e-5, 0.0)
    close(y, wy, by + R.half_step(F16) * wy.abs() + R.tiny(F16), "y")


@pytest.mark.parametrize("lens", [[40, 3, 0, 1000], [17]])
def test_the_python_and_the_compiled_calls_are_the_same(lens, monkeypatch):
    say(f"case both-bindings {lens}")
    assert S._fast is not None
    n, H, K, D, P = len(lens), 8, 2, 64, 16
    c = AttnCase(lens, H, K, D, P, F16, seed=31, garbage=False)
    qkv = torch.randn(n, (H + 2 * K) * D, device="cuda").half()
    res, w = torch.randn(n, 512, device="cuda").half(), torch.randn(512, device="cuda").half()
    gate, gi = torch.randn(3, 512, device="cuda").half(), ints([i % 4 - 1 for i in range(n)])
    rope, pos, slots = S.Rope.base(D), ints([[5 * i for i in range(n)]]), ints([P * i for i in range(n)])
    table, ln, work = c.table.cuda(), ints(lens), S.attention_workspace(n, H, c.cache)

    def all_calls():
        kc, vc = c.cache.k.clone(), c.cache.v.clone()
        cache = S.PagedKV(kc, vc)
        q_out, out, lse = torch.empty(n, H * D, dtype=F16, device="cuda"), torch.empty(n, H * D, dtype=F16, device="cuda"), torch.empty(n, H, device="cuda")
        S.lora_rope_append(q_out, qkv[:, :H * D], qkv[:, H * D:(H + K) * D], qkv[:, (H + K) * D:], cache, slots, rope=rope, positions=pos)
        S.lora_rope_append(None, None, qkv[:, H * D:(H + K) * D], qkv[:, (H + K) * D:], cache, ints([P * i + 1 for i in range(n)]))
        S.lora_paged_attention(out, q_out, cache, table, ln, work, window=100, lse=lse, req=ints(list(range(n))))
        y, ro, y2 = torch.empty_like(res), torch.empty_like(res), torch.empty_like(res)
        S.lora_residual_norm(y, res, w, x=y2.copy_(res).mul_(2), res_out=ro, post_w=w, gate=gate, gate_idx=gi, alpha=0.5, w_offset=1.0)
        S.lora_residual_norm(y2, res, w)
        pages = S.KVPages.fresh(n, 70, 80 * n, P)
        plan = S.KVPlan(n, 64 * n)
        S.lora_kv_plan(plan, pages, ints([0] * n), ints([3 + i for i in range(n)]), req_slot=gi)
        torch.cuda.synchronize()
        return [kc, vc, q_out, out, lse, y, ro, y2, plan.status, plan.slots, plan.idx, pages.block_table]

    fast = all_calls()
    monkeypatch.setattr(S, "_fast", None)
    slow = all_calls()
    for i, (a, b) in enumerate(zip(fast, slow)):
        assert torch.equal(a, b), i


def test_a_refused_call_says_why_either_way(monkeypatch):
    say("case refusals-on-the-gpu")
    c = AttnCase([5, 6], 4, 2, 64, 16, F16, seed=1)
    q, tab, ln, work = c.q.cuda(), c.table.cuda(), ints([5, 6]), S.attention_workspace(2, 4, c.cache)
    out = torch.zeros_like(q)
    for again in range(2):
        for kw, msg in ((dict(kv_len=ln.long()), "dtype"), (dict(out=out[:1]), "at least"), (dict(out=out.cpu()), "GPU tensor"),
                        (dict(lse=torch.zeros(3, device="cuda")), "elements"), (dict(block_table=tab.cpu()), "GPU tensor")):
            with pytest.raises(ValueError, match=msg):
                S.lora_paged_attention(**{**dict(out=out, q=q, cache=c.cache, block_table=tab, kv_len=ln, work=work), **kw})
        for kw, code in ((dict(out=q), B.LORA_E_SHAPE), (dict(window=-1), B.LORA_E_SHAPE), (dict(work=work[:64]), B.LORA_E_SHAPE),
                         (dict(scale=float("nan")), B.LORA_E_SHAPE)):
            with pytest.raises(B.LoraError) as e:
                S.lora_paged_attention(**{**dict(out=out, q=q, cache=c.cache, block_table=tab, kv_len=ln, work=work), **kw})
            assert e.value.code == code
        monkeypatch.setattr(S, "_fast", None)
    torch.cuda.synchronize()
    assert not out.any()


# ------------------------------------------------------------------ streams
def test_calls_on_a_side_stream():
    say("case side-stream")
    c = AttnCase([300, 5, 1200], 8, 2, 128, 16, F16, seed=6)
    want = c.want()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out, lse = c.run()
    c.check(out, lse, want, "torch's current stream")
    out2 = torch.zeros_like(out)
    work = S.attention_workspace(3, 8, c.cache)
    args = (c.q.cuda(), c.cache, c.table.cuda(), ints(c.lens), work)
    torch.cuda.synchronize()
    S.lora_paged_attention(out2, *args, stream=side)
    side.synchronize()
    assert torch.equal(out2, out)


class Compiled:
    """The compiled module, keeping what each of its calls answered."""

    def __init__(self):
        self.answers, self.module = [], S._fast

    def __getattr__(self, name):
        fn = getattr(self.module, name)
        if name not in ("append", "attention", "norm", "plan"):
            return fn

        def call(*args):
            self.answers.append((name, fn(*args)))
            return self.answers[-1][1]

        return call


@pytest.mark.parametrize("n", [1, 5, 64])
def test_one_axis_positions_take_the_compiled_call(n, monkeypatch):
    """Positions [n_rows] and [1, n_rows] of one axis are one call, made by the compiled module, also
    for a longer array and a view of one; what it leaves to Python is refused there."""
    say(f"case compiled-append n={n}")
    H, K, D, P = 4, 2, 64, 16
    rope, slots = S.Rope.base(D), ints([3 * i for i in range(n)])
    qkv = torch.randn(n, (H + 2 * K) * D, device="cuda").half()
    q, k, v = qkv[:, :H * D], qkv[:, H * D:(H + K) * D], qkv[:, (H + K) * D:]
    pos = ints([7 * i + 1 for i in range(n + 3)])
    seen = Compiled()
    monkeypatch.setattr(S, "_fast", seen)

    def call(positions, axes=rope):
        cache = S.PagedKV(torch.zeros(3 * n // P + 1, P, K, D, dtype=F16, device="cuda"),
                          torch.zeros(3 * n // P + 1, P, K, D, dtype=F16, device="cuda"))
        q_out = torch.zeros(n, H * D, dtype=F16, device="cuda")
        S.lora_rope_append(q_out, q, k, v, cache, slots, rope=axes, positions=positions)
        torch.cuda.synchronize()
        return q_out, cache.k, cache.v

    want = call(pos[None, :n])
    assert want[0].any() and want[1].any()
    later = torch.cat([pos.new_full((2,), 99), pos])
    for p in (pos[:n], pos, later[2:], later[2:2 + n]):
        for a, b in zip(call(p), want):
            assert torch.equal(a, b)
    assert seen.answers == [("append", 0)] * 5, seen.answers
    if n > 1:
        for bad, msg in ((pos[:n - 1], "at least"), (later.repeat(2)[::2], "stride"), (pos[:n].long(), "dtype"),
                         (pos.cpu(), "GPU tensor")):
            with pytest.raises(ValueError, match=msg):
                call(bad)
    with pytest.raises(ValueError, match="at least"):
        call(pos, S.Rope(rope.inv_freq, axes=2))


def test_the_layers_append_takes_the_compiled_call(monkeypatch):
    """Every call of the decoder layer's paged step is made by the compiled module."""
    from segmented_gather_matmul_amd import layer as LY
    say("case compiled-layer")
    shape = LY.LlamaShape("case", 256, 512, 4, 64, kv_heads=2)
    layer = LY.random_layer(shape, 2, 8, 8, torch.Generator(device="cuda").manual_seed(0))
    step = LY.PagedStep(shape, 2, 8, 3, 6, 8, rope=S.Rope.base(64))
    cache, meta = step.new_cache(), LY.BatchMeta.of_step(step, 2)
    seen = Compiled()
    monkeypatch.setattr(S, "_fast", seen)
    step.begin(ints([5, 2]))
    layer.forward_paged(torch.randn(8, 256, device="cuda").half(), cache, step, meta)
    torch.cuda.synchronize()
    assert seen.answers == [(c, 0) for c in ("plan", "norm", "append", "attention", "norm", "norm")], seen.answers


def test_other_threads_run_while_a_compiled_call_waits():
    """The library's call may wait for room in the launch queue: it is made without the
    interpreter's lock.  In its place here the C library's sleep, whose argument takes the
    stream's and which answers 0, from each compiled call."""
    import ctypes
    import threading
    import time
    say("case compiled-lock")
    sleep = ctypes.cast(ctypes.CDLL(None).usleep, ctypes.c_void_p).value
    c = AttnCase([5, 6], 4, 2, 64, 16, F16, seed=1)
    q, tab, ln, work = c.q.cuda(), c.table.cuda(), ints([5, 6]), S.attention_workspace(2, 4, c.cache)
    kv, none = torch.zeros(2, 128, dtype=F16, device="cuda"), S._NoRope
    pages, plan = S.KVPages.fresh(2, 3, 6, 16), S.KVPlan(2, 8)
    us, dev = 200000, torch.cuda.current_device()
    calls = dict(norm=lambda: S._fast.norm(sleep, us, dev, None, q, None, None, torch.empty_like(q), None, None, None, 1.0, 1e-5, 0.0),
                 attention=lambda: S._fast.attention(sleep, us, dev, torch.empty_like(q), q, c.cache.address, c.cache.k, tab, ln, work,
                                                     None, 1.0, 0, None),
                 append=lambda: S._fast.append(sleep, us, dev, None, None, kv, kv, c.cache.address, c.cache.k, ln, none.address,
                                               None, None, None),
                 plan=lambda: S._fast.plan(sleep, us, dev, plan.address, pages.address, ln, ln, None))
    torch.cuda.synchronize()
    for name, call in calls.items():
        ticks, stop = [], threading.Event()

        def count():
            while not stop.is_set():
                ticks.append(time.perf_counter())
                time.sleep(0.002)

        other = threading.Thread(target=count)
        other.start()
        while not ticks:
            time.sleep(0.001)
        begin = time.perf_counter()
        assert call() == 0, name
        end = time.perf_counter()
        stop.set()
        other.join()
        assert end - begin > us * 0.9e-6, name
        inside = [t for t in ticks if begin + 0.02 < t < end - 0.02]
        assert len(inside) >= 5, (name, len(inside))


def test_an_lse_of_other_columns_is_refused_either_way(monkeypatch):
    say("case lse-columns")
    c = AttnCase([5, 6], 4, 2, 64, 16, F16, seed=1, garbage=False)
    q, tab, ln, work = c.q.cuda(), c.table.cuda(), ints([5, 6]), S.attention_workspace(2, 4, c.cache)
    out, lse = torch.zeros_like(q), torch.zeros(2, 4, device="cuda")
    S.lora_paged_attention(out, q, c.cache, tab, ln, work, lse=lse)
    for again in range(2):
        for shape in ((3, 4), (8,), (2, 2, 2)):
            got = torch.zeros(shape, device="cuda")
            S.lora_paged_attention(out, q, c.cache, tab, ln, work, lse=got)
            assert torch.equal(got.flatten()[:8], lse.flatten())
        for shape in ((2, 8), (4, 2), (1, 8)):
            with pytest.raises(ValueError, match="lse is"):
                S.lora_paged_attention(out, q, c.cache, tab, ln, work, lse=torch.zeros(shape, device="cuda"))
        monkeypatch.setattr(S, "_fast", None)
