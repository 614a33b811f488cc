"""GPU: the decode-step operators run together as a server uses them -- the decoder layer's
paged step over several steps of one batch (prompts admitted beside decoding requests,
requests that end, rows that pad the batch, rows without an adapter), against a CPU
reference of the same steps; captured in a graph and replayed; and refused steps."""
import math

import numpy as np
import pytest
import torch

from tests import layer_ref as R
from tests import step_ref as SR
from tests.gpu_cases import say

pytestmark = pytest.mark.gpu
TOL = 5e-3   # relative Frobenius per tensor, as for the dense step: fp16 storage roundings
F64 = np.float64

H, KV, DH, HID, FFN, EPS = 4, 2, 128, 512, 1376, 1e-5
RANKS = (16, 0, 8, 64, 3)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from segmented_gather_matmul_amd import binding as B
    B.lib()
    yield


@pytest.fixture(scope="module")
def case():
    from segmented_gather_matmul_amd import workloads as wl
    rank = np.asarray(RANKS, np.int32)
    scale = wl.scale_for_rank(rank)
    kvw = KV * DH
    dims = {"q": (HID, HID), "k": (HID, kvw), "v": (HID, kvw), "o": (HID, HID), "gate": (HID, FFN), "up": (HID, FFN),
            "down": (FFN, HID)}
    stores = {p: wl.dense_store(77, wl.PROJ_IDS[p], len(rank), di, do, rank, scale, r_max=64) for p, (di, do) in dims.items()}
    w = lambda k, sh: wl.normal16(wl.rng_for(77, 7, k), sh)
    bb = dict(w_qkv=w(0, (HID, HID + 2 * kvw)), w_o=w(1, (HID, HID)), w_gu=w(2, (HID, 2 * FFN)), w_d=w(3, (FFN, HID)),
              norm1=(1.0 + 5.0 * w(4, (HID,)).astype(F64)).astype(np.float16),
              norm2=(1.0 + 5.0 * w(5, (HID,)).astype(F64)).astype(np.float16))
    return dict(rank=rank, scale=scale, stores=stores, bb=bb)


def _layer(case, max_rows, **kw):
    from segmented_gather_matmul_amd import layer as LY
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    shape = LY.LlamaShape("case", HID, FFN, H, DH, EPS, kv_heads=KV)
    return LY.LoraDecoderLayer(shape, {k: dev(v) for k, v in case["bb"].items()},
                               {p: (dev(s.a_t), dev(s.b)) for p, s in case["stores"].items()}, dev(case["rank"]),
                               dev(case["scale"]), max_rows, **kw)


class Reference:
    """The same steps on the CPU: one list of cached k and v per request."""

    def __init__(self, case, n_req):
        self.case, self.kv = case, [([], []) for _ in range(n_req)]
        self.inv = np.array([10000.0 ** (-2.0 * i / DH) for i in range(DH // 2)], np.float32)

    def step(self, hidden, new, slot):
        c, bb = self.case, self.case["bb"]
        req = [r for r, m in enumerate(new) for _ in range(max(m, 0))]
        for r, m in enumerate(new):
            if m < 0:
                self.kv[r] = ([], [])
        idx = np.asarray([slot[r] for r in req], np.int32)
        x = hidden[:len(req)]
        outs = {}
        kvw = KV * DH

        def add(p, a, y):
            outs[p] = R.lora16(c["stores"][p], a, np.ascontiguousarray(y), idx)
            return outs[p]

        a = R.rms_norm(x, bb["norm1"], EPS)
        qkv = R.mm16(a, bb["w_qkv"])
        q, k, v = add("q", a, qkv[:, :HID]), add("k", a, qkv[:, HID:HID + kvw]), add("v", a, qkv[:, HID + kvw:])
        attn = np.zeros_like(x)
        for i, r in enumerate(req):
            pos = torch.tensor([[len(self.kv[r][0])]])
            turn = lambda t, n: SR.rotate(torch.from_numpy(t.reshape(1, n, DH).copy()), pos, self.inv, None, 1, False)[0][0]
            qr = turn(q[i], H).half().numpy()
            self.kv[r][0].append(turn(k[i], KV).half().numpy())
            self.kv[r][1].append(v[i].reshape(KV, DH).copy())
            kk, vv = (np.stack(t).astype(F64) for t in self.kv[r])
            for h in range(H):
                s = kk[:, h // (H // KV)] @ qr[h].astype(F64) / math.sqrt(DH)
                p = np.exp(s - s.max())
                attn[i, h * DH:(h + 1) * DH] = (p / p.sum()) @ vv[:, h // (H // KV)]
        o = add("o", attn, R.mm16(attn, bb["w_o"]))
        full = x.astype(F64) + o.astype(F64)
        a2 = (full / np.sqrt((full * full).mean(-1, keepdims=True) + EPS) * bb["norm2"].astype(F64)).astype(np.float16)
        gu = R.mm16(a2, bb["w_gu"])
        g, u = add("gate", a2, gu[:, :FFN]), add("up", a2, gu[:, FFN:])
        act = (R.silu16(g).astype(F64) * u.astype(F64)).astype(np.float16)
        d = add("down", act, R.mm16(act, bb["w_d"]))
        outs["out"] = (full.astype(np.float16).astype(F64) + d.astype(F64)).astype(np.float16)
        return outs


# new tokens of each request, step by step: prompts beside decoding rows, an idle request,
# requests that end and whose pages and table rows are used again
STEPS = [[5, 17, 0, 1], [1, 1, 20, 0], [1, -1, 1, 1], [1, 9, 1, 1], [-1, 1, 1, 1], [3, 1, -1, 0], [1, 1, 16, 1]]
SLOT = [0, 3, -1, 4]


def _steps(n, seed):
    g = np.random.default_rng(seed)
    return [g.standard_normal((n, HID)).astype(np.float16) for _ in STEPS]


@pytest.mark.parametrize("form", ["bgmv", "sgmv"])
@pytest.mark.parametrize("page", [1, 8, 16])
def test_steps_match_the_reference(case, form, page):
    from segmented_gather_matmul_amd import layer as LY
    from segmented_gather_matmul_amd import step as S
    say(f"case step-layer form={form} page={page}")
    T = 24
    layer = _layer(case, T)
    step = LY.PagedStep(layer.shape, 4, T, -(-40 // page), 4 * -(-40 // page), page, rope=S.Rope.base(DH))
    step.req_slot.copy_(torch.tensor(SLOT, dtype=torch.int32))
    cache = step.new_cache()
    for t in (cache.k, cache.v):
        t.fill_(float("nan"))               # pages hold whatever was there
    meta = LY.BatchMeta.of_step(step, len(RANKS), form)
    ref = Reference(case, 4)
    for i, (new, hidden) in enumerate(zip(STEPS, _steps(T, 3))):
        want = ref.step(hidden, new, SLOT)
        step.begin(torch.tensor(new, dtype=torch.int32, device="cuda"))
        trace = {}
        out = layer.forward_paged(torch.from_numpy(hidden).cuda(), cache, step, meta, trace=trace)
        torch.cuda.synchronize()
        assert step.plan.status.tolist()[0] == 0
        n = sum(max(m, 0) for m in new)
        for p in R.PROJS + ("out",):
            got = (out if p == "out" else trace[p]).cpu().numpy()[:n]
            assert np.isfinite(got).all(), f"step {i} {p}: not finite"
            rel = R.rel_fro(got, want[p])
            assert rel <= TOL, f"step {i} {p}: relative Frobenius {rel}"
        assert step.kv_len.tolist() == [len(k) for k, _ in ref.kv]


def test_reference_detects_a_missing_rotation_and_a_wrong_page(case):
    """What the comparison above can see: positions off by one, or one token's cell lost, moves
    the output of the attention projection far outside its tolerance."""
    new, hidden = [7, 9, 1, 3], _steps(24, 9)[0]
    base = Reference(case, 4).step(hidden, new, SLOT)
    ref = Reference(case, 4)
    ref.inv = ref.inv * 0
    assert R.rel_fro(ref.step(hidden, new, SLOT)["o"], base["o"]) > 4 * TOL
    ref = Reference(case, 4)
    ref.kv[1] = ([np.zeros((KV, DH), np.float16)], [np.zeros((KV, DH), np.float16)])
    assert R.rel_fro(ref.step(hidden, new, SLOT)["o"], base["o"]) > 4 * TOL


def test_captured_step_replays_on_new_lengths(case):
    """Plan and layer captured once; each replay gets its own lengths, adapters and hidden state
    and equals an eager run of the same steps bit for bit."""
    from segmented_gather_matmul_amd import layer as LY
    from segmented_gather_matmul_amd import step as S
    say("case step-layer-graph")
    T = 24
    layer = _layer(case, T)

    def fresh():
        st = LY.PagedStep(layer.shape, 4, T, 5, 20, 8, rope=S.Rope.base(DH))
        st.req_slot.copy_(torch.tensor(SLOT, dtype=torch.int32))
        return st, st.new_cache(), LY.BatchMeta.of_step(st, len(RANKS))

    eager_step, eager_cache, eager_meta = fresh()
    step, cache, meta = fresh()
    new = torch.zeros(4, dtype=torch.int32, device="cuda")
    hid = torch.zeros(T, HID, dtype=torch.float16, device="cuda")

    def one():
        step.begin(new)
        return layer.forward_paged(hid, cache, step, meta)

    one()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = one()
    for i, (m, hidden) in enumerate(zip(STEPS, _steps(T, 5))):
        new.copy_(torch.tensor(m, dtype=torch.int32))
        hid.copy_(torch.from_numpy(hidden))
        g.replay()
        torch.cuda.synchronize()
        eager_step.begin(new)
        want = layer.forward_paged(hid, eager_cache, eager_step, eager_meta)
        torch.cuda.synchronize()
        n = sum(max(v, 0) for v in m)
        assert torch.equal(out[:n], want[:n]), f"replay {i}"
        assert torch.equal(step.kv_len, eager_step.kv_len)
        assert torch.equal(cache.k, eager_cache.k) and torch.equal(cache.v, eager_cache.v), f"replay {i}: cache"
    del g


@pytest.mark.parametrize("kw", [dict(overlap=True), dict(handoff=False)])
def test_the_layers_other_forms_give_the_same_bits(case, kw):
    """The add-ons' shrinks on a second stream, or in launches of their own."""
    from segmented_gather_matmul_amd import layer as LY
    from segmented_gather_matmul_amd import step as S
    say(f"case step-layer-forms {kw}")
    T, outs = 24, []
    for layer in (_layer(case, T), _layer(case, T, **kw)):
        step = LY.PagedStep(layer.shape, 4, T, 5, 20, 8, rope=S.Rope.base(DH))
        step.req_slot.copy_(torch.tensor(SLOT, dtype=torch.int32))
        cache, meta = step.new_cache(), LY.BatchMeta.of_step(step, len(RANKS))
        for new, hidden in zip(STEPS[:3], _steps(T, 11)):
            step.begin(torch.tensor(new, dtype=torch.int32, device="cuda"))
            out = layer.forward_paged(torch.from_numpy(hidden).cuda(), cache, step, meta)
            outs.append(out[:sum(max(v, 0) for v in new)].clone())
        torch.cuda.synchronize()
    for a, b in zip(outs[:3], outs[3:]):
        assert torch.equal(a, b)


def test_a_step_that_does_not_fit_leaves_the_caches(case):
    from segmented_gather_matmul_amd import layer as LY
    from segmented_gather_matmul_amd import step as S
    T = 24
    layer = _layer(case, T)
    step = LY.PagedStep(layer.shape, 4, T, 5, 4, 8, rope=S.Rope.base(DH))
    cache = step.new_cache()
    new = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    hidden = torch.randn(T, HID, device="cuda").half()
    step.begin(new([8, 8, 0, 1]))
    layer.forward_paged(hidden, cache, step, None)
    k, v, ln = cache.k.clone(), cache.v.clone(), step.kv_len.clone()
    step.begin(new([9, 9, 0, 0]))          # needs four pages, one is free
    layer.forward_paged(hidden, cache, step, None)
    torch.cuda.synchronize()
    assert step.plan.status.tolist() == [S.KV_NO_PAGES, 18, 4, 0]
    assert torch.equal(cache.k, k) and torch.equal(cache.v, v) and torch.equal(step.kv_len, ln)
    step.begin(new([1, 0, 0, 1]))          # fits again
    layer.forward_paged(hidden, cache, step, None)
    torch.cuda.synchronize()
    assert step.plan.status.tolist()[0] == 0 and step.kv_len.tolist() == [9, 8, 0, 2]


def test_dense_step_refuses_grouped_heads(case):
    from segmented_gather_matmul_amd import layer as LY
    layer = _layer(case, 4)
    cache = LY.KVCache(torch.zeros(4, H, DH, 8, device="cuda").half(), torch.zeros(4, H, 8, DH, device="cuda").half())
    with pytest.raises(ValueError, match="forward_paged"):
        layer.forward(torch.zeros(4, HID, device="cuda").half(), cache, None)
    step = LY.PagedStep(layer.shape, 2, 3, 4, 8, 8)
    with pytest.raises(ValueError, match="does not fit"):
        layer.forward_paged(torch.zeros(4, HID, device="cuda").half(), step.new_cache(), step, None)
