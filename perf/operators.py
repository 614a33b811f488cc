"""Timing cases of the decode-step operators, with their plain forms in torch.

Four operators of one serving step around the LoRA add-ons:

  plan       pages, slots and token maps of a step from the requests' lengths (lora_kv_plan)
  append     rotary positions of q and k, k and v written into their pages (lora_rope_append)
  attention  one query token per row over the paged cache (lora_paged_attention)
  norm       residual add with an optional norm, gate and scale, and the next norm (lora_residual_norm)

``run`` computes an operator in elementary torch operations (32-bit, rounded once at the
end; angles in 64 bits), or with ``own`` set through the package's entry points.
"""
import math
import random

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-5


def listed():
    return [
        # a decode step of the 7B batch: one new token for each of 32 requests
        dict(name="plan_decode_32", op="plan", requests=32, lo=64, ctx=4096, page=16, prefill=0, chunk=1, retire=0),
        # a step that admits prompts beside decoding requests and returns the pages of finished ones
        dict(name="plan_mixed_509", op="plan", requests=509, lo=1, ctx=8191, page=32, prefill=61, chunk=1021, retire=31),
        # Llama-2-7B decode, 32 rows
        dict(name="append_7b_decode", op="append", dtype="fp16", tokens=32, pad=0, heads=32, kv_heads=32, dim=128,
             rot=128, axes=1, interleaved=False, page=16, decode=True, far=4096),
        # Llama-2-7B prefill of 12,907 rows (16 prompts)
        dict(name="append_7b_prefill", op="append", dtype="fp16", tokens=12907, pad=0, heads=32, kv_heads=32, dim=128,
             rot=128, axes=1, interleaved=False, page=16, decode=False, far=4096),
        # the 70B head layout on image and video tokens (time, height, width), far positions, a padded batch
        dict(name="append_70b_3axes", op="append", dtype="bf16", tokens=4001, pad=95, heads=64, kv_heads=8, dim=128,
             rot=128, axes=3, interleaved=True, page=32, decode=False, far=1000000),
        # the first tokens of one 7B request: latency
        dict(name="attention_first_17", op="attention", dtype="fp16", rows=1, pad=0, heads=32, kv_heads=32, dim=128,
             lo=17, ctx=17, page=16, window=0),
        # Llama-2-7B decode, 32 requests up to the model's full length
        dict(name="attention_7b_32", op="attention", dtype="fp16", rows=32, pad=0, heads=32, kv_heads=32, dim=128,
             lo=64, ctx=4096, page=16, window=0),
        # 70B grouped-query decode, 61 requests in a batch padded to 64, very unequal lengths
        dict(name="attention_70b_61", op="attention", dtype="bf16", rows=61, pad=3, heads=64, kv_heads=8, dim=128,
             lo=1, ctx=16381, page=32, window=0),
        # one long request on one GPU's shard of 70B
        dict(name="attention_tp8_long", op="attention", dtype="fp16", rows=1, pad=0, heads=8, kv_heads=1, dim=128,
             lo=131071, ctx=131071, page=64, window=0),
        # Llama-2-7B decode: residual add and the next norm
        dict(name="norm_7b_decode", op="norm", dtype="fp16", rows=32, hidden=4096, post=False, gates=0, alpha=1.0),
        # Llama-2-7B prefill of 12,907 rows
        dict(name="norm_7b_prefill", op="norm", dtype="fp16", rows=12907, hidden=4096, post=False, gates=0, alpha=1.0),
        # norms on both sides of a block, per-request gates and a residual scale, at the 70B width
        dict(name="norm_gated_8192", op="norm", dtype="bf16", rows=4001, hidden=8192, post=True, gates=16, alpha=0.75),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng: random.Random):
    op = rng.choice(["plan", "append", "attention", "norm"])
    while True:
        if op == "plan":
            requests = _log_int(rng, 1, 1024)
            prefill = rng.choice([0, 0, requests // 8, requests // 2])
            ctx = _log_int(rng, 1, 16384)
            case = dict(op=op, requests=requests, lo=_log_int(rng, 1, ctx), ctx=ctx, page=rng.choice([1, 8, 16, 32, 64]),
                        prefill=prefill, chunk=_log_int(rng, 1, 2048),
                        retire=rng.choice([0, (requests - prefill) // 8]))
        elif op == "append":
            heads, kv, dim, rot = rng.choice([(32, 32, 128, 128), (40, 40, 128, 128), (64, 8, 128, 128),
                                              (8, 1, 128, 128), (16, 2, 64, 64), (12, 4, 80, 80), (8, 4, 256, 64)])
            decode = rng.random() < 0.5
            case = dict(op=op, dtype=rng.choice(["fp16", "bf16"]), tokens=_log_int(rng, 1, 512 if decode else 16384),
                        pad=rng.choice([0, rng.randint(1, 64)]), heads=heads, kv_heads=kv, dim=dim, rot=rot,
                        axes=rng.choice([1, 2, 3]), interleaved=rng.random() < 0.5, page=rng.choice([1, 8, 16, 32, 64]),
                        decode=decode, far=rng.choice([4096, 131072, 1000000]))
        elif op == "attention":
            heads, kv, dim = rng.choice([(32, 32, 128), (40, 40, 128), (64, 8, 128), (8, 1, 128), (16, 2, 64),
                                         (12, 4, 80), (8, 4, 256)])
            ctx = _log_int(rng, 1, 131072)
            case = dict(op=op, dtype=rng.choice(["fp16", "bf16"]), rows=_log_int(rng, 1, 256),
                        pad=rng.choice([0, rng.randint(1, 8)]), heads=heads, kv_heads=kv, dim=dim,
                        lo=_log_int(rng, 1, ctx), ctx=ctx, page=rng.choice([1, 8, 16, 32, 64]),
                        window=rng.choice([0, 0, _log_int(rng, 1, 4096)]))
            if (case["rows"] + case["pad"]) * ctx * kv * dim > 1 << 29:  # the padded batch of the plain form
                continue
        else:
            case = dict(op=op, dtype=rng.choice(["fp16", "bf16"]), rows=_log_int(rng, 1, 16384),
                        hidden=8 * _log_int(rng, 8, 2048), post=rng.random() < 0.5, gates=rng.choice([0, 1, 16]),
                        alpha=rng.choice([1.0, 0.5, 0.22]))
        if work(case)["bytes"] <= 480e6:
            return case


# ------------------------------------------------------------------------------ sizes
def _spread(n, lo, hi):
    """n whole numbers from lo to hi, evenly spaced on a logarithmic scale."""
    return [int(round(lo * (hi / lo) ** ((i + 0.5) / n))) for i in range(n)]


def _plan_requests(case):
    """(cached tokens, new tokens) of each request; -1 new tokens: the request has ended."""
    n, p, r = case["requests"], case["prefill"], case["retire"]
    old = _spread(n, case["lo"], case["ctx"])
    new = [1] * (n - p - r) + [-1] * r + _spread(p, 1, case["chunk"])
    old = old[:n - p] + [0 if i % 2 else o for i, o in enumerate(old[n - p:])]  # half of the prompts are new requests
    return old, new


def _pages(tokens, page):
    return -(-tokens // page)


def work(case):
    op = case["op"]
    if op == "plan":
        old, new = _plan_requests(case)
        P = case["page"]
        tokens = sum(max(c, 0) for c in new)
        taken = sum(_pages(o + c, P) - _pages(o, P) for o, c in zip(old, new) if c > 0)
        given = sum(_pages(o, P) for o, c in zip(old, new) if c < 0)
        # lengths, adapter slots, lengths after and offsets; four maps a token; ids moved once
        return dict(bytes=20 * len(old) + 4 + 16 * tokens + 8 * (taken + given), flops=0)
    if op == "append":
        T, H, K, D = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
        return dict(bytes=2 * 2 * T * (H + 2 * K) * D + 4 * T * (case["axes"] + 1) + 4 * case["rot"],
                    flops=3 * T * (H + K) * case["rot"])
    if op == "attention":
        span = [min(n, case["window"]) if case["window"] else n for n in _spread(case["rows"], case["lo"], case["ctx"])]
        K, H, D = case["kv_heads"], case["heads"], case["dim"]
        return dict(bytes=4 * sum(span) * K * D + 4 * case["rows"] * H * D + 4 * sum(_pages(s, case["page"]) for s in span)
                    + 4 * (case["rows"] + case["pad"]) * (1 + H), flops=4 * sum(span) * H * D)
    n, h = case["rows"], case["hidden"]
    return dict(bytes=2 * h * (4 * n + 1 + (1 if case["post"] else 0) + case["gates"]) + (4 * n if case["gates"] > 1 else 0),
                flops=n * h * (5 + (4 if case["post"] else 0) + (1 if case["gates"] else 0)))


# ------------------------------------------------------------------------------ inputs
class State:
    """What a serving program holds before the call."""


def _gen(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    return g


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEVICE)


def prepare(case, seed):
    s = State()
    s.case = case
    {"plan": _prepare_plan, "append": _prepare_append, "attention": _prepare_attention,
     "norm": _prepare_norm}[case["op"]](s, case, seed)
    return s


def _prepare_plan(s, case, seed):
    old, new = _plan_requests(case)
    order = list(range(len(old)))
    random.Random(seed).shuffle(order)
    old, new = [old[i] for i in order], [new[i] for i in order]
    P, n = case["page"], len(old)
    s.tokens = -(-max(1, sum(max(c, 0) for c in new)) // 8) * 8  # the batch's rows, padded to a multiple of 8
    blocks = [_pages(o, P) for o in old]
    s.max_blocks = max(_pages(o + max(c, 0), P) for o, c in zip(old, new)) + 1
    taken = sum(_pages(o + c, P) - b for o, c, b in zip(old, new, blocks) if c > 0)
    g = _gen(seed)
    used = sum(blocks)
    s.num_pages = used + taken + 64
    ids = torch.randperm(s.num_pages, generator=g, device=DEVICE).int()
    s.table = torch.full((n, s.max_blocks), -1, dtype=torch.int32, device=DEVICE)
    cols = torch.arange(s.max_blocks, device=DEVICE)
    s.table[cols[None, :] < _ints(blocks)[:, None]] = ids[:used]
    s.free = torch.full((s.num_pages,), -1, dtype=torch.int32, device=DEVICE)
    s.free[:s.num_pages - used] = ids[used:]
    s.top = _ints([s.num_pages - used])
    s.old, s.new = _ints(old), _ints(new)
    s.adapter = torch.randint(-1, 32, (n,), generator=g, device=DEVICE, dtype=torch.int32)
    if own:
        from segmented_gather_matmul_amd import step
        s.pages = step.KVPages(s.table, s.free, s.top, P)
        s.plan = step.KVPlan(n, s.tokens, device=DEVICE)


def _inv_freq(rot, theta=10000.0):
    return torch.tensor([theta ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float32, device=DEVICE)


def _prepare_append(s, case, seed):
    g = _gen(seed)
    dt, T, pad, H, K, D, P = (TYPES[case["dtype"]], case["tokens"], case["pad"], case["heads"], case["kv_heads"],
                              case["dim"], case["page"])
    n = T + pad
    qkv = torch.randn((n, (H + 2 * K) * D), generator=g, device=DEVICE, dtype=torch.float32).to(dt)
    # the projections' columns of one product
    s.q, s.k, s.v = qkv[:, :H * D], qkv[:, H * D:(H + K) * D], qkv[:, (H + K) * D:]
    s.q_out = torch.randn((n, H * D), generator=g, device=DEVICE, dtype=torch.float32).to(dt)
    if case["decode"]:  # every token in a page of its own
        page = torch.randperm(T + 3, generator=g, device=DEVICE)[:T]
        slot = page * P + torch.randint(0, P, (T,), generator=g, device=DEVICE)
        num_pages = T + 3
        first = torch.randint(0, case["far"], (T,), generator=g, device=DEVICE)
    else:  # prompts: runs of tokens, pages in any order
        num_pages = _pages(T, P) + 3
        t = torch.arange(T, device=DEVICE)
        slot = torch.randperm(num_pages, generator=g, device=DEVICE)[t // P] * P + t % P
        first = (t + torch.randint(0, case["far"], (1,), generator=g, device=DEVICE)) % case["far"]
    s.slots = torch.full((n,), -1, dtype=torch.int32, device=DEVICE)
    s.slots[:T] = slot.int()
    s.pos = torch.full((case["axes"], n), -1, dtype=torch.int32, device=DEVICE)
    s.pos[0, :T] = first.int()
    for a in range(1, case["axes"]):  # rows and columns of a picture
        s.pos[a, :T] = torch.randint(0, 128, (T,), generator=g, device=DEVICE).int()
    s.kc = torch.randn((num_pages, P, K, D), generator=g, device=DEVICE, dtype=torch.float32).to(dt)
    s.vc = torch.randn((num_pages, P, K, D), generator=g, device=DEVICE, dtype=torch.float32).to(dt)
    s.inv_freq = _inv_freq(case["rot"])
    half = case["rot"] // 2
    s.axis = _ints([i * case["axes"] // half for i in range(half)])  # the axes share the frequencies in sections
    if own:
        from segmented_gather_matmul_amd import step
        s.cache = step.PagedKV(s.kc, s.vc)
        s.rope = step.Rope(s.inv_freq, axis=s.axis, axes=case["axes"], interleaved=case["interleaved"])


def _prepare_attention(s, case, seed):
    g = _gen(seed)
    dt, n, pad, H, K, D, P = (TYPES[case["dtype"]], case["rows"], case["pad"], case["heads"], case["kv_heads"],
                              case["dim"], case["page"])
    lens = _spread(n, case["lo"], case["ctx"])
    random.Random(seed).shuffle(lens)
    s.max_len = max(lens)
    lens += [-1] * pad  # rows without a request
    blocks = [_pages(max(c, 0), P) for c in lens]
    num_pages = sum(blocks) + 2
    s.kc = torch.randn((num_pages, P, K, D), generator=g, device=DEVICE, dtype=dt)
    s.vc = torch.randn((num_pages, P, K, D), generator=g, device=DEVICE, dtype=dt)
    s.table = torch.full((n + pad, max(blocks) + 1), -1, dtype=torch.int32, device=DEVICE)
    cols = torch.arange(s.table.shape[1], device=DEVICE)
    s.table[cols[None, :] < _ints(blocks)[:, None]] = torch.randperm(num_pages, generator=g, device=DEVICE)[:sum(blocks)].int()
    s.lens = _ints(lens)
    s.q = (2.0 * torch.randn((n + pad, H * D), generator=g, device=DEVICE, dtype=torch.float32)).to(dt)
    s.out = torch.randn((n + pad, H * D), generator=g, device=DEVICE, dtype=torch.float32).to(dt)
    s.lse = torch.randn((n + pad, H), generator=g, device=DEVICE, dtype=torch.float32)
    if own:
        from segmented_gather_matmul_amd import step
        s.cache = step.PagedKV(s.kc, s.vc)
        s.work = step.attention_workspace(n + pad, H, s.cache)


def _prepare_norm(s, case, seed):
    g = _gen(seed)
    dt, n, h = TYPES[case["dtype"]], case["rows"], case["hidden"]
    rnd = lambda *sh: torch.randn(sh, generator=g, device=DEVICE, dtype=torch.float32)
    s.x, s.res = rnd(n, h).to(dt), (4.0 * rnd(n, h)).to(dt)
    s.w = (1.0 + 0.1 * rnd(h)).to(dt)
    s.post = (1.0 + 0.1 * rnd(h)).to(dt) if case["post"] else None
    s.gate = torch.tanh(rnd(case["gates"], h)).to(dt) if case["gates"] else None
    # rows of one request share a gate; some rows have none
    s.gate_idx = None
    if case["gates"] > 1:
        s.gate_idx = torch.randint(-1, case["gates"], (n,), generator=g, device=DEVICE, dtype=torch.int32)
    s.y, s.res_out = torch.empty_like(s.x), torch.empty_like(s.x)


# ------------------------------------------------------------------------------ one pass
def run(s):
    return {"plan": _run_plan, "append": _run_append, "attention": _run_attention, "norm": _run_norm}[s.case["op"]](s)


def _run_plan(s):
    P = s.case["page"]
    if own:
        from segmented_gather_matmul_amd import step
        p = s.plan
        step.lora_kv_plan(p, s.pages, s.old, s.new, req_slot=s.adapter)
        return [p.status, p.q_ptr, p.kv_end, p.free_top, p.tok_req, p.tok_pos, p.slots, p.idx, s.table, s.free]
    n, T = s.old.numel(), s.tokens
    old, ended, new = s.old.long(), s.new < 0, s.new.clamp(min=0).long()
    end = torch.where(ended, 0, old + new)
    had = (old + P - 1) // P
    grown = torch.where(ended, 0, (end + P - 1) // P - had)
    given = torch.where(ended, had, 0)
    cols = torch.arange(s.max_blocks, device=old.device)
    # pages of ended requests go on top of the free list, in order
    top = s.top.long()
    at = top + (given.cumsum(0) - given)[:, None] + cols
    put = ended[:, None] & (cols < had[:, None])
    free = torch.cat([s.free, s.free.new_zeros(1)])
    free[torch.where(put, at, s.num_pages)] = s.table
    s.free.copy_(free[:-1])
    top = top + given.sum()
    # growing requests take pages from the top, in order
    take = top - 1 - ((grown.cumsum(0) - grown)[:, None] + cols - had[:, None])
    got = (cols >= had[:, None]) & (cols < (had + grown)[:, None])
    s.table.copy_(torch.where(got, s.free[take.clamp(0, s.num_pages - 1)], s.table))
    taken, tokens = grown.sum(), new.sum()
    # token maps; the rows behind the last token belong to nobody
    q_ptr = torch.cat([new.new_zeros(1), new.cumsum(0)])
    req = torch.repeat_interleave(torch.arange(n + 1, device=old.device), torch.cat([new, (T - tokens)[None]]), output_size=T)
    live = req < n
    r = req.clamp(max=n - 1)
    pos = torch.arange(T, device=old.device) - q_ptr[r] + old[r]
    slot = s.table[r, torch.where(live, pos // P, 0)].long() * P + pos % P
    mark = lambda t: torch.where(live, t, -1).int()
    status = torch.stack([torch.zeros_like(tokens), tokens, taken, given.sum()]).int()
    return [status, q_ptr.int(), end.int(), (top - taken).int(), mark(r), mark(pos), mark(slot),
            mark(s.adapter[r].long()), s.table, s.free]


def _run_append(s):
    c = s.case
    if own:
        from segmented_gather_matmul_amd import step
        step.lora_rope_append(s.q_out, s.q, s.k, s.v, s.cache, s.slots, rope=s.rope, positions=s.pos)
        return [s.q_out, s.kc, s.vc]
    n, H, K, D, rot = s.q.shape[0], c["heads"], c["kv_heads"], c["dim"], c["rot"]
    live = (s.slots >= 0).nonzero()[:, 0] if c["pad"] else slice(None)
    angle = s.pos[s.axis.long()].T.double() * s.inv_freq.double()  # [n, rot / 2]
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]

    def turn(x, heads):
        x = x.reshape(n, heads, D).float()
        if c["interleaved"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).reshape(n, heads, rot)
        else:
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            y = torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)
        return torch.cat([y, x[..., rot:]], dim=-1)

    dt = s.q.dtype
    s.q_out[live] = turn(s.q, H).to(dt).reshape(n, H * D)[live]
    at = s.slots[live].long()
    s.kc.view(-1, K, D)[at] = turn(s.k, K).to(dt)[live]
    s.vc.view(-1, K, D)[at] = s.v.reshape(n, K, D)[live]
    return [s.q_out, s.kc, s.vc]


def _run_attention(s):
    c = s.case
    if own:
        from segmented_gather_matmul_amd import step
        step.lora_paged_attention(s.out, s.q, s.cache, s.table, s.lens, s.work, window=c["window"], lse=s.lse)
        return [s.out, s.lse]
    n, H, K, D, P = s.q.shape[0], c["heads"], c["kv_heads"], c["dim"], c["page"]
    G = H // K
    wide = _pages(s.max_len, P)
    ids = s.table[:, :wide].long().clamp(min=0)
    t = torch.arange(wide * P, device=s.q.device)
    seen = t < s.lens[:, None]
    if c["window"]:
        seen = seen & (t >= s.lens[:, None] - c["window"])
    k = s.kc[ids].float().reshape(n, wide * P, K, D).permute(0, 2, 3, 1).reshape(n * K, D, wide * P).contiguous()
    score = torch.bmm(s.q.float().reshape(n * K, G, D), k).reshape(n, K * G, wide * P) * (1.0 / math.sqrt(D))
    del k
    score = score.masked_fill(~seen[:, None, :], -math.inf)
    most = score.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(score - most)
    total = p.sum(-1, keepdim=True)
    v = s.vc[ids].float().reshape(n, wide * P, K, D).permute(0, 2, 1, 3).reshape(n * K, wide * P, D).contiguous()
    o = torch.bmm((p / total).nan_to_num(0.0).reshape(n * K, G, wide * P), v).reshape(n, H * D).to(s.out.dtype)
    live = s.lens >= 0
    s.out.copy_(torch.where(live[:, None], o, s.out))
    s.lse.copy_(torch.where(live[:, None], (most + total.log())[:, :, 0], s.lse))
    return [s.out, s.lse]


def _run_norm(s):
    c = s.case
    if own:
        from segmented_gather_matmul_amd import step
        step.lora_residual_norm(s.y, s.res, s.w, x=s.x, res_out=s.res_out, post_w=s.post, gate=s.gate,
                                gate_idx=s.gate_idx, alpha=c["alpha"], eps=EPS)
        return [s.y, s.res_out]
    x = s.x.float()
    if s.post is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s.post.float()
    if s.gate_idx is not None:
        i = s.gate_idx.long()
        x = torch.where(i[:, None] < 0, x, x * s.gate.float()[i.clamp(min=0)])
    elif s.gate is not None:
        x = x * s.gate.float()
    h = s.res.float() + c["alpha"] * x
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s.w.float()
    s.res_out.copy_(h)
    s.y.copy_(y)
    return [s.y, s.res_out]


# ------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """The outputs from the operators' definitions in 64 bits (whole numbers have none)."""
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    return {"append": _exact_append, "attention": _exact_attention, "norm": _exact_norm}[case["op"]](s, case)


def _exact_append(s, c):
    H, K, D, half = c["heads"], c["kv_heads"], c["dim"], c["rot"] // 2
    T = c["tokens"]
    q, kc, vc = s.q_out.double(), s.kc.double(), s.vc.double()
    at = s.slots[:T].long()
    kc.view(-1, K, D)[at] = s.k[:T].double().reshape(T, K, D)
    vc.view(-1, K, D)[at] = s.v[:T].double().reshape(T, K, D)
    q[:T] = s.q[:T].double()
    qh, kh = q.view(-1, H, D), s.k[:T].double().reshape(T, K, D)
    flat = kc.view(-1, K, D)
    for i in range(half):  # one frequency after another, as complex numbers turned by e^(i angle)
        a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, half + i)
        angle = s.pos[int(s.axis[i]), :T].double() * float(s.inv_freq[i])
        turn = torch.polar(torch.ones_like(angle), angle)[:, None]
        z = torch.complex(qh[:T, :, a].clone(), qh[:T, :, b].clone()) * turn
        qh[:T, :, a], qh[:T, :, b] = z.real, z.imag
        z = torch.complex(kh[:, :, a].contiguous(), kh[:, :, b].contiguous()) * turn
        flat[at, :, a], flat[at, :, b] = z.real, z.imag
    return [q, kc, vc]


def _exact_attention(s, c):
    H, K, D, P = c["heads"], c["kv_heads"], c["dim"], c["page"]
    out, lse = s.out.double(), s.lse.double()
    for r, length in enumerate(s.lens.tolist()):
        if length < 0:
            continue
        first = max(0, length - c["window"]) if c["window"] else 0
        t = torch.arange(first, length, device=out.device)
        page, off = s.table[r].long()[t // P], t % P
        k, v = s.kc[page, off].double(), s.vc[page, off].double()
        q = s.q[r].double().reshape(K, H // K, D)
        for h in range(K):
            z = (q[h] @ k[:, h].T.contiguous()) / math.sqrt(D)
            lse[r, h * (H // K):(h + 1) * (H // K)] = torch.logsumexp(z, -1)
            out[r].view(K, H // K, D)[h] = torch.softmax(z, -1) @ v[:, h].contiguous()
    return [out, lse]


def _exact_norm(s, c):
    x = s.x.double()
    if s.post is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / c["hidden"] + EPS) * s.post.double()
    if s.gate is not None:
        gate = torch.cat([s.gate.double(), torch.ones_like(s.gate[:1], dtype=torch.float64)])
        x = x * (gate[0] if s.gate_idx is None else gate[s.gate_idx.long()])  # the last row stands for -1
    h = s.res.double() + c["alpha"] * x
    return [h / torch.sqrt((h * h).sum(-1, keepdim=True) / c["hidden"] + EPS) * s.w.double(), h]
