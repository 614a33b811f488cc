"""Timing cases of the quantised cache's operators and of sampling, with their plain forms in torch.

  append     rotary positions of q and k, k and v quantised into their pages (lora_quant_append), and read
             back as the values that they now stand for (lora_quant_read): what a prompt's own attention needs
  read       the cells of many tokens as 16-bit rows (lora_quant_read)
  attention  one query token per row over the quantised cache (lora_quant_attention)
  sample     temperature, top-k, top-p, min-p and the draw from given random numbers (lora_sample)

A cell is blocks of 32 columns: codes of 4 (E2M1) or 8 bits (E4M3) and one exponent byte e, value code * 2^(e - 127).

``run`` computes an operator in elementary torch operations (32-bit, rounded once at the end; 64-bit for angles, for
what is rounded to codes, and for the masses of a draw), or with ``own`` set through the package's entry points.
"""
import math
import random

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
UNIT = 2.0 ** 40  # the largest weight of a draw


def listed():
    return [
        # Llama-2-7B decode, 32 rows: latency
        dict(name="append_q4_7b_decode", op="append", dtype="fp16", bits=4, tokens=32, pad=0, heads=32, kv_heads=32,
             dim=128, rot=128, axes=1, interleaved=False, page=16, decode=True, far=4096),
        # Llama-2-7B prefill of 12,907 rows (16 prompts)
        dict(name="append_q4_7b_prefill", op="append", dtype="fp16", bits=4, tokens=12907, pad=0, heads=32, kv_heads=32,
             dim=128, rot=128, axes=1, interleaved=False, page=16, decode=False, far=4096),
        # the 70B head layout on image and video tokens, far positions, a padded batch, 8 bits
        dict(name="append_q8_70b_3axes", op="append", dtype="bf16", bits=8, tokens=4001, pad=95, heads=64, kv_heads=8,
             dim=128, rot=128, axes=3, interleaved=True, page=32, decode=False, far=1000000),
        # a cached prefix of one 7B request as 16-bit rows
        dict(name="read_q4_7b_prefix", op="read", dtype="fp16", bits=4, tokens=4096, pad=0, kv_heads=32, dim=128, page=16),
        # long prefixes in the 70B layout, an odd number of rows, some of them without a token
        dict(name="read_q8_70b_long", op="read", dtype="bf16", bits=8, tokens=32749, pad=19, kv_heads=8, dim=128, page=32),
        # the first tokens of one 7B request: latency
        dict(name="attention_q4_first_17", op="attention", dtype="fp16", bits=4, rows=1, pad=0, heads=32, kv_heads=32,
             dim=128, lo=17, ctx=17, page=16, window=0),
        # Llama-2-7B decode, 32 requests up to the model's full length
        dict(name="attention_q4_7b_32", op="attention", dtype="fp16", bits=4, rows=32, pad=0, heads=32, kv_heads=32,
             dim=128, lo=64, ctx=4096, page=16, window=0),
        # 70B grouped-query decode, 61 requests in a batch padded to 64, very unequal lengths
        dict(name="attention_q4_70b_61", op="attention", dtype="bf16", bits=4, rows=61, pad=3, heads=64, kv_heads=8,
             dim=128, lo=1, ctx=16381, page=32, window=0),
        # one long request on one GPU's shard of 70B
        dict(name="attention_q4_tp8_long", op="attention", dtype="fp16", bits=4, rows=1, pad=0, heads=8, kv_heads=1,
             dim=128, lo=131071, ctx=131071, page=64, window=0),
        # one request's next token: latency
        dict(name="sample_1", op="sample", dtype="fp16", rows=1, extra=0, vocab=32000, filters="both"),
        # Llama-2-7B decode, 32 requests, each with settings of its own; a step's logits of 64 token rows
        dict(name="sample_7b_32", op="sample", dtype="fp16", rows=32, extra=32, vocab=32000, filters="mixed"),
        # a large batch over a large vocabulary of odd size
        dict(name="sample_251_wide", op="sample", dtype="bf16", rows=251, extra=0, vocab=128257, filters="mixed"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


LAYOUTS = [(32, 32, 128, 128), (40, 40, 128, 128), (64, 8, 128, 128), (8, 1, 128, 128), (16, 2, 64, 64), (12, 4, 80, 80),
           (8, 4, 256, 64)]


def draw(rng: random.Random):
    op = rng.choice(["append", "read", "attention", "attention", "sample"])
    while True:
        heads, kv, dim, rot = rng.choice(LAYOUTS)
        bits, page, dtype = rng.choice([4, 4, 8]), rng.choice([1, 8, 16, 32, 64]), rng.choice(["fp16", "bf16"])
        if op == "append":
            decode = rng.random() < 0.5
            case = dict(op=op, dtype=dtype, bits=bits, tokens=_log_int(rng, 1, 512 if decode else 16384),
                        pad=rng.choice([0, rng.randint(1, 64)]), heads=heads, kv_heads=kv, dim=dim, rot=rot,
                        axes=rng.choice([1, 2, 3]), interleaved=rng.random() < 0.5, page=page, decode=decode,
                        far=rng.choice([4096, 131072, 1000000]))
        elif op == "read":
            case = dict(op=op, dtype=dtype, bits=bits, tokens=_log_int(rng, 1, 65536),
                        pad=rng.choice([0, rng.randint(1, 64)]), kv_heads=kv, dim=dim, page=page)
        elif op == "attention":
            ctx = _log_int(rng, 1, 131072)
            case = dict(op=op, dtype=dtype, bits=bits, rows=_log_int(rng, 1, 256), pad=rng.choice([0, rng.randint(1, 8)]),
                        heads=heads, kv_heads=kv, dim=dim, lo=_log_int(rng, 1, ctx), ctx=ctx, page=page,
                        window=rng.choice([0, 0, _log_int(rng, 1, 4096)]))
            if (case["rows"] + case["pad"]) * ctx * kv * dim > 1 << 29:  # the padded batch of the plain form
                continue
        else:
            case = dict(op=op, dtype=rng.choice(["fp16", "bf16", "fp32"]), rows=_log_int(rng, 1, 256),
                        extra=rng.choice([0, rng.randint(1, 16)]), vocab=_log_int(rng, 1000, 200000),
                        filters=rng.choice(["none", "greedy", "both", "mixed", "mixed"]))
            if case["rows"] * case["vocab"] > 1 << 25:
                continue
        if work(case)["bytes"] <= 480e6:
            return case


# ------------------------------------------------------------------------------ sizes
def _spread(n, lo, hi):
    """n whole numbers from lo to hi, evenly spaced on a logarithmic scale."""
    return [int(round(lo * (hi / lo) ** ((i + 0.5) / n))) for i in range(n)]


def _pages(tokens, page):
    return -(-tokens // page)


def _padded(dim):
    return -(-dim // 32) * 32


def _cell_bytes(case):
    """Bytes of one token's k or v."""
    return case["kv_heads"] * (_padded(case["dim"]) * case["bits"] // 8 + _padded(case["dim"]) // 32)


def work(case):
    op = case["op"]
    if op == "append":
        T, H, K, D = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
        # q, k, v and q_out; the cells written and read; k and v read back
        return dict(bytes=2 * T * (2 * H + 2 * K) * D + 4 * T * _cell_bytes(case) + 4 * T * K * D
                    + 4 * T * (case["axes"] + 1) + 4 * case["rot"], flops=3 * T * (H + K) * case["rot"])
    if op == "read":
        T = case["tokens"]
        return dict(bytes=2 * T * _cell_bytes(case) + 4 * T * case["kv_heads"] * case["dim"] + 4 * T, flops=0)
    if op == "attention":
        span = [min(n, case["window"]) if case["window"] else n for n in _spread(case["rows"], case["lo"], case["ctx"])]
        H, D = case["heads"], case["dim"]
        return dict(bytes=2 * sum(span) * _cell_bytes(case) + 4 * case["rows"] * H * D
                    + 4 * sum(_pages(s, case["page"]) for s in span) + 4 * (case["rows"] + case["pad"]) * (1 + H),
                    flops=4 * sum(span) * H * D)
    n, V = case["rows"], case["vocab"]
    return dict(bytes=n * V * (4 if case["dtype"] == "fp32" else 2) + 28 * n, flops=12 * n * V)


# ------------------------------------------------------------------------------ the format
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _exponents(dtype, bits):
    """Least and largest exponent of a block whose values the 16-bit type holds."""
    least, most = (-24, 15) if dtype is torch.float16 else (-126, 127)
    return (least + 1, most - 2) if bits == 4 else (least + 9, most - 8)


def _quantise(x, bits, dtype):
    """x [..., D] in 32 bits -> (codes uint8 [..., Dp * bits / 8], exponents uint8 [..., Dp / 32])."""
    x = torch.nn.functional.pad(x, (0, _padded(x.shape[-1]) - x.shape[-1]))
    x = x.reshape(*x.shape[:-1], -1, 32)
    most = x.abs().amax(-1)
    exp = ((most.view(torch.int32) + (0x200000 if bits == 4 else 0x180000)) >> 23) - 127 - (2 if bits == 4 else 8)
    exp = exp.clamp(*_exponents(dtype, bits))
    q = x * ((127 - exp) << 23).view(torch.float32)[..., None]
    if bits == 8:
        code = q.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        a = q.abs()
        code = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte()
                + (a >= 3.5).byte() + (a > 5.0).byte() + 8 * torch.signbit(q).byte())
        code = code[..., 0::2] | (code[..., 1::2] << 4)
    return code.flatten(-2), (exp + 127).to(torch.uint8)


def _values(code, exp, bits, dim):
    """What codes and exponents stand for, in 32 bits."""
    if bits == 8:
        x = code.view(torch.float8_e4m3fn).float()
    else:
        lut = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float32, device=code.device)
        x = torch.stack([lut[(code & 15).int()], lut[(code >> 4).int()]], dim=-1).flatten(-2)
    x = x.reshape(*exp.shape, 32) * (exp.int() << 23).view(torch.float32)[..., None]
    return x.flatten(-2)[..., :dim]


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
    {"append": _prepare_append, "read": _prepare_read, "attention": _prepare_attention,
     "sample": _prepare_sample}[case["op"]](s, case, seed)
    return s


def _empty_cache(s, case, num_pages):
    """Codes and exponents [page, token, head, ...], heads before tokens in memory."""
    K, P, Dp = case["kv_heads"], case["page"], _padded(case["dim"])
    new = lambda n: torch.zeros((num_pages, K, P, n), dtype=torch.uint8, device=DEVICE).transpose(1, 2)
    s.kc, s.vc, s.ks, s.vs = new(Dp * case["bits"] // 8), new(Dp * case["bits"] // 8), new(Dp // 32), new(Dp // 32)
    if own:
        from segmented_gather_matmul_amd import quant
        s.cache = quant.QuantKV(s.kc, s.vc, s.ks, s.vs, case["dim"], TYPES[case["dtype"]])


def _fill_cache(s, case, num_pages, g):
    """Cells of normal values; a few columns of k are much larger than the others, as they are in earnest."""
    _empty_cache(s, case, num_pages)
    K, P, D, dt = case["kv_heads"], case["page"], case["dim"], TYPES[case["dtype"]]
    wide = 1.0 + 7.0 * (torch.rand((K, D), generator=g, device=DEVICE) < 0.03).float()
    step = max(1, (1 << 26) // (P * K * D))
    for i in range(0, num_pages, step):
        n = min(step, num_pages - i)
        for codes, exps, gain in ((s.kc, s.ks, wide), (s.vc, s.vs, 1.0)):
            x = torch.randn((n, P, K, D), generator=g, device=DEVICE, dtype=torch.float32) * gain
            codes[i:i + n], exps[i:i + n] = _quantise(x.to(dt).float(), case["bits"], dt)


def _prepare_append(s, case, seed):
    g = _gen(seed)
    dt, T, pad, H, K, D, P = (TYPES[case["dtype"]], case["tokens"], case["pad"], case["heads"], case["kv_heads"],
                              case["dim"], case["page"])
    n = T + pad
    qkv = torch.randn((n, (H + 2 * K) * D), generator=g, device=DEVICE, dtype=torch.float32)
    qkv[:, H * D:(H + K) * D] *= 1.0 + 7.0 * (torch.rand((K * D,), generator=g, device=DEVICE) < 0.03).float()
    qkv = qkv.to(dt)
    # the projections' columns of one product
    s.q, s.k, s.v = qkv[:, :H * D], qkv[:, H * D:(H + K) * D], qkv[:, (H + K) * D:]
    rnd = lambda cols: torch.randn((n, cols), generator=g, device=DEVICE, dtype=torch.float32).to(dt)
    s.q_out, s.k_out, s.v_out = rnd(H * D), rnd(K * D), rnd(K * D)
    if case["decode"]:  # every token in a page of its own
        num_pages = T + 3
        page = torch.randperm(num_pages, generator=g, device=DEVICE)[:T]
        slot = page * P + torch.randint(0, P, (T,), generator=g, device=DEVICE)
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
    s.inv_freq = torch.tensor([10000.0 ** (-2.0 * i / case["rot"]) for i in range(case["rot"] // 2)],
                              dtype=torch.float32, device=DEVICE)
    half = case["rot"] // 2
    s.axis = _ints([i * case["axes"] // half for i in range(half)])  # the axes share the frequencies in sections
    _empty_cache(s, case, num_pages)
    if own:
        from segmented_gather_matmul_amd import step
        s.rope = step.Rope(s.inv_freq, axis=s.axis, axes=case["axes"], interleaved=case["interleaved"])


def _prepare_read(s, case, seed):
    g = _gen(seed)
    T, P, K, D, dt = case["tokens"], case["page"], case["kv_heads"], case["dim"], TYPES[case["dtype"]]
    n, num_pages = T + case["pad"], _pages(T, P) + 3
    _fill_cache(s, case, num_pages, g)
    t = torch.arange(T, device=DEVICE)
    slot = torch.randperm(num_pages, generator=g, device=DEVICE)[t // P] * P + t % P
    s.slots = torch.full((n,), -1, dtype=torch.int32, device=DEVICE)
    s.slots[torch.randperm(n, generator=g, device=DEVICE)[:T].sort()[0]] = slot.int()
    rnd = lambda: torch.randn((n, K * D), generator=g, device=DEVICE, dtype=torch.float32).to(dt)
    s.k_out, s.v_out = rnd(), rnd()


def _prepare_attention(s, case, seed):
    g = _gen(seed)
    dt, n, pad, H, D, P = (TYPES[case["dtype"]], case["rows"], case["pad"], case["heads"], case["dim"], case["page"])
    lens = _spread(n, case["lo"], case["ctx"])
    random.Random(seed).shuffle(lens)
    s.max_len = max(lens)
    lens += [-1] * pad  # rows without a request
    blocks = [_pages(max(c, 0), P) for c in lens]
    num_pages = sum(blocks) + 2
    _fill_cache(s, case, num_pages, g)
    s.table = torch.full((n + pad, max(blocks) + 1), -1, dtype=torch.int32, device=DEVICE)
    cols = torch.arange(s.table.shape[1], device=DEVICE)
    s.table[cols[None, :] < _ints(blocks)[:, None]] = torch.randperm(num_pages, generator=g, device=DEVICE)[:sum(blocks)].int()
    s.lens = _ints(lens)
    s.q = torch.randn((n + pad, H * D), generator=g, device=DEVICE, dtype=torch.float32).to(dt)
    s.out = torch.randn((n + pad, H * D), generator=g, device=DEVICE, dtype=torch.float32).to(dt)
    s.lse = torch.randn((n + pad, H), generator=g, device=DEVICE, dtype=torch.float32)
    if own:
        from segmented_gather_matmul_amd import quant
        s.work = quant.attention_workspace(n + pad, H, s.cache)


def _prepare_sample(s, case, seed):
    g, r = _gen(seed), random.Random(seed)
    n, m, V, kind = case["rows"], case["rows"] + case["extra"], case["vocab"], case["filters"]
    x = 2.0 * torch.randn((m, V), generator=g, device=DEVICE, dtype=torch.float32)
    # a few likely tokens in every row
    x.scatter_add_(1, torch.randint(0, V, (m, 24), generator=g, device=DEVICE),
                   3.0 + 6.0 * torch.rand((m, 24), generator=g, device=DEVICE))
    # rows held to a grammar: most of the vocabulary is masked
    held = torch.arange(m, device=DEVICE)[:, None] % 8 == 5
    x.masked_fill_(held & (torch.rand((m, V), generator=g, device=DEVICE) < 0.9), -math.inf)
    s.logits = x.to(TYPES[case["dtype"]])
    pick = {"none": ([1.0, 0.7, 1.3], [0], [1.0], [0.0]), "greedy": ([0.0], [0], [1.0], [0.0]),
            "both": ([0.8], [50], [0.95], [0.0]),
            "mixed": ([0.0, 0.6, 0.8, 1.0, 1.5], [0, 0, 1, 40, 1000], [1.0, 0.9, 0.95, 0.5], [0.0, 0.0, 0.05, 0.3])}[kind]
    t, k, p, q = ([r.choice(v) for _ in range(n)] for v in pick)
    real = lambda v: torch.tensor(v, dtype=torch.float32, device=DEVICE)
    s.temperature, s.top_k, s.top_p, s.min_p = real(t), _ints(k), real(p), real(q)
    s.u = torch.rand((n,), generator=g, device=DEVICE, dtype=torch.float32)
    s.rows = torch.randperm(m, generator=g, device=DEVICE)[:n].int() if case["extra"] else None
    s.token = torch.full((n,), -7, dtype=torch.int32, device=DEVICE)
    s.logprob = torch.zeros((n,), dtype=torch.float32, device=DEVICE)
    if own:
        from segmented_gather_matmul_amd import sample
        s.work = sample.sample_workspace(n, V, device=DEVICE)


# ------------------------------------------------------------------------------ one pass
def run(s):
    return {"append": _run_append, "read": _run_read, "attention": _run_attention, "sample": _run_sample}[s.case["op"]](s)


def _run_append(s):
    c = s.case
    if own:
        from segmented_gather_matmul_amd import quant
        quant.lora_quant_append(s.q_out, s.q, s.k, s.v, s.cache, s.slots, rope=s.rope, positions=s.pos)
        quant.lora_quant_read(s.k_out, s.v_out, s.cache, s.slots)
        return [s.q_out, s.k_out, s.v_out]
    n, H, K, D, P, rot = s.q.shape[0], c["heads"], c["kv_heads"], c["dim"], c["page"], c["rot"]
    live = (s.slots >= 0).nonzero()[:, 0] if c["pad"] else slice(None)
    angle = s.pos[s.axis.long()].T.double() * s.inv_freq.double()  # [n, rot / 2]
    cos, sin = angle.cos()[:, None, :], angle.sin()[:, None, :]

    def turn(x, heads):
        x = x.reshape(n, heads, D).double()
        if c["interleaved"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).reshape(n, heads, rot)
        else:
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            y = torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)
        return torch.cat([y, x[..., rot:]], dim=-1).float()

    dt = s.q.dtype
    s.q_out[live] = turn(s.q, H).to(dt).reshape(n, H * D)[live]
    at = s.slots[live].long()
    s.kc[at // P, at % P], s.ks[at // P, at % P] = _quantise(turn(s.k, K)[live], c["bits"], dt)
    s.vc[at // P, at % P], s.vs[at // P, at % P] = _quantise(s.v.reshape(n, K, D).float()[live], c["bits"], dt)
    return [s.q_out, *_run_read(s)]


def _run_read(s):
    c = s.case
    if own:
        from segmented_gather_matmul_amd import quant
        quant.lora_quant_read(s.k_out, s.v_out, s.cache, s.slots)
        return [s.k_out, s.v_out]
    live = (s.slots >= 0).nonzero()[:, 0] if c["pad"] else slice(None)
    at = s.slots[live].long()
    page, off = at // c["page"], at % c["page"]
    s.k_out[live] = _values(s.kc[page, off], s.ks[page, off], c["bits"], c["dim"]).flatten(1).to(s.k_out.dtype)
    s.v_out[live] = _values(s.vc[page, off], s.vs[page, off], c["bits"], c["dim"]).flatten(1).to(s.v_out.dtype)
    return [s.k_out, s.v_out]


def _run_attention(s):
    c = s.case
    if own:
        from segmented_gather_matmul_amd import quant
        quant.lora_quant_attention(s.out, s.q, s.cache, s.table, s.lens, s.work, window=c["window"], lse=s.lse)
        return [s.out, s.lse]
    n, H, K, D, P = s.q.shape[0], c["heads"], c["kv_heads"], c["dim"], c["page"]
    G = H // K
    wide = _pages(s.max_len, P)
    ids = s.table[:, :wide].long().clamp(min=0)
    t = torch.arange(wide * P, device=s.q.device)
    seen = t < s.lens[:, None]
    if c["window"]:
        seen = seen & (t >= s.lens[:, None] - c["window"])
    k = _values(s.kc[ids], s.ks[ids], c["bits"], D).reshape(n, wide * P, K, D).permute(0, 2, 3, 1)
    k = k.reshape(n * K, D, wide * P).contiguous()
    score = torch.bmm(s.q.float().reshape(n * K, G, D), k).reshape(n, K * G, wide * P) * (1.0 / math.sqrt(D))
    del k
    score = score.masked_fill(~seen[:, None, :], -math.inf)
    most = score.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(score - most)
    total = p.sum(-1, keepdim=True)
    v = _values(s.vc[ids], s.vs[ids], c["bits"], D).reshape(n, wide * P, K, D).permute(0, 2, 1, 3)
    v = v.reshape(n * K, wide * P, D).contiguous()
    o = torch.bmm((p / total).nan_to_num(0.0).reshape(n * K, G, wide * P), v).reshape(n, H * D).to(s.out.dtype)
    live = s.lens >= 0
    s.out.copy_(torch.where(live[:, None], o, s.out))
    s.lse.copy_(torch.where(live[:, None], (most + total.log())[:, :, 0], s.lse))
    return [s.out, s.lse]


def _run_sample(s):
    if own:
        from segmented_gather_matmul_amd import sample
        sample.lora_sample(s.token, s.logits, s.u, s.work, temperature=s.temperature, top_k=s.top_k, top_p=s.top_p,
                           min_p=s.min_p, rows=s.rows, logprob=s.logprob)
        return [s.token, s.logprob]
    x = (s.logits if s.rows is None else s.logits[s.rows.long()]).double()
    V = x.shape[1]
    x, order = torch.sort(x, dim=-1, descending=True, stable=True)  # equal ones by their index
    cold = s.temperature[:, None] == 0
    z = (x - x[:, :1]) / torch.where(cold, 1.0, s.temperature[:, None].double())
    weight = (torch.exp(z) * UNIT).floor().long()  # whole numbers: their sums are exact
    rank = torch.arange(V, device=x.device)
    top_k = torch.where(s.top_k == 0, V, s.top_k)[:, None]
    weight = torch.where(rank < torch.where(cold, 1, top_k), weight, 0)
    before = weight.cumsum(-1) - weight
    total = weight.sum(-1, keepdim=True)
    keep = (before.double() < s.top_p[:, None].double() * total.double()) | (rank == 0)
    keep = keep & (weight.double() >= s.min_p[:, None].double() * UNIT)
    weight = torch.where(keep, weight, 0)
    line = torch.zeros_like(weight).scatter_(1, order, weight).cumsum(-1)
    total = line[:, -1:]
    at = torch.minimum((s.u[:, None].double() * total.double()).floor().long(), total - 1)
    token = (line <= at).sum(-1, keepdim=True)
    s.token.copy_(token[:, 0])
    z = torch.where(order == token, z, 0.0).sum(-1)
    s.logprob.copy_(z - (total[:, 0].double() / UNIT).log())
    return [s.token, s.logprob]


# ------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """The outputs from the operators' definitions in 64 bits (tokens have none)."""
    s = prepare(case, seed)
    return {"append": _exact_append, "read": _exact_read, "attention": _exact_attention,
            "sample": _exact_sample}[case["op"]](s, case)


def _grid(bits):
    """Every magnitude that a code stands for, from 0 up."""
    if bits == 4:
        return torch.tensor(E2M1, dtype=torch.float64, device=DEVICE)
    sub = [m * 2.0 ** -9 for m in range(8)]
    return torch.tensor(sub + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1],
                        dtype=torch.float64, device=DEVICE)


def _exact_rounded(x, c):
    """x [n, K, D] in 64 bits, block by block, on the nearest point of the block's grid (the even one of two)."""
    least, most = _exponents(TYPES[c["dtype"]], c["bits"])
    grid, edge = _grid(c["bits"]), 7.0 if c["bits"] == 4 else 464.0
    y = torch.empty_like(x)
    for d in range(0, c["dim"], 32):
        b = x[..., d:d + 32]
        top = b.abs().amax(-1, keepdim=True)
        e = torch.full_like(top, least)
        for i in range(least, most):  # one step up for as long as the block does not fit
            e += (top >= edge * 2.0 ** i).double()
        unit = torch.exp2(e)
        a = (b.abs() / unit).clamp(max=float(grid[-1]))
        hi = torch.searchsorted(grid, a.contiguous()).clamp(1, grid.numel() - 1)
        down, up = a - grid[hi - 1], grid[hi] - a
        pick = torch.where((down < up) | ((down == up) & (hi % 2 == 1)), hi - 1, hi)
        y[..., d:d + 32] = torch.copysign(grid[pick] * unit, b)
    return y


def _exact_append(s, c):
    H, K, D, half, T = c["heads"], c["kv_heads"], c["dim"], c["rot"] // 2, c["tokens"]
    outs = []
    for x, heads, out, cell in ((s.q, H, s.q_out, False), (s.k, K, s.k_out, True), (s.v, K, s.v_out, True)):
        y = x[:T].double().reshape(T, heads, D).clone()
        if x is not s.v:
            for i in range(half):  # one frequency after another, as complex numbers turned by e^(i angle)
                a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, half + i)
                angle = s.pos[int(s.axis[i]), :T].double() * float(s.inv_freq[i])
                z = torch.complex(y[:, :, a].contiguous(), y[:, :, b].contiguous())
                z = z * torch.polar(torch.ones_like(angle), angle)[:, None]
                y[:, :, a], y[:, :, b] = z.real, z.imag
        y = _exact_rounded(y, c) if cell else y
        outs.append(torch.cat([y.reshape(T, heads * D), out[T:].double()]))
    return outs


def _exact_cells(codes, exps, c):
    """Values of codes [..., bytes] in 64 bits, from the bits of each code."""
    codes = codes.long()
    if c["bits"] == 4:
        codes = torch.stack([codes % 16, codes // 16], dim=-1).flatten(-2)
        sign, mag = codes // 8, codes % 8
    else:
        sign, mag = codes // 128, codes % 128
    x = _grid(c["bits"])[mag] * (1 - 2 * sign)
    return (x * torch.exp2(exps.double() - 127).repeat_interleave(32, dim=-1))[..., :c["dim"]]


def _exact_read(s, c):
    outs = []
    for out, codes, exps in ((s.k_out, s.kc, s.ks), (s.v_out, s.vc, s.vs)):
        y = out.double()
        live = (s.slots >= 0).nonzero()[:, 0]
        at = s.slots[live].long()
        page, off = at // c["page"], at % c["page"]
        y[live] = _exact_cells(codes[page, off], exps[page, off], c).flatten(1)
        outs.append(y)
    return outs


def _exact_attention(s, c):
    H, K, D, P = c["heads"], c["kv_heads"], c["dim"], c["page"]
    out, lse = s.out.double(), s.lse.double()
    for r, length in enumerate(s.lens.tolist()):
        if length < 0:
            continue
        first = max(0, length - c["window"]) if c["window"] else 0
        t = torch.arange(first, length, device=out.device)
        page, off = s.table[r].long()[t // P], t % P
        q = s.q[r].double().reshape(K, H // K, D)
        for h in range(K):
            k = _exact_cells(s.kc[page, off, h], s.ks[page, off, h], c)
            v = _exact_cells(s.vc[page, off, h], s.vs[page, off, h], c)
            z = (q[h] @ k.T.contiguous()) / math.sqrt(D)
            lse[r, h * (H // K):(h + 1) * (H // K)] = torch.logsumexp(z, -1)
            out[r].view(K, H // K, D)[h] = torch.softmax(z, -1) @ v
    return [out, lse]


def _exact_sample(s, c):
    """No value for the tokens; the drawn token's log-probability from the definition, one row after another."""
    logprob = torch.zeros((c["rows"],), dtype=torch.float64)
    for r in range(c["rows"]):
        x = s.logits[r if s.rows is None else int(s.rows[r])].double()
        t, k, p, q = float(s.temperature[r]), int(s.top_k[r]), float(s.top_p[r]), float(s.min_p[r])
        if t == 0.0:
            continue
        order = torch.argsort(x, descending=True, stable=True)[:k or None]
        prob = torch.softmax(x[order] / t, 0)
        before = prob.cumsum(0) - prob
        on = ((before < p) | (torch.arange(order.numel(), device=x.device) == 0)) & (prob >= q * prob[0])
        chosen = order[on].sort()[0]
        prob = torch.softmax(x[chosen] / t, 0)
        i = int((prob.cumsum(0) <= float(s.u[r])).sum().clamp(max=chosen.numel() - 1))
        logprob[r] = prob[i].log()
    return [None, logprob]
