"""GPU: attention over a quantised cache where every wavefront has parts of its own (many rows or many heads), and steps
captured and replayed with other lengths, in both ways to split the rows.  Tolerances are derived in quant_ref."""
import math
import random

import pytest
import torch

from segmented_gather_matmul_amd import binding as B
from segmented_gather_matmul_amd import quant as Q
from segmented_gather_matmul_amd import step as S
from tests import quant_ref as QR
from tests.gpu_cases import say
from tests.test_gpu_quant import Attn, bytes_of, cells
from tests.test_gpu_step import close, ints

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
COUNTERS = 2 * (4 * 256 + 4096)     # first in a workspace


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()
    yield


def alone(n, H, K, D):
    """Whether such a call is split by wavefronts: its workspace has more parts than one row's."""
    size = B.lib().lora_quant_attention_bytes
    return size(n, H, K, D) > size(1, H, K, D)


def spread(lens, n, seed):
    """Those lengths in order among n rows, the others not active."""
    at = sorted(random.Random(seed).sample(range(n), len(lens)))
    rows = [-1] * n
    for i, x in zip(at, lens):
        rows[i] = x
    return rows


LONG = [300, 9000, 1, 0, 64, 2500, 65, 17, 5003, 256, 128, 129]     # parts of 4 tiles: up to 36 of them
# active rows' lengths, rows, heads, kv_heads, D, page
ALONE = [(LONG, 1024, 3, 1, 128, 16), (LONG, 1030, 7, 1, 64, 8), (LONG, 1024, 16, 1, 128, 64), (LONG, 350, 34, 1, 96, 32),
         (LONG[:6], 512, 10, 2, 40, 1), (LONG, 600, 5, 1, 256, 16), (LONG[:8], 300, 36, 2, 160, 4),
         ([20011, 700], 1024, 8, 1, 128, 16), ([1, 40000, 33], 1024, 4, 1, 32, 1024),
         ([1500, 700, 64, 1], 4, 256, 256, 16, 16), ([900, 300], 2, 512, 512, 8, 8), ([130, 2000, 0, 513], 8, 512, 128, 32, 16),
         ([64, 1500, 3, 200, 1025] * 2, 64, 16, 16, 128, 16), ([777, 64, 1400, 31], 32, 32, 32, 128, 8),
         ([1000, 65], 22, 34 * 16, 16, 48, 16), ([700, 129, 2000], 32, 16, 16, 256, 32)]


@pytest.mark.parametrize("case", ALONE, ids=lambda c: f"{len(c[0])}of{c[1]}x{max(c[0])}-" + "-".join(map(str, c[2:])))
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dt", [F16, BF16], ids=["f16", "bf16"])
def test_rows_of_many_tiles_and_parts(case, bits, dt):
    lens, n, H, K, D, P = case
    say(f"case quant-alone {case} bits={bits} {dt}")
    assert alone(n, H, K, D)
    layout = ("heads", "tokens", "gaps", "record")[(H + D + bits) % 4]
    a = Attn(spread(lens, n, H + D), H, K, D, P, dt, bits, layout, seed=H + n)
    a.poison()
    a.run().check(what="call")


@pytest.mark.parametrize("window", [63, 1000, 4000])
@pytest.mark.parametrize("bits,P", [(4, 16), (8, 4)])
def test_windows(window, bits, P):
    say(f"case quant-alone-window {window} bits={bits}")
    a = Attn(spread(LONG, 520, window), 10, 2, 64, P, BF16, bits, seed=window)
    assert alone(520, 10, 2, 64)
    a.poison()
    a.run(window=window).check(window=window, what="window")


def test_pages_that_are_none_and_rows_that_share_a_request():
    say("case quant-alone-pages")
    n = 1024
    a = Attn([3000, 700], 6, 1, 128, 16, F16, 4, seed=3)
    a.table[0, 3:40], a.table[0, 100], a.table[1, 43] = -1, a.c.num_pages, 2 ** 31 - 1
    a.poison()
    req = [(i // 100) % 3 - 1 if i % 50 == 7 else -1 for i in range(n)]
    req[5] = 2 ** 31 - 1
    lens = [(3000, 2999, 64 * 3 + 1, 640)[i % 4] if req[i] == 0 else 700 - i % 60 for i in range(n)]
    lens[7] = -1
    q = torch.randn(n, 6 * 128, generator=torch.Generator().manual_seed(1)).to(F16)
    a.run(req=ints(req), kv_len=ints(lens), q=q.cuda()).check(req=req, kv_len=lens, q=q, what="pages")


def test_results_are_the_same_every_time_and_the_workspace_is_left_clean():
    """Calls of both splits, and of the 16-bit attention, in one workspace."""
    say("case quant-alone-repeat")
    many = [Attn(spread(LONG + [20011], 1024, 1), 8, 1, 128, 16, F16, 4, seed=1),
            Attn(spread([1500, 700, 900], 4, 2), 256, 256, 16, 8, BF16, 8, seed=2), Attn([9000, 3, 700], 8, 2, 128, 16, F16, 4, seed=3)]
    assert [alone(len(a.lens), a.H, a.c.kv_heads, a.D) for a in many] == [True, True, False]
    paged = S.PagedKV(*(v.cuda() for v in many[0].val))
    work = torch.zeros(max([Q.attention_workspace(len(a.lens), a.H, a.c).numel() for a in many]
                           + [S.attention_workspace(1024, 8, paged).numel()]), dtype=torch.int32, device="cuda")
    first, out = [], torch.empty(1024, 8 * 128, dtype=F16, device="cuda")
    for a in many:
        a.run(work=work).check(what="first")
        first.append((a.out.clone(), a.lse.clone()))
    for _ in range(3):
        for a, (o, lse) in zip(many, first):
            a.run(work=work)
            assert torch.equal(a.out, o) and torch.equal(a.lse, lse)
            assert not bool(work[:COUNTERS].any())
        S.lora_paged_attention(out, many[0].q.cuda(), paged, many[0].table.cuda(), ints(many[0].lens), work)
        assert not bool(work[:COUNTERS].any())


def test_two_streams_with_workspaces_of_their_own():
    say("case quant-alone-streams")
    cases = [Attn(spread(LONG, 1024, i), 8, 1, 128, 16, F16, 4, seed=20 + i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in cases]
    works = [Q.attention_workspace(1024, 8, a.c) for a in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for a, st, w in zip(cases, streams, works):
            with torch.cuda.stream(st):
                a.run(work=w)
    torch.cuda.synchronize()
    for a in cases:
        a.check(what="stream")


# rows, requests, heads, kv_heads, tokens a request has room for
@pytest.mark.parametrize("bits,dt", [(4, F16), (8, BF16)], ids=["4-f16", "8-bf16"])
@pytest.mark.parametrize("n,n_req,H,K,most", [(6, 6, 8, 2, 4096), (1024, 12, 8, 1, 4096), (64, 16, 16, 16, 512)])
def test_steps_captured_and_replayed_with_other_lengths(n, n_req, H, K, most, bits, dt):
    """Append, read and attention as one graph over a filled cache.  Between replays lengths go up and down, from none to
    rows of many parts, and rows come and go, so that the schedule of each replay is another one and its joins
    count from what the one before has left; eager work in between."""
    say(f"case quant-replay n={n} heads={H}/{K} bits={bits}")
    D, P = 128, 16
    blocks = most // P
    caches = [Q.QuantKV.zeros(n_req * blocks, P, K, D, dt, bits) for _ in range(2)]
    c = caches[0]
    table = torch.randperm(n_req * blocks, generator=torch.Generator().manual_seed(n)).int().view(n_req, blocks)
    dev_table = table.cuda()
    g = torch.Generator(device="cuda").manual_seed(0)
    fill = torch.randn(n_req * most, 2 * K * D, generator=g, device="cuda").to(dt)
    for cache in caches:
        Q.lora_quant_append(None, None, fill[:, :K * D], fill[:, K * D:], cache, torch.arange(n_req * most, dtype=torch.int32, device="cuda"))
    rope, works = S.Rope.base(D), [Q.attention_workspace(n, H, c) for _ in range(2)]
    x = torch.zeros(n, (H + 2 * K) * D, dtype=dt, device="cuda")
    lens, slots, pos, req = (torch.zeros(n, dtype=torch.int32, device="cuda") for _ in range(4))
    q, k, v = x[:, :H * D], x[:, H * D:(H + K) * D], x[:, (H + K) * D:]
    bufs = [[torch.zeros(n, w, dtype=dt, device="cuda") for w in (H * D, K * D, K * D, H * D)] +
            [torch.zeros(n, H, device="cuda")] for _ in range(2)]

    def step(i):
        qo, ko, vo, out, lse = bufs[i]
        Q.lora_quant_append(qo, q, k, v, caches[i], slots, rope=rope, positions=pos)
        Q.lora_quant_read(ko, vo, caches[i], slots)
        Q.lora_quant_attention(out, qo, caches[i], dev_table, lens, works[i], req=req, lse=lse)

    r = random.Random(n)
    now = {}

    def tokens(i):
        x.copy_(torch.randn(n, (H + 2 * K) * D, generator=g, device="cuda").to(dt))
        rows = r.sample(range(n), min(n, n_req))
        who = r.sample(range(n_req), len(rows))
        ln, rq = [-1] * n, [-1] * n
        for row, w in zip(rows, who):
            if r.random() < 0.8:
                rq[row], ln[row] = w, r.choice([1, 17, 64, 65, 300, most, most - 1, r.randrange(1, most + 1)])
        now.update(lens=ln, req=rq)
        p = [max(a - 1, 0) for a in ln]
        for t, values in ((lens, ln), (req, rq), (pos, p),
                          (slots, [int(table[w, a // P]) * P + a % P if w >= 0 else -1 for w, a in zip(rq, p)])):
            t.copy_(ints(values))

    tokens(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(0)
    torch.cuda.current_stream().wait_stream(side)
    step(1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(0)
    seen = set()
    for i in range(1, 13):
        tokens(i)
        seen.add(tuple(now["lens"]))
        graph.replay()
        step(1)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(*bufs)), i
        assert all(torch.equal(s, t) for s, t in zip(*map(bytes_of, caches)))
        assert not any(bool(w[:COUNTERS].any()) for w in works)
    assert len(seen) == 12
    want = QR.attention(bufs[0][0].cpu().reshape(n, H, D), *(cells(c, what).to(dt) for what in "kv"), table, now["lens"],
                        now["req"], 1 / math.sqrt(D), 0, H)
    for i, w in enumerate(want):
        if w is not None:
            close(bufs[0][3][i].cpu().reshape(H, D), w[0], w[2], f"row {i} out")
            close(bufs[0][4][i].cpu(), w[1], w[3], f"row {i} lse")
    assert any(w is not None for w in want)
