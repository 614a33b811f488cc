"""GPU: sampling (lora_sample.h) against its definition, at the sizes, settings and values where it can go wrong."""
import decimal
import math
import random

import pytest
import torch

from segmented_gather_matmul_amd import binding as B
from segmented_gather_matmul_amd import sample as SA
from segmented_gather_matmul_amd import step as S
from tests import sample_ref as SR
from tests.gpu_cases import say
from tests.test_gpu_step import ints

pytestmark = pytest.mark.gpu
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()
    yield


def real(v):
    return torch.tensor(v, dtype=torch.float32, device="cuda")


class Draw:
    """Rows of logits and settings; every output entry starts as a mark."""

    def __init__(self, logits, t=None, k=None, p=None, m=None, u=None, rows=None):
        self.x, self.rows = logits, rows
        n = logits.shape[0] if rows is None else len(rows)
        fill = lambda v, d: [d] * n if v is None else list(v) if isinstance(v, (list, tuple)) else [v] * n
        g = random.Random(n * 7 + logits.shape[1])
        self.t, self.k, self.p, self.m = fill(t, 1.0), fill(k, 0), fill(p, 1.0), fill(m, 0.0)
        self.u = [g.random() for _ in range(n)] if u is None else fill(u, 0.0)
        f = lambda v: [float(torch.tensor(x, dtype=torch.float32)) for x in v]      # as the kernel gets them
        self.t, self.p, self.m, self.u = f(self.t), f(self.p), f(self.m), f([min(x, 1 - 2.0 ** -24) if 0 <= x < 1 else x for x in self.u])
        self.n = n

    def run(self, dev=None, work=None):
        self.token = torch.full((self.n + 3,), -77, dtype=torch.int32, device="cuda")
        self.logprob = torch.full((self.n + 3,), 55.0, device="cuda")
        x = self.x.cuda() if dev is None else dev
        work = SA.sample_workspace(self.n, x.shape[1]) if work is None else work
        SA.lora_sample(self.token[:self.n], x, real(self.u), work, temperature=real(self.t), top_k=ints(self.k),
                       top_p=real(self.p), min_p=real(self.m), rows=None if self.rows is None else ints(self.rows),
                       logprob=self.logprob[:self.n])
        return self

    def check(self, what=""):
        torch.cuda.synchronize()
        tok, lp = self.token.tolist(), self.logprob.double().tolist()
        for i in range(self.n):
            src = i if self.rows is None else self.rows[i]
            want = SR.sample(self.x[src], self.t[i], self.k[i], self.p[i], self.m[i], self.u[i]) if 0 <= src < self.x.shape[0] else None
            case = f"{what} row {i}: t={self.t[i]} k={self.k[i]} p={self.p[i]} m={self.m[i]} u={self.u[i]}"
            if want is None:
                assert (tok[i], lp[i]) == (-77, 55.0), case
                continue
            assert tok[i] == want[0], f"{case}: {tok[i]}, not {want[0]}"
            assert lp[i] == want[1] or abs(lp[i] - want[1]) <= want[2], f"{case}: logprob {lp[i]}, not {want[1]}"
        assert tok[self.n:] == [-77] * 3 and lp[self.n:] == [55.0] * 3
        return self


def settings(n, seed):
    g = random.Random(seed)
    return dict(t=[g.choice([0.0, 0.1, 0.6, 0.8, 1.0, 1.0, 1.5, 5.0]) for _ in range(n)],
                k=[g.choice([0, 0, 1, 2, 40, 50, 1000, 10 ** 6, 2 ** 31 - 1]) for _ in range(n)],
                p=[g.choice([1.0, 1.0, 0.95, 0.9, 0.5, 0.1, 0.0, 1e-6]) for _ in range(n)],
                m=[g.choice([0.0, 0.0, 0.02, 0.3, 1.0]) for _ in range(n)])


def logits(n, V, dt, seed, spikes=8, gain=2.0):
    g = torch.Generator().manual_seed(seed)
    x = gain * torch.randn(n, V, generator=g)
    for _ in range(spikes):
        x[torch.arange(n), torch.randint(0, V, (n,), generator=g)] += 8 * torch.rand(n, generator=g)
    return x.to(dt)


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 63, 64, 65, 511, 512, 513, 1000, 4097, 32000, 50257, 131072])
def test_draws_match_the_definition(V, dt):
    say(f"case sample V={V} {dt}")
    n = 48 if V <= 4097 else 16
    Draw(logits(n, V, TYPES[dt], V), **settings(n, V)).run().check(f"V={V}")


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("kind", ["none", "k", "p", "m", "kp"])
def test_one_filter_at_a_time_over_flat_and_peaked_rows(kind, dt):
    say(f"case sample-filter {kind} {dt}")
    g = random.Random(1)
    for gain in (0.0, 0.01, 0.5, 3.0, 30.0):
        n = 24
        kw = {}
        if "k" in kind:
            kw["k"] = [g.choice([1, 2, 3, 17, 100, 999, 1000, 1500, 2999, 3000, 3001]) for _ in range(n)]
        if "p" in kind:
            kw["p"] = [g.choice([0.0, 1e-7, 0.01, 0.25, 0.5, 0.9, 0.99, 0.999999, 1.0]) for _ in range(n)]
        if kind == "m":
            kw["m"] = [g.choice([1e-12, 1e-6, 0.01, 0.5, 0.99, 1.0]) for _ in range(n)]
        Draw(logits(n, 3000, TYPES[dt], 5, gain=gain), t=[g.choice([0.3, 1.0, 4.0]) for _ in range(n)], **kw).run().check(f"gain {gain}")


@pytest.mark.parametrize("dt", list(TYPES))
def test_equal_logits_go_by_index(dt):
    """Rows of few values: borders inside classes of equals, -0 among 0."""
    say(f"case sample-ties {dt}")
    g = torch.Generator().manual_seed(3)
    r = random.Random(3)
    n, V = 64, 2500
    x = torch.randint(-2, 3, (n, V), generator=g).float() * 0.5
    x[:8] = 0.0
    x[8:16] = torch.where(torch.rand(8, V, generator=g) < 0.5, 0.0, -0.0)
    x[16:24] = -1.0
    x[20:24, 700:710] = 3.0
    kw = dict(k=[r.choice([0, 1, 2, 5, 500, 1249, 1250, 1251, 2499]) for _ in range(n)],
              p=[r.choice([1.0, 0.999, 0.5, 0.25, 0.0004, 0.3]) for _ in range(n)],
              u=[r.choice([0.0, 0.25, 0.5, 0.75, 1 - 2.0 ** -24, r.random()]) for _ in range(n)],
              t=[r.choice([0.0, 0.5, 1.0, 2.0]) for _ in range(n)], m=[r.choice([0.0, 0.5, 1.0]) for _ in range(n)])
    Draw(x.to(TYPES[dt]), **kw).run().check("ties")


@pytest.mark.parametrize("dt", list(TYPES))
def test_masked_infinite_and_nan_logits(dt):
    say(f"case sample-masked {dt}")
    inf, nan, V = math.inf, math.nan, 700
    x = logits(24, V, torch.float32, 9)
    x[0] = -inf
    x[1] = nan
    x[2, ::2], x[2, 1::2] = nan, -inf
    x[3] = -inf
    x[3, 699] = -5.0
    x[4, 17] = inf
    x[5, 100:200] = inf
    x[6, 3], x[6, 4] = inf, nan
    x[7:12][torch.rand(5, V, generator=torch.Generator().manual_seed(1)) < 0.97] = -inf
    x[12:16, 5:] = nan
    x[16] = torch.finfo(TYPES[dt]).max
    x[17] = torch.finfo(TYPES[dt]).min
    x[17, 9] = torch.finfo(TYPES[dt]).max
    x[18] = torch.finfo(TYPES[dt]).smallest_normal * torch.rand(V)
    x[19] = inf
    x[20, 5] = -nan
    for seed in range(3):
        kw = settings(24, seed)
        if seed == 0:
            kw = {}
        if seed == 1:
            kw["k"], kw["p"], kw["t"] = [50] * 24, [0.9] * 24, [1.0] * 24
        Draw(x.to(TYPES[dt]), **kw).run().check(f"seed {seed}")


@pytest.mark.parametrize("t", [1e-45, 1e-38, 1e-6, 0.01, 100.0, 1e10, 3e38])
def test_extreme_temperatures(t):
    say(f"case sample-temperature {t}")
    for dt in TYPES.values():
        Draw(logits(12, 2000, dt, 4), t=t, k=[0, 50, 0] * 4, p=[1.0, 0.9, 0.5, 1.0] * 3).run().check(f"t={t}")


def test_rows_with_settings_out_of_range_are_left_alone():
    say("case sample-range")
    nan, inf = math.nan, math.inf
    t = [-1.0, nan, inf, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0, -0.0]
    k = [0, 0, 0, -1, 0, 0, 0, 0, 0, 0, 0, 0, 3, 0]
    p = [1.0] * 4 + [-0.1, 1.0001, nan] + [1.0] * 7
    m = [0.0] * 7 + [-0.5, 1.5, nan] + [0.0] * 4
    u = [0.5] * 10 + [1.0, -0.5, 0.5, 0.5]
    Draw(logits(14, 300, torch.float16, 1), t, k, p, m, u).run().check("range")
    d = Draw(logits(14, 300, torch.float16, 1), u=[nan] * 13 + [0.0])
    d.u[:13] = [nan] * 13
    d.run().check("u")
    rows = [0, -1, 14, 13, 2 ** 31 - 1, -(2 ** 31), 5, 5, 0]
    Draw(logits(14, 300, torch.bfloat16, 2), rows=rows, t=[1.0] * 9).run().check("rows")


@pytest.mark.parametrize("dt", list(TYPES))
def test_unaligned_and_strided_rows(dt):
    """Rows of any alignment inside a buffer whose other entries must not be read as logits."""
    say(f"case sample-strides {dt}")
    for V, ld, off in ((1001, 1009, 3), (64, 67, 1), (513, 1024, 7), (5, 6, 1), (9, 11, 2), (1, 3, 1)):
        n = 11
        x = logits(n, V, TYPES[dt], V + ld)
        buf = torch.full((off + n * ld + 64,), math.inf).to(TYPES[dt]).cuda()
        dev = buf[off:off + n * ld].view(n, ld)[:, :V]
        dev.copy_(x)
        Draw(x, **settings(n, V)).run(dev).check(f"ld {ld}")


def test_the_largest_vocabulary_and_one_beyond_a_segment_table():
    say("case sample-large")
    for V in (SA.MAX_VOCAB, 600001):
        x = logits(3, V, torch.float16, 1)
        Draw(x, t=[1.0, 0.8, 1.2], k=[0, 1000, 0], p=[1.0, 1.0, 0.9], u=[0.999, 0.5, 0.75]).run().check(f"V={V}")


def test_rows_beyond_32_bit_offsets():
    say("case sample-offsets")
    V, ld = 1000, (1 << 31) + 24
    buf = torch.zeros(2 * ld + V, dtype=torch.float16, device="cuda")
    dev = buf.as_strided((3, V), (ld, 1))
    x = logits(3, V, torch.float16, 2)
    dev.copy_(x)
    Draw(x, k=[0, 5, 0], p=[1.0, 1.0, 0.7]).run(dev).check("far")


def test_draws_follow_the_distribution():
    """Over evenly spread u, each token is drawn as often as its share of the mass says: exactly, to one draw a border."""
    say("case sample-share")
    V, n = 40, 4000
    x = logits(1, V, torch.float32, 6, spikes=0, gain=1.0)
    d = Draw(x, t=0.9, u=[(i + 0.5) / n for i in range(n)], rows=[0] * n).run()
    torch.cuda.synchronize()
    got = torch.bincount(d.token[:n].long().cpu(), minlength=V).double()
    want = n * torch.softmax(x[0].double() / d.t[0], 0)
    assert bool(((got - want).abs() <= 1.0 + 1e-6).all())


def test_calls_on_no_rows_and_without_options():
    e = lambda dt: torch.empty(0, dtype=dt, device="cuda")
    SA.lora_sample(e(torch.int32), torch.empty(0, 50, device="cuda"), e(torch.float32), SA.sample_workspace(0, 50))
    x = logits(5, 333, torch.float32, 3)
    token, u = torch.zeros(5, dtype=torch.int32, device="cuda"), [0.1, 0.3, 0.5, 0.7, 0.9]
    SA.lora_sample(token, x.cuda(), real(u), SA.sample_workspace(5, 333))
    u32 = real(u).double().tolist()
    assert token.tolist() == [SR.sample(x[i], 1.0, 0, 1.0, 0.0, u32[i])[0] for i in range(5)]


def test_the_python_and_the_compiled_calls_are_the_same(monkeypatch):
    say("case sample-python")
    got = []
    for fast in (S._fast, None):
        monkeypatch.setattr(S, "_fast", fast)
        for dt in TYPES.values():
            d = Draw(logits(9, 1001, dt, 3), rows=[8, 7, 6, 5, 4, 3, 2, 1, 0], **settings(9, 3)).run().check("python")
            got.append((d.token.tolist(), d.logprob.tolist()))
    assert got[:3] == got[3:]


def test_repeated_and_concurrent_calls_are_the_same():
    say("case sample-streams")
    draws = [Draw(logits(20, 40000, torch.bfloat16, i), **settings(20, i)) for i in range(3)]
    dev, works = [d.x.cuda() for d in draws], [SA.sample_workspace(20, 40000) for _ in draws]
    streams = [torch.cuda.Stream() for _ in draws]
    first = None
    torch.cuda.synchronize()
    for _ in range(3):
        for d, x, w, st in zip(draws, dev, works, streams):
            with torch.cuda.stream(st):
                d.run(x, w)
        torch.cuda.synchronize()
        now = [(d.token.tolist(), d.logprob.tolist()) for d in draws]
        first = first or now
        assert now == first
    for d in draws:
        d.check("stream")


def test_captured_and_replayed_with_other_logits_and_settings():
    say("case sample-graph")
    n, V = 6, 5003
    d = [Draw(logits(n, V, torch.float16, i), **settings(n, i)) for i in range(6)]
    x, work = torch.empty(n, V, dtype=torch.float16, device="cuda"), SA.sample_workspace(n, V)
    t, k, p, m, u = (torch.zeros(n, dtype=dt, device="cuda") for dt in (torch.float32, torch.int32) + (torch.float32,) * 3)
    token, lp = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros(n, device="cuda")
    call = lambda: SA.lora_sample(token, x, u, work, temperature=t, top_k=k, top_p=p, min_p=m, logprob=lp)

    def fill(c):
        for a, v in ((x, c.x.cuda()), (t, real(c.t)), (k, ints(c.k)), (p, real(c.p)), (m, real(c.m)), (u, real(c.u))):
            a.copy_(v)

    fill(d[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for c in d:
        fill(c)
        graph.replay()
        torch.cuda.synchronize()
        got = token.tolist()
        c.run().check("eager")
        assert got == c.token[:n].tolist() and lp.tolist() == c.logprob[:n].tolist()


# (logit, temperature, u): with the largest logit 0 behind it, floor(u M) lies below the logit's weight by so little that
# one smaller by 2^-36.62 of itself (nine terms of the series) gives the other token, and by so much that none right to
# 2^-37 does.
NEAR_A_BORDER = [("-0x1.f8939cp-3", "0x1.6cp-1", "0x1.a8291cp-2"), ("-0x1.c0d9a8p-3", "0x1.44p-1", "0x1.a836c6p-2"),
                 ("-0x1.94834cp-3", "0x1.24p-1", "0x1.a83720p-2"), ("-0x1.6aef60p-2", "0x1.06p+0", "0x1.a8383cp-2"),
                 ("-0x1.811fd2p-2", "0x1.16p+0", "0x1.a836cap-2"), ("-0x1.9d14bcp-2", "0x1.2ap+0", "0x1.a82974p-2"),
                 ("-0x1.ad7650p-2", "0x1.36p+0", "0x1.a8366ep-2"), ("-0x1.df4ceep-2", "0x1.5ap+0", "0x1.a83806p-2"),
                 ("-0x1.e4b824p-2", "0x1.5ep+0", "0x1.a83d94p-2"), ("-0x1.110d7ap-1", "0x1.8ap+0", "0x1.a82b6cp-2"),
                 ("-0x1.50a33ep-1", "0x1.e6p+0", "0x1.a836c6p-2"), ("-0x1.b7361ep-1", "0x1.3dp+1", "0x1.a833d6p-2")]


@pytest.mark.parametrize("V,k,p", [(2, 0, 1.0), (3, 2, 1.0), (700, 0, 0.99999994), (900, 200, 1.0), (40000, 0, 1.0), (40000, 40, 1.0)])
def test_weights_are_right_to_their_bound_where_the_series_ends(V, k, p):
    """Half way between two powers of 2, where the exponential's series is furthest off."""
    say(f"case sample-weight V={V} k={k} p={p}")
    with decimal.localcontext() as ctx:
        ctx.prec = 50
        dec, unit = decimal.Decimal, decimal.Decimal(2) ** 40
        l, t, u = ([float.fromhex(c[i]) for c in NEAR_A_BORDER] for i in range(3))
        for a, b, c in zip(l, t, u):
            assert [float(torch.tensor(x, dtype=torch.float32)) for x in (a, b, c)] == [a, b, c]
            w = (dec(a) / dec(b)).exp() * unit
            least, most = int(w * (1 - dec(2) ** -37)), int(w * (1 + dec(2) ** -37))
            assert all(int(dec(c) * (unit + m)) < m for m in range(least, most + 1))
            low = int(w * (1 - dec("9.44e-12")))
            assert int(dec(c) * (unit + low)) >= low
    x = torch.full((len(l), V), -math.inf)
    x[:, 0], x[:, 1] = torch.tensor(l), 0.0
    d = Draw(x, t=t, k=k, p=p, u=u).run()
    torch.cuda.synchronize()
    assert d.token[:len(l)].tolist() == [0] * len(l)
