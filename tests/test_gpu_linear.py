"""moe_linear_q against the formats' definition in 64 bits: bit for bit where
every sum is exact in fp32, within the derived bound on random inputs, and the
calls that the documentation allows (strides, captured graphs, streams)."""
import numpy as np
import pytest
import torch

import synth
from oracle import moe_oracle as mo
from sparse_moe_router_amd import api
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu
FORMATS = ("q4_sym_g32", "q3_sym_g32", "q2_asym_g32")
PACK = {"q4_sym_g32": synth.pack_q4, "q3_sym_g32": synth.pack_q3, "q2_asym_g32": synth.pack_q2}
TOP = {"q4_sym_g32": 15, "q3_sym_g32": 7, "q2_asym_g32": 3}
DT = {"f32": torch.float32, "bf16": torch.bfloat16}

# (tokens, rows, cols): one token to a prompt, one group to many, odd sizes
SIZES = [(1, 1, 32), (1, 17, 96), (1, 300, 2048), (2, 33, 64), (3, 100, 160), (4, 70, 2048), (5, 129, 2016), (8, 64, 768),
         (13, 257, 224), (16, 100, 1024), (17, 61, 544), (33, 130, 512), (64, 96, 4096), (65, 200, 160), (130, 257, 96),
         (300, 129, 2080)]
# sizes that take the kernels of many rows: several rounds of a block, tiles of two row groups, x that does not fit LDS
MANY = [(1, 70001, 96), (3, 40001, 64), (4, 33, 20000), (6, 8200, 96), (16, 9001, 544), (12, 8200, 1664), (130, 4200, 96),
        (1030, 4100, 64), (20, 12300, 96), (16, 8193, 3712), (9, 8192, 1280), (4, 4200, 2048), (3, 40001, 288),
        (2, 9000, 2080), (16, 4100, 544), (6, 8200, 704), (11, 8200, 2592), (7, 8193, 7200), (20, 33000, 96),
        (70, 12300, 160), (200, 5000, 96), (64, 17000, 96), (500, 1030, 288), (100, 40000, 64)]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    api.lib()


def bf16_dev(v):
    return torch.from_numpy(synth.f32_to_bf16_bits(v.astype(np.float32)).view(np.int16)).to(gu.DEV).view(torch.bfloat16)


class Case:
    """One projection: codes, scales, minima and bias in fp64 and on the device."""

    def __init__(self, qfmt, n, k, seed, exact, act="bf16", out="f32", bias=True):
        r = np.random.default_rng(seed)
        self.qfmt, self.n, self.k, self.act = qfmt, n, k, act
        u = r.integers(0, TOP[qfmt] + 1, (n, k)).astype(np.uint8)
        g = k // 32
        if exact:  # scales and minima with the full 11 bits of fp16 (or a power of two for wide fp32 x)
            s = (2.0 ** r.integers(-3, 1, (n, g)) if act == "f32" else r.integers(1, 2048, (n, g)) / 1024.0)
            m = (2.0 ** r.integers(-3, 1, (n, g)) if act == "f32" else r.integers(-2047, 2048, (n, g)) / 1024.0)
            b = r.integers(-1000, 1001, n) / 8.0
        else:
            s = 0.02 * (0.5 + r.random((n, g)))
            m = -1.5 * s * (0.9 + 0.2 * r.random((n, g)))
            b = r.standard_normal(n)
        s16, m16 = s.astype(np.float16), m.astype(np.float16) if qfmt == "q2_asym_g32" else None
        codes = PACK[qfmt](u)
        self.w = mo.dequant(codes, s16.view(np.uint16), None if m16 is None else m16.view(np.uint16), qfmt)
        self.s, self.m = s16.astype(np.float64), 0.0 if m16 is None else np.abs(m16.astype(np.float64))
        self.b = b.astype(np.float32).astype(np.float64) if bias else np.zeros(n)
        dev = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(gu.DEV)
        self.lin = api.Linear(rows=n, cols=k, qfmt=qfmt, act=act, out=out, codes=dev(codes), scales=dev(s16.view(np.int16)),
                              mins=None if m16 is None else dev(m16.view(np.int16)),
                              bias=dev(b.astype(np.float32)) if bias else None)

    def x_dev(self, v):
        return bf16_dev(v) if self.act == "bf16" else torch.from_numpy(v.astype(np.float32)).to(gu.DEV)

    def ref(self, x):
        return x @ self.w.T + self.b

    def bound(self, x):
        """Worst case of an fp32 evaluation of the group form.  The terms of one
        weight are at most F s |x| (+ 2 |m| |x|): the code with its offset,
        s (2^bits + u), and the offset taken off again (4-bit: 16 + 15 + 24 = 55,
        3-bit: 8 + 7 + 12 = 27, 2-bit: 4 + 3 + 4 = 11).  A sum of j fp32 terms in
        any order is off by at most (j - 1) 2^-24 sum |terms| (1 + small); here
        j <= 3 x 32 + 32 within a group (three parts of an fp32 x and the offset),
        one per group, and at most 20 more for the joins, the scale's product,
        the bias and the one rounding of a 2-bit weight in the definition."""
        f = {"q4_sym_g32": 55, "q3_sym_g32": 27, "q2_asym_g32": 11}[self.qfmt]
        ax = np.abs(x).reshape(x.shape[0], -1, 32).sum(axis=2)  # [T][G]
        mag = ax @ (f * self.s + 2 * self.m).T + np.abs(self.b)
        return (128 + self.k // 32 + 20) * 2.0 ** -24 * 1.01 * mag


def call(c, xd, T, out="f32", ldy=None, fill=7.0):
    ldy = ldy or c.n
    y = torch.full((T, ldy), fill, dtype=DT[out], device=gu.DEV)
    api.moe_linear_q(c.lin, xd, T, y[:, :c.n])
    torch.cuda.synchronize()
    return y


def sparse_x(r, T, k, act):
    """A few small whole numbers a row (bf16), or one of 18 bits (fp32, three bf16 parts): every sum is exact."""
    x = np.zeros((T, k))
    for t in range(T):
        at = r.choice(k, size=1 if act == "f32" else min(12, k), replace=False)
        x[t, at] = r.integers(-(1 << 18) + 1, 1 << 18) | 1 if act == "f32" else r.choice([-2, -1, 1, 2], size=at.size)
    return x


@pytest.mark.parametrize("act", ("bf16", "f32"))
@pytest.mark.parametrize("qfmt", FORMATS)
def test_exact_sums(qfmt, act):
    """Inputs whose every partial sum fits 24 bits: y equals the definition bit
    for bit, so no weight or activation lost a bit on the way.  (bf16: at most
    12 x 2 x 2047 x 31 < 2^24 units of 2^-14; fp32: 2^18 x 31 < 2^23 units.)"""
    for i, (T, n, k) in enumerate(SIZES + MANY):
        gu.say(f"linear exact {qfmt} {act} T={T} N={n} K={k}")
        c = Case(qfmt, n, k, 100 + i, True, act, bias=False)
        x = sparse_x(np.random.default_rng(i), T, k, act)
        y = call(c, c.x_dev(x), T).cpu().numpy().astype(np.float64)
        assert np.array_equal(y, c.ref(x)), (T, n, k, np.abs(y - c.ref(x)).max())


@pytest.mark.parametrize("act,out", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("qfmt", FORMATS)
def test_random_values(qfmt, act, out):
    """Normal x with a few large channels and a mean: within the fp32 bound, plus
    half a step of bf16 (2^-8 of the value) where y is bf16."""
    for i, (T, n, k) in enumerate(SIZES):
        gu.say(f"linear random {qfmt} {act}->{out} T={T} N={n} K={k}")
        r = np.random.default_rng(500 + i)
        c = Case(qfmt, n, k, 200 + i, False, act, out)
        x = (0.3 + r.standard_normal((T, k))) * np.where(r.random(k) < 0.02, 10.0, 1.0)
        x = mo.round_act(x, act)
        y = call(c, c.x_dev(x), T, out).float().cpu().numpy().astype(np.float64)
        want = c.ref(x)
        lim = c.bound(x)
        if out == "bf16":
            lim = lim + 2.0 ** -8 * (np.abs(want) + lim)
        else:
            lim = lim + 2.0 ** -24 * (np.abs(want) + lim)
        worst = (np.abs(y - want) / lim).max()
        assert worst <= 1.0, (T, n, k, worst)


@pytest.mark.parametrize("act", ("bf16", "f32"))
@pytest.mark.parametrize("qfmt", FORMATS)
def test_random_values_many_rows(qfmt, act):
    for i, (T, n, k) in enumerate(MANY):
        gu.say(f"linear random {qfmt} {act} T={T} N={n} K={k}")
        r = np.random.default_rng(700 + i)
        c = Case(qfmt, n, k, 300 + i, False, act, "f32")
        x = mo.round_act(0.3 + r.standard_normal((T, k)), act)
        y = call(c, c.x_dev(x), T).cpu().numpy().astype(np.float64)
        want = c.ref(x)
        lim = c.bound(x)
        assert (np.abs(y - want) <= lim + 2.0 ** -24 * (np.abs(want) + lim)).all(), (T, n, k)


@pytest.mark.parametrize("T,n,k", ((1, 75, 160), (4, 75, 160), (7, 75, 160), (40, 75, 160), (130, 75, 160), (4, 8201, 1056),
                                   (7, 8201, 608), (14, 8201, 608), (16, 4101, 544)))
def test_strides_and_untouched_bytes(T, n, k):
    """x and y inside wider buffers (rows of x at odd multiples of 16 bytes, y at
    an odd element): same values, and nothing between the rows or behind them is
    written."""
    for act, out in (("bf16", "bf16"), ("f32", "f32")):
        c = Case("q4_sym_g32", n, k, 3, False, act, out)
        x = mo.round_act(np.random.default_rng(T).standard_normal((T, k)), act)
        plain = call(c, c.x_dev(x), T, out)
        wide = torch.full((T, k + 24), float("nan"), dtype=DT[act], device=gu.DEV)
        wide[:, 8:8 + k] = c.x_dev(x)
        y = torch.full((T + 2, n + 6), 7.0, dtype=DT[out], device=gu.DEV)
        api.moe_linear_q(c.lin, wide[:, 8:8 + k], T, y[1:, 3:3 + n])
        torch.cuda.synchronize()
        assert torch.equal(y[1:T + 1, 3:3 + n], plain)
        y[1:T + 1, 3:3 + n] = 7.0
        assert torch.all(y == 7.0)


@pytest.mark.parametrize("T,n,k", ((2, 130, 96), (4, 130, 96), (16, 130, 96), (30, 130, 96), (100, 130, 96), (4, 8200, 1056),
                                   (8, 8200, 544), (16, 8200, 544), (16, 4100, 544)))
@pytest.mark.parametrize("act", ("bf16", "f32"))
def test_bad_rows_stay_alone(T, n, k, act):
    """A NaN or an infinity in one token's x leaves the other tokens' rows with the bits they have without it."""
    for qfmt in FORMATS:
        c = Case(qfmt, n, k, 11, False, act)
        x = mo.round_act(np.random.default_rng(T).standard_normal((T, k)), act)
        want = call(c, c.x_dev(x), T)
        bad = x.copy()
        bad[0, 40], bad[T - 1, k - 1] = np.nan, np.inf
        got = call(c, c.x_dev(bad), T)
        assert torch.equal(got[1:T - 1], want[1:T - 1])
        assert not torch.isfinite(got[0]).any() and not torch.isfinite(got[T - 1]).any()


def test_rows_do_not_depend_on_the_batch_inside_one_kernel():
    """The same token gives the same bits at every position of a batch."""
    for qfmt in FORMATS:
        c = Case(qfmt, 200, 512, 5, False)
        x = mo.round_act(np.random.default_rng(1).standard_normal((1, 512)), "bf16")
        for T in (3, 16, 64, 150):
            y = call(c, c.x_dev(np.repeat(x, T, axis=0)), T)
            assert torch.equal(y, y[:1].expand_as(y))


def test_large_rows_of_codes():
    """More rows than 2^31 bytes of fp32 weights would hold in one matrix (offsets past 31 bits): the last rows are right."""
    n, k = 600_000, 8192  # 2.46 GB of 4-bit codes
    r = np.random.default_rng(9)
    codes = torch.zeros((n, k // 2), dtype=torch.uint8, device=gu.DEV)
    codes.fill_(0x88)  # u = 8: weight 0
    scales = torch.zeros((n, k // 32), dtype=torch.float16, device=gu.DEV)
    rows = [0, 299_999, 524_287, 524_288, n - 1]
    u = r.integers(0, 16, (len(rows), k)).astype(np.uint8)
    s = (0.02 * (0.5 + r.random((len(rows), k // 32)))).astype(np.float16)
    for i, row in enumerate(rows):
        codes[row] = torch.from_numpy(synth.pack_q4(u[i:i + 1])[0]).to(gu.DEV)
        scales[row] = torch.from_numpy(s[i]).to(gu.DEV)
    lin = api.Linear(rows=n, cols=k, qfmt="q4_sym_g32", act="bf16", codes=codes, scales=scales.view(torch.int16))
    w = mo.dequant(synth.pack_q4(u), s.view(np.uint16), None, "q4_sym_g32")
    for T in (1, 6, 70):
        x = mo.round_act(r.standard_normal((T, k)), "bf16")
        y = torch.full((T, n), float("nan"), dtype=torch.float32, device=gu.DEV)
        gu.say(f"large T={T}")
        api.moe_linear_q(lin, bf16_dev(x), T, y)
        got = y[:, torch.tensor(rows, device=gu.DEV)].cpu().numpy()
        want = x @ w.T
        assert np.abs(got - want).max() <= 1e-3 * np.sqrt(np.mean(want ** 2))  # a wrong row is off by the RMS itself
        rest = torch.ones(n, dtype=torch.bool, device=gu.DEV)
        rest[rows] = False
        assert torch.all(y[:, rest] == 0.0)
        del y


@pytest.mark.parametrize("n,k", ((300, 512), (8300, 2080), (4300, 2112)))
def test_graph_replays_and_streams(n, k):
    """Captured calls of every kernel, replayed with new inputs and the eager call in between; two streams at once."""
    c = Case("q4_sym_g32", n, k, 21, False)
    r = np.random.default_rng(2)
    bufs = {T: (bf16_dev(mo.round_act(r.standard_normal((T, k)), "bf16")),
                torch.zeros((T, n), device=gu.DEV)) for T in (1, 4, 8, 12, 60, 140)}
    for T, (x, y) in bufs.items():
        api.moe_linear_q(c.lin, x, T, y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        for T, (x, y) in bufs.items():
            api.moe_linear_q(c.lin, x, T, y)
    for rep in range(4):
        for T, (x, y) in bufs.items():
            x.copy_(bf16_dev(mo.round_act(r.standard_normal((T, k)), "bf16")))
            y.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        for T, (x, y) in bufs.items():
            assert torch.equal(call(c, x, T), y), (rep, T)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    want = {T: call(c, x, T) for T, (x, _) in bufs.items()}
    outs = {T: [torch.zeros((T, n), device=gu.DEV) for _ in range(6)] for T in bufs}
    torch.cuda.synchronize()
    for i in range(6):
        for T, (x, _) in bufs.items():
            api.moe_linear_q(c.lin, x, T, outs[T][i], stream=(s1, s2)[(i + T) % 2])
    torch.cuda.synchronize()
    for T in bufs:
        for y in outs[T]:
            assert torch.equal(y, want[T])


def test_bound_call_and_an_expert_matrix():
    """bind_linear_q gives the call's bits again and again; one expert's gate matrix of a layer is a projection as it is
    and agrees with moe_dequant."""
    spec = synth.LayerSpec("lin", 256, 4, 2, 96, 3, "q3_sym_g32", "bf16", 256 ** -0.5, 1.1, family=301)
    ld = synth.gen_layer(spec)
    p = ld.routed.gate
    codes = torch.from_numpy(p.codes[2:3]).to(gu.DEV)
    scales = torch.from_numpy(p.scales[2:3].view(np.int16)).to(gu.DEV)
    lin = api.Linear(rows=96, cols=256, qfmt=spec.qfmt, act="bf16", codes=codes, scales=scales)
    w = torch.empty((96, 256), device=gu.DEV)
    api.moe_dequant(codes, scales, None, spec.qfmt, 96, 256, w)
    x = synth.gen_x(spec)
    xd = gu.x_dev(x, spec.act)
    y = torch.zeros((3, 96), device=gu.DEV)
    f = api.bind_linear_q(lin, xd, 3, y)
    f()
    first = y.clone()
    y.zero_()
    f()
    torch.cuda.synchronize()
    assert torch.equal(first, y)
    want = x.values.astype(np.float64) @ w.cpu().numpy().astype(np.float64).T
    assert np.abs(y.cpu().numpy() - want).max() <= 1e-4 * np.sqrt(np.mean(want ** 2))
