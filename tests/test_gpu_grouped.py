"""GPU parity of the int8 products, the products grouped by expert with their gradients, and
the expert combine, against float64 (or exact integer) computations of their definitions.

Tolerance of a 16-bit product: the products of two bf16 / fp16 values are exact in fp32, so
a sum of C of them has at most C roundings of half a step of a partial sum, each at most
S = sum |a||b|: C * 2^-24 * S; then one rounding to the output type, half a step of the
result (plus half the smallest subnormal in fp16). Int8 sums and small-integer sums are exact,
so those tests ask for equal bits."""
import numpy as np
import pytest
import torch

from gpu_util import DEV

pytestmark = pytest.mark.gpu
nv = pytest.importorskip("nvfp4_quantized_moe_02_amd")

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
SENTINEL = 77.0


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def half_step(t):
    return torch.finfo(t).eps / 2


def rounding(ref, t):
    return ref.abs() * half_step(t) + (2.0 ** -25 if t == F16 else 0.0)


def close(got, ref, S, C, extra=0.0):
    """|got - ref| within C fp32 roundings of sums up to S and one rounding to got's type."""
    assert torch.isfinite(got).all()
    got, t = got.double().cpu(), got.dtype
    ref, S = ref.cpu(), S.cpu()
    acc = (C + extra) * 2.0 ** -24 * S
    bound = acc + (0.0 if t == F32 else 1.0) * rounding(ref.abs() + acc, t)
    err = (got - ref).abs()
    assert bool((err <= bound).all()), float((err / bound.clamp_min(1e-300)).max())


class Routing:
    """Sorted pairs with given numbers of rows per expert; the rest of T * topk are dropped."""

    def __init__(self, sizes, T, topk, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.sizes, self.T, self.topk, self.E = list(sizes), T, topk, len(sizes)
        self.rows, self.used = T * topk, sum(sizes)
        assert self.used <= self.rows
        perm = torch.randperm(self.rows, generator=g).to(torch.int32)
        pairs = torch.full((self.rows,), -1, dtype=torch.int32)
        at = 0
        for n in self.sizes:
            pairs[at:at + n] = torch.sort(perm[at:at + n]).values
            at += n
        off = torch.zeros(self.E + 1, dtype=torch.int32)
        off[1:] = torch.cumsum(torch.tensor(self.sizes), 0)
        self.pairs_cpu, self.off_cpu = pairs, off
        self.pairs, self.off = pairs.to(DEV), off.to(DEV)

    def spans(self):
        at = 0
        for e, n in enumerate(self.sizes):
            yield e, at, at + n
            at += n

    def src(self, gather):
        return (self.pairs_cpu[:self.used] // self.topk).long() if gather else torch.arange(self.used)


def draw(shape, t, seed, ints=False):
    g = torch.Generator().manual_seed(seed)
    v = torch.randint(-3, 4, shape, generator=g).float() if ints else torch.randn(shape, generator=g)
    return v.to(t)


def fwd_ref(x, w, r, src):
    out = torch.zeros(r.used, w.shape[1], dtype=torch.float64)
    S = torch.zeros_like(out)
    for e, a, b in r.spans():
        xe, we = x[src[a:b]].double(), w[e].double()
        out[a:b] = xe @ we.t()
        S[a:b] = xe.abs() @ we.abs().t()
    return out, S


def dx_ref(dy, w, r):
    out = torch.zeros(r.used, w.shape[2], dtype=torch.float64)
    S = torch.zeros_like(out)
    for e, a, b in r.spans():
        out[a:b] = dy[a:b].double() @ w[e].double()
        S[a:b] = dy[a:b].double().abs() @ w[e].double().abs()
    return out, S


def dw_ref(dy, x, r, src, N, K):
    out = torch.zeros(r.E, N, K, dtype=torch.float64)
    S = torch.zeros_like(out)
    for e, a, b in r.spans():
        d, xe = dy[a:b].double(), x[src[a:b]].double()
        out[e] = d.t() @ xe
        S[e] = d.abs().t() @ xe.abs()
    return out, S


# (rows per expert, topk, N, K): empty experts, single rows, tile edges, one expert, more
# experts than a block has threads, contraction lengths inside and across a K-block
CASES = [
    ([1], 1, 8, 8),
    ([0, 1, 0, 2], 1, 16, 40),
    ([5, 0, 17, 33], 2, 264, 72),
    ([128, 129, 127, 0, 64], 2, 136, 320),
    ([300, 0, 1], 1, 520, 264),
    ([31, 32, 33, 63, 65, 96, 97], 3, 80, 2056),
    ([1, 0] * 160, 1, 24, 96),
    ([0] * 700 + [3] + [0] * 299 + [2], 1, 56, 48),
    ([1100, 40], 4, 72, 136),
]
IDS = [f"E{len(c[0])}r{sum(c[0])}N{c[2]}K{c[3]}" for c in CASES]


def routing_of(case, drop=7, seed=1):
    sizes, topk, _, _ = case
    rows = sum(sizes) + drop
    return Routing(sizes, -(-rows // topk), topk, seed)


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("t", [BF16, F16])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_grouped_exact_on_small_integers(case, t, gather):
    """Forward and both gradients on integers of at most 3: every sum is exact in fp32."""
    r, (N, K) = routing_of(case), case[2:]
    x = draw((r.T if gather else r.rows, K), t, 2, ints=True)
    w, dy = draw((r.E, N, K), t, 3, ints=True), draw((r.rows, N), t, 4, ints=True)
    src, pairs = r.src(gather), r.pairs if gather else None
    xd, wd, dyd = x.to(DEV), w.to(DEV), dy.to(DEV)
    out = torch.full((r.rows, N), SENTINEL, device=DEV)
    nv.grouped_linear(xd, wd, r.off, pairs, r.topk, out=out)
    dx = torch.full((r.rows, K), SENTINEL, device=DEV)
    nv.grouped_linear_dx(dyd, wd, r.off, out=dx)
    dw = torch.full((r.E, N, K), SENTINEL, device=DEV)
    nv.grouped_linear_dw(dyd, xd, r.off, pairs, r.topk, out=dw)
    assert torch.equal(out[:r.used].double().cpu(), fwd_ref(x, w, r, src)[0]), "forward"
    assert torch.equal(dx[:r.used].double().cpu(), dx_ref(dy, w, r)[0]), "dx"
    assert torch.equal(dw.double().cpu(), dw_ref(dy, x, r, src, N, K)[0]), "dw"
    assert bool((out[r.used:] == SENTINEL).all()) and bool((dx[r.used:] == SENTINEL).all()), "rows behind the last"


# Loads that reach every tile of the forward product and of the gradients, with partial row
# tiles, column tiles and K-blocks in each: (rows per expert, topk, N, K)
LOADS = {
    "stream two groups": ([1, 2, 0, 1] * 15, 1, 520, 264),
    "stream 32 rows": ([20, 0, 31, 33, 100], 1, 136, 264),
    "64 x 64": ([200, 0, 65, 250, 1], 2, 264, 2056),
    "64 x 128": ([40, 1, 0, 33, 65, 2, 64, 7] * 5, 2, 1032, 136),
    "128 x 256": ([300, 60, 130, 1, 0, 515], 2, 5128, 328),
    "256 x 256": ([700, 2101], 1, 5640, 200),
    "256 x 256, one K-block": ([513, 1500], 1, 8200, 48),
    "gradients of few rows": ([1, 0, 3] * 80, 1, 264, 520),
    "gradients of many rows": ([1029, 2300, 31], 1, 520, 5640),
    "weights, 128 x 128": ([1100, 3000, 0], 1, 776, 1032),
    "weights of many experts": ([1, 0, 70] * 90 + [2113], 1, 136, 72),
}


@pytest.mark.parametrize("load", LOADS.values(), ids=LOADS.keys())
def test_every_tile_exact(load):
    r, (N, K) = routing_of(load), load[2:]
    src = r.src(True)
    for t in (BF16, F16):
        x, w, dy = draw((r.T, K), t, 2, ints=True), draw((r.E, N, K), t, 3, ints=True), draw((r.rows, N), t, 4, ints=True)
        xd, wd, dyd = x.to(DEV), w.to(DEV), dy.to(DEV)
        out = torch.full((r.rows, N), SENTINEL, device=DEV)
        nv.grouped_linear(xd, wd, r.off, r.pairs, r.topk, out=out)
        dx = torch.full((r.rows, K), SENTINEL, device=DEV)
        nv.grouped_linear_dx(dyd, wd, r.off, out=dx)
        dw = nv.grouped_linear_dw(dyd, xd, r.off, r.pairs, r.topk, out_dtype=F32)
        # sums of integers below 2^24: float32 products on the CPU are exact too
        for e, a, b in r.spans():
            xe, de = x[src[a:b]].float(), dy[a:b].float()
            assert torch.equal(out[a:b].cpu(), xe @ w[e].float().t()), ("forward", e)
            assert torch.equal(dx[a:b].cpu(), de @ w[e].float()), ("dx", e)
            assert torch.equal(dw[e].cpu(), de.t() @ xe), ("dw", e)
        assert bool((out[r.used:] == SENTINEL).all()) and bool((dx[r.used:] == SENTINEL).all())
    K = -(-K // 16) * 16
    q, sx = quantized(r.T, K, 3)
    w8, sw = quantized(r.E * (N + 1), K, 4)
    w8, sw = w8.reshape(r.E, N + 1, K), sw.reshape(r.E, N + 1)
    for od in (F32, F16):
        y = nv.grouped_linear_i8(q.to(DEV), sx.to(DEV), w8.to(DEV), sw.to(DEV), r.off, r.pairs, r.topk, out_dtype=od)
        for e, a, b in r.spans():
            acc = (q[src[a:b]].double() @ w8[e].double().t()).to(torch.int32)
            assert torch.equal(y[a:b].cpu(), scaled(acc, sx[src[a:b]], sw[e], od)), (e, od)


@pytest.mark.parametrize("T,N,K", [(2049, 4100, 144), (700, 9001, 528), (8200, 2048, 64)])
def test_linear_i8_of_many_rows(T, N, K):
    """The larger tiles with one expert (no offsets)."""
    x, sx = quantized(T, K, 1)
    w, sw = quantized(N, K, 2)
    for od in (BF16, F32):
        y = nv.linear_i8(x.to(DEV), sx.to(DEV), w.to(DEV), sw.to(DEV), out_dtype=od)
        # sums up to 528 * 2^14 < 2^24: exact in fp32
        assert torch.equal(y.cpu(), scaled((x.float() @ w.float().t()).to(torch.int32), sx, sw, od))


@pytest.mark.parametrize("od", [F32, BF16, F16])
@pytest.mark.parametrize("t", [BF16, F16])
@pytest.mark.parametrize("case", [CASES[i] for i in (2, 3, 5)], ids=[IDS[i] for i in (2, 3, 5)])
def test_grouped_against_float64(case, t, od):
    r, (N, K) = routing_of(case), case[2:]
    x, w, dy = draw((r.T, K), t, 5), draw((r.E, N, K), t, 6), draw((r.rows, N), t, 7)
    src = r.src(True)
    xd, wd, dyd = x.to(DEV), w.to(DEV), dy.to(DEV)
    y = nv.grouped_linear(xd, wd, r.off, r.pairs, r.topk, out_dtype=od)
    close(y[:r.used], *fwd_ref(x, w, r, src), K)
    close(nv.grouped_linear_dx(dyd, wd, r.off, out_dtype=od)[:r.used], *dx_ref(dy, w, r), N)
    close(nv.grouped_linear_dw(dyd, xd, r.off, r.pairs, r.topk, out_dtype=od), *dw_ref(dy, x, r, src, N, K),
          max(r.sizes))
    assert torch.equal(y[:r.used], nv.grouped_linear(xd, wd, r.off, r.pairs, r.topk, out_dtype=od)[:r.used])


@pytest.mark.parametrize("K,N", [(40, 24), (72, 264), (264, 136)])
def test_foreign_nans_stay_out(K, N):
    """NaN in dropped rows, in unused experts and behind each operand's used part never
    reaches an output (tails of tiles are cleared, not multiplied by zero)."""
    r = Routing([0, 3, 0, 140, 1, 0], 200, 1)
    nan = float("nan")
    x, w, dy = draw((r.rows, K), BF16, 1), draw((r.E, N, K), BF16, 2), draw((r.rows, N), BF16, 3)
    x[r.used:], dy[r.used:] = nan, nan
    for e, n in enumerate(r.sizes):
        if n == 0:
            w[e] = nan
    xd, wd, dyd = x.to(DEV), w.to(DEV), dy.to(DEV)
    src = r.src(False)
    close(nv.grouped_linear(xd, wd, r.off, out_dtype=F32)[:r.used], *fwd_ref(x, w, r, src), K)
    close(nv.grouped_linear_dx(dyd, wd, r.off, out_dtype=F32)[:r.used], *dx_ref(dy, w, r), N)
    close(nv.grouped_linear_dw(dyd, xd, r.off, out_dtype=F32), *dw_ref(dy, x, r, src, N, K), max(r.sizes))


def test_non_finite_values_propagate():
    r = Routing([4, 4], 8, 1)
    x, w = draw((8, 64), BF16, 1).to(DEV), draw((2, 16, 64), BF16, 2).abs().to(DEV)
    x[1, 5], x[6, 60] = float("nan"), float("inf")
    y = nv.grouped_linear(x, w, r.off)
    assert torch.isnan(y[1]).all() and torch.isfinite(y[[0, 2, 3, 4, 5, 7]]).all()
    assert not torch.isfinite(y[6]).any()
    dy = draw((8, 16), BF16, 3).to(DEV)
    dw = nv.grouped_linear_dw(dy, x, r.off)
    assert torch.isnan(dw[0, :, 5]).all() and torch.isfinite(dw[0, :, :5]).all()


def test_experts_without_any_row():
    off = torch.zeros(4, dtype=torch.int32, device=DEV)
    pairs = torch.full((6,), -1, dtype=torch.int32, device=DEV)
    x, w = draw((6, 32), BF16, 1).to(DEV), draw((3, 16, 32), BF16, 2).to(DEV)
    out = torch.full((6, 16), SENTINEL, device=DEV)
    nv.grouped_linear(x, w, off, pairs, 1, out=out)
    assert bool((out == SENTINEL).all())
    dw = torch.full((3, 16, 32), SENTINEL, device=DEV)
    nv.grouped_linear_dw(out.to(BF16), x, off, pairs, 1, out=dw)
    assert bool((dw == 0).all())
    empty = torch.empty((0, 16), dtype=BF16, device=DEV)
    dw.fill_(SENTINEL)
    nv.grouped_linear_dw(empty, torch.empty((0, 32), dtype=BF16, device=DEV), off, out=dw)
    assert bool((dw == 0).all())
    assert nv.grouped_linear(torch.empty((0, 32), dtype=BF16, device=DEV), w, off).shape == (0, 16)


def test_offsets_outside_the_rows_stay_in_bounds():
    """Offsets and pairs outside their ranges are clamped: the call ends, and what lies
    around the output is left alone."""
    x, w = draw((40, 32), BF16, 1).to(DEV), draw((3, 16, 32), BF16, 2).to(DEV)
    raw = torch.full((40 + 64, 16), SENTINEL, device=DEV)
    out = raw[32:72]
    for off in ([-5, 10, 50, 1 << 30], [30, 10, 20, 5], [0, 1 << 30, -(1 << 30), 40]):
        o = torch.tensor(off, dtype=torch.int32, device=DEV)
        pairs = torch.tensor([7, -9, 1 << 30, -(1 << 31), 39] * 8, dtype=torch.int32, device=DEV)
        nv.grouped_linear(x, w, o, pairs, 1, out=out)
        nv.grouped_linear_dw(draw((40, 16), BF16, 3).to(DEV), x, o, pairs, 1)
        nv.grouped_linear_dx(draw((40, 16), BF16, 3).to(DEV), w, o)
        torch.cuda.synchronize()
        assert bool((raw[:32] == SENTINEL).all()) and bool((raw[72:] == SENTINEL).all())


def quantized(rows, K, seed):
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(-128, 128, (rows, K), generator=g, dtype=torch.int16).to(torch.int8)
    return q, torch.rand(rows, generator=g) * 1e-2


def scaled(acc, sx, sw, t):
    """The definition's fp32 products, rounded to t."""
    return ((acc.float() * sx.unsqueeze(1)) * sw).to(t)


@pytest.mark.parametrize("od", [F32, BF16, F16])
@pytest.mark.parametrize("T,N,K", [(1, 1, 16), (1, 2048, 2048), (3, 7, 48), (16, 33, 80), (17, 130, 4096), (64, 64, 64),
                                   (65, 257, 144), (128, 256, 1024), (200, 1001, 1040), (333, 515, 272)])
def test_linear_i8_exact(T, N, K, od):
    x, sx = quantized(T, K, 1)
    w, sw = quantized(N, K, 2)
    y = nv.linear_i8(x.to(DEV), sx.to(DEV), w.to(DEV), sw.to(DEV), out_dtype=od)
    acc = (x.double() @ w.double().t()).to(torch.int64)  # below 2^53: exact
    assert torch.equal(y.cpu(), scaled(acc.to(torch.int32), sx, sw, od))


def test_linear_i8_largest_sum():
    """K at its limit with every product -128 * -128: the int32 sum just fits."""
    K = 131056
    x = torch.full((2, K), -128, dtype=torch.int8, device=DEV)
    w = torch.full((3, K), -128, dtype=torch.int8, device=DEV)
    one = torch.ones(3, device=DEV)
    assert bool((nv.linear_i8(x, one[:2], w, one, out_dtype=F32) == float(K * 16384)).all())
    x[1] = 127
    y = nv.linear_i8(x, one[:2], w, one, out_dtype=F32)
    assert bool((y[1] == torch.tensor(float(-K * 128 * 127), device=DEV)).all())


def test_linear_i8_non_finite_scales():
    x, sx = quantized(4, 64, 1)
    w, sw = quantized(8, 64, 2)
    x[1] = 0
    sx[0], sx[1] = float("nan"), float("inf")
    y = nv.linear_i8(x.to(DEV), sx.to(DEV), w.to(DEV), sw.to(DEV), out_dtype=F32)
    assert torch.isnan(y[:2]).all() and torch.isfinite(y[2:]).all()


def test_linear_i8_after_the_quantizer():
    """The pair as it is used: quant_rows_i8, then the product, against float64 on its codes."""
    x = torch.randn(50, 256, device=DEV, dtype=BF16)
    q, s = nv.quant_rows_i8(x)
    w, sw = quantized(96, 256, 3)
    y = nv.linear_i8(q, s, w.to(DEV), sw.to(DEV), out_dtype=F32)
    acc = (q.cpu().double() @ w.double().t()).to(torch.int32)
    assert torch.equal(y.cpu(), scaled(acc, s.cpu(), sw, F32))


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("case", [c[:2] + (c[2] + odd, -(-c[3] // 16) * 16) for c, odd in zip(CASES, (0, 1, 2, 3, 0, 5, 1, 0, 7))],
                         ids=IDS)
def test_grouped_i8_exact(case, gather):
    r, (N, K) = routing_of(case), case[2:]
    x, sx = quantized(r.T if gather else r.rows, K, 3)
    w, sw = quantized(r.E * N, K, 4)
    w, sw = w.reshape(r.E, N, K), sw.reshape(r.E, N)
    src = r.src(gather)
    for od in (F32, BF16):
        out = torch.full((r.rows, N), SENTINEL, device=DEV, dtype=od)
        nv.grouped_linear_i8(x.to(DEV), sx.to(DEV), w.to(DEV), sw.to(DEV), r.off, r.pairs if gather else None, r.topk,
                             out=out)
        acc = fwd_ref(x, w, r, src)[0].to(torch.int32)
        for e, a, b in r.spans():
            assert torch.equal(out[a:b].cpu(), scaled(acc[a:b], sx[src[a:b]], sw[e], od)), e
        assert bool((out[r.used:] == SENTINEL).all())


def test_outputs_and_weights_past_32_bits():
    """Row and weight offsets beyond 2^31 elements (and 2^32 bytes)."""
    rows, N = (1 << 20) + 5, 2056
    x = torch.zeros((rows, 8), dtype=BF16, device=DEV)
    x[:, 0] = (torch.arange(rows, device=DEV) % 7).to(BF16)
    w = torch.ones((2, N, 8), dtype=BF16, device=DEV)
    w[1] *= 2
    off = torch.tensor([0, rows - 3, rows], dtype=torch.int32, device=DEV)
    y = nv.grouped_linear(x, w, off)
    assert bool((y[:, 0].float() == x[:, 0].float() * torch.where(torch.arange(rows, device=DEV) < rows - 3, 1., 2.)).all())
    assert bool((y[-5:] == y[-5:, :1]).all()) and bool((y[1_044_500:1_044_600] == y[1_044_500:1_044_600, :1]).all())
    dw = nv.grouped_linear_dw(y[:, :8].contiguous(), x, off, out_dtype=F32)
    assert dw[1, 0, 0].item() == float((x[-3:, 0].float() ** 2).sum() * 2)
    del y, x, w, dw
    E, N, K = 520, 2048, 2056
    w = torch.zeros((E, N, K), dtype=BF16, device=DEV)
    w[E - 1, :, K - 1], w[E - 2, N - 1, 0] = 3.0, 5.0
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    off[E - 1], off[E] = 1, 3
    x = torch.ones((3, K), dtype=BF16, device=DEV)
    y = nv.grouped_linear(x, w, off, out_dtype=F32)
    assert bool((y[1:] == 3.0).all()) and y[0, N - 1].item() == 5.0 and bool((y[0, :-1] == 0).all())
    dx = nv.grouped_linear_dx(torch.ones((3, N), dtype=BF16, device=DEV), w, off, out_dtype=F32)
    assert bool((dx[1:, K - 1] == 3.0 * N).all()) and dx[0, 0].item() == 5.0


@pytest.mark.parametrize("t", [F32, BF16, F16])
@pytest.mark.parametrize("T,topk,H,drop", [(1, 8, 2048, 0), (1, 1, 8, 1), (5, 3, 17, 4), (130, 8, 64, 40), (200, 9, 520, 3),
                                           (64, 2, 1000, 0), (3, 17, 4104, 20), (1500, 2, 24, 700)])
def test_combine(T, topk, H, drop, t):
    P = T * topk
    r = Routing([P - drop], T, topk, 3)
    y, dout = draw((P, H), t, 1), draw((T, H), t, 2)
    y[P - drop:] = float("nan")  # rows no pair has
    w = torch.rand(T, topk, generator=torch.Generator().manual_seed(3))
    pr = r.pairs_cpu[:r.used].long()
    tok, slot = pr // topk, pr % topk
    wr = w[tok, slot].double().unsqueeze(1)
    yu = y[:r.used].double()
    ref = torch.zeros(T, H, dtype=torch.float64).index_add_(0, tok, yu * wr)
    S = torch.zeros(T, H, dtype=torch.float64).index_add_(0, tok, (yu * wr).abs())
    yd, wd, dd = y.to(DEV), w.to(DEV), dout.to(DEV)
    for od in (F32, BF16, F16):
        # topk products and sums, each within half a step of a partial sum
        close(nv.moe_combine(yd, r.pairs, topk, wd, out_dtype=od), ref, S, 2 * topk)
    # without weights: the sum over slots
    ones = torch.zeros(T, H, dtype=torch.float64).index_add_(0, tok, yu)
    So = torch.zeros(T, H, dtype=torch.float64).index_add_(0, tok, yu.abs())
    close(nv.moe_combine(yd, r.pairs, topk, out_dtype=F32), ones, So, 2 * topk)
    # the gradients, on a workspace of any contents
    dy = torch.full((P, H), SENTINEL, dtype=t, device=DEV)
    for fill in (0, 255):
        ws = torch.full((max(nv.combine_workspace_size(T, topk), 16),), fill, dtype=torch.uint8, device=DEV)
        _, dw = nv.moe_combine_grad(dd, yd, r.pairs, wd, dy=dy, ws=ws)
        d = dout[tok].double()
        # one fp32 product, then one rounding to the type
        close(dy[:r.used], d * wr, (d * wr).abs(), 1)
        assert bool((dy[r.used:] == SENTINEL).all())
        full, Sf = torch.zeros(P, dtype=torch.float64), torch.zeros(P, dtype=torch.float64)
        full[pr], Sf[pr] = (d * yu).sum(1), (d * yu).abs().sum(1)
        close(dw.reshape(-1), full, Sf, H + 8)
        assert bool((dw.reshape(-1).cpu()[full == 0] == 0).all())


def test_combine_of_repeated_and_foreign_entries_stays_in_bounds():
    y = draw((12, 16), F32, 1).to(DEV)
    pairs = torch.tensor([0, 0, 5, -7, 1 << 30, 11, 2, 12, -1, -1, 3, 3], dtype=torch.int32, device=DEV)
    out = nv.moe_combine(y, pairs, 3)
    assert torch.equal(out[3], y[5]) and torch.isfinite(out).all()


# ------------------------------------------------------------------ streams, graphs, together
def test_another_stream_and_a_replayed_graph():
    r = Routing([3, 0, 150, 40], 97, 2)
    x, w = draw((r.T, 72), BF16, 1).to(DEV), draw((4, 264, 72), BF16, 2).to(DEV)
    wts = torch.rand(r.T, 2, device=DEV)
    ws = torch.empty(max(nv.combine_workspace_size(r.T, 2), 16), dtype=torch.uint8, device=DEV)
    y, out = torch.zeros((r.rows, 264), dtype=BF16, device=DEV), torch.zeros((r.T, 264), dtype=BF16, device=DEV)
    dw = torch.zeros((4, 264, 72), dtype=BF16, device=DEV)

    def step():
        nv.grouped_linear(x, w, r.off, r.pairs, 2, out=y)
        nv.moe_combine(y, r.pairs, 2, wts, out=out, ws=ws)
        nv.grouped_linear_dw(y, x, r.off, r.pairs, 2, out=dw)

    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (y[:r.used], out, dw)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out.zero_(), dw.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (y[:r.used], out, dw)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(4):
        x.copy_(draw((r.T, 72), BF16, 10 + k))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y[:r.used], out, dw)]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (y[:r.used], out, dw))), k


def _layer_gpu(x, wgu, wd, wts, off, pairs, topk, dout):
    """One expert layer, forward and backward, as a training step calls it."""
    gu = nv.grouped_linear(x, wgu, off, pairs, topk, out_dtype=F32)
    g, u = gu.chunk(2, dim=1)
    s = torch.sigmoid(g)
    h = (g * s * u).to(x.dtype)
    y = nv.grouped_linear(h, wd, off, out_dtype=F32)
    out = nv.moe_combine(y, pairs, topk, wts)
    dy, dwts = nv.moe_combine_grad(dout, y, pairs, wts)
    dy = dy.to(x.dtype)
    dwd = nv.grouped_linear_dw(dy, h, off, out_dtype=F32)
    dh = nv.grouped_linear_dx(dy, wd, off, out_dtype=F32)
    dgu = torch.cat([dh * u * s * (1 + g * (1 - s)), dh * g * s], dim=1).to(x.dtype)
    dwgu = nv.grouped_linear_dw(dgu, x, off, pairs, topk, out_dtype=F32)
    dxp = nv.grouped_linear_dx(dgu, wgu, off, out_dtype=F32)
    dx = nv.moe_combine(dxp, pairs, topk)
    return out, dx, dwgu, dwd, dwts


def _layer_f64(x, wgu, wd, wts, ids):
    out = []
    for t in range(x.shape[0]):
        acc = 0
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if 0 <= e < wgu.shape[0]:
                g, u = (wgu[e] @ x[t]).chunk(2)
                acc = acc + wts[t, j] * (wd[e] @ (g * torch.sigmoid(g) * u))
        out.append(acc if not isinstance(acc, int) else torch.zeros(wd.shape[1], dtype=x.dtype))
    return torch.stack(out)


def test_a_layer_with_its_gradients():
    """route -> gathered gate/up -> SwiGLU -> down -> combine and the backward pass, from the
    framework's routing (dropped and repeated ids, an unused expert), against float64
    autograd and against differences. Bound: the intermediate roundings to fp16 (h, dy, dgu),
    each half a step 2^-11 of a term of the sums, 4 of them on the longest path."""
    T, topk, E, H, I = 37, 3, 6, 64, 40
    ids = torch.randint(0, E - 1, (T, topk), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    ids[3, 1], ids[4] = -1, torch.tensor([-1, E, 900], dtype=torch.int32)
    ids[5, 0] = ids[5, 1]
    x = draw((T, H), F16, 1)
    wgu, wd = (draw((E, 2 * I, H), F16, 2) / 8).to(F16), (draw((E, H, I), F16, 3) / 6).to(F16)
    wts = torch.softmax(draw((T, topk), F32, 4), dim=1)
    dout = draw((T, H), F32, 5)
    off, pairs, _ = nv.route(ids.to(DEV), E)
    got = _layer_gpu(x.to(DEV), wgu.to(DEV), wd.to(DEV), wts.to(DEV), off, pairs, topk, dout.to(DEV))
    leaves = [v.double().requires_grad_() for v in (x, wgu, wd, wts)]
    ref = _layer_f64(*leaves, ids)
    (ref * dout.double()).sum().backward()
    want = (ref.detach(), leaves[0].grad, leaves[1].grad, leaves[2].grad, leaves[3].grad)
    for name, a, b in zip(("out", "dx", "dwgu", "dwd", "dwts"), got, want):
        rel = float((a.double().cpu() - b).norm() / b.norm())
        assert rel <= 4 * 2.0 ** -11, (name, rel)
    assert bool((got[0][4] == 0).all()) and bool((got[1][4] == 0).all())
    assert bool((got[2][E - 1] == 0).all()) and bool((got[3][E - 1] == 0).all())
    assert bool((got[4].cpu()[(ids < 0) | (ids >= E)] == 0).all())
    # differences of the float64 layer along one direction per input
    f = lambda *v: float((_layer_f64(*v, ids) * dout.double()).sum())  # noqa: E731
    base = [v.detach() for v in leaves]
    for k, grad in enumerate(got[1:]):
        d = torch.randn(base[k].shape, dtype=torch.float64, generator=torch.Generator().manual_seed(k))
        step = 1e-5
        hi, lo = list(base), list(base)
        hi[k], lo[k] = base[k] + step * d, base[k] - step * d
        slope = (f(*hi) - f(*lo)) / (2 * step)
        dot = float((grad.double().cpu() * d).sum())
        scale = float(grad.double().cpu().norm() * d.norm())
        assert abs(dot - slope) <= 4 * 2.0 ** -11 * scale, (k, dot, slope)


def test_int8_experts_together():
    """quant_rows_i8 -> int8 gate/up over the routing -> SwiGLU -> quant_rows_i8 -> int8 down ->
    combine, against float64 on the same codes (the requantized h is the library's own)."""
    T, topk, E, H, I = 21, 2, 5, 128, 96
    ids = torch.randint(0, E, (T, topk), generator=torch.Generator().manual_seed(2), dtype=torch.int32)
    x = draw((T, H), BF16, 1).to(DEV)
    wts = torch.softmax(draw((T, topk), F32, 4), dim=1).to(DEV)
    w1, s1 = quantized(E * 2 * I, H, 5)
    w2, s2 = quantized(E * H, I, 6)
    w1, s1, w2, s2 = w1.reshape(E, 2 * I, H), s1.reshape(E, -1), w2.reshape(E, H, I), s2.reshape(E, -1)
    off, pairs, _ = nv.route(ids.to(DEV), E)
    q, s = nv.quant_rows_i8(x)
    gu = nv.grouped_linear_i8(q, s, w1.to(DEV), s1.to(DEV), off, pairs, topk, out_dtype=F32)
    g, u = gu.chunk(2, dim=1)
    qh, sh = nv.quant_rows_i8((torch.nn.functional.silu(g) * u).contiguous())
    out = nv.moe_combine(nv.grouped_linear_i8(qh, sh, w2.to(DEV), s2.to(DEV), off, out_dtype=F32), pairs, topk, wts)
    hd = (qh.double() * sh.double().unsqueeze(1)).cpu()
    ref = torch.zeros(T, H, dtype=torch.float64)
    S = torch.zeros_like(ref)
    pos = {int(p): k for k, p in enumerate(pairs.cpu())}
    for t in range(T):
        for j in range(topk):
            e = int(ids[t, j])
            y = (w2[e].double() * s2[e].double().unsqueeze(1)) @ hd[pos[t * topk + j]]
            ref[t] += float(wts[t, j]) * y
            S[t] += float(wts[t, j]) * y.abs()
    # per term: int32 -> fp32, two scale products, the weighted sum
    close(out, ref, S, 3 + 2 * topk)
