"""The grouped products (zi_grouped_fwd, zi_grouped_dx, zi_grouped_dw): exactly on small whole numbers, and against
their formulas in 64 bits.

Tolerances.  u = 2^-24 is fp32's half step; a sum of n products in fp32, in any order and with additions that truncate,
is off by at most n 2 u of the sum of their magnitudes; a stored value adds half a step of its type.  GeLU: Phi is off
by 1e-6 of its tail (the polynomial) and by the roundings of its exponent, 1.5 a^2 u, and of some 20 operations; an
exponential below fp32's normal range, 2^-126, counts as zero (as the hardware's exp2 gives it)."""
import math

import pytest
import torch

from zi_testlib import say

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
U = 2.0 ** -24
INF = float("inf")


def half(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def matrix(g, rows, cols, dtype, pad, whole, std=1.0):
    """[rows, cols] with NaN between its rows."""
    buf = torch.full((rows, cols + pad), float("nan"), dtype=dtype, device="cuda")
    if whole:
        buf[:, :cols] = torch.randint(-3, 4, (rows, cols), generator=g, device="cuda").to(dtype)
    else:
        buf[:, :cols] = torch.randn((rows, cols), generator=g, device="cuda").mul_(std).to(dtype)
    return buf[:, :cols]


def blank(rows, cols, dtype, pad):
    buf = torch.full((rows, cols + pad), -7.0, dtype=dtype, device="cuda")
    return buf[:, :cols], buf


def close(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), "%s: %d of %d outside, worst %.3g of tolerance" % (
        what, int(bad.sum()), bad.numel(), float(((got.double() - want).abs() / tol).nan_to_num(INF).max()))


def cdf(a):
    return 0.5 * torch.erfc(a * -math.sqrt(0.5))  # torch.special.ndtr has no digits below -8


def pdf(a):
    return torch.exp(-a * a / 2) / math.sqrt(2 * math.pi)


def cdf_off(a):
    """How far Phi in fp32 may be off."""
    return cdf(-a.abs()) * (1e-6 + (1.5 * a * a + 20) * U) + 2.0 ** -126 + torch.where(a > 0, 2 * U, 0.0)


class Case:
    """Groups of the given sizes after `front` rows of nobody's, and as many behind."""

    def __init__(self, sizes, K, M, dtype, pad=0, whole=False, front=0, seed=1):
        g = gen(seed)
        self.dt, self.K, self.M, self.pad = DT[dtype], K, M, pad
        self.E, self.R = len(sizes), sum(sizes) + 2 * front
        edge = [front]
        for n in sizes:
            edge.append(edge[-1] + n)
        self.edge = edge
        self.offsets = torch.tensor(edge, dtype=torch.int32, device="cuda")
        self.X = matrix(g, self.R, K, self.dt, pad, whole)
        self.dY = matrix(g, self.R, M, self.dt, 2 * pad, whole)
        w = torch.full((self.E, M + (2 if pad else 0), K + pad), float("nan"), dtype=self.dt, device="cuda")
        self.W = w[:, :M, :K]
        for e in range(self.E):
            self.W[e] = matrix(g, M, K, self.dt, 0, whole, 1 / math.sqrt(K))
        self.A = matrix(g, self.R, K, self.dt, pad, False)
        self.mine = torch.zeros(self.R, dtype=torch.bool, device="cuda")
        self.mine[edge[0]:edge[-1]] = True
        self.X[~self.mine] = float("nan")
        self.dY[~self.mine] = float("nan")

    def product(self, X, W):
        """The sums of X_e W_e and of their magnitudes, in 64 bits."""
        out = torch.zeros((self.R, W(0).shape[1]), dtype=torch.float64, device="cuda")
        size = torch.zeros_like(out)
        for e in range(self.E):
            a, b = self.edge[e], self.edge[e + 1]
            if b > a:
                x, w = X[a:b].double(), W(e).double().contiguous()
                out[a:b] = x @ w
                size[a:b] = x.abs() @ w.abs()
        return out, size

    def check(self, got, buf, want, tol, what, exact=False):
        m = self.mine
        assert (buf[~m] == -7.0).all() and (buf[:, got.shape[1]:] == -7.0).all(), what + ": wrote elsewhere"
        if exact:
            assert torch.equal(got[m], want[m].to(got.dtype)), what
        else:
            close(got[m], want[m], tol[m], what)

    def fwd(self, layers, out, gelu=False, keep=False, exact=False):
        Y, yb = blank(self.R, self.M, DT[out], self.pad)
        A, ab = blank(self.R, self.M, self.dt, 2 * self.pad) if keep else (None, None)
        layers.grouped_fwd(self.X, self.W, self.offsets, Y, A=A, gelu=gelu)
        torch.cuda.synchronize()
        a, size = self.product(self.X, lambda e: self.W[e].t())
        off = self.K * 2 * U * size
        if keep:
            self.check(A, ab, a, off + half(self.dt) * a.abs() + tiny(self.dt), "A", exact)
        if gelu:
            want = a * cdf(a)
            off = 1.13 * off + a.abs() * cdf_off(a) + 2 * U * want.abs()
        else:
            want = a
        self.check(Y, yb, want, (off + half(DT[out]) * want.abs()) * 1.01 + tiny(DT[out]), "Y", exact and not gelu)

    def dx(self, layers, out, gelu=False, exact=False):
        dX, db = blank(self.R, self.K, DT[out], self.pad)
        layers.grouped_dx(self.dY, self.W, self.offsets, dX, A=self.A if gelu else None)
        torch.cuda.synchronize()
        want, size = self.product(self.dY, lambda e: self.W[e])
        off = self.M * 2 * U * size
        if gelu:
            a = self.A.double()
            slope = cdf(a) + a * pdf(a)
            slope_off = cdf_off(a) + a.abs() * (pdf(a) * (1.5 * a * a + 10) * U + 2.0 ** -126) + 2 * U * slope.abs()
            off = off * (slope.abs() + slope_off) + want.abs() * slope_off
            want = want * slope
            off = off + U * want.abs()
        self.check(dX, db, want, (off + half(DT[out]) * want.abs()) * 1.01 + tiny(DT[out]), "dX", exact and not gelu)

    def dw(self, layers, out, accumulate=False, exact=False):
        buf = torch.full((self.E, self.M + 1, self.K + self.pad), -7.0, dtype=DT[out], device="cuda")
        dW = buf[:, :self.M, :self.K]
        before = None
        if accumulate:
            before = torch.randint(-3, 4, dW.shape, generator=gen(4), device="cuda").to(DT[out])
            dW.copy_(before)
        layers.grouped_dw(self.X, self.dY, self.offsets, dW, accumulate=accumulate)
        torch.cuda.synchronize()
        assert (buf[:, self.M:] == -7.0).all() and (buf[:, :, self.K:] == -7.0).all(), "dW: wrote elsewhere"
        for e in range(self.E):
            a, b = self.edge[e], self.edge[e + 1]
            x, d = self.X[a:b].double(), self.dY[a:b].double()
            want, size = d.t().contiguous() @ x, d.abs().t().contiguous() @ x.abs()
            if accumulate:
                want, size = want + before[e].double(), size + before[e].double().abs()
            if exact:
                assert torch.equal(dW[e], want.to(dW.dtype)), "dW of group %d" % e
            else:
                close(dW[e], want, ((b - a + 2) * 2 * U * size + half(DT[out]) * want.abs()) * 1.01 + tiny(DT[out]), "dW of group %d" % e)


# sizes of the groups, K, M: none, one and odd numbers of rows; reductions and widths that end inside a step or a tile
CASES = [
    ([1], 8, 8), ([3], 64, 64), ([0, 1, 0, 2, 0], 40, 72), ([5, 0, 17, 1], 128, 200), ([16, 33, 7], 264, 136),
    ([0, 0, 70], 96, 320), ([64, 65, 63, 1, 0, 130], 192, 264), ([300, 2, 0, 257], 320, 520), ([128] * 9, 64, 136),
    ([1000, 24, 513], 1032, 776), ([1] * 70, 72, 88), ([0] * 130 + [40] + [0] * 70 + [9], 136, 96),
]


@pytest.mark.parametrize("sizes,K,M", CASES)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_whole_numbers(sizes, K, M, dtype):
    """Small whole numbers, whose sums fp32 holds exactly: any element out of place shows."""
    from offload_memory_centric_amd import layers
    say("grouped exact", sizes[:8], K, M, dtype)
    c = Case(sizes, K, M, dtype, pad=8, whole=True, front=3)
    for out in (dtype, "f32"):
        c.fwd(layers, out, exact=True)
        c.dx(layers, out, exact=True)
        c.dw(layers, out, exact=True)
    c.dw(layers, "f32", accumulate=True, exact=True)
    c.fwd(layers, dtype, gelu=True, keep=True, exact=True)


@pytest.mark.parametrize("sizes,K,M", CASES[2:11])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_formulas(sizes, K, M, dtype):
    from offload_memory_centric_amd import layers
    say("grouped", sizes[:8], K, M, dtype)
    c = Case(sizes, K, M, dtype, seed=3)
    c.fwd(layers, dtype, gelu=True, keep=True)
    c.fwd(layers, dtype, gelu=True)
    c.fwd(layers, "f32")
    c.dx(layers, dtype, gelu=True)
    c.dx(layers, "f32")
    c.dw(layers, "f32")
    c.dw(layers, dtype)


# tiles of 256, of 128 and of 64; whole and ragged reductions; experts of very different sizes
@pytest.mark.parametrize("sizes,K,M", [([4096, 3000, 1, 5000], 512, 2048), ([700, 900, 1100, 0], 456, 1024),
                                       ([2500], 512, 2048), ([90, 120, 30, 400, 8, 77, 64, 200], 1000, 1408),
                                       ([20, 40, 25, 33, 0, 9, 16, 48], 2048, 1408), ([8, 0, 3, 2, 9, 1], 2056, 712)])
def test_larger(sizes, K, M):
    from offload_memory_centric_amd import layers
    say("grouped larger", sizes, K, M)
    c = Case(sizes, K, M, "bf16", whole=True, front=1)
    c.fwd(layers, "bf16", exact=True)
    c.fwd(layers, "bf16", gelu=True, keep=True, exact=True)
    c.dx(layers, "bf16", exact=True)
    c.dw(layers, "f32", exact=True)
    c.dw(layers, "f32", accumulate=True, exact=True)
    c = Case(sizes, K, M, "f16")
    c.fwd(layers, "f16", gelu=True, keep=True)
    c.dx(layers, "f16", gelu=True)
    c.dw(layers, "f16")


# input gradients of few rows over a long reduction: one tile and several, ends inside a step of 32 and a tile of 16 x 32
@pytest.mark.parametrize("sizes,K,M", [([21], 160, 5000), ([3, 0, 16, 17, 1, 40], 88, 1704), ([1], 520, 4104), ([9, 2], 1032, 2000),
                                       ([2, 5, 0, 1], 8, 648), ([16], 2048, 2048)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_input_gradient_of_few_rows(sizes, K, M, dtype):
    from offload_memory_centric_amd import layers
    say("grouped dX of few rows", sizes, K, M, dtype)
    c = Case(sizes, K, M, dtype, pad=8, whole=True, front=3)
    for out in (dtype, "f32"):
        c.dx(layers, out, exact=True)
    c = Case(sizes, K, M, dtype, pad=16, seed=5)
    c.dx(layers, dtype, gelu=True)
    c.dx(layers, dtype)
    c.dx(layers, "f32")


def test_gelu_over_its_range():
    """Every finite fp16 value as A, forward and backward, by products with one."""
    from offload_memory_centric_amd import layers
    bits = torch.arange(-32768, 32768, dtype=torch.int32, device="cuda").to(torch.int16)
    a = bits.view(torch.float16)
    a = a[torch.isfinite(a)]
    n = a.numel()
    for dt in (torch.float16, torch.bfloat16):
        X = torch.zeros((n, 8), dtype=dt, device="cuda")
        X[:, 0] = a.to(dt)
        W = torch.zeros((1, 8, 8), dtype=dt, device="cuda")
        W[0, :, 0] = 1.0
        offsets = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        Y, A = torch.empty_like(X), torch.empty_like(X)
        layers.grouped_fwd(X, W, offsets, Y, A=A, gelu=True)
        assert torch.equal(A, X[:, :1].expand(n, 8))
        x = X[:, :1].double()
        want = x * cdf(x)
        close(Y, want.expand(n, 8), (half(dt) * want.abs() + x.abs() * cdf_off(x) + 2 * U * want.abs()) * 1.01 + tiny(dt), "GeLU")
        dX = torch.empty_like(X)
        one = torch.zeros_like(X)
        one[:, 0] = 1.0
        layers.grouped_dx(one, W.transpose(1, 2).contiguous(), offsets, dX, A=A)
        slope = cdf(x) + x * pdf(x)
        off = cdf_off(x) + x.abs() * (pdf(x) * (1.5 * x * x + 10) * U + 2.0 ** -126) + 3 * U * slope.abs()
        close(dX, slope.expand(n, 8), (half(dt) * slope.abs() + off) * 1.01 + tiny(dt), "GeLU'")


def test_special_values_stay_in_their_rows():
    from offload_memory_centric_amd import layers
    for sizes in ([40, 50, 30], [5, 6, 3]):
        c = Case(sizes, 72, 136, "bf16")
        c.X[2, 7] = INF
        c.X[sizes[0] + 1, 0] = float("nan")
        c.W[2, 5, 6] = float("nan")
        Y = torch.zeros((c.R, c.M), dtype=torch.bfloat16, device="cuda")
        layers.grouped_fwd(c.X, c.W, c.offsets, Y)
        bad = ~torch.isfinite(Y)
        rows = bad.any(1).nonzero().flatten().tolist()
        third = list(range(sizes[0] + sizes[1], c.R))
        assert rows == [2, sizes[0] + 1] + third
        assert bad[third].sum() == len(third) and bad[third, 5].all()
        dX = torch.zeros((c.R, c.K), dtype=torch.bfloat16, device="cuda")
        layers.grouped_dx(c.dY, c.W, c.offsets, dX)
        bad = ~torch.isfinite(dX)
        assert bad.sum() == len(third) and bad[third, 6].all()


def test_offsets_outside_the_rows():
    """Offsets that are not what they should be leave rows out; nothing outside is read or written."""
    from offload_memory_centric_amd import layers
    R, K, M = 100, 64, 64
    g = gen(2)
    X = matrix(g, R, K, torch.bfloat16, 0, True)
    W = torch.ones((4, M, K), dtype=torch.bfloat16, device="cuda")
    want = X.double().sum(1, keepdim=True)
    for edge in ([-50, 20, 40, 60, 1000], [0, 60, 30, 90, 100], [200, 300, 400, 500, 600]):
        offsets = torch.tensor(edge, dtype=torch.int32, device="cuda")
        Y = torch.full((R, M), -7.0, dtype=torch.float32, device="cuda")
        layers.grouped_fwd(X, W, offsets, Y)
        torch.cuda.synchronize()
        assert ((Y == want.float()) | (Y == -7.0)).all()
        if edge[0] == -50:
            assert (Y == want.float()).all()
        if edge[0] == 200:
            assert (Y == -7.0).all()


def test_no_rows():
    from offload_memory_centric_amd import layers
    offsets = torch.zeros(4, dtype=torch.int32, device="cuda")
    X, dY = (torch.empty((0, n), dtype=torch.bfloat16, device="cuda") for n in (64, 72))
    for dt in (torch.bfloat16, torch.float32):
        dW = torch.full((3, 72, 64), 2.0, dtype=dt, device="cuda")
        layers.grouped_dw(X, dY, offsets, dW)
        assert (dW == 0).all()
    dW.fill_(2.0)
    layers.grouped_dw(X, dY, offsets, dW, accumulate=True)
    assert (dW == 2.0).all()
    layers.grouped_fwd(X, dW.bfloat16(), offsets, dY)
    layers.grouped_dx(dY, dW.bfloat16(), offsets, X)


def test_many_groups():
    """More groups than a wave has lanes many times over, few with rows."""
    from offload_memory_centric_amd import layers
    E, K, M = 4096, 64, 40
    for rows in (1, 40):
        sizes = [0] * E
        for e in (0, 63, 64, 1000, 4095):
            sizes[e] = rows
        c = Case(sizes, K, M, "bf16", whole=True)
        c.fwd(layers, "bf16", exact=True)
        c.dx(layers, "f32", exact=True)
        c.dw(layers, "f32", exact=True)


def test_far_rows():
    """Rows and weights past 2^32 bytes."""
    from offload_memory_centric_amd import layers
    K, M, R = 8192, 64, 300000
    X = torch.zeros((R, K), dtype=torch.bfloat16, device="cuda")
    X[R - 300:] = 1.0
    E = 5000 // 8
    W = torch.zeros((E, 512, K), dtype=torch.bfloat16, device="cuda")
    W[E - 1, :, :2] = 3.0
    offsets = torch.full((E + 1,), R - 300, dtype=torch.int32, device="cuda")
    offsets[0], offsets[E] = 0, R
    Y = torch.empty((R, M), dtype=torch.bfloat16, device="cuda")
    layers.grouped_fwd(X, W[:, :M], offsets, Y)
    assert (Y[R - 300:] == 6.0).all() and (Y[:R - 300] == 0.0).all()
    dX = torch.full((R, K), 9.0, dtype=torch.bfloat16, device="cuda")
    layers.grouped_dx(Y, W[:, :M], offsets, dX)
    assert (dX[R - 300:, :2] == 18.0 * M).all() and (dX[R - 300:, 2:] == 0).all() and (dX[:R - 300] == 0).all()
    dW = W[:, :M]
    layers.grouped_dw(X, Y, offsets, dW)
    assert (dW[E - 1] == 1800.0).all() and (dW[:E - 1] == 0).all() and (W[:, M:, 2:] == 0).all()
