"""The adapters (zi_adapters_fwd, zi_adapters_bwd) against their formulas in 64 bits.

Tolerances.  u = 2^-24 is fp32's half step; a sum of n products in fp32, in any order and with additions that truncate,
is off by at most n 2 u of the sum of their magnitudes; an error of U goes through the second product with the
magnitudes of B; a stored value adds half a step of its type."""
import math

import pytest
import torch

from zi_testlib import say

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
U2 = 2.0 ** -23
INF = float("inf")


def half(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def matrix(g, rows, cols, dtype, pad, std=1.0):
    buf = torch.full((rows, cols + pad), float("nan"), dtype=dtype, device="cuda")
    buf[:, :cols] = torch.randn((rows, cols), generator=g, device="cuda").mul_(std).to(dtype)
    return buf[:, :cols]


def close(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), "%s: %d of %d outside, worst %.3g of tolerance" % (
        what, int(bad.sum()), bad.numel(), float(((got.double() - want).abs() / tol).nan_to_num(INF).max()))


class Case:
    """Segments of the given lengths after `front` rows of nobody's, and as many behind; ids by segment."""

    def __init__(self, lengths, ids, N, r, K, M, dtype, out, pad=0, front=0, seed=1):
        g = gen(seed)
        self.dt, self.out, self.pad = DT[dtype], DT[out], pad
        self.T, self.K, self.M, self.N, self.r, self.S = sum(lengths) + 2 * front, K, M, N, r, len(lengths)
        self.edge = [front]
        for n in lengths:
            self.edge.append(self.edge[-1] + n)
        self.ids_list = ids
        self.offsets = torch.tensor(self.edge, dtype=torch.int32, device="cuda")
        self.ids = torch.tensor(ids, dtype=torch.int32, device="cuda")
        self.scales = torch.rand(N, generator=g, device="cuda") + 0.5
        self.X = matrix(g, self.T, K, self.dt, pad)
        self.dY = matrix(g, self.T, M, self.dt, pad)
        self.Y0 = matrix(g, self.T, M, self.out, 2 * pad)
        self.dX0 = matrix(g, self.T, K, self.out, 2 * pad)
        self.A = matrix(g, N * r, K, self.dt, 0, 1 / math.sqrt(K)).view(N, r, K)
        self.B = matrix(g, N * r, M, self.dt, 0, 1 / math.sqrt(r)).view(N, r, M)

    def runs(self):
        for n, a, b in zip(self.ids_list, self.edge, self.edge[1:]):
            if 0 <= n < self.N and b > a:
                yield n, a, b

    def fwd(self, layers, base="other", keep=True):
        work = layers.workspace(layers.adapters_fwd_bytes(self.T, self.r))
        U = torch.full((self.r, self.T), float("nan"), device="cuda") if keep else None
        yb = torch.full((self.T, self.M + self.pad), -7.0, dtype=self.out, device="cuda")
        Y, Y0 = yb[:, :self.M], self.Y0
        if base == "same":
            Y.copy_(self.Y0)
            Y0 = Y
        elif base is None:
            Y0 = None
        layers.adapters_fwd(self.X, self.A, self.B, self.offsets, self.ids, self.scales, Y, work, Y0=Y0, U=U)
        torch.cuda.synchronize()
        assert (yb[:, self.M:] == -7.0).all(), "wrote between the rows"
        u = torch.zeros((self.r, self.T), dtype=torch.float64, device="cuda")
        uoff = torch.zeros_like(u)
        y = torch.zeros((self.T, self.M), dtype=torch.float64, device="cuda") if base is None else self.Y0.double()
        off = U2 * y.abs()
        for n, a, b in self.runs():
            x, A, B, s = self.X[a:b].double(), self.A[n].double(), self.B[n].double(), float(self.scales[n])
            un, size = A @ x.t().contiguous(), A.abs() @ x.abs().t().contiguous()
            u[:, a:b], uoff[:, a:b] = un, self.K * U2 * size
            y[a:b] += s * (un.t().contiguous() @ B)
            off[a:b] += s * ((uoff[:, a:b] + (self.r + 6) * U2 * un.abs()).t().contiguous() @ B.abs())
        if keep:
            close(U, u, uoff * 1.01, "U")
        close(Y, y, (off + (half(self.out) + U2) * y.abs()) * 1.01 + tiny(self.out), "Y")
        return U

    def bwd(self, layers, base="other", accumulate=False, form_dx=True, exact_u=None):
        r, T, N, K, M = self.r, self.T, self.N, self.K, self.M
        U = torch.zeros((r, T), device="cuda")
        for n, a, b in self.runs():
            U[:, a:b] = (self.A[n].double() @ self.X[a:b].double().t().contiguous()).float()
        work = layers.workspace(layers.adapters_bwd_bytes(T, r))
        dA, dB = torch.full((N, r, K), 2.0, device="cuda"), torch.full((N, r, M), 3.0, device="cuda")
        xb = torch.full((T, K + self.pad), -7.0, dtype=self.out, device="cuda")
        dX, dX0 = xb[:, :K], self.dX0
        if base == "same":
            dX.copy_(self.dX0)
            dX0 = dX
        elif base is None:
            dX0 = None
        if not form_dx:
            dX = dX0 = None
        layers.adapters_bwd(self.X, self.dY, U, self.A, self.B, self.offsets, self.ids, self.scales, dA, dB, work, dX=dX, dX0=dX0,
                            accumulate=accumulate)
        torch.cuda.synchronize()
        dx = torch.zeros((T, K), dtype=torch.float64, device="cuda") if base is None else self.dX0.double()
        off = U2 * dx.abs()
        start = (2.0, 3.0) if accumulate else (0.0, 0.0)
        da, db = torch.full((N, r, K), start[0], dtype=torch.float64, device="cuda"), torch.full((N, r, M), start[1], dtype=torch.float64, device="cuda")
        da_off, db_off, rows = da * 4 * U2, db * 4 * U2, [0] * N
        da_size, db_size = torch.zeros_like(da), torch.zeros_like(db)
        for n, a, b in self.runs():
            d, x, A, B, s = self.dY[a:b].double(), self.X[a:b].double(), self.A[n].double(), self.B[n].double(), float(self.scales[n])
            du, du_size = s * (B @ d.t().contiguous()), s * (B.abs() @ d.abs().t().contiguous())
            du_off = (M + 2) * U2 * du_size
            dx[a:b] += du.t().contiguous() @ A
            off[a:b] += (du_off + (r + 6) * U2 * du.abs()).t().contiguous() @ A.abs()
            u = U[:, a:b].double()
            da[n] += du @ x
            da_off[n] += du_off @ x.abs()
            da_size[n] += du.abs() @ x.abs()
            db[n] += s * (u @ d)
            db_size[n] += s * (u.abs() @ d.abs())
            rows[n] += b - a
        n_rows = torch.tensor(rows, device="cuda", dtype=torch.float64)[:, None, None] + 8
        close(dA, da, (da_off + n_rows * U2 * da_size) * 1.01 + tiny(torch.float32), "dA")
        close(dB, db, (db_off + n_rows * U2 * db_size) * 1.01 + tiny(torch.float32), "dB")
        if form_dx:
            assert (xb[:, K:] == -7.0).all(), "wrote between the rows"
            close(dX, dx, (off + (half(self.out) + U2) * dx.abs()) * 1.01 + tiny(self.out), "dX")


# lengths, ids, adapters: none, one and odd numbers of rows, segments that cross blocks of 16 and 64, requests without an
# adapter, several of one adapter, adapters of nobody
CASES = [
    ([1], [0], 1, 1, 8, 8), ([3], [0], 2, 4, 64, 40), ([1] * 9, [0, 3, -1, 1, 1, 2, 7, 0, 2], 4, 8, 136, 264),
    ([1, 2, 0, 1, 3, 1], [2, 0, 1, 2, -1, 2], 3, 16, 520, 2056), ([20, 0, 7, 40, 1], [1, 0, 0, 1, 5], 2, 16, 72, 512),
    ([5, 60, 64, 70, 128, 1], [0, 1, 2, 1, -1, 0], 4, 24, 264, 520), ([300], [0], 1, 17, 1032, 136),
    ([33, 200, 31], [1, 0, 1], 2, 64, 128, 640), ([90, 75], [0, 1], 2, 100, 200, 104), ([130], [0], 1, 256, 96, 88),
    ([700, 0, 900, 65], [2, 1, 2, 0], 3, 32, 2048, 1024), ([64] * 3, [-1, -1, 5], 2, 8, 64, 64),
]


@pytest.mark.parametrize("lengths,ids,N,r,K,M", CASES)
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f16", "f32")])
def test_formulas(lengths, ids, N, r, K, M, dtype, out):
    from offload_memory_centric_amd import layers
    say("adapters", lengths[:8], ids[:8], N, r, K, M, dtype, out)
    c = Case(lengths, ids, N, r, K, M, dtype, out, pad=8, front=2)
    c.fwd(layers)
    c.bwd(layers)


@pytest.mark.parametrize("lengths", [[1] * 70, [100, 17, 60]])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f16", "f32")])
def test_bases_and_accumulation(lengths, dtype, out):
    from offload_memory_centric_amd import layers
    ids = [(7 * i) % 5 - 1 for i in range(len(lengths))]
    c = Case(lengths, ids, 4, 16, 264, 328, dtype, out)
    for base in ("other", "same", None):
        c.fwd(layers, base=base)
        c.bwd(layers, base=base)
    c.fwd(layers, keep=False)
    c.bwd(layers, accumulate=True)
    c.bwd(layers, form_dx=False)


@pytest.mark.parametrize("lengths,N,r,K,M", [([1] * 200, 64, 16, 8192, 4096), ([512], 1, 16, 8192, 2048), ([1], 1, 64, 8192, 8192),
                                             ([3000, 2000], 2, 8, 1024, 4096), ([1] * 3000, 7, 8, 256, 256)])
def test_larger(lengths, N, r, K, M):
    from offload_memory_centric_amd import layers
    say("adapters larger", len(lengths), lengths[:3], N, r, K, M)
    c = Case(lengths, [(3 * i) % (N + 1) - (1 if N > 1 else 0) for i in range(len(lengths))], N, r, K, M, "bf16", "bf16")
    c.fwd(layers)
    c.bwd(layers)


def test_no_rows_and_no_segments():
    from offload_memory_centric_amd import layers
    c = Case([], [], 2, 8, 64, 72, "bf16", "bf16", front=5)
    c.fwd(layers)
    c.bwd(layers)
    c = Case([0, 0], [0, 1], 2, 8, 64, 72, "bf16", "f32")
    dA, dB = torch.full((2, 8, 64), 2.0, device="cuda"), torch.full((2, 8, 72), 2.0, device="cuda")
    U = torch.empty((8, 0), device="cuda")
    layers.adapters_bwd(c.X, c.dY, U, c.A, c.B, c.offsets, c.ids, c.scales, dA, dB, None)
    assert (dA == 0).all() and (dB == 0).all()


@pytest.mark.parametrize("lengths", [[1, 1, 1, 1, 1, 1], [30, 20, 1, 50, 40, 3]])
def test_requests_do_not_reach_each_other(lengths):
    """NaN and infinities in one request's rows, and in one adapter, stay there."""
    from offload_memory_centric_amd import layers
    c = Case(lengths, [0, 1, 2, 0, 1, -1], 3, 16, 136, 200, "bf16", "bf16")
    good = torch.empty((c.T, c.M), dtype=torch.bfloat16, device="cuda")
    got, U = torch.empty_like(good), torch.empty((16, c.T), device="cuda")
    work = layers.workspace(layers.adapters_fwd_bytes(c.T, 16))
    layers.adapters_fwd(c.X, c.A, c.B, c.offsets, c.ids, c.scales, good, work, Y0=c.Y0)
    c.X[c.edge[3]] = float("nan")             # one row of the fourth request
    c.X[c.edge[5]:] = INF                     # a request without an adapter
    c.A[1, 3], c.B[1, 0, 0], c.scales[1] = float("nan"), INF, INF  # the second and fifth requests' adapter
    layers.adapters_fwd(c.X, c.A, c.B, c.offsets, c.ids, c.scales, got, work, Y0=c.Y0, U=U)
    bad = torch.zeros(c.T, dtype=torch.bool, device="cuda")
    bad[c.edge[3]] = True
    bad[c.edge[1]:c.edge[2]] = bad[c.edge[4]:c.edge[5]] = True
    assert torch.equal(got[~bad], good[~bad])
    assert not torch.isfinite(got[bad]).all(1).any()
    work = layers.workspace(layers.adapters_bwd_bytes(c.T, 16))
    dA, dB = torch.empty((3, 16, c.K), device="cuda"), torch.empty((3, 16, c.M), device="cuda")
    dX = torch.empty((c.T, c.K), dtype=torch.bfloat16, device="cuda")
    c.dY[c.edge[5]:] = INF
    layers.adapters_bwd(c.X, c.dY, U, c.A, c.B, c.offsets, c.ids, c.scales, dA, dB, work, dX=dX, dX0=c.dX0)
    bad[c.edge[3]] = False  # its dY and its adapter are sound
    assert torch.isfinite(dX[~bad]).all() and torch.isfinite(dA[2]).all() and torch.isfinite(dB[2]).all()
    assert torch.equal(dX[c.edge[5]:], c.dX0[c.edge[5]:])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_infinities_beside_finite_values(dtype):
    """An infinity and finite values of the other sign in one sum: the sum is the infinity, not NaN."""
    from offload_memory_centric_amd import layers
    T, K, M, r = 40, 64, 72, 2
    one = lambda *shape: torch.ones(shape, dtype=DT[dtype], device="cuda")
    X, dY, A, B = one(T, K), one(T, M), one(1, r, K), one(1, r, M)
    A[0, 1] = -0.125
    offsets, ids = torch.tensor([0, T], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    # U = 64 and -8 times 6e36: the first is past fp32's range where it is scaled
    scales = torch.full((1,), 6e36, device="cuda")
    U, Y = torch.empty((r, T), device="cuda"), torch.empty((T, M), device="cuda")
    layers.adapters_fwd(X, A, B, offsets, ids, scales, Y, layers.workspace(layers.adapters_fwd_bytes(T, r)), U=U)
    assert torch.equal(U, torch.tensor([[64.0], [-8.0]], device="cuda").expand(r, T))
    assert (Y == INF).all()
    U = torch.full((r, T), -4.0, device="cuda")
    U[0, 3] = INF
    dA, dB = torch.empty((1, r, K), device="cuda"), torch.empty((1, r, M), device="cuda")
    layers.adapters_bwd(X, dY, U, A, B, offsets, ids, torch.ones(1, device="cuda"), dA, dB,
                        layers.workspace(layers.adapters_bwd_bytes(T, r)))
    assert (dB[0, 0] == INF).all() and (dB[0, 1] == -4.0 * T).all()
    assert (dA == 1.0 * M * T).all()


def test_offsets_outside_the_rows():
    """Offsets that are not what they should be give rows another adapter or none; nothing outside is read or written."""
    from offload_memory_centric_amd import layers
    T, K, M, r = 200, 64, 72, 8
    for S in (3, 100):
        for edges in ([-50] + [70] * (S - 1) + [1000], [500] * (S + 1), list(range(0, 2 * (S + 1), 2))[::-1]):
            c = Case([T], [0], 1, r, K, M, "bf16", "bf16")
            offsets = torch.tensor(edges, dtype=torch.int32, device="cuda")
            ids = torch.zeros(S, dtype=torch.int32, device="cuda")
            buf = torch.full((T + 8, M), -7.0, dtype=torch.bfloat16, device="cuda")
            work = layers.workspace(layers.adapters_bwd_bytes(T, r))
            U = torch.empty((r, T), device="cuda")
            layers.adapters_fwd(c.X, c.A, c.B, offsets, ids, c.scales, buf[:T], work, Y0=None, U=U)
            dA, dB = torch.empty((1, r, K), device="cuda"), torch.empty((1, r, M), device="cuda")
            layers.adapters_bwd(c.X, c.dY, U, c.A, c.B, offsets, ids, c.scales, dA, dB, work)
            torch.cuda.synchronize()
            full = float(c.scales[0]) * (c.X.double() @ c.A[0].double().t().contiguous() @ c.B[0].double())
            near = (buf[:T].double() - full).abs() <= 0.02 * full.abs() + 0.05
            assert (near | (buf[:T] == 0)).all() and (buf[T:] == -7.0).all()
            assert torch.isfinite(dA).all() and torch.isfinite(dB).all()


def test_far_rows():
    """Rows past 2^32 bytes."""
    from offload_memory_centric_amd import layers
    T, K, M, r = 280000, 8192, 64, 4
    X = torch.zeros((T, K), dtype=torch.bfloat16, device="cuda")
    X[T - 100:, K - 1] = 2.0
    A = torch.zeros((1, r, K), dtype=torch.bfloat16, device="cuda")
    A[0, :, K - 1] = 1.0
    B = torch.ones((1, r, M), dtype=torch.bfloat16, device="cuda")
    offsets, ids = torch.tensor([0, T], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    scales = torch.full((1,), 0.5, device="cuda")
    Y, U = torch.empty((T, M), dtype=torch.bfloat16, device="cuda"), torch.empty((r, T), device="cuda")
    work = layers.workspace(max(layers.adapters_fwd_bytes(T, r), layers.adapters_bwd_bytes(T, r)))
    layers.adapters_fwd(X, A, B, offsets, ids, scales, Y, work, U=U)
    assert (Y[T - 100:] == 4.0).all() and (Y[:T - 100] == 0).all()
    dX = torch.empty((T, K), dtype=torch.bfloat16, device="cuda")
    dA, dB = torch.empty((1, r, K), device="cuda"), torch.empty((1, r, M), device="cuda")
    layers.adapters_bwd(X, Y, U, A, B, offsets, ids, scales, dA, dB, work, dX=dX)
    assert (dX[T - 100:, K - 1] == 512.0).all() and (dX[:, :K - 1] == 0).all() and (dX[:T - 100] == 0).all()
    assert (dA[0, :, K - 1] == 128.0 * 2 * 100).all() and (dB == 0.5 * 2 * 4 * 100).all()
