"""Infinities, unused adapters and values at the ends of the types' ranges in the adapters (zi_adapters_fwd,
zi_adapters_bwd), against their formulas in 64 bits.

Where the formula's sum has one infinite product the result is that infinity, where it has 0 times infinity or
infinities of both signs it is NaN, in every kernel that the lengths of the segments choose; the other elements of Y
are the same bits as without the infinity.  Tolerances of finite values: u2 = 2^-23 covers an fp32 operation that truncates; a
sum of n products, three for each factor of U (its planes), is off by n u2 of the sum of their magnitudes, and in fp16
a factor of U is off by 2^-22 of itself (two roundings to 11 bits, 2^-11 each) or by 2^-39 of the largest that shares
its scale (half of the last unit, 2^-24, where that largest is 2^14 or more)."""
import pytest
import torch

from zi_testlib import say

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
U2 = 2.0 ** -23
INF, NAN = float("inf"), float("nan")


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def index(*values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def product(a, b):
    """a^T b in 64 bits, elementwise products (so that infinities meet what they meet), and the sum of their magnitudes."""
    p = a.double()[:, :, None] * b.double()[:, None, :]
    return p.sum(0), p.abs().sum(0)


def same(got, want, tol, what):
    """Infinities and NaN in the same places, finite values within tol."""
    assert torch.equal(torch.isnan(got), torch.isnan(want)), "%s: NaN at %d places, expected at %d" % (
        what, int(torch.isnan(got).sum()), int(torch.isnan(want).sum()))
    inf = torch.isinf(want)
    assert torch.equal(torch.isinf(got), inf) and torch.equal(got[inf].double(), want[inf]), what + ": infinities"
    ok = torch.isfinite(want)
    bad = (got[ok].double() - want[ok]).abs() > (tol[ok] if torch.is_tensor(tol) else tol)
    assert not bad.any(), "%s: %d finite values outside" % (what, int(bad.sum()))


# expand_row_kernel (segments of a row) and expand_kernel with one held step, two, and more ranks than it holds
LENGTHS = [([1] * 5, 24), ([37], 3), ([40, 9], 48), ([50], 70)]


@pytest.mark.parametrize("lengths,r", LENGTHS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_infinite_b_reaches_its_column_as_an_infinity(lengths, r, dtype):
    from offload_memory_centric_amd import layers
    say("infinite B", lengths, r, dtype)
    g, T, K, M, S = gen(3), sum(lengths), 64, 136, len(lengths)
    X = torch.randn((T, K), generator=g, device="cuda").to(DT[dtype])
    A = torch.randn((1, r, K), generator=g, device="cuda").to(DT[dtype])
    B = torch.randn((1, r, M), generator=g, device="cuda").to(DT[dtype])
    A[0, 1] = 0  # a rank whose U is zero
    X[:, 0] = X[:, 1] = 0
    X[2, 0], A[0, 0, 0] = 2.0 ** -24, 2.0 ** -24  # and one far below its row's largest, 2^-48
    A[0, 0, 1:] = 0
    edges = [0]
    for n in lengths:
        edges.append(edges[-1] + n)
    offsets, ids = index(*edges), index(*[0] * S)
    scales = torch.full((1,), 0.75, device="cuda")
    U, Y, good = torch.empty((r, T), device="cuda"), torch.empty((T, M), device="cuda"), torch.empty((T, M), device="cuda")
    work = layers.workspace(layers.adapters_fwd_bytes(T, r))
    layers.adapters_fwd(X, A, B, offsets, ids, scales, good, work)
    B[0, 2, 0], B[0, 2, 9], B[0, 2, 130] = INF, -INF, INF  # a column each
    B[0, 0, 17], B[0, 1, 33], B[0, 2, 47], B[0, 1, 47] = INF, INF, INF, 1.0
    layers.adapters_fwd(X, A, B, offsets, ids, scales, Y, work, U=U)
    assert float(U[0, 2]) == 2.0 ** -48 and (U[1] == 0).all()
    want, size = product(U.double() * 0.75, B[0])
    assert torch.isnan(want[:, 33]).all() and torch.isinf(want[:, 0]).all() and float(want[2, 17]) == INF
    largest = (U.double().abs() * 0.75).amax(0)[:, None] * 2.0 ** -39 * B[0].double().abs().nan_to_num(posinf=0).sum(0)[None]
    same(Y, want, (3 * r + 8) * U2 * size + largest, "Y")
    for m in set(range(M)) - {0, 9, 130, 17, 33, 47}:
        assert torch.equal(Y[:, m], good[:, m])


@pytest.mark.parametrize("lengths,r", LENGTHS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_infinite_a_reaches_its_column_of_dx(lengths, r, dtype):
    from offload_memory_centric_amd import layers
    say("infinite A", lengths, r, dtype)
    g, T, K, M, S = gen(4), sum(lengths), 136, 64, len(lengths)
    X = torch.randn((T, K), generator=g, device="cuda").to(DT[dtype])
    dY = torch.randn((T, M), generator=g, device="cuda").to(DT[dtype])
    A = torch.randn((1, r, K), generator=g, device="cuda").to(DT[dtype])
    B = torch.zeros((1, r, M), dtype=DT[dtype], device="cuda")
    for q in range(r):
        B[0, q, q % M] = 0.5 + q / 256  # dU is a product each, exact in fp32
    edges = [0]
    for n in lengths:
        edges.append(edges[-1] + n)
    offsets, ids, scales = index(*edges), index(*[0] * S), torch.ones(1, device="cuda")
    dX, dA, dB = torch.empty((T, K), device="cuda"), torch.empty((1, r, K), device="cuda"), torch.empty((1, r, M), device="cuda")
    U = torch.zeros((r, T), device="cuda")
    A[0, 0, 0], A[0, 2, 9], A[0, 1, 135] = INF, -INF, INF
    layers.adapters_bwd(X, dY, U, A, B, offsets, ids, scales, dA, dB, layers.workspace(layers.adapters_bwd_bytes(T, r)), dX=dX)
    dU = (B[0].double() @ dY.double().t().contiguous()).float()
    want, size = product(dU, A[0])
    assert int(torch.isinf(want).sum()) == 3 * T - int((dU[:3] == 0).sum())
    largest = dU.double().abs().amax(0)[:, None] * 2.0 ** -39 * A[0].double().abs().nan_to_num(posinf=0).sum(0)[None]
    same(dX, want, (3 * r + 8) * U2 * size + largest, "dX")


@pytest.mark.parametrize("r", [3, 24, 40])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_infinite_rows_reach_the_gradients_as_infinities(r, dtype):
    from offload_memory_centric_amd import layers
    say("infinite X, dY", r, dtype)
    g, T, K, M = gen(5), 75, 136, 72
    X = torch.randn((T, K), generator=g, device="cuda").to(DT[dtype])
    dY = torch.randn((T, M), generator=g, device="cuda").to(DT[dtype])
    A = torch.randn((1, r, K), generator=g, device="cuda").to(DT[dtype])
    B = torch.zeros((1, r, M), dtype=DT[dtype], device="cuda")
    for q in range(r):
        B[0, q, q] = 0.5 + q / 256  # dU is a product each, exact in fp32
    U = torch.randn((r, T), generator=g, device="cuda") * 0.1
    U[0, 7], U[1, 7], U[2, 7] = 0.1, 0.0, 1e-14
    offsets, ids, scales = index(0, T), index(0), torch.full((1,), 0.5, device="cuda")
    dA, dB = torch.empty((1, r, K), device="cuda"), torch.empty((1, r, M), device="cuda")
    work = layers.workspace(layers.adapters_bwd_bytes(T, r))

    def gradients():
        layers.adapters_bwd(X, dY, U, A, B, offsets, ids, scales, dA, dB, work)

    X[70, 0], X[7, 100], X[8, 100] = INF, -INF, 1.0
    gradients()
    dU = (0.5 * (B[0].double() @ dY.double().t().contiguous())).float()
    want, size = product(dU.t().contiguous(), X)
    assert torch.isinf(want[:, 0]).sum() + torch.isnan(want[:, 0]).sum() == r
    largest = dU.double().abs().amax(1)[:, None] * 2.0 ** -39 * X.double().abs().nan_to_num(posinf=0).sum(0)[None]
    same(dA[0], want, (3 * T + 12) * U2 * size + largest, "dA")
    X[70, 0] = X[7, 100] = 1.0
    dY[7, 3], dY[60, 71] = INF, -INF
    gradients()
    want, size = product(U.t().contiguous(), dY)
    want, size = 0.5 * want, 0.5 * size
    assert float(want[0, 3]) == INF and torch.isnan(want[1, 3]) and float(want[2, 3]) == INF
    largest = U.double().abs().amax(1)[:, None] * 2.0 ** -39 * dY.double().abs().nan_to_num(posinf=0).sum(0)[None]
    same(dB[0], want, (3 * T + 12) * U2 * size + largest, "dB")


@pytest.mark.parametrize("scale", [INF, NAN])
@pytest.mark.parametrize("lengths", [[40, 0, 25], [2000, 0, 1000]])  # one split of the rows, several
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_scales_of_adapters_without_rows(scale, lengths, dtype):
    """An adapter that no segment names, and one whose segment is empty: zero gradients, or what was there, whatever
    their scales."""
    from offload_memory_centric_amd import layers
    say("scales without rows", scale, lengths, dtype)
    g, T, K, M, N, r = gen(6), sum(lengths), 72, 136, 4, 8
    X = torch.randn((T, K), generator=g, device="cuda").to(DT[dtype])
    dY = torch.randn((T, M), generator=g, device="cuda").to(DT[dtype])
    A = torch.randn((N, r, K), generator=g, device="cuda").to(DT[dtype])
    B = torch.randn((N, r, M), generator=g, device="cuda").to(DT[dtype])
    U = torch.randn((r, T), generator=g, device="cuda")
    offsets, ids = index(0, lengths[0], lengths[0], T), index(0, 1, 2)
    work = layers.workspace(layers.adapters_bwd_bytes(T, r))
    scales = torch.full((N,), 0.5, device="cuda")
    for accumulate in (False, True):
        out = []
        for bad in (False, True):
            s = scales.clone()
            if bad:
                s[1] = s[3] = scale
            dA, dB = torch.full((N, r, K), 2.0, device="cuda"), torch.full((N, r, M), 3.0, device="cuda")
            dA[1, 0, :5] = dB[1, 0, :5] = dB[3, 7, 9:] = -0.0
            kept = dA.clone(), dB.clone()
            layers.adapters_bwd(X, dY, U, A, B, offsets, ids, s, dA, dB, work, accumulate=accumulate)
            for n in (1, 3):
                for got, was in zip((dA, dB), kept):
                    want = was[n] if accumulate else torch.zeros_like(was[n])
                    assert torch.equal(got[n].view(torch.int32), want.view(torch.int32)), (n, accumulate, bad)
            out.append((dA, dB))
        assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])


@pytest.mark.parametrize("lengths", [[1] * 5, [40]])
def test_bf16_values_at_the_end_of_fp32s_range(lengths):
    """A finite factor that rounds to bf16's infinity is still finite: Y and the gradients are, too."""
    from offload_memory_centric_amd import layers
    say("end of the range", lengths)
    T, K, M, r, S = sum(lengths), 64, 72, 2, len(lengths)
    top = float(torch.finfo(torch.float32).max)
    bf = torch.bfloat16
    X, dY = torch.zeros((T, K), dtype=bf, device="cuda"), torch.zeros((T, M), dtype=bf, device="cuda")
    A, B = torch.zeros((1, r, K), dtype=bf, device="cuda"), torch.zeros((1, r, M), dtype=bf, device="cuda")
    X[:, 0], A[0, 0, 0], B[0, 0] = 1.0, 1.0, 2.0 ** -10
    offsets, ids = index(*range(0, T, 1), T) if S > 1 else index(0, T), index(*[0] * S)
    Y = torch.empty((T, M), device="cuda")
    layers.adapters_fwd(X, A, B, offsets, ids, torch.full((1,), top, device="cuda"), Y,
                        layers.workspace(layers.adapters_fwd_bytes(T, r)))
    assert torch.isfinite(Y).all() and ((Y.double() / (top * 2.0 ** -10) - 1).abs() <= 4 * U2).all()
    U = torch.zeros((r, T), device="cuda")
    U[0, T - 1] = -top
    dY[:, 0] = 2.0 ** -10
    dA, dB = torch.empty((1, r, K), device="cuda"), torch.empty((1, r, M), device="cuda")
    layers.adapters_bwd(X, dY, U, A, B, offsets, ids, torch.ones(1, device="cuda"), dA, dB,
                        layers.workspace(layers.adapters_bwd_bytes(T, r)))
    assert torch.isfinite(dB).all() and abs(float(dB[0, 0, 0]) / (-top * 2.0 ** -10) - 1) <= 4 * U2
    assert (dB[0, 1] == 0).all() and (dB[0, 0, 1:] == 0).all()
