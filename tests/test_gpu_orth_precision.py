"""The precision of the orthogonalised update (zi_orthogonalize), where its input has directions that are nearly or
wholly empty, or is far smaller than eps, or zero.

Tolerance, relative to the result's norm.  The bf16 result is off by its rounding, at most half a step (2^-8) of
each element, and by the error before it; what |O - exact| leaves above 2^-8 |exact|, element by element, is at most
1 + 2^-8 times the second.  A step rounds three fp16 operands, by 2^-11 of an element at most and 0.42 * 2^-11 in the
root mean square.  Over hundreds of rows these roundings are independent and no step's polynomial enlarges what
they leave in G's own directions by more than it shrinks it in the next, so fifteen of them add up like
sqrt(15) * 0.42 * 2^-11, 0.8 * 2^-10: 2^-10 is taken."""
import pytest
import torch

from zi_testlib import say

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
COEFFS = (3.4445, -4.7750, 2.0315)
MANY = 2.0 ** -10


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def polynomial(G, steps=5, coeffs=COEFFS, eps=1e-7):
    a, b, c, eps = (float(torch.tensor(v, dtype=torch.float32)) for v in (*coeffs, eps))
    X = G.double()
    flip = X.shape[0] > X.shape[1]
    if flip:
        X = X.t().contiguous()
    X = X / (X.square().sum().sqrt() + eps)
    for _ in range(steps):
        A = torch.mm(X, X.t().contiguous())
        X = a * X + torch.mm(b * A + c * torch.mm(A, A), X)
    return X.t().contiguous() if flip else X


def orth(layers, G, **kw):
    M, K = G.shape
    out = torch.full((M, K), float("nan"), dtype=torch.bfloat16, device="cuda")
    layers.orthogonalize(G, out, layers.workspace(layers.orthogonalize_bytes(M, K)).fill_(255), **kw)
    torch.cuda.synchronize()
    return out


def error(got, want):
    """The norm of what got is off by past bf16's rounding, relative to want's."""
    assert torch.isfinite(got).all()
    past = ((got.double() - want).abs() - 2.0 ** -8 * want.abs()).clamp_(min=0)
    return float(past.norm() / want.norm()) / (1 + 2.0 ** -8)


def low_rank(g, M, K, rank, noise=0.0, dtype="f32"):
    G = torch.mm(torch.randn((M, rank), generator=g, device="cuda"), torch.randn((rank, K), generator=g, device="cuda"))
    if noise:
        G.add_(torch.randn((M, K), generator=g, device="cuda"), alpha=noise)
    return G.to(DT[dtype])


@pytest.mark.parametrize("M,K", [(1024, 4096), (2048, 4096), (4096, 2048), (2048, 8192), (4096, 4096), (5700, 6100)])
@pytest.mark.parametrize("rank,noise,dtype", [(1, 0.0, "f32"), (1, 0.0, "bf16"), (16, 0.0, "f32"), (16, 0.01, "bf16"),
                                              (4, 1e-4, "f16")])
def test_low_rank(M, K, rank, noise, dtype):
    """A gradient from fewer tokens than the weight has rows: what the planes of X lose in its empty directions,
    the steps would enlarge nearly 500 times."""
    from offload_memory_centric_amd import layers
    G = low_rank(gen(M + rank), M, K, rank, noise, dtype)
    e = error(orth(layers, G), polynomial(G))
    say("orthogonalise", M, K, "rank", rank, "noise", noise, dtype, "error %.2g" % e)
    assert e <= MANY, e


@pytest.mark.parametrize("M,K", [(300, 1000), (1024, 4096), (2000, 700)])
@pytest.mark.parametrize("norm", [1e-6, 1e-8, 1e-10, 1e-12, 1e-20, 1e-30])
def test_far_below_eps(M, K, norm):
    """X_0 is then far smaller than one, and stays so: every step takes it up by a."""
    from offload_memory_centric_amd import layers
    g = gen(K)
    for rank in (1, min(M, K)):
        G = low_rank(g, M, K, rank)
        G.mul_(norm / float(G.double().norm()))
        e = error(orth(layers, G), polynomial(G))
        say("orthogonalise", M, K, "rank", rank, "norm", norm, "error %.2g" % e)
        assert e <= MANY, e


@pytest.mark.parametrize("coeffs,steps", [((1.5, -0.5, 0.0), 9), ((1.875, -1.25, 0.375), 7), ((3.0, -3.0, 1e-30), 3),
                                          ((1.0, 0.0, 0.0), 4), ((2.0, 0.0, -1.0), 3), ((5.0, 0.0, 0.0), 4),
                                          ((0.25, 0.0, 0.0), 40)])
def test_other_polynomials(coeffs, steps):
    """The largest singular value that X can have, by which its planes are scaled, is the polynomial's: cubic,
    quintic, with two, one or no peak, growing or shrinking without end."""
    from offload_memory_centric_amd import layers
    M, K = 400, 900
    G = low_rank(gen(steps), M, K, M)
    e = error(orth(layers, G, steps=steps, coeffs=coeffs), polynomial(G, steps, coeffs))
    say("orthogonalise", coeffs, steps, "error %.2g" % e)
    assert e <= MANY, e


# Few elements: fifteen roundings need not average out.  2^-11 each; from one step to the next the polynomial's slope
# at the singular values near one (-1.7 to 2.3, alternating) leaves them as large.
FEW = 15 * 2.0 ** -11


@pytest.mark.parametrize("M,K", [(1, 1), (1, 7), (3, 5), (5, 3), (9, 16), (16, 9), (40, 24), (64, 64), (70, 130)])
@pytest.mark.parametrize("rank", [1, 3])
def test_low_rank_small(M, K, rank):
    from offload_memory_centric_amd import layers
    worst = 0.0
    for seed in range(8):
        G = low_rank(gen(seed), M, K, min(rank, M, K))
        worst = max(worst, error(orth(layers, G), polynomial(G)))
    say("orthogonalise", M, K, "rank", rank, "error %.2g" % worst)
    assert worst <= FEW, worst


@pytest.mark.parametrize("M,K", [(70, 90), (90, 70), (1, 1)])
@pytest.mark.parametrize("eps", [0.0, 1e-42, 1e-39])
def test_zero_with_next_to_no_eps(M, K, eps):
    """A zero gradient has no direction: its update is zero, whatever eps."""
    from offload_memory_centric_amd import layers
    Z = torch.zeros((M, K), device="cuda")
    assert not orth(layers, Z, eps=eps).any()


@pytest.mark.parametrize("K", [2000, 20000])
@pytest.mark.parametrize("flip", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_one_row(K, flip, dtype):
    """A single row is multiplied by numbers alone: no element's rounding stays with it, and in the number, a sum over
    the row, they average out.  Fifteen of 0.42 * 2^-11, each over 2000 elements of either weight at least, come to less
    than 2^-12: of elements a step of 2^-8 or more apart, at most one in sixteen falls to the other side."""
    from offload_memory_centric_amd import layers
    for seed in range(3):
        G = torch.randn((1, K), generator=gen(seed), device="cuda").to(DT[dtype])
        G = G.t().contiguous() if flip else G
        off = float((orth(layers, G) != polynomial(G).to(torch.bfloat16)).float().mean())
        say("orthogonalise one row", K, flip, dtype, "not the nearest: %.2g" % off)
        assert off <= 1 / 16, off
