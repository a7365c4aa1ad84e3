"""The precision of the orthogonalised update (zi_orthogonalize), where its input has directions that are nearly or
wholly empty, or is far smaller than eps.

Tolerance, relative to the result's norm.  The bf16 result is off by its rounding, at most half a step (2^-8) of
each element, and by the error before it; what |O - exact| leaves above 2^-8 |exact|, element by element, is at most
1 + 2^-8 times the second.  A step rounds three fp16 operands, by 2^-11 of an element at most."""
import pytest
import torch

from zi_testlib import say

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
COEFFS = (3.4445, -4.7750, 2.0315)


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
