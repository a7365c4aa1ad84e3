"""Grouped products whose smaller tiles would be more workgroups than a launch has: exactly, on small whole numbers."""
import pytest
import torch

from zi_testlib import say

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def whole(g, *shape):
    return torch.randint(-3, 4, shape, generator=g, device="cuda", dtype=torch.int8).to(BF)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def index(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def test_half_a_billion_rows():
    """2^29 rows of eight columns: the forward and dX."""
    from offload_memory_centric_amd import layers
    g, R, block = gen(1), 1 << 29, 1 << 20
    say("grouped rows", R)
    W, part = whole(g, 1, 8, 8), whole(g, block, 8)
    X = torch.empty((R, 8), dtype=BF, device="cuda")
    X.view(R // block, block, 8).copy_(part.expand(R // block, block, 8))
    out = torch.full((R, 8), -77.0, dtype=BF, device="cuda")
    offsets = index([3, R - 2])
    for run, w in ((layers.grouped_fwd, W[0].float().t().contiguous()), (layers.grouped_dx, W[0].float())):
        out.fill_(-77.0)
        run(X, W, offsets, out)
        want = (part.float() @ w).to(BF)
        assert (out[:3] == -77.0).all() and (out[R - 2:] == -77.0).all()
        out[:3], out[R - 2:] = want[:3], want[block - 2:]
        for k in range(R // block):
            assert torch.equal(out[k * block:(k + 1) * block], want), k


def test_many_wide_experts_of_a_row():
    """4096 experts of a row each, 8 -> 131072: the forward, and dX of 131072 -> 8."""
    from offload_memory_centric_amd import layers
    g, E, K, M = gen(2), 4096, 8, 131072
    say("grouped experts", E, K, M)
    X, offsets = whole(g, E, K), index(list(range(E + 1)))
    W, Y = whole(g, E, M, K), torch.empty((E, M), dtype=BF, device="cuda")
    layers.grouped_fwd(X, W, offsets, Y)
    for e0 in range(0, E, 64):
        want = (W[e0:e0 + 64].float() * X[e0:e0 + 64].float()[:, None, :]).sum(2)
        assert torch.equal(Y[e0:e0 + 64].float(), want), e0
    V = W.view(E, K, M)  # the same elements as weights of 131072 -> 8
    layers.grouped_dx(X, V, offsets, Y)
    for e0 in range(0, E, 64):
        want = (V[e0:e0 + 64].float() * X[e0:e0 + 64].float()[:, :, None]).sum(1)
        assert torch.equal(Y[e0:e0 + 64].float(), want), e0


def test_weight_gradients_of_many_experts():
    """4096 gradients of 131072 x 8, most of them of no row."""
    from offload_memory_centric_amd import layers
    g, E, K, M, R = gen(3), 4096, 8, 131072, 768
    say("grouped gradients", E, K, M, R)
    edges = [min(R, e // 5) for e in range(E)] + [R]
    X, dY, dW = whole(g, R, K), whole(g, R, M), torch.full((E, M, K), 5.0, dtype=BF, device="cuda")
    layers.grouped_dw(X, dY, index(edges), dW)
    for e in range(E):
        a, b = edges[e], edges[e + 1]
        if a == b:
            assert not dW[e].any(), e
        else:
            want = (dY[a:b].float()[:, :, None] * X[a:b].float()[:, None, :]).sum(0)
            assert torch.equal(dW[e].float(), want), e
