"""One workspace, made for the largest call, for smaller ones."""
import pytest
import torch

from zi_testlib import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,D", [(8000, 1024), (8193, 1024), (9000, 500), (16384, 512), (300, 1024), (1, 8)])
def test_embedding_gradient(T, D):
    """The sums of whole numbers are exact in any order."""
    from offload_memory_centric_amd import layers
    V = 40
    say("embedding gradient", T, D, "in the workspace of 16384 x 1024")
    work = layers.workspace(layers.embedding_bwd_bytes(16384, V, 1024)).fill_(255)
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    ids = torch.randint(-2, V, (T,), generator=g, device="cuda")
    dX = torch.randint(-8, 9, (T, D), generator=g, device="cuda").float()
    dW = torch.full((V, D), float("nan"), device="cuda")
    layers.embedding_bwd(ids, dX, dW, work)
    torch.cuda.synchronize()
    at = ids >= 0
    assert torch.equal(dW, torch.zeros((V, D), device="cuda").index_add_(0, ids[at], dX[at]))


@pytest.mark.parametrize("T,D", [(2000, 4096), (2000, 4097), (2000, 8192), (2000, 8193), (600, 4000), (3, 8)])
def test_norm_backward(T, D):
    """dbeta, the sum of dY, is exact for whole numbers; the same bits as with a workspace of the call's own."""
    from offload_memory_centric_amd import layers
    say("layer norm backward", T, D, "in the workspace of 2000 x 8193")
    work = layers.workspace(layers.layer_norm_bwd_bytes(2000, 8193)).fill_(255)
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    S = torch.randn((T, D), generator=g, device="cuda")
    dY = torch.randint(-8, 9, (T, D), generator=g, device="cuda").float()
    mean, rstd = S.mean(1), (S.var(1, correction=0) + 1e-5).rsqrt()
    out = []
    for w in (work, layers.workspace(layers.layer_norm_bwd_bytes(T, D))):
        dX, dg, db = torch.empty_like(S), torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
        layers.layer_norm_bwd(dY, S, None, mean, rstd, dX, dg, db, w)
        torch.cuda.synchronize()
        out.append((dX, dg, db))
    assert torch.equal(out[0][2], dY.sum(0))
    assert all(torch.equal(a, b) for a, b in zip(*out))
