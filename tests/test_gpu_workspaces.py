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
