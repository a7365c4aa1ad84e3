"""The layer norm's backward of rows so long that one thread for each of their columns' partial sums would be more
than a launch can have."""
import pytest
import torch

from zi_testlib import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.mark.parametrize("T", [1, 2])
def test_rows_past_2_27(T):
    """Sums over the rows of dY h and dY: of one row dbeta is dY itself; a product and a difference more, and a sum
    with a second row, add u of each result.  A row's own sums are as long as the row and not compared here."""
    from offload_memory_centric_amd import layers
    D = (1 << 27) + 5
    say("layer norm backward", T, D)
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    S, dY = (torch.empty((T, D), dtype=torch.float16, device="cuda").normal_(generator=g) for _ in range(2))
    mean, rstd = torch.full((T,), 0.25, device="cuda"), torch.full((T,), 0.75, device="cuda")
    dX, dg, db = torch.empty_like(S), torch.full((D,), float("nan"), device="cuda"), torch.full((D,), float("nan"), device="cuda")
    layers.layer_norm_bwd(dY, S, None, mean, rstd, dX, dg, db, layers.workspace(layers.layer_norm_bwd_bytes(T, D)))
    torch.cuda.synchronize()
    for first in range(0, D, 1 << 24):
        at = slice(first, first + (1 << 24))
        d = dY[:, at].double()
        p = d * (S[:, at].double() - 0.25) * 0.75
        assert ((dg[at].double() - p.sum(0)).abs() <= (3 + T) * U * p.abs().sum(0) * 1.01).all(), first
        assert ((db[at].double() - d.sum(0)).abs() <= T * U * d.abs().sum(0)).all(), first
    assert torch.isfinite(dX[:, ::1 << 20]).all() and torch.isfinite(dX[:, -8:]).all()
