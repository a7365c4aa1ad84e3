"""The layer norm's backward in place, where a workgroup has several rows at a time and the last has fewer left: the
threads without a row have no part in the sums, whatever becomes of the other rows meanwhile."""
import pytest
import torch

from zi_testlib import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,D", [(1, 8), (17, 100), (17, 128), (33, 128), (5, 130), (6, 512), (7, 513), (13, 1000), (9, 1024),
                                 (20481, 128)])
@pytest.mark.parametrize("over", ["S", "dS", "dY"])
def test_last_row_overflows(T, D, over):
    """dX of the last row is past fp16's range: infinite where it is stored, and no other result's business."""
    from offload_memory_centric_amd import layers
    say("layer norm backward in place", T, D, over)
    g = torch.Generator(device="cuda")
    g.manual_seed(T + D)
    t = {k: torch.randn((T, D), generator=g, device="cuda").half() for k in ("S", "dS", "dY")}
    t["dS"][-1] = 65504.0
    t["dY"][-1] *= 1000
    S = t["S"].float()
    mean, rstd = S.mean(1), (S.var(1, correction=0) + 1e-5).rsqrt()
    gamma = torch.randn(D, generator=g, device="cuda")
    work = layers.workspace(layers.layer_norm_bwd_bytes(T, D))

    def run(t, dX):
        dg, db = torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
        layers.layer_norm_bwd(t["dY"], t["S"], gamma, mean, rstd, dX, dg, db, work, dS=t["dS"])
        torch.cuda.synchronize()
        return dX, dg, db

    dX, dg, db = run(t, torch.empty_like(t["S"]))
    assert D < 100 or torch.isinf(dX[-1]).any()
    assert torch.isfinite(dg).all() and torch.isfinite(db).all()
    for _ in range(4):
        u = {k: v.clone() for k, v in t.items()}
        x, g1, b1 = run(u, u[over])
        assert torch.equal(x, dX) and torch.equal(g1, dg) and torch.equal(b1, db)


@pytest.mark.parametrize("T,D", [(17, 100), (33, 128), (5, 130), (13, 1000)])
def test_forward_last_row(T, D):
    from offload_memory_centric_amd import layers
    say("layer norm forward in place", T, D)
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    X, R = torch.randn((T, D), generator=g, device="cuda").half(), torch.randn((T, D), generator=g, device="cuda").half()
    gamma = torch.full((D,), 65504.0, device="cuda")
    out = [torch.empty_like(X), torch.empty_like(X), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")]
    layers.layer_norm_fwd(X, gamma, None, out[1], out[2], out[3], R=R, S=out[0])
    for _ in range(4):
        x, r, m, s = X.clone(), R.clone(), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
        layers.layer_norm_fwd(x, gamma, None, r, m, s, R=r, S=x)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((x, r, m, s), out))
