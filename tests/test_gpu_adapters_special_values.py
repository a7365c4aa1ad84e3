"""Infinities, unused adapters and values at the ends of the types' ranges in the adapters (zi_adapters_fwd,
zi_adapters_bwd)."""
import pytest
import torch

from zi_testlib import say

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
INF, NAN = float("inf"), float("nan")


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def index(*values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


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
