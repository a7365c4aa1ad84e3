"""Token embedding (zi_embedding_fwd, zi_embedding_bwd) against its formulas in 64 bits.

Tolerances.  u = 2^-24 is fp32's half step.  The gradient of a row with c
tokens adds at most 64 of them in a row, then its pieces, at most c / 64 + 2:
its error is at most (c / 64 + 70) u sum|dX|, scaled, plus u of the product
and of the sum with the old value; a stored value adds half a step of its
type."""
import pytest
import torch

from zi_testlib import say

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
U = 2.0 ** -24


def half(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rows(g, T, D, dtype, pad=0):
    buf = torch.full((T, D + pad), float("nan"), dtype=dtype, device="cuda")
    buf[:, :D] = torch.randn((T, D), generator=g, device="cuda").to(dtype)
    return buf[:, :D], buf


def make_ids(g, T, V, kind, dtype=torch.int64):
    if kind == "zipf":
        ids = ((V + 1.0) ** torch.rand(T, generator=g, device="cuda", dtype=torch.float64)).long().sub_(1).clamp_(0, V - 1)
    elif kind == "same":
        ids = torch.full((T,), V // 2, dtype=torch.int64, device="cuda")
    elif kind == "padding":
        ids = torch.full((T,), -1, dtype=torch.int64, device="cuda")
    elif kind == "falling":
        ids = torch.arange(T - 1, -1, -1, device="cuda") * V // max(T, 1)
    else:  # uniform, with padding and ids outside the table on both sides
        ids = torch.randint(-3, V + 3, (T,), generator=g, device="cuda")
    return ids.to(dtype)


def close(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), "%s: %d of %d outside" % (what, int(bad.sum()), bad.numel())


@pytest.mark.parametrize("T,V,D", [(1, 1, 1), (1, 5, 8192), (3, 7, 9), (100, 50, 127), (33, 40, 129), (65, 30, 512),
                                   (20, 9, 1000), (7, 100, 16385), (5, 3, 40000), (70000, 11, 8)])
@pytest.mark.parametrize("w,x", [("f16", "f16"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "f16"), ("f32", "bf16"),
                                 ("f16", "f32"), ("bf16", "f16")])
def test_forward(T, V, D, w, x):
    from offload_memory_centric_amd import layers
    say("embedding forward", T, V, D, w, x)
    g = gen(T + D)
    for kind, dtype, pad, scale in (("uniform", torch.int64, 0, 1.0), ("zipf", torch.int32, 3, 1.7)):
        ids = make_ids(g, T, V, kind, dtype)
        W, wb = rows(g, V, D, DT[w], pad)
        X = torch.full((T, D + 2 * pad), float("nan"), dtype=DT[x], device="cuda")
        layers.embedding_fwd(ids, W, X[:, :D], scale=scale)
        torch.cuda.synchronize()
        assert torch.isnan(X[:, D:]).all()
        ok = (ids >= 0) & (ids < V)
        sc = float(torch.tensor(scale, dtype=torch.float32))
        want = W.double()[ids.long().clamp(0, V - 1)] * sc * ok[:, None]
        close(X[:, :D], want, half(DT[x]) * want.abs() + U * want.abs() * 1.01 + tiny(DT[x]) * (want != 0), "X")
        assert not X[:, :D][~ok].any()


def check_bwd(layers, T, V, D, kind, dx="f32", dw="f32", pad=0, acc=False, scale=1.0, dtype=torch.int64, seed=3):
    g = gen(seed)
    ids = make_ids(g, T, V, kind, dtype)
    dX, xb = rows(g, T, D, DT[dx], pad)
    buf = torch.full((V, D + 2 * pad), float("nan"), dtype=DT[dw], device="cuda")
    dW = buf[:, :D]
    if acc:
        dW.copy_(torch.randn((V, D), generator=g, device="cuda"))
    before = dW.double() if acc else torch.zeros((V, D), dtype=torch.float64, device="cuda")
    work = layers.workspace(layers.embedding_bwd_bytes(T, V, D)).fill_(0)
    layers.embedding_bwd(ids, dX, dW, work, scale=scale, accumulate=acc)
    torch.cuda.synchronize()
    if pad:
        assert torch.isnan(buf[:, D:]).all(), "wrote between the rows"
    at = torch.nonzero((ids >= 0) & (ids < V)).squeeze(1)
    i = ids[at].long()
    sc = float(torch.tensor(scale, dtype=torch.float32))
    total, size = torch.zeros((V, D), dtype=torch.float64, device="cuda"), torch.zeros((V, D), dtype=torch.float64, device="cuda")
    total.index_add_(0, i, dX[at].double())
    size.index_add_(0, i, dX[at].double().abs())
    count = torch.bincount(i, minlength=V).double()[:, None]
    want = before + total * sc
    tol = (count / 64 + 72) * U * size * abs(sc) * 1.01 + (half(DT[dw]) + U) * want.abs() + tiny(DT[dw]) * (size > 0)
    close(dW, want, tol, "dW")
    assert torch.equal(dW[count[:, 0] == 0].double(), before[count[:, 0] == 0]), "rows without a token"
    # again, over a workspace full of ones and of places in the list: the same bits
    for fill in (255, 1):
        out = torch.empty_like(dW)
        if acc:
            out.copy_(before)
        work.fill_(fill)
        layers.embedding_bwd(ids, dX, out, work, scale=scale, accumulate=acc)
        torch.cuda.synchronize()
        assert torch.equal(out, dW), "not the same twice"


BWD = [(1, 1, 1), (1, 9, 100), (2, 3, 7), (63, 5, 8), (64, 5, 9), (65, 70, 33), (128, 2, 512), (129, 1000, 100), (1000, 37, 65),
       (1023, 10, 16), (1024, 2000, 16), (1025, 10, 16), (2047, 5000, 40), (4096, 300, 24), (32767, 900, 8), (32768, 60000, 8),
       (32769, 100, 8), (40001, 7, 8), (300, 20, 2049), (40, 6, 9000)]


@pytest.mark.parametrize("T,V,D", BWD)
@pytest.mark.parametrize("kind", ["uniform", "zipf", "same", "padding", "falling"])
def test_backward(T, V, D, kind):
    from offload_memory_centric_amd import layers
    say("embedding backward", T, V, D, kind)
    check_bwd(layers, T, V, D, kind)


@pytest.mark.parametrize("dx", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("dw", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("acc", [False, True])
def test_backward_types(dx, dw, acc):
    from offload_memory_centric_amd import layers
    say("embedding backward types", dx, dw, acc)
    check_bwd(layers, 777, 200, 130, "zipf", dx, dw, pad=3, acc=acc, scale=-2.3, dtype=torch.int32)
    check_bwd(layers, 3000, 50, 24, "uniform", dx, dw, acc=acc, scale=11.3)


def test_backward_two_merges_and_wide_ids():
    from offload_memory_centric_amd import layers
    check_bwd(layers, 1_100_003, 50257, 8, "zipf", "bf16", "f32")
    g = gen(4)  # ids far outside 32 bits are padding, not wrapped
    ids = torch.tensor([0, 1 << 32, (1 << 32) + 1, -(1 << 40), 1, (1 << 62)], device="cuda")
    dX = torch.randn((6, 16), generator=g, device="cuda")
    dW = torch.empty((3, 16), device="cuda")
    layers.embedding_bwd(ids, dX, dW, layers.workspace(layers.embedding_bwd_bytes(6, 3, 16)))
    X = torch.empty_like(dX)
    layers.embedding_fwd(ids, dW, X)
    torch.cuda.synchronize()
    assert torch.equal(dW, torch.stack([dX[0], dX[4], torch.zeros_like(dX[0])]))
    assert torch.equal(X, torch.where((ids < 2)[:, None] & (ids >= 0)[:, None], dX, torch.zeros_like(dX)))


def test_backward_without_tokens():
    from offload_memory_centric_amd import layers
    ids, dX = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty((0, 40), device="cuda")
    dW = torch.full((5, 40), 3.0, device="cuda")
    layers.embedding_bwd(ids, dX, dW, None, accumulate=True)
    torch.cuda.synchronize()
    assert (dW == 3).all()
    layers.embedding_bwd(ids, dX, dW, None)
    torch.cuda.synchronize()
    assert not dW.any()


def test_special_values_stay_in_their_rows():
    from offload_memory_centric_amd import layers
    ids = torch.tensor([1, 2, -1, 1], device="cuda")
    dX = torch.ones((4, 24), device="cuda")
    dX[1, 3], dX[2, 5] = float("inf"), float("nan")   # the second is a padding position
    dW = torch.empty((4, 24), device="cuda")
    layers.embedding_bwd(ids, dX, dW, layers.workspace(layers.embedding_bwd_bytes(4, 4, 24)))
    torch.cuda.synchronize()
    want = torch.zeros((4, 24), device="cuda")
    want[1], want[2], want[2, 3] = 2, 1, float("inf")
    assert torch.equal(dW, want)


def test_streams_and_graph():
    from offload_memory_centric_amd import layers
    g = gen(7)
    T, V, D = 3000, 700, 264
    ids = make_ids(g, T, V, "zipf")
    W, dX = torch.randn((V, D), generator=g, device="cuda"), torch.randn((T, D), generator=g, device="cuda")
    work = layers.workspace(layers.embedding_bwd_bytes(T, V, D))
    X, dW = torch.zeros_like(dX), torch.zeros_like(W)
    X0, dW0 = torch.zeros_like(dX), torch.zeros_like(W)

    def both(x, w, stream=None):
        layers.embedding_fwd(ids, W, x, scale=3.0, stream=stream)
        layers.embedding_bwd(ids, dX, w, work, scale=3.0, stream=stream)

    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    both(X, dW, side)
    side.synchronize()
    both(X0, dW0)
    torch.cuda.synchronize()
    assert torch.equal(X, X0) and torch.equal(dW, dW0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(X, dW)
    for k in range(4):
        ids.copy_(make_ids(g, T, V, "uniform"))
        both(X0, dW0)
        torch.cuda.synchronize()
        X.fill_(float("nan"))
        dW.fill_(float("nan"))
        work.fill_(k)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(X, X0) and torch.equal(dW, dW0), k


def test_offsets_past_32_bits():
    """A table of more than 2^32 bytes and 2^31 elements: its first and last rows."""
    from offload_memory_centric_amd import layers
    V, D, T = 270000, 8200, 300
    g = gen(12)
    W = torch.empty((V, D), dtype=torch.float16, device="cuda")
    W[:100].normal_(generator=g)
    W[-100:].normal_(generator=g)
    ids = torch.randint(0, 100, (T,), generator=g, device="cuda")
    ids[::2] += V - 100
    X = torch.empty((T, D), dtype=torch.float16, device="cuda")
    layers.embedding_fwd(ids, W, X)
    torch.cuda.synchronize()
    assert torch.equal(X, W[ids])
    W.fill_(7)
    layers.embedding_bwd(ids, X, W, layers.workspace(layers.embedding_bwd_bytes(T, V, D)))
    low = torch.where(ids >= 100, ids - (V - 200), ids)
    small = torch.empty((200, D), dtype=torch.float16, device="cuda")
    layers.embedding_bwd(low, X, small, layers.workspace(layers.embedding_bwd_bytes(T, 200, D)))
    torch.cuda.synchronize()
    assert torch.equal(W[:100], small[:100]) and torch.equal(W[-100:], small[-100:])
    assert not W[100:-100].any()
