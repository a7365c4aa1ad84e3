"""The orthogonalised update (zi_orthogonalize) against its polynomial in 64 bits.

Tolerances, relative to the result's norm.  The bf16 result is rounded by half
a step, 2^-8 at most.  A step rounds three fp16 operands by 2^-11 at most; what
that adds is carried on by the later steps, whose polynomial's slope at the
singular values near one is between -1.7 and 2.3 (it takes the small ones up
by 3.4, but a rounding meets those through b A + c A^2, which vanishes there):
8 * 2^-11 is taken for all of it.  An element may be six times that, relative
to the root mean square."""
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
    a, b, c = (float(torch.tensor(v, dtype=torch.float32)) for v in coeffs)
    X = G.double()
    flip = X.shape[0] > X.shape[1]
    if flip:
        X = X.t().contiguous()
    X = X / (X.square().sum().sqrt() + eps)
    for _ in range(steps):
        A = torch.mm(X, X.t().contiguous())
        X = a * X + torch.mm(b * A + c * torch.mm(A, A), X)
    return X.t().contiguous() if flip else X


def orth(layers, G, pad=0, **kw):
    M, K = G.shape
    buf = torch.full((M, K + pad), float("nan"), dtype=torch.bfloat16, device="cuda")
    work = layers.workspace(layers.orthogonalize_bytes(M, K)).fill_(255)
    layers.orthogonalize(G, buf[:, :K], work, **kw)
    torch.cuda.synchronize()
    assert torch.isnan(buf[:, K:]).all(), "wrote between the rows"
    again = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    work.fill_(85)
    layers.orthogonalize(G, again, work, **kw)
    torch.cuda.synchronize()
    assert torch.equal(again.view(torch.int16), buf[:, :K].contiguous().view(torch.int16)), "not the same twice"
    return again


def close(got, want, steps=5):
    d = got.double() - want
    own = 8 * 2.0 ** -11
    norm, rms = float(want.norm()), float(want.norm()) / want.numel() ** 0.5
    assert torch.isfinite(got).all()
    assert float(d.norm()) <= (2.0 ** -8 + own) * norm, float(d.norm()) / norm
    worst = float(((d.abs() - 2.0 ** -8 * want.abs()) / rms).max())
    assert worst <= 6 * own, worst


def gradient(g, M, K, dtype, std=0.01):
    r = max(1, min(16, M // 2, K // 2))
    lead = torch.randn((M, r), generator=g, device="cuda") / torch.arange(1, r + 1, device="cuda").sqrt()
    G = torch.mm(lead, torch.randn((r, K), generator=g, device="cuda")) + torch.randn((M, K), generator=g, device="cuda")
    return G.mul_(std).to(DT[dtype])


SHAPES = [(1, 1), (1, 7), (9, 1), (3, 5), (5, 3), (63, 64), (64, 64), (65, 65), (64, 200), (130, 65), (127, 300), (300, 129),
          (128, 128), (129, 1000), (256, 256), (257, 511), (512, 2048), (2048, 512), (1001, 1531), (640, 130), (1500, 1500),
          (16, 20000), (20000, 16), (2000, 4100)]


@pytest.mark.parametrize("M,K", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_shapes(M, K, dtype):
    from offload_memory_centric_amd import layers
    say("orthogonalise", M, K, dtype)
    G = gradient(gen(M + 3 * K), M, K, dtype)
    close(orth(layers, G), polynomial(G))


@pytest.mark.parametrize("M,K", [(5700, 6100), (6016, 5889)])
def test_large_tiles(M, K):
    from offload_memory_centric_amd import layers
    say("orthogonalise", M, K)
    G = gradient(gen(1), M, K, "bf16")
    close(orth(layers, G), polynomial(G))


@pytest.mark.parametrize("steps", [1, 2, 3, 7])
def test_steps_and_coefficients(steps):
    from offload_memory_centric_amd import layers
    G = gradient(gen(steps), 200, 333, "f32")
    close(orth(layers, G, steps=steps), polynomial(G, steps))
    cubic = (1.5, -0.5, 0.0)
    close(orth(layers, G, steps=steps, coeffs=cubic), polynomial(G, steps, cubic))


@pytest.mark.parametrize("M,K", [(150, 260), (260, 150)])
def test_strides(M, K):
    from offload_memory_centric_amd import layers
    g = gen(3)
    for dtype, pad in (("bf16", 3), ("f32", 5), ("f16", 8)):
        buf = torch.full((M, K + pad), float("nan"), dtype=DT[dtype], device="cuda")
        buf[:, :K] = gradient(g, M, K, dtype)
        G = buf[:, :K]
        close(orth(layers, G, pad=2 * pad), polynomial(G))


@pytest.mark.parametrize("M,K", [(300, 700), (900, 400)])
def test_one_direction(M, K):
    """Rank one, exactly: the directions that G does not have stay empty.  (A rounding beside a direction that
    is not there would be multiplied by nearly 500.)"""
    from offload_memory_centric_amd import layers
    g = gen(4)
    u = torch.randint(0, 2, (M, 1), generator=g, device="cuda") * 2.0 - 1
    v = torch.randint(0, 2, (1, K), generator=g, device="cuda") * 2.0 - 1
    G = (u * v).to(torch.bfloat16)
    close(orth(layers, G), polynomial(G))


def test_scale_does_not_matter():
    """Times a power of two, without eps: the same bits, over fp32's range."""
    from offload_memory_centric_amd import layers
    G = gradient(gen(5), 100, 170, "f32", std=1.0)
    want = orth(layers, G, eps=0.0)
    close(want, polynomial(G, eps=0.0))
    for e in (-100, -40, 30, 120):
        got = orth(layers, G * 2.0 ** e, eps=0.0)
        assert torch.equal(got, want), e


def test_zero_nan_and_infinity():
    from offload_memory_centric_amd import layers
    for M, K in ((70, 90), (90, 70), (1, 1)):
        Z = torch.zeros((M, K), device="cuda")
        assert not orth(layers, Z).any()
        for bad in (float("nan"), float("inf"), -float("inf")):
            G = torch.ones((M, K), device="cuda")
            G[M // 2, K // 3] = bad
            assert torch.isnan(orth(layers, G)).all()


def test_singular_values():
    """They lie where the polynomial takes them: near one."""
    from offload_memory_centric_amd import layers
    G = gradient(gen(6), 256, 1024, "f32")
    s = torch.linalg.svdvals(orth(layers, G).float())
    assert 0.6 < float(s.min()) and float(s.max()) < 1.3


def test_streams_and_graph():
    from offload_memory_centric_amd import layers
    g = gen(7)
    M, K = 300, 1000
    G = gradient(g, M, K, "f32")
    work = layers.workspace(layers.orthogonalize_bytes(M, K))
    O, O0 = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda"), torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    layers.orthogonalize(G, O, work, stream=side)
    side.synchronize()
    layers.orthogonalize(G, O0, work)
    torch.cuda.synchronize()
    assert torch.equal(O, O0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layers.orthogonalize(G, O, work)
    for k in range(4):
        G.copy_(gradient(g, M, K, "f32"))
        layers.orthogonalize(G, O0, work)
        torch.cuda.synchronize()
        O.fill_(float("nan"))
        work.fill_(k)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(O, O0), k
