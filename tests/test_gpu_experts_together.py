"""The operators of a mixture of experts together, as a training step runs them; adapters beside the tiled linear; both
on another stream, replayed from a graph, and twice with the same bits.

Tolerance of the step.  Against the same formulas in 64 bits on the same (16-bit) inputs, every tensor that is stored in
16 bits on the way adds half a step of its type, h = 2^-9 relative for bf16 and 2^-12 for fp16 (as a norm: a rounding is
at most half a step of its element), to everything that follows; the fp32 sums add far less.  A result that n stored
tensors come before, itself among them, is off by at most n h of its norm times the products' growth of a relative
error, which is about one here (random signs); twice that is allowed."""
import math

import pytest
import torch

from zi_testlib import say

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, std=1.0, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda").mul_(std).to(dtype)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32, device="cuda")


class Experts:
    """E experts W2 GeLU(W1 x) behind a router, k of them for each of T tokens."""

    def __init__(self, layers, T, E, k, D, F, dtype, seed=0):
        self.layers, self.T, self.E, self.k, self.normalize = layers, T, E, k, True
        g, dt = gen(seed), DT[dtype]
        R = T * k
        self.X = randn(g, T, D, dtype=dt)
        self.W1, self.W2 = randn(g, E, F, D, std=D ** -0.5, dtype=dt), randn(g, E, D, F, std=F ** -0.5, dtype=dt)
        self.logits = randn(g, T, E)
        self.logits[T // 3] = -math.inf  # a padding position
        self.dY = randn(g, T, D, dtype=dt)
        self.ids, self.slots, self.rows, self.offsets = i32(T, k), i32(T, k), i32(R), i32(E + 1)
        self.weights, self.dweights, self.ones = (torch.ones((T, k), device="cuda") for _ in range(3))

        def lo(*shape):
            return torch.zeros(shape, dtype=dt, device="cuda")
        self.Xs, self.A, self.H, self.Z, self.Y = lo(R, D), lo(R, F), lo(R, F), lo(R, D), lo(T, D)
        self.dZ, self.dA, self.dXs, self.dX = lo(R, D), lo(R, F), lo(R, D), lo(T, D)
        self.dW1, self.dW2 = torch.zeros_like(self.W1, dtype=torch.float32), torch.zeros_like(self.W2, dtype=torch.float32)
        self.dlogits = torch.zeros_like(self.logits)
        self.work = layers.workspace(layers.route_fwd_bytes(T, E, k))

    def forward(self):
        L = self.layers
        L.route_fwd(self.logits, self.ids, self.weights, self.offsets, self.rows, self.slots, self.work, normalize=self.normalize)
        L.embedding_fwd(self.rows, self.X, self.Xs)
        L.grouped_fwd(self.Xs, self.W1, self.offsets, self.H, A=self.A)
        L.grouped_fwd(self.H, self.W2, self.offsets, self.Z)
        L.combine_fwd(self.Z, self.slots, self.weights, self.Y)

    def backward(self):
        L = self.layers
        L.combine_bwd(self.dY, self.Z, self.slots, self.weights, self.dZ, self.dweights)
        L.route_bwd(self.logits, self.ids, self.weights, self.dweights, self.dlogits, normalize=self.normalize)
        L.grouped_dw(self.H, self.dZ, self.offsets, self.dW2)
        L.grouped_dx(self.dZ, self.W2, self.offsets, self.dA, A=self.A)
        L.grouped_dw(self.Xs, self.dA, self.offsets, self.dW1)
        L.grouped_dx(self.dA, self.W1, self.offsets, self.dXs)
        L.combine_fwd(self.dXs, self.slots, self.ones, self.dX)  # the gather's gradient: the sum of a token's rows

    def outputs(self):
        return [self.Y, self.dX, self.dW1, self.dW2, self.dlogits, self.dweights, self.ids, self.rows, self.slots, self.offsets]

    def reference(self):
        """Y and the gradients by torch's autograd in 64 bits, expert by expert."""
        X, W1, W2, logits = (t.double().requires_grad_() for t in (self.X, self.W1, self.W2, self.logits))
        live = self.ids[:, 0] >= 0
        at = self.ids.clamp(min=0).long()
        w = torch.softmax(logits[live].gather(1, at[live]), 1)
        Y = torch.zeros_like(X)
        full = torch.zeros((self.T, self.k), dtype=torch.float64, device="cuda")
        full = full.index_put((torch.nonzero(live).squeeze(1),), w)
        for e in range(self.E):
            t, j = torch.nonzero((self.ids == e), as_tuple=True)
            if t.numel():
                a = X[t] @ W1[e].t()
                h = a * 0.5 * torch.erfc(-a * math.sqrt(0.5))
                Y = Y.index_add(0, t, full[t, j].unsqueeze(1) * (h @ W2[e].t()))
        grads = torch.autograd.grad(Y, (X, W1, W2, logits), self.dY.double())
        return [Y.detach()] + [g.nan_to_num(0.0) for g in grads]


@pytest.mark.parametrize("T,E,k,D,F,dtype", [(37, 6, 2, 64, 136, "bf16"), (300, 8, 3, 264, 520, "f16"), (3, 16, 4, 512, 256, "bf16"),
                                             (2000, 4, 2, 512, 1024, "bf16")])
def test_training_step(T, E, k, D, F, dtype):
    from offload_memory_centric_amd import layers
    say("experts step", T, E, k, D, F, dtype)
    m = Experts(layers, T, E, k, D, F, dtype)
    m.forward()
    m.backward()
    torch.cuda.synchronize()
    h = torch.finfo(DT[dtype]).eps / 2
    # tensors stored before each result, itself among them: Y: H, Z, Y; dX: A, dZ, dA, dXs, dX; dW1: A, dZ, dA;
    # dW2: H, dZ; dlogits: H, Z
    for name, got, want, n in zip(("Y", "dX", "dW1", "dW2", "dlogits"), (m.Y, m.dX, m.dW1, m.dW2, m.dlogits), m.reference(),
                                  (3, 5, 3, 2, 2)):
        off = float((got.double() - want).norm() / want.norm())
        assert off <= 2 * n * h, (name, off, 2 * n * h)


def test_another_stream_and_the_same_bits():
    from offload_memory_centric_amd import layers
    m = Experts(layers, 700, 12, 4, 256, 520, "bf16")
    m.forward()
    m.backward()
    torch.cuda.synchronize()
    first = [t.clone() for t in m.outputs()]
    for t in m.outputs():
        t.fill_(1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        m.forward()
        m.backward()
    s.synchronize()
    for a, b in zip(first, m.outputs()):
        assert torch.equal(a, b)


class Tuned:
    """Requests of a batch with adapters beside a projection whose output is Y0."""

    def __init__(self, layers, lengths, N, r, K, M, dtype, seed=0):
        self.layers = layers
        g, dt = gen(seed), DT[dtype]
        T = sum(lengths)
        self.X, self.dY = randn(g, T, K, dtype=dt), randn(g, T, M, dtype=dt)
        self.A, self.B = randn(g, N, r, K, std=K ** -0.5, dtype=dt), randn(g, N, r, M, std=r ** -0.5, dtype=dt)
        self.offsets = torch.tensor([0] + list(lengths), device="cuda").cumsum(0).int()
        self.ids = torch.randint(-1, N, (len(lengths),), generator=g, device="cuda").int()
        self.scales = torch.rand(N, generator=g, device="cuda") + 0.5
        self.Y0, self.Y, self.U = randn(g, T, M, dtype=dt), torch.zeros((T, M), dtype=dt, device="cuda"), torch.zeros((r, T), device="cuda")
        self.dX0, self.dX = randn(g, T, K), torch.zeros((T, K), device="cuda")
        self.dA, self.dB = torch.zeros((N, r, K), device="cuda"), torch.zeros((N, r, M), device="cuda")
        self.work = layers.workspace(max(layers.adapters_fwd_bytes(T, r), layers.adapters_bwd_bytes(T, r)))

    def forward(self):
        self.layers.adapters_fwd(self.X, self.A, self.B, self.offsets, self.ids, self.scales, self.Y, self.work, Y0=self.Y0, U=self.U)

    def backward(self):
        self.layers.adapters_bwd(self.X, self.dY, self.U, self.A, self.B, self.offsets, self.ids, self.scales, self.dA, self.dB,
                                 self.work, dX=self.dX, dX0=self.dX0)

    def outputs(self):
        return [self.Y, self.U, self.dX, self.dA, self.dB]


@pytest.mark.parametrize("kind", ["experts", "experts_few", "adapters", "adapters_rows"])
def test_replayed_from_a_graph(kind):
    """A captured step, replayed several times on other inputs with eager work between, gives what eager calls give."""
    from offload_memory_centric_amd import layers

    def make(seed):
        if kind == "experts":
            return Experts(layers, 700, 12, 4, 256, 520, "bf16", seed)
        if kind == "experts_few":
            return Experts(layers, 5, 16, 2, 512, 256, "f16", seed)
        if kind == "adapters":
            return Tuned(layers, [100, 3, 64, 200, 17], 3, 16, 520, 776, "bf16", seed)
        return Tuned(layers, [1] * 50, 7, 16, 2048, 776, "f16", seed)
    say("graph", kind)
    m, other = make(0), make(100)
    m.forward()  # once outside, as torch asks for
    m.backward()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.forward()
        m.backward()
    for seed in (1, 2, 3):
        new = make(seed)
        for name in ("X", "logits", "dY", "W1", "W2", "A0", "Y0", "dX0", "ids", "offsets", "scales"):
            if kind.startswith("experts") and name in ("ids", "offsets"):
                continue  # what the router writes
            if hasattr(new, name):
                getattr(m, name).copy_(getattr(new, name))
        if kind.startswith("adapters"):
            m.A.copy_(new.A)
            m.B.copy_(new.B)
        graph.replay()
        other.forward()  # eager work of another step between the replays
        other.backward()
        graph.replay()
        torch.cuda.synchronize()
        new.forward()
        new.backward()
        torch.cuda.synchronize()
        for a, b in zip(m.outputs(), new.outputs()):
            assert torch.equal(a, b)


def test_adapters_beside_the_tiled_linear():
    """Y = X W + adapters and its gradients, W staged tile by tile: what the adapters add to, they take from the tiled
    linear where it left it."""
    from offload_memory_centric_amd import layers, tiling
    T, K, M, N, r = 200, 512, 1024, 3, 8
    dt = torch.float16
    g = gen(5)
    W = randn(g, M, K, std=K ** -0.5, dtype=dt)
    Wt, dWt = tiling.host_tensor((M, K), dt), tiling.host_tensor((M, K), dt)
    Wt.copy_(W)
    plan = tiling.Plan(T, K, M, 4, 2, "f16", Wt, dWt)
    ctx = tiling.Context(plan)
    stream = torch.cuda.ExternalStream(ctx.streams[0])
    m = Tuned(layers, [60, 1, 100, 39], N, r, K, M, "f16", 6)
    m.ids = torch.tensor([1, -1, 0, 1], dtype=torch.int32, device="cuda")
    Y, dX = torch.empty((T, M), dtype=dt, device="cuda"), torch.empty((T, K), device="cuda")
    torch.cuda.synchronize()
    ctx.fwd(plan, m.X, Y)
    layers.adapters_fwd(m.X, m.A, m.B, m.offsets, m.ids, m.scales, Y, m.work, Y0=Y, U=m.U, stream=stream)
    ctx.bwd(plan, m.X, m.dY, dX)
    layers.adapters_bwd(m.X, m.dY, m.U, m.A, m.B, m.offsets, m.ids, m.scales, m.dA, m.dB, m.work, dX=dX, dX0=dX, stream=stream)
    ctx.sync()
    torch.cuda.synchronize()
    X, A, B = (t.double().requires_grad_() for t in (m.X, m.A, m.B))
    want = X @ W.double().t()
    parts = []
    for s, n in enumerate(m.ids.tolist()):
        a, b = int(m.offsets[s]), int(m.offsets[s + 1])
        x = want[a:b]
        parts.append(x + m.scales[n].double() * (X[a:b] @ A[n].t() @ B[n]) if n >= 0 else x)
    want = torch.cat(parts)
    dx, da, db = torch.autograd.grad(want, (X, A, B), m.dY.double())
    h = torch.finfo(dt).eps / 2
    # Y is stored twice (the projection's and the sum); the gradients are fp32 sums of 16-bit inputs and of fp32 U, dU
    for name, got, ref, tol in (("Y", Y, want.detach(), 2 * h), ("dX", dX, dx, 1e-5), ("dA", m.dA, da, 1e-5), ("dB", m.dB, db, 1e-5)):
        off = float((got.double() - ref).norm() / ref.norm())
        assert off <= tol, (name, off)
    ctx.close()
    plan.close()
