"""The router and the combination (zi_route_fwd, zi_route_bwd, zi_combine_fwd, zi_combine_bwd) against their formulas
in 64 bits.

Tolerances.  u = 2^-24 is fp32's half step.  exp(x - top) has the rounding of the difference, |x - top| u as a relative
error, and 4 u of its own; a sum of n terms adds at most n u of the sum of their magnitudes; every other operation u of
its result; a stored value half a step of its type."""
import pytest
import torch

from zi_testlib import say

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
U = 2.0 ** -24
INF = float("inf")
GUARD = 17  # elements behind every output, which stay as they were


def half(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def guarded(shape, dtype, fill):
    n = 1
    for s in shape:
        n *= s
    buf = torch.full((n + GUARD,), fill, dtype=dtype, device="cuda")
    return buf[:n].view(shape), buf[n:], fill


def close(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), "%s: %d of %d outside, worst %.3g of tolerance" % (
        what, int(bad.sum()), bad.numel(), float(((got.double() - want).abs() / tol).nan_to_num(INF).max()))


def logits_of(g, T, E, dtype, ld=None, ties=False):
    buf = torch.full((T, ld or E), float("nan"), dtype=dtype, device="cuda")
    x = torch.randn((T, E), generator=g, device="cuda") * 2
    buf[:, :E] = (x.round() if ties else x).to(dtype)
    return buf[:, :E]


def route(layers, logits, k, normalize):
    T, E = logits.shape
    outs = {"ids": guarded((T, k), torch.int32, -77), "weights": guarded((T, k), torch.float32, -77.0),
            "offsets": guarded((E + 1,), torch.int32, -77), "rows": guarded((T * k,), torch.int32, -77),
            "slots": guarded((T, k), torch.int32, -77)}
    work = layers.workspace(layers.route_fwd_bytes(T, E, k)) if T > 64 else None
    layers.route_fwd(logits, work=work, normalize=normalize, **{n: o[0] for n, o in outs.items()})
    torch.cuda.synchronize()
    for n, (_, behind, fill) in outs.items():
        assert (behind == fill).all(), "wrote behind " + n
    return {n: o[0] for n, o in outs.items()}


def check_route(layers, logits, k, normalize):
    T, E = logits.shape
    got = route(layers, logits, k, normalize)
    z = logits.double()
    choosable = torch.where(torch.isnan(z), -INF, z)
    order = torch.sort(choosable, dim=1, descending=True, stable=True)
    ids = torch.where(order.values[:, :k] > -INF, order.indices[:, :k], -1)
    assert torch.equal(got["ids"].long(), ids), "ids"
    chosen = ids >= 0
    # the places: by expert, in it by token
    flat = ids.flatten()
    key = torch.where(flat >= 0, flat, E)
    at = torch.sort(key, stable=True)
    n = int((flat >= 0).sum())
    counts = torch.bincount(key, minlength=E + 1)[:E]
    assert torch.equal(got["offsets"].long(), torch.cat([counts.new_zeros(1), counts.cumsum(0)])), "offsets"
    rows = torch.where(torch.arange(T * k, device="cuda") < n, at.indices // k, -1)
    assert torch.equal(got["rows"].long(), rows), "rows"
    slots = torch.full_like(flat, -1)
    slots[at.indices[:n]] = torch.arange(n, device="cuda")
    assert torch.equal(got["slots"].long(), slots.view(T, k)), "slots"
    # the weights
    top = order.values[:, :1]
    over = torch.where(chosen, z.gather(1, ids.clamp(min=0)), -INF) if normalize else z
    e = (over - top).exp()
    w = torch.where(chosen, (z.gather(1, ids.clamp(min=0)) - top).exp() / e.sum(1, keepdim=True), 0.0)
    nan = chosen & (torch.isnan(z).any(1, keepdim=True) | torch.isinf(top))
    assert torch.equal(torch.isnan(got["weights"]), nan), "NaN"
    far = torch.where(torch.isfinite(z), (z - top).abs(), 0.0)
    # a term of the sum that is far below the largest is off by more, and counts for less
    spread = torch.where(e > 0, e * far.gather(1, ids.clamp(min=0)) if normalize else e * far, 0.0).sum(1, keepdim=True) / e.sum(1, keepdim=True)
    rel = (far.gather(1, ids.clamp(min=0)) + spread + (k if normalize else E) + 16) * U
    ok = ~nan
    tol = torch.where(chosen, rel * w + tiny(torch.float32), 0.0)
    close(got["weights"][ok], w[ok], tol[ok], "weights")
    return got


SIZES = [(1, 1, 1), (1, 64, 6), (2, 3, 3), (7, 64, 32), (31, 65, 4), (64, 128, 8), (65, 129, 8), (63, 256, 8), (100, 257, 5),
         (129, 512, 16), (300, 513, 2), (1000, 1024, 32), (257, 1000, 1), (5000, 160, 6), (4097, 8, 2), (70000, 16, 2)]


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("dtype,normalize", [("f32", True), ("bf16", False)])
def test_route_sizes(T, E, k, dtype, normalize):
    from offload_memory_centric_amd import layers
    say("route", T, E, k, dtype, normalize)
    check_route(layers, logits_of(gen(T + E), T, E, DT[dtype]), k, normalize)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("T", [40, 200])
def test_route_ties_strides_and_masks(T, dtype, normalize):
    from offload_memory_centric_amd import layers
    E, k = 37, 5
    x = logits_of(gen(3), T, E, DT[dtype], ld=E + 6, ties=True)
    x[x == 0] *= -1.0                       # zeros of both signs tie
    x[3] = -INF                             # nothing to choose
    x[5, 2:] = -INF                         # fewer than k
    x[7, ::2] = torch.finfo(DT[dtype]).min  # the lowest finite value can be chosen
    x[8] = torch.finfo(DT[dtype]).min
    x[9] = 1.0                              # all equal
    x[10, 4] = float("nan")
    x[11] = float("nan")
    x[12, 6] = INF
    x[T - 1] = -INF
    check_route(layers, x, k, normalize)


def test_route_many_blocks():
    from offload_memory_centric_amd import layers
    check_route(layers, logits_of(gen(9), 150001, 12, torch.float16, ties=True), 3, True)


def test_route_no_tokens():
    from offload_memory_centric_amd import layers
    got = route(layers, torch.empty((0, 5), device="cuda"), 2, True)
    assert (got["offsets"] == 0).all()


def check_route_bwd(layers, logits, k, normalize, seed=5):
    T, E = logits.shape
    z = logits.double()
    order = torch.sort(z, dim=1, descending=True, stable=True)
    ids = torch.where(order.values[:, :k] > -INF, order.indices[:, :k], -1)
    chosen = ids >= 0
    p = torch.where(chosen[:, :1], torch.softmax(z, 1), 0.0)
    w = torch.where(chosen, p.gather(1, ids.clamp(min=0)), 0.0)
    if normalize:
        w = torch.where(chosen, w / w.sum(1, keepdim=True), 0.0)
    w = w.float()
    d = torch.randn((T, k), generator=gen(seed), device="cuda")
    d[~chosen] = float("nan")  # not read
    buf = torch.full((T, E + 5), 7.0, dtype=logits.dtype, device="cuda")
    layers.route_bwd(logits, ids.int(), w, d, buf[:, :E], normalize=normalize)
    torch.cuda.synchronize()
    assert (buf[:, E:] == 7.0).all(), "wrote between the rows"
    zero = torch.zeros_like(z)
    at = ids.clamp(min=0)
    g = zero.scatter_add(1, at, torch.where(chosen, d.double(), 0.0))
    if normalize:
        p = zero.scatter_add(1, at, w.double())
    along = (p * g).sum(1, keepdim=True)
    want = p * (g - along)
    far = torch.where(torch.isfinite(z) & chosen[:, :1], (z - order.values[:, :1]).abs(), 0.0)
    rel = 0.0 if normalize else (far + (p * far).sum(1, keepdim=True) + E + 20) * U
    size = (p * g.abs()).sum(1, keepdim=True)
    off = (rel * p * g.abs()).sum(1, keepdim=True) if not normalize else 0.0
    tol = p * (rel * (g - along).abs() + off + (E + 8) * U * size + 4 * U * (g.abs() + along.abs()))
    close(buf[:, :E], want, tol + half(logits.dtype) * want.abs() + tiny(logits.dtype), "dlogits")


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 64, 6), (17, 65, 1), (130, 128, 32), (33, 200, 8), (40, 300, 3), (21, 1024, 16),
                                   (70000, 8, 2)])
@pytest.mark.parametrize("dtype,normalize", [("f32", True), ("f32", False), ("bf16", True), ("f16", False)])
def test_route_bwd(T, E, k, dtype, normalize):
    from offload_memory_centric_amd import layers
    say("route backward", T, E, k, dtype, normalize)
    x = logits_of(gen(T), T, E, DT[dtype], ld=E + 3)
    if T > 10:
        x[4] = -INF
        x[6, 1:] = -INF
        x[7, ::2] = torch.finfo(DT[dtype]).min
    check_route_bwd(layers, x, k, normalize)


@pytest.mark.parametrize("normalize", [True, False])
def test_route_gradient_by_differences(normalize):
    """The gradient of sum(weights d) along random directions against differences of the forward's formula in 64 bits."""
    from offload_memory_centric_amd import layers
    T, E, k = 9, 21, 4
    g = gen(11)
    x = logits_of(g, T, E, torch.float32)
    d = torch.randn((T, k), generator=g, device="cuda")
    got = route(layers, x, k, normalize)
    dl = torch.empty_like(x)
    layers.route_bwd(x, got["ids"], got["weights"], d, dl, normalize=normalize)
    at = got["ids"].long()

    def value(z):
        p = torch.softmax(z, 1).gather(1, at)
        return ((p / p.sum(1, keepdim=True) if normalize else p) * d.double()).sum()
    h = 1e-5
    for s in range(3):
        v = torch.randn((T, E), generator=g, device="cuda").double()
        diff = (value(x.double() + h * v) - value(x.double() - h * v)) / (2 * h)
        along = (dl.double() * v).sum()
        # the difference is off by h^2 times a third derivative of the order of the values
        assert abs(float(diff - along)) <= 1e-4 * float((dl.double() * v).abs().sum()) + 1e-6


# ---- combination -----------------------------------------------------------------------------

def rows(g, T, D, dtype, pad, std=1.0):
    buf = torch.full((T, D + pad), float("nan"), dtype=dtype, device="cuda")
    buf[:, :D] = torch.randn((T, D), generator=g, device="cuda").mul_(std).to(dtype)
    return buf[:, :D], buf


def check_combine(layers, T, k, D, dtype, pad=0, holes=True, seed=2):
    g, dt = gen(seed), DT[dtype]
    R = T * k + 3  # three rows that no slot names
    Z, _ = rows(g, R, D, dt, pad)
    dY, _ = rows(g, T, D, dt, 2 * pad)
    slots = torch.randperm(R, generator=g, device="cuda")[:T * k].view(T, k).int()
    weights = torch.randn((T, k), generator=g, device="cuda")
    if holes:
        drop = torch.rand((T, k), generator=g, device="cuda") < 0.2
        lost = slots[drop].long()
        Z[lost] = float("nan")           # a row that nobody names reaches nothing
        slots[drop] = torch.where(torch.rand(len(lost), generator=g, device="cuda") < 0.5, -1, R).int()
        weights[drop] = float("nan")     # nor does its weight
        slots[T // 2], weights[T // 2] = -1, float("nan")
    live = (slots >= 0) & (slots < R)
    at = torch.where(live, slots, 0).long()
    w = torch.where(live, weights, 0.0).double()
    z = torch.where(live[:, :, None], Z[at].double(), 0.0)
    _, yb = rows(g, T, D, dt, pad + 1)
    yb.fill_(float("nan"))
    layers.combine_fwd(Z, slots, weights, yb[:, :D])
    torch.cuda.synchronize()
    assert torch.isnan(yb[:, D:]).all(), "wrote between the rows"
    want = (w[:, :, None] * z).sum(1)
    size = (w[:, :, None] * z).abs().sum(1)
    close(yb[:, :D], want, half(dt) * want.abs() + tiny(dt) + (k + 2) * U * size * 1.01, "Y")

    zb = torch.full((R, D + pad + 2), -3.0, dtype=dt, device="cuda")
    dw, behind, fill = guarded((T, k), torch.float32, -77.0)
    layers.combine_bwd(dY, Z, slots, weights, zb[:, :D], dw)
    torch.cuda.synchronize()
    assert (behind == fill).all() and (zb[:, D:] == -3.0).all(), "wrote elsewhere"
    d = dY.double()[:, None]
    dot, size = (z * d).sum(2), (z * d).abs().sum(2)
    close(dw, dot, (32 + D / 128) * U * size * 1.01 + tiny(torch.float32), "dweights")
    named = torch.zeros(R, dtype=torch.bool, device="cuda")
    named[at[live]] = True
    assert (zb[~named][:, :D] == -3.0).all(), "a row that no slot names was written"
    dz = torch.zeros((R, D), dtype=torch.float64, device="cuda")
    dz[at[live]] = (w[:, :, None] * d)[live]
    close(zb[:, :D][named], dz[named], (half(dt) + U) * dz[named].abs() * 1.01 + tiny(dt), "dZ")


@pytest.mark.parametrize("T,k,D", [(1, 1, 1), (3, 2, 7), (5, 3, 8), (4, 1, 9), (17, 5, 63), (33, 2, 64), (9, 6, 513), (7, 4, 1000),
                                   (6, 8, 2048), (3, 9, 2049), (2, 3, 8192), (5, 2, 25600), (3, 40, 100), (3000, 2, 24)])
@pytest.mark.parametrize("dtype", list(DT))
def test_combine(T, k, D, dtype):
    from offload_memory_centric_amd import layers
    say("combine", T, k, D, dtype)
    check_combine(layers, T, k, D, dtype, pad=3)
    check_combine(layers, T, k, D, dtype, holes=False, seed=8)


def test_combine_without_rows():
    from offload_memory_centric_amd import layers
    Z, Y = torch.empty((0, 16), device="cuda"), torch.full((4, 16), 5.0, device="cuda")
    slots, w = torch.full((4, 2), -1, dtype=torch.int32, device="cuda"), torch.full((4, 2), float("nan"), device="cuda")
    dw = torch.full_like(w, 3.0)
    layers.combine_fwd(Z, slots, w, Y)
    layers.combine_bwd(torch.ones_like(Y), Z, slots, w, torch.empty_like(Z), dw)
    assert (Y == 0).all() and (dw == 0).all()


def test_combine_far_rows():
    """Rows past 2^32 bytes of Z."""
    from offload_memory_centric_amd import layers
    D, R = 25600, 90000
    Z = torch.zeros((R, D), dtype=torch.bfloat16, device="cuda")
    Z[R - 1], Z[1] = 2.0, 3.0
    slots = torch.tensor([[R - 1, 1], [1, -1]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[1.0, 2.0], [4.0, 1.0]], device="cuda")
    Y = torch.empty((2, D), dtype=torch.bfloat16, device="cuda")
    layers.combine_fwd(Z, slots, w, Y)
    assert (Y[0] == 8.0).all() and (Y[1] == 12.0).all()
    dw = torch.empty_like(w)
    slots[1, 0] = 5
    dZ = torch.zeros_like(Z)
    layers.combine_bwd(Y, Z, slots, w, dZ, dw)
    assert (dZ[R - 1] == 8.0).all() and (dZ[1] == 16.0).all() and (dZ[5] == 48.0).all()
    assert dw.tolist() == [[16.0 * D, 24.0 * D], [0.0, 0.0]]
