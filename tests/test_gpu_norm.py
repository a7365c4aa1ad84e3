"""Layer norm (zi_layer_norm_fwd, zi_layer_norm_bwd) against its formulas in 64 bits.

Tolerances.  u = 2^-24 is fp32's half step.  A row's sum has at most
n = 64 + D / 1024 additions in a row (vectors of a thread, lanes, waves), so its
error is at most n u sum|.|; every other operation adds at most u of its
result; a stored value adds half a step of its type."""
import pytest
import torch

from zi_testlib import say

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
U = 2.0 ** -24
EPS = 1e-5


def half(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps


def depth(D):
    return 64 + D / 1024


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rows(g, T, D, dtype, ld=None, std=1.0, mean=0.0):
    """A [T, D] tensor of row stride ld, with NaN between its rows."""
    ld = ld or D
    buf = torch.full((T, ld), float("nan"), dtype=dtype, device="cuda")
    buf[:, :D] = torch.randn((T, D), generator=g, device="cuda").mul_(std).add_(mean).to(dtype)
    return buf[:, :D], buf


def blank(T, D, dtype, ld=None):
    buf = torch.full((T, ld or D), float("nan"), dtype=dtype, device="cuda")
    return buf[:, :D], buf


def untouched(buf, D):
    assert torch.isnan(buf[:, D:]).all(), "wrote between the rows"


def close(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), "%s: %d of %d outside, worst %.3g of tolerance" % (
        what, int(bad.sum()), bad.numel(), float(((got.double() - want).abs() / tol).nan_to_num(float("inf")).max()))


def check_fwd(layers, T, D, x, y, p, res, keep=True, pad=0, mean=0.3, std=1.5, seed=1, affine=True):
    g = gen(seed)
    xt, yt = DT[x], DT[y]
    X, xb = rows(g, T, D, xt, D + pad, std, mean)
    R, rb = rows(g, T, D, yt, D + 2 * pad, 0.5) if res else (None, None)
    S, sb = blank(T, D, xt, D + 3 * pad) if res and keep else (None, None)
    Y, yb = blank(T, D, yt, D + pad)
    gamma = torch.randn(D, generator=g, device="cuda").mul_(0.2).add_(1).to(DT[p]) if affine else None
    beta = torch.randn(D, generator=g, device="cuda").mul_(0.1).to(DT[p]) if affine else None
    m, r = torch.full((T,), float("nan"), device="cuda"), torch.full((T,), float("nan"), device="cuda")
    layers.layer_norm_fwd(X, gamma, beta, Y, m, r, eps=EPS, R=R, S=S)
    torch.cuda.synchronize()
    for buf in (xb, rb, sb, yb):
        if buf is not None:
            untouched(buf, D)
    want = X if not res else (X.float() + R.float()).to(xt)
    if S is not None:
        assert torch.equal(S, want), "S is RNE(X + R)"
    s = want.double()
    mu = s.mean(1, keepdim=True)
    var = (s - mu).square().mean(1, keepdim=True)
    rs = (var + EPS).rsqrt()
    h = (s - mu) * rs
    G = gamma.double() if affine else torch.ones(D, dtype=torch.float64, device="cuda")
    B = beta.double() if affine else torch.zeros(D, dtype=torch.float64, device="cuda")
    n, big = depth(D), s.abs().mean(1, keepdim=True)
    dmean = (n + 2) * U * big                 # error of a mean
    # relative error of rstd: half that of var, whose differences are off by dmean
    drel = 0.5 * (n + 6) * U + dmean.square() * rs.square() + dmean * rs * U + 3 * U
    close(m[:, None], mu, dmean + tiny(torch.float32), "mean")
    close(r[:, None], rs, drel * rs, "rstd")
    want = h * G + B
    tol = half(yt) * want.abs() + tiny(yt) + G.abs() * (dmean * rs * 1.01 + h.abs() * (drel + 3 * U)) + U * (want.abs() + B.abs())
    close(Y, want, tol * 1.01, "Y")


FWD = [  # T, D: one row; odd widths; each side of every shape's border
    (1, 1), (3, 2), (5, 7), (17, 8), (2, 9), (33, 127), (16, 128), (31, 129), (7, 511), (9, 512), (5, 513), (4, 1000),
    (3, 1024), (6, 1025), (1, 2048), (2, 2049), (3, 4096), (2, 4097), (1, 8192), (3, 8193), (2, 16384), (2, 16387),
    (1, 25600), (2, 24577), (1, 32768), (2, 32769), (1, 50001),
]


@pytest.mark.parametrize("T,D", FWD)
@pytest.mark.parametrize("x,y,p,res", [("bf16", "bf16", "bf16", True), ("f32", "f16", "f32", False)])
def test_forward_widths(T, D, x, y, p, res):
    from offload_memory_centric_amd import layers
    say("layer norm forward", T, D, x, y, p, res)
    check_fwd(layers, T, D, x, y, p, res)


@pytest.mark.parametrize("x,y", [("f16", "f16"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "f16"), ("f32", "bf16"),
                                 ("f16", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("p", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("res,keep", [(False, False), (True, True), (True, False)])
def test_forward_types(x, y, p, res, keep):
    from offload_memory_centric_amd import layers
    say("layer norm forward types", x, y, p, res, keep)
    check_fwd(layers, 37, 1000, x, y, p, res, keep=keep, pad=3)
    check_fwd(layers, 3, 40000, x, y, p, res, keep=keep, pad=5)


def test_forward_no_affine_large_mean_and_many_rows():
    from offload_memory_centric_amd import layers
    check_fwd(layers, 11, 777, "f32", "f32", "f32", False, affine=False)
    check_fwd(layers, 5, 5000, "f32", "f32", "f32", True, mean=1000.0, std=0.01)
    check_fwd(layers, 70000, 24, "bf16", "bf16", "f32", True)
    check_fwd(layers, 5000, 5000, "f16", "f16", "f32", True)


def test_forward_constant_rows_and_specials():
    from offload_memory_centric_amd import layers
    X = torch.full((4, 300), 3.0, device="cuda")
    X[1, 5] = float("nan")
    X[2, 7] = float("inf")
    Y, m, r = torch.empty_like(X), torch.empty(4, device="cuda"), torch.empty(4, device="cuda")
    one, zero = torch.ones(300, device="cuda"), torch.full((300,), 0.25, device="cuda")
    layers.layer_norm_fwd(X, one, zero, Y, m, r, eps=EPS)
    torch.cuda.synchronize()
    assert torch.equal(Y[0], zero) and torch.equal(Y[3], zero)   # a constant row: beta
    assert torch.isnan(Y[1]).all() and torch.isnan(Y[2]).all()   # only its own row
    assert float(m[0]) == 3.0


@pytest.mark.parametrize("D", [100, 3000, 40000])
def test_forward_in_place(D):
    from offload_memory_centric_amd import layers
    g = gen(5)
    X, R = torch.randn((6, D), generator=g, device="cuda"), torch.randn((6, D), generator=g, device="cuda")
    gam, bet = torch.randn(D, generator=g, device="cuda"), torch.randn(D, generator=g, device="cuda")
    S, Y = torch.empty_like(X), torch.empty_like(X)
    layers.layer_norm_fwd(X, gam, bet, Y, R=R, S=S)
    X1, R1 = X.clone(), R.clone()
    layers.layer_norm_fwd(X1, gam, bet, R1, R=R1, S=X1)   # S over X, Y over R
    X2 = X.clone()
    layers.layer_norm_fwd(X2, gam, bet, X2, R=R)          # Y over X
    torch.cuda.synchronize()
    assert torch.equal(X1, S) and torch.equal(R1, Y) and torch.equal(X2, Y)


def reference_bwd(dY, S, gamma, mean, rstd, dS):
    s, dy = S.double(), dY.double()
    h = (s - mean.double()[:, None]) * rstd.double()[:, None]
    G = torch.ones(s.shape[1], dtype=torch.float64, device="cuda") if gamma is None else gamma.double()
    g = dy * G
    dX = rstd.double()[:, None] * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
    if dS is not None:
        dX = dX + dS.double()
    return h, g, dX, (dy * h).sum(0), dy.sum(0)


def check_bwd(layers, T, D, x, y, p, res, pad=0, seed=2, affine=True):
    g = gen(seed)
    xt, yt = DT[x], DT[y]
    S, sb = rows(g, T, D, xt, D + pad, 1.5, 0.3)
    dY, yb = rows(g, T, D, yt, D + 2 * pad, 0.1)
    dS, db = rows(g, T, D, xt, D + 3 * pad, 0.1) if res else (None, None)
    dX, xb = blank(T, D, xt, D + pad)
    gamma = torch.randn(D, generator=g, device="cuda").mul_(0.2).add_(1).to(DT[p]) if affine else None
    mean = S.double().mean(1).float()
    rstd = (S.double().var(1, correction=0) + EPS).rsqrt().float()
    dgamma, dbeta = torch.full((D,), float("nan"), device="cuda"), torch.full((D,), float("nan"), device="cuda")
    work = layers.workspace(layers.layer_norm_bwd_bytes(T, D)).fill_(255)
    layers.layer_norm_bwd(dY, S, gamma, mean, rstd, dX, dgamma, dbeta, work, dS=dS)
    torch.cuda.synchronize()
    for buf in (sb, yb, db, xb):
        if buf is not None:
            untouched(buf, D)
    h, gg, want, wg, wb = reference_bwd(dY, S, gamma, mean, rstd, dS)
    n, r = depth(D), rstd.double()[:, None]
    gh = (gg * h).abs().mean(1, keepdim=True)
    tol = half(xt) * want.abs() + tiny(xt) + U * (
        r * (8 * gg.abs() + (n + 8) * (gg.abs().mean(1, keepdim=True) + h.abs() * gh)) + 2 * want.abs())
    if dS is not None:
        tol = tol + 2 * U * dS.double().abs()
    close(dX, want, tol * 1.01, "dX")
    m = T / 64 + 100  # rows of a workgroup, and the workgroups
    close(dgamma, wg, (m + 6) * U * (dY.double() * h).abs().sum(0) * 1.01 + tiny(torch.float32), "dgamma")
    close(dbeta, wb, m * U * dY.double().abs().sum(0) * 1.01 + tiny(torch.float32), "dbeta")
    again_g, again_b, again_x = torch.empty_like(dgamma), torch.empty_like(dbeta), torch.empty_like(dX)
    work.fill_(255)
    layers.layer_norm_bwd(dY, S, gamma, mean, rstd, again_x, again_g, again_b, work, dS=dS)
    torch.cuda.synchronize()
    assert torch.equal(again_g, dgamma) and torch.equal(again_b, dbeta) and torch.equal(again_x, dX), "not the same twice"


BWD = [(1, 1), (3, 2), (40, 7), (17, 8), (100, 128), (33, 129), (300, 512), (700, 513), (600, 1024), (9, 1025), (520, 2048),
       (3, 2049), (1100, 4096), (2, 4097), (530, 8192), (3, 8193), (514, 16384), (5, 16385), (600, 25600), (2, 24576),
       (520, 28672), (3, 28673), (4, 32768), (3, 32769), (70, 50001)]


@pytest.mark.parametrize("T,D", BWD)
@pytest.mark.parametrize("x,y,p,res", [("f16", "f32", "f32", True), ("bf16", "bf16", "bf16", False), ("f32", "f32", "f32", True)])
def test_backward_widths(T, D, x, y, p, res):
    from offload_memory_centric_amd import layers
    say("layer norm backward", T, D, x, y, p, res)
    check_bwd(layers, T, D, x, y, p, res)


@pytest.mark.parametrize("x,y", [("f16", "f16"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "f16"), ("f32", "bf16"),
                                 ("f16", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("p", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("res", [False, True])
def test_backward_types(x, y, p, res):
    from offload_memory_centric_amd import layers
    say("layer norm backward types", x, y, p, res)
    check_bwd(layers, 37, 1000, x, y, p, res, pad=3)
    check_bwd(layers, 20, 9001, x, y, p, res, pad=1)
    check_bwd(layers, 3, 40000, x, y, p, res, pad=5)


def test_backward_many_rows():
    from offload_memory_centric_amd import layers
    check_bwd(layers, 70001, 24, "bf16", "f32", "f32", True)
    check_bwd(layers, 9000, 300, "f32", "f32", "f32", False, affine=False)


@pytest.mark.parametrize("D", [100, 3000, 40000])
def test_backward_in_place_and_parts(D):
    from offload_memory_centric_amd import layers
    g = gen(6)
    T = 9
    S, dY, dS = (torch.randn((T, D), generator=g, device="cuda") for _ in range(3))
    gamma = torch.randn(D, generator=g, device="cuda")
    mean, rstd = S.mean(1), (S.var(1, correction=0) + EPS).rsqrt()
    work = layers.workspace(layers.layer_norm_bwd_bytes(T, D))
    dX, dg, db = torch.empty_like(S), torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
    layers.layer_norm_bwd(dY, S, gamma, mean, rstd, dX, dg, db, work, dS=dS)
    for over in ("dS", "dY", "S"):
        t = {"S": S.clone(), "dY": dY.clone(), "dS": dS.clone()}
        g1, b1 = torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
        layers.layer_norm_bwd(t["dY"], t["S"], gamma, mean, rstd, t[over], g1, b1, work, dS=t["dS"])
        torch.cuda.synchronize()
        assert torch.equal(t[over], dX) and torch.equal(g1, dg) and torch.equal(b1, db), over
    only, none = torch.empty(D, device="cuda"), torch.empty_like(S)
    layers.layer_norm_bwd(dY, S, gamma, mean, rstd, none, None, only, work, dS=dS)
    torch.cuda.synchronize()
    assert torch.equal(only, db) and torch.equal(none, dX)
    none.fill_(0)
    layers.layer_norm_bwd(dY, S, gamma, mean, rstd, none, None, None, None, dS=dS)
    torch.cuda.synchronize()
    assert torch.equal(none, dX)


def test_backward_without_rows():
    from offload_memory_centric_amd import layers
    e = torch.empty((0, 40), device="cuda")
    v = torch.empty(0, device="cuda")
    dg, db = torch.full((40,), 7.0, device="cuda"), torch.full((40,), 7.0, device="cuda")
    layers.layer_norm_bwd(e, e, None, v, v, e, dg, db, None)
    torch.cuda.synchronize()
    assert not dg.any() and not db.any()


def test_backward_against_differences():
    """dX and dgamma against central differences of the forward's formula in 64 bits."""
    from offload_memory_centric_amd import layers
    g = gen(8)
    T, D = 3, 37
    S, dY = torch.randn((T, D), generator=g, device="cuda"), torch.randn((T, D), generator=g, device="cuda")
    gamma, beta = torch.randn(D, generator=g, device="cuda"), torch.zeros(D, device="cuda")
    Y, mean, rstd = torch.empty_like(S), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    layers.layer_norm_fwd(S, gamma, beta, Y, mean, rstd, eps=EPS)
    dX, dg, db = torch.empty_like(S), torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
    layers.layer_norm_bwd(dY, S, gamma, mean, rstd, dX, dg, db, layers.workspace(layers.layer_norm_bwd_bytes(T, D)))
    torch.cuda.synchronize()
    s, w, d = S.cpu().double(), gamma.cpu().double(), dY.cpu().double()

    def loss(s, w):
        c = s - s.mean(1, keepdim=True)
        return float((d * (c * (c.square().mean(1, keepdim=True) + EPS).rsqrt() * w)).sum())

    e = 1e-5
    for t in range(T):
        for i in range(0, D, 5):
            a, b = s.clone(), s.clone()
            a[t, i] += e
            b[t, i] -= e
            # differences: e^2 of the third derivative, and 2^-53 of the loss over e
            assert abs((loss(a, w) - loss(b, w)) / (2 * e) - float(dX[t, i])) < 1e-4
    for i in range(0, D, 5):
        a, b = w.clone(), w.clone()
        a[i] += e
        b[i] -= e
        assert abs((loss(s, a) - loss(s, b)) / (2 * e) - float(dg[i])) < 1e-4


def test_streams_and_graph():
    """On another stream, and captured: every replay gives the eager result for new inputs."""
    from offload_memory_centric_amd import layers
    g = gen(9)
    T, D = 200, 1500
    S, dY, R = (torch.randn((T, D), generator=g, device="cuda") for _ in range(3))
    gamma, beta = torch.randn(D, generator=g, device="cuda"), torch.randn(D, generator=g, device="cuda")
    work = layers.workspace(layers.layer_norm_bwd_bytes(T, D))
    outs = [torch.zeros_like(S), torch.zeros_like(S), torch.zeros(T, device="cuda"), torch.zeros(T, device="cuda"),
            torch.zeros_like(S), torch.zeros(D, device="cuda"), torch.zeros(D, device="cuda")]

    def both(o, stream=None):
        layers.layer_norm_fwd(S, gamma, beta, o[1], o[2], o[3], R=R, S=o[0], stream=stream)
        layers.layer_norm_bwd(dY, o[0], gamma, o[2], o[3], o[4], o[5], o[6], work, stream=stream)

    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    both(outs, side)
    side.synchronize()
    eager = [torch.zeros_like(o) for o in outs]
    both(eager)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, eager))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(outs)
    for k in range(4):
        S.copy_(torch.randn((T, D), generator=g, device="cuda"))
        both(eager)
        torch.cuda.synchronize()
        for o in outs:
            o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, eager)), k


def test_offsets_past_32_bits():
    """More than 2^32 bytes and 2^31 elements: the last rows."""
    from offload_memory_centric_amd import layers
    T, D = 90000, 25000
    g = gen(11)
    X = torch.empty((T, D), dtype=torch.bfloat16, device="cuda")
    X[:50].normal_(generator=g)
    X[50:-50].fill_(1.0)
    X[-50:].normal_(generator=g)
    Y = torch.empty_like(X)
    mean, rstd = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    gamma = torch.randn(D, generator=g, device="cuda")
    layers.layer_norm_fwd(X, gamma, None, Y, mean, rstd, eps=EPS)
    part = torch.cat([X[:50], X[-50:]])
    y, m, r = torch.empty_like(part), torch.empty(100, device="cuda"), torch.empty(100, device="cuda")
    layers.layer_norm_fwd(part, gamma, None, y, m, r, eps=EPS)
    torch.cuda.synchronize()
    assert torch.equal(torch.cat([Y[:50], Y[-50:]]), y) and torch.equal(torch.cat([mean[:50], mean[-50:]]), m)
    assert not Y[1000:1010].any() and float(mean[45000]) == 1.0
    dX = Y  # reused: the gradient of the constant rows is rstd (g - mean(g)), of the others as alone
    dY = X
    dg, db = torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
    layers.layer_norm_bwd(dY, X, gamma, mean, rstd, dX, dg, db, layers.workspace(layers.layer_norm_bwd_bytes(T, D)))
    dx, dg1, db1 = torch.empty_like(part), torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
    layers.layer_norm_bwd(part, part, gamma, m, r, dx, dg1, db1, layers.workspace(layers.layer_norm_bwd_bytes(100, D)))
    torch.cuda.synchronize()
    assert torch.equal(torch.cat([dX[:50], dX[-50:]]), dx)
    want = part.double().sum(0) + (T - 100)
    close(db, want, (T / 64 + 100) * U * (part.double().abs().sum(0) + T), "dbeta")
