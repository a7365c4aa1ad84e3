"""Operators of a pre-norm feed-forward training step, as a user's program calls them.

Three operators stand next to the tiled feed-forward block: the token embedding that makes the block's
input, the layer norm in front of it (with the residual sum), and the orthogonalised update of a weight's
gradient.  Each case is one pass through one of them.  `run` computes the plain form in elementary torch
operations where `own` is false, and calls the framework where it is true.
"""
from __future__ import annotations

import math

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}
EPS = 1e-5                          # layer norm
NS_COEFFS = (3.4445, -4.7750, 2.0315)   # one step: X <- a X + (b A + c A^2) X, A = X X^T
NS_EPS = 1e-7
NS_STEPS = 5


def listed():
    return [
        # one token at a time: the norm before a block of width 8192, where only latency counts
        dict(name="norm_fwd_one_token", op="norm_fwd", T=1, D=8192, x="bf16", y="bf16", p="bf16", res=True),
        # a ragged batch of an odd width, an fp32 residual stream feeding fp16 products
        dict(name="norm_fwd_ragged", op="norm_fwd", T=1777, D=5003, x="f32", y="f16", p="f32", res=False),
        # the input of the 1T model's feed-forward block at the benchmark's token count
        dict(name="norm_fwd_block", op="norm_fwd", T=32768, D=25600, x="f16", y="f16", p="f32", res=True),
        # backward before the mid up-projection: dY is the fp32 dX of the tiled linear, residual gradient in bf16
        dict(name="norm_bwd_mid", op="norm_bwd", T=4096, D=8192, x="bf16", dy="f32", p="f32", res=True),
        # backward of the 1T model's block at the benchmark's token count
        dict(name="norm_bwd_block", op="norm_bwd", T=32768, D=25600, x="f16", dy="f32", p="f32", res=True),
        # the embedding of one new token
        dict(name="embed_fwd_one_token", op="embed_fwd", T=1, V=50257, D=8192, w="bf16", x="bf16", ids="i32", pad=False),
        # the embedding of a full batch at the 1T model's width
        dict(name="embed_fwd_block", op="embed_fwd", T=32768, V=50257, D=25600, w="f16", x="f16", ids="i64", pad=True),
        # the gradient of a small model's table: nearly every row of it is zero
        dict(name="embed_bwd_small", op="embed_bwd", T=2047, V=50257, D=512, dx="f32", dw="f32", ids="i64", pad=True, acc=False),
        # the gradient of a full batch at width 8192: frequent tokens' sums are long
        dict(name="embed_bwd_mid", op="embed_bwd", T=32768, V=50257, D=8192, dx="bf16", dw="f32", ids="i32", pad=True, acc=False),
        # the weight of the tiny tiled linear (W^t is 2048 x 512): launches are most of it
        dict(name="orth_tiny", op="orth", M=2048, K=512, g="f16"),
        # an odd shape in fp32
        dict(name="orth_ragged", op="orth", M=1001, K=1531, g="f32"),
        # the mid feed-forward up-projection (W^t is 32768 x 8192)
        dict(name="orth_mid", op="orth", M=32768, K=8192, g="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "embed_fwd", "embed_bwd", "orth"])
    lp = rng.choice(["f16", "bf16"])
    if op in ("norm_fwd", "norm_bwd"):
        x = rng.choice([lp, lp, "f32"])
        y = rng.choice([lp, "f32"]) if x == "f32" else lp
        D = _log(rng, 8, 25600)
        most = 32768 * 25600 // (1 if x != "f32" else 2)
        T = _log(rng, 1, min(32768, most // D))
        c = dict(op=op, T=T, D=D, x=x, p=rng.choice(["f32", y]), res=rng.random() < 0.5)
        c["y" if op == "norm_fwd" else "dy"] = y if op == "norm_fwd" else rng.choice([y, "f32"])
        return c
    if op in ("embed_fwd", "embed_bwd"):
        D = _log(rng, 8, 25600 if op == "embed_fwd" else 16384)
        V = _log(rng, 16, min(131072, 400_000_000 // D))
        T = _log(rng, 1, 32768 if op == "embed_fwd" else min(32768, 32768 * 8192 // D))
        c = dict(op=op, T=T, V=V, D=D, ids=rng.choice(["i32", "i64"]), pad=rng.random() < 0.5)
        if op == "embed_fwd":
            w = rng.choice([lp, "f32"])
            return dict(c, w=w, x=lp if w != "f32" else rng.choice([lp, "f32"]))
        return dict(c, dx=rng.choice([lp, "f32"]), dw=rng.choice([lp, "f32"]), acc=rng.random() < 0.3)
    M = _log(rng, 1, 32768)
    K = _log(rng, 1, 32768)
    while min(M, K) ** 2 * max(M, K) > 4096 ** 2 * 16384:
        M, K = _log(rng, 1, 32768), _log(rng, 1, 32768)
    return dict(op=op, M=M, K=K, g=rng.choice([lp, lp, "f32"]))


def _randn(g, shape, dtype, std=1.0, mean=0.0):
    return torch.randn(shape, generator=g, device="cuda").mul_(std).add_(mean).to(DT[dtype])


def _ids(g, case):
    """Token ids by Zipf's law (p(i) ~ 1 / (i + 1)); -1 marks a padding position."""
    T, V = case["T"], case["V"]
    u = torch.rand(T, generator=g, device="cuda", dtype=torch.float64)
    ids = ((V + 1.0) ** u).floor().long().sub_(1).clamp_(0, V - 1)
    if case["pad"]:
        ids[torch.rand(T, generator=g, device="cuda") < 0.05] = -1
    return ids.to(torch.int32 if case["ids"] == "i32" else torch.int64)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    s = {"case": case}
    if op == "norm_fwd":
        T, D = case["T"], case["D"]
        s["X"] = _randn(g, (T, D), case["x"], 1.5, 0.25)
        s["R"] = _randn(g, (T, D), case["y"], 0.5) if case["res"] else None
        s["gamma"] = _randn(g, (D,), case["p"], 0.2, 1.0)
        s["beta"] = _randn(g, (D,), case["p"], 0.1)
        s["S"] = torch.empty_like(s["X"]) if case["res"] else None
        s["Y"] = torch.empty((T, D), dtype=DT[case["y"]], device="cuda")
        s["mean"] = torch.empty(T, device="cuda")
        s["rstd"] = torch.empty(T, device="cuda")
    elif op == "norm_bwd":
        T, D = case["T"], case["D"]
        s["S"] = _randn(g, (T, D), case["x"], 1.5, 0.25)
        s["dY"] = _randn(g, (T, D), case["dy"], 1e-2)
        s["dS"] = _randn(g, (T, D), case["x"], 1e-2) if case["res"] else None
        s["gamma"] = _randn(g, (D,), case["p"], 0.2, 1.0)
        f = s["S"].float()
        s["mean"] = f.mean(1)
        s["rstd"] = (f.var(1, correction=0) + EPS).rsqrt()
        del f
        s["dX"] = torch.empty_like(s["S"])
        s["dgamma"] = torch.empty(D, device="cuda")
        s["dbeta"] = torch.empty(D, device="cuda")
        if own:
            from offload_memory_centric_amd import layers

            s["work"] = layers.workspace(layers.layer_norm_bwd_bytes(T, D))
    elif op == "embed_fwd":
        s["W"] = _randn(g, (case["V"], case["D"]), case["w"], 0.02)
        s["ids"] = _ids(g, case)
        s["X"] = torch.empty((case["T"], case["D"]), dtype=DT[case["x"]], device="cuda")
        s["scale"] = math.sqrt(case["D"])
    elif op == "embed_bwd":
        T, V, D = case["T"], case["V"], case["D"]
        s["ids"] = _ids(g, case)
        s["dX"] = _randn(g, (T, D), case["dx"], 1e-2)
        s["scale"] = math.sqrt(D)
        s["dW"] = torch.empty((V, D), dtype=DT[case["dw"]], device="cuda")
        # an accumulated gradient keeps what an earlier micro-batch left
        s["before"] = _randn(g, (V, D), case["dw"], 1e-2) if case["acc"] else None
        if own:
            from offload_memory_centric_amd import layers

            s["work"] = layers.workspace(layers.embedding_bwd_bytes(T, V, D))
    else:
        # a gradient X^T dY: a few directions carry most of it, over a floor of noise
        M, K = case["M"], case["K"]
        r = max(1, min(64, M // 2, K // 2))
        lead = torch.randn((M, r), generator=g, device="cuda") / torch.arange(1, r + 1, device="cuda").sqrt()
        G = lead @ torch.randn((r, K), generator=g, device="cuda")
        s["G"] = G.add_(torch.randn((M, K), generator=g, device="cuda")).mul_(0.01).to(DT[case["g"]])
        s["O"] = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
        if own:
            from offload_memory_centric_amd import layers

            s["work"] = layers.workspace(layers.orthogonalize_bytes(M, K))
    return s


def _run_own(s):
    from offload_memory_centric_amd import layers

    op = s["case"]["op"]
    if op == "norm_fwd":
        layers.layer_norm_fwd(s["X"], s["gamma"], s["beta"], s["Y"], s["mean"], s["rstd"], eps=EPS, R=s["R"], S=s["S"])
        return {"S": s["S"], "Y": s["Y"], "mean": s["mean"], "rstd": s["rstd"]}
    if op == "norm_bwd":
        layers.layer_norm_bwd(s["dY"], s["S"], s["gamma"], s["mean"], s["rstd"], s["dX"], s["dgamma"], s["dbeta"],
                              s["work"], dS=s["dS"])
        return {"dX": s["dX"], "dgamma": s["dgamma"], "dbeta": s["dbeta"]}
    if op == "embed_fwd":
        layers.embedding_fwd(s["ids"], s["W"], s["X"], scale=s["scale"])
        return s["X"]
    if op == "embed_bwd":
        # an fp32 gradient is accumulated where the earlier micro-batch left it, as the plain form does; one in
        # 16 bits, which the plain form rounds into a new tensor, into a copy
        acc, dW = s["before"] is not None, s["dW"]
        if acc and s["before"].dtype == torch.float32:
            dW = s["before"]
        elif acc:
            dW.copy_(s["before"])
        layers.embedding_bwd(s["ids"], s["dX"], dW, s["work"], scale=s["scale"], accumulate=acc)
        return dW
    layers.orthogonalize(s["G"], s["O"], s["work"], steps=NS_STEPS, coeffs=NS_COEFFS, eps=NS_EPS)
    return s["O"]


def run(s):
    if own:
        return _run_own(s)
    case = s["case"]
    op = case["op"]
    if op == "norm_fwd":
        if s["R"] is None:
            S, x = None, s["X"].float()
        else:
            S = (s["X"].float() + s["R"].float()).to(s["X"].dtype)
            x = S.float()
        mean = x.mean(1)
        x = x - mean[:, None]
        rstd = (x.square().mean(1) + EPS).rsqrt()
        Y = (x * rstd[:, None] * s["gamma"].float() + s["beta"].float()).to(s["Y"].dtype)
        return {"S": S, "Y": Y, "mean": mean, "rstd": rstd}
    if op == "norm_bwd":
        xhat = (s["S"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        dy = s["dY"].float()
        g = dy * s["gamma"].float()
        dx = (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True)) * s["rstd"][:, None]
        if s["dS"] is not None:
            dx = dx + s["dS"].float()
        return {"dX": dx.to(s["S"].dtype), "dgamma": (dy * xhat).sum(0), "dbeta": dy.sum(0)}
    if op == "embed_fwd":
        ids = s["ids"].long()
        x = s["W"][ids.clamp(min=0)].float() * s["scale"]
        return torch.where((ids >= 0)[:, None], x, 0.0).to(s["X"].dtype)
    if op == "embed_bwd":
        ids = s["ids"].long()
        dx = torch.where((ids >= 0)[:, None], s["dX"].float() * s["scale"], 0.0)
        dW = torch.zeros((case["V"], case["D"]), device="cuda") if s["before"] is None else s["before"].float()
        return dW.index_add_(0, ids.clamp(min=0), dx).to(s["dW"].dtype)
    G = s["G"].float()
    x = G if case["M"] <= case["K"] else G.t().contiguous()
    x = x / (x.double().square().sum().sqrt() + NS_EPS).float()
    x = _steps(x, NS_STEPS)
    return (x if case["M"] <= case["K"] else x.t()).to(torch.bfloat16).contiguous()


def _steps(x, n):
    """n Newton-Schulz steps on x in its own precision."""
    if n == 0:
        return x
    a, b, c = NS_COEFFS
    A = x @ x.t().contiguous()
    return _steps(a * x + (b * A + c * (A @ A)) @ x, n - 1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm_fwd":
        # the residual sum is defined as stored: the norm reads S in X's type
        src = s["X"] if s["R"] is None else (s["X"].double() + s["R"].double()).to(s["X"].dtype)
        var, mean = torch.var_mean(src.double(), dim=1, correction=0)
        inv = 1.0 / torch.sqrt(var + EPS)
        y = torch.addcmul(s["beta"].double(), (src.double() - mean.unsqueeze(1)).mul_(inv.unsqueeze(1)), s["gamma"].double())
        return {"S": None if s["R"] is None else src, "Y": y, "mean": mean, "rstd": inv}
    if op == "norm_bwd":
        r = s["rstd"].double().unsqueeze(1)
        h = s["S"].double().sub_(s["mean"].double().unsqueeze(1)).mul_(r)   # normalised values
        n = case["D"]
        d = s["dY"].double()
        dbeta = torch.ones(case["T"], dtype=torch.float64, device="cuda") @ d
        dgamma = torch.linalg.vecdot(d, h, dim=0)
        d *= s["gamma"].double()
        along = (d * h).sum(1, keepdim=True)
        total = d.sum(1, keepdim=True)
        out = (n * d - total - h * along) * (r / n)
        return {"dX": out if s["dS"] is None else out.add_(s["dS"].double()), "dgamma": dgamma, "dbeta": dbeta}
    if op == "embed_fwd":
        rows = torch.zeros((case["T"], case["D"]), dtype=torch.float64, device="cuda")
        at = torch.nonzero(s["ids"] >= 0).squeeze(1)
        rows[at] = s["W"].index_select(0, s["ids"][at].long()).double() * s["scale"]
        return rows
    if op == "embed_bwd":
        # sums over runs of equal ids in sorted order
        order = torch.sort(s["ids"].long(), stable=True).indices
        keys, counts = torch.unique_consecutive(s["ids"].long()[order], return_counts=True)
        run_of = torch.repeat_interleave(torch.arange(keys.numel(), device="cuda"), counts)
        sums = torch.zeros((keys.numel(), case["D"]), dtype=torch.float64, device="cuda")
        sums.index_add_(0, run_of, s["dX"][order].double())
        out = torch.zeros((case["V"], case["D"]), dtype=torch.float64, device="cuda") if s["before"] is None else s["before"].double()
        out[keys[keys >= 0]] += sums[keys >= 0] * s["scale"]
        return out
    # odd polynomial of the singular values, by products on the shorter side
    a, b, c = NS_COEFFS
    X = s["G"].double()
    X = X / (torch.linalg.vector_norm(X) + NS_EPS)
    wide = case["M"] <= case["K"]
    eye = torch.eye(min(case["M"], case["K"]), dtype=torch.float64, device="cuda")
    for _ in range(NS_STEPS):
        P = torch.mm(X, X.mT.contiguous()) if wide else torch.mm(X.mT.contiguous(), X)
        Q = a * eye + torch.mm(P, b * eye + c * P)
        X = torch.mm(Q, X) if wide else torch.mm(X, Q)
    return X


def _distinct(T, V):
    """Expected number of different ids among T drawn by _ids."""
    return sum(-math.expm1(T * math.log1p(-min(1 - 1e-12, math.log((i + 2) / (i + 1)) / math.log(V + 1)))) for i in range(V))


def work(case):
    op = case["op"]
    if op == "norm_fwd":
        T, D, x, y, p = case["T"], case["D"], SIZE[case["x"]], SIZE[case["y"]], SIZE[case["p"]]
        per = x + y + (y + x if case["res"] else 0)
        return {"bytes": T * D * per + 2 * D * p + 8 * T, "flops": 8 * T * D}
    if op == "norm_bwd":
        T, D, x, dy, p = case["T"], case["D"], SIZE[case["x"]], SIZE[case["dy"]], SIZE[case["p"]]
        per = x + dy + x + (x if case["res"] else 0)
        return {"bytes": T * D * per + D * p + 8 * D + 8 * T, "flops": 14 * T * D}
    ids = 8 if case.get("ids") == "i64" else 4
    if op == "embed_fwd":
        T, V, D = case["T"], case["V"], case["D"]
        return {"bytes": T * ids + _distinct(T, V) * D * SIZE[case["w"]] + T * D * SIZE[case["x"]], "flops": T * D}
    if op == "embed_bwd":
        T, V, D = case["T"], case["V"], case["D"]
        before = V * D * SIZE[case["dw"]] if case["acc"] else 0
        return {"bytes": T * ids + T * D * SIZE[case["dx"]] + V * D * SIZE[case["dw"]] + before, "flops": T * D}
    # X X^T and its square are symmetric: half of each product
    m, k = min(case["M"], case["K"]), max(case["M"], case["K"])
    return {"bytes": m * k * (SIZE[case["g"]] + 2), "flops": NS_STEPS * (m * m * k + m * m * m + 2 * m * m * k)}
