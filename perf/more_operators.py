"""Operators of mixture-of-experts and adapter layers next to the tiled linear, as a user's program calls them.

A router picks experts for every token and groups the rows by expert; the grouped products multiply each
expert's rows by its own weight (forward with GeLU, input gradient, weight gradient); the combination sums the
experts' rows for every token.  Low-rank adapters add to the output of a shared projection what each request's
own adapter gives.  Each case is one pass through one of them.  `run` computes the plain form in elementary
torch operations where `own` is false, and calls the framework where it is true.
"""
from __future__ import annotations

import math

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}


def listed():
    return [
        # the router of one new token: only latency counts
        dict(name="route_one_token", op="route_fwd", T=1, E=64, k=6, l="bf16", norm=True, pad=False),
        # the router of a full batch (the benchmark's token count) over many experts, some positions padding
        dict(name="route_block", op="route_fwd", T=32768, E=256, k=8, l="f32", norm=True, pad=True),
        # its backward where the weights are probabilities over all experts
        dict(name="route_bwd_block", op="route_bwd", T=32768, E=128, k=6, l="bf16", norm=False, pad=True),
        # serving: a handful of tokens, most experts without a row; the experts' weights are what is read
        dict(name="grouped_fwd_decode", op="grouped_fwd", R=32, E=64, K=2048, M=1408, x="bf16", y="bf16", gelu=True, keep=False),
        # the mid up-projection (8192 to 32768) as eight experts over a full batch, with what the backward needs
        dict(name="grouped_fwd_block", op="grouped_fwd", R=32768, E=8, K=8192, M=32768, x="bf16", y="bf16", gelu=True, keep=True),
        # backward through GeLU of many smaller experts, odd counts of rows
        dict(name="grouped_dx_ragged", op="grouped_dx", R=14211, E=24, K=5000, M=2048, x="f16", y="f16", gelu=True),
        # the weight gradient of experts with few hundred to some thousand rows each, into fp32
        dict(name="grouped_dw_block", op="grouped_dw", R=32768, E=16, K=2048, M=8192, x="bf16", y="f32", acc=False),
        # the sum over each token's experts at width 8192
        dict(name="combine_fwd_block", op="combine_fwd", T=32768, k=4, D=8192, x="bf16", pad=True),
        # its backward at an odd width
        dict(name="combine_bwd_ragged", op="combine_bwd", T=4099, k=6, D=5003, x="f16", pad=True),
        # serving: 64 requests of one token each, nearly all with an adapter of their own
        dict(name="adapters_decode", op="adapters_fwd", T=64, S=64, N=64, r=16, K=8192, M=8192, x="bf16", y="bf16"),
        # prompts of different lengths behind one shared projection
        dict(name="adapters_prompts", op="adapters_fwd", T=20011, S=29, N=12, r=16, K=8192, M=8192, x="f16", y="f16"),
        # a training step of a few adapters over a full batch; dX is the tiled linear's, in fp32
        dict(name="adapters_bwd_block", op="adapters_bwd", T=32768, S=8, N=4, r=32, K=8192, M=8192, x="bf16", y="f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route_fwd", "route_bwd", "grouped_fwd", "grouped_fwd", "grouped_dx", "grouped_dw", "combine_fwd",
                     "combine_bwd", "adapters_fwd", "adapters_fwd", "adapters_bwd"])
    lp = rng.choice(["f16", "bf16"])
    if op in ("route_fwd", "route_bwd"):
        E, norm = _log(rng, 2, 512), rng.random() < 0.5
        # one expert's normalised weight is one, whatever the logits
        return dict(op=op, T=_log(rng, 1, 32768), E=E, k=min(E, _log(rng, 2 if norm else 1, 16)), l=rng.choice([lp, "f32"]),
                    norm=norm, pad=rng.random() < 0.5)
    if op in ("combine_fwd", "combine_bwd"):
        k, D = _log(rng, 1, 8), _log(rng, 64, 25600)
        return dict(op=op, T=_log(rng, 1, min(32768, 32768 * 8192 * 4 // (k * D))), k=k, D=D, x=rng.choice([lp, lp, "f32"]),
                    pad=rng.random() < 0.5)
    if op in ("adapters_fwd", "adapters_bwd"):
        K, M = 8 * _log(rng, 8, 1024), 8 * _log(rng, 8, 1024)
        T = _log(rng, 1, 32768)
        S = _log(rng, 1, min(T, 128))
        return dict(op=op, T=T, S=S, N=_log(rng, 1, min(64, S + 3)), r=rng.choice([4, 8, 16, 16, 24, 32, 64]), K=K, M=M, x=lp,
                    y=rng.choice([lp, "f32"]))
    E = _log(rng, 1, 64)
    K, M = 8 * _log(rng, 8, 1024), 8 * _log(rng, 8, 4096)
    while E * K * M > 1 << 31:
        K, M = 8 * _log(rng, 8, 1024), 8 * _log(rng, 8, 4096)
    c = dict(op=op, R=_log(rng, 1, min(32768, (1 << 43) // (K * M))), E=E, K=K, M=M, x=lp)
    if op == "grouped_dw":
        return dict(c, y=rng.choice([lp, "f32"]), acc=False)
    gelu = rng.random() < 0.5
    c = dict(c, y=lp if gelu else rng.choice([lp, lp, "f32"]), gelu=gelu)
    return dict(c, keep=gelu and rng.random() < 0.5) if op == "grouped_fwd" else c


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, shape, dtype, std=1.0):
    return torch.randn(shape, generator=g, device="cuda").mul_(std).to(DT[dtype])


def _int(*shape):
    return torch.zeros(shape, dtype=torch.int32, device="cuda")


def _split(g, total, parts):
    """int32 offsets of `parts` groups of uneven sizes that cover `total` rows."""
    share = (torch.randn(parts, generator=g, device="cuda") * 0.7).exp().double()
    edge = (share.cumsum(0) / share.sum() * total).round().int().clamp_(0, total)
    edge[-1] = total
    return torch.cat([edge.new_zeros(1), edge])


def _logits(g, case):
    """Logits of experts of different popularity; -inf in the rows of padding positions."""
    T, E = case["T"], case["E"]
    x = torch.randn((T, E), generator=g, device="cuda") * 1.5 + torch.randn(E, generator=g, device="cuda") * 0.5
    if case["pad"]:
        x[torch.rand(T, generator=g, device="cuda") < 0.03] = -math.inf
    return x.to(DT[case["l"]])


def _slots(g, case):
    """Where each token's experts left their rows: a permutation, -1 for the positions without experts."""
    T, k = case["T"], case["k"]
    live = torch.randperm(T, generator=g, device="cuda") >= (T // 32 if case["pad"] else 0)
    n = (T - T // 32 if case["pad"] else T) * k
    slots = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    slots[live] = torch.randperm(n, generator=g, device="cuda").view(-1, k).int()
    return slots, n


def _top(logits, k):
    """The k largest of every row, ties to the lowest index; -1 for those at -inf."""
    val, at = torch.sort(logits.float(), dim=1, descending=True, stable=True)
    return torch.where(val[:, :k] > -math.inf, at[:, :k], -1)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op == "route_fwd":
        T, E, k = case["T"], case["E"], case["k"]
        s["logits"] = _logits(g, case)
        s["ids"], s["slots"], s["rows"], s["offsets"] = _int(T, k), _int(T, k), _int(T * k), _int(E + 1)
        s["weights"] = torch.zeros((T, k), device="cuda")
        if own:
            from offload_memory_centric_amd import layers

            s["work"] = layers.workspace(layers.route_fwd_bytes(T, E, k))
    elif op == "route_bwd":
        T, E, k = case["T"], case["E"], case["k"]
        s["logits"] = _logits(g, case)
        s["ids"] = _top(s["logits"], k).int()
        p = torch.softmax(s["logits"].double(), 1).nan_to_num(0.0).gather(1, s["ids"].clamp(min=0).long())
        p = torch.where(s["ids"] >= 0, p, 0.0)
        s["weights"] = (p / p.sum(1, keepdim=True).clamp(min=1e-300) if case["norm"] else p).float()
        s["dweights"] = torch.randn((T, k), generator=g, device="cuda")
        s["dlogits"] = torch.empty_like(s["logits"])
    elif op in ("combine_fwd", "combine_bwd"):
        T, k, D, x = case["T"], case["k"], case["D"], case["x"]
        s["slots"], n = _slots(g, case)
        s["Z"] = _randn(g, (n, D), x)
        s["weights"] = torch.rand((T, k), generator=g, device="cuda")
        s["weights"] /= s["weights"].sum(1, keepdim=True)
        if op == "combine_fwd":
            s["Y"] = torch.empty((T, D), dtype=DT[x], device="cuda")
        else:
            s["dY"] = _randn(g, (T, D), x, 1e-2)
            s["dZ"] = torch.empty_like(s["Z"])
            s["dweights"] = torch.empty_like(s["weights"])
    elif op in ("adapters_fwd", "adapters_bwd"):
        T, S, N, r, K, M, x = (case[n] for n in ("T", "S", "N", "r", "K", "M", "x"))
        s["offsets"] = _split(g, T, S) if S < T else torch.arange(T + 1, dtype=torch.int32, device="cuda")
        # every adapter at most a few times; now and then a request without one
        s["ids"] = torch.arange(S, device="cuda")[torch.randperm(S, generator=g, device="cuda")].remainder_(N + 1).sub_(
            (torch.rand(S, generator=g, device="cuda") < 0.05).long()).int()
        s["ids"][s["ids"] == N] = -1 if S > 4 else 0
        s["scales"] = torch.rand(N, generator=g, device="cuda") + 0.5
        s["X"] = _randn(g, (T, K), x)
        s["A"] = _randn(g, (N, r, K), x, 1 / math.sqrt(K))
        s["B"] = _randn(g, (N, r, M), x, 0.5 / math.sqrt(r))
        if op == "adapters_fwd":
            s["Y0"] = _randn(g, (T, M), case["y"])
            s["Y"] = torch.empty_like(s["Y0"])
            s["U"] = torch.zeros((r, T), device="cuda")
        else:
            s["dY"] = _randn(g, (T, M), x, 1e-2)
            s["U"] = _hidden(s, s["X"]).float()
            s["dX0"] = _randn(g, (T, K), case["y"], 1e-2)
            s["dX"] = torch.empty_like(s["dX0"])
            s["dA"], s["dB"] = torch.empty((N, r, K), device="cuda"), torch.empty((N, r, M), device="cuda")
        if own:
            from offload_memory_centric_amd import layers

            size = layers.adapters_fwd_bytes if op == "adapters_fwd" else layers.adapters_bwd_bytes
            s["work"] = layers.workspace(size(T, r))
    else:
        R, E, K, M, x, y = (case[n] for n in ("R", "E", "K", "M", "x", "y"))
        s["offsets"] = _split(g, R, E)
        s["at"] = s["offsets"].tolist()
        if op == "grouped_dw":
            s["X"], s["dY"] = _randn(g, (R, K), x), _randn(g, (R, M), x, 1e-2)
            s["dW"] = torch.empty((E, M, K), dtype=DT[y], device="cuda")
            return s
        s["W"] = torch.empty((E, M, K), dtype=DT[x], device="cuda")
        for w in s["W"]:
            w.copy_(torch.randn((M, K), generator=g, device="cuda").mul_(1 / math.sqrt(K)))
        if op == "grouped_fwd":
            s["X"], s["Y"] = _randn(g, (R, K), x), torch.empty((R, M), dtype=DT[y], device="cuda")
            s["A"] = torch.empty((R, M), dtype=DT[x], device="cuda") if case["keep"] else None
        else:
            s["dY"], s["dX"] = _randn(g, (R, M), x, 1e-2), torch.empty((R, K), dtype=DT[y], device="cuda")
            s["A"] = _randn(g, (R, K), x) if case["gelu"] else None
    return s


def _run_own(s):
    from offload_memory_centric_amd import layers

    case = s["case"]
    op = case["op"]
    if op == "route_fwd":
        layers.route_fwd(s["logits"], s["ids"], s["weights"], s["offsets"], s["rows"], s["slots"], s["work"],
                         normalize=case["norm"])
        return {n: s[n] for n in ("ids", "weights", "offsets", "rows", "slots")}
    if op == "route_bwd":
        layers.route_bwd(s["logits"], s["ids"], s["weights"], s["dweights"], s["dlogits"], normalize=case["norm"])
        return s["dlogits"]
    if op == "grouped_fwd":
        layers.grouped_fwd(s["X"], s["W"], s["offsets"], s["Y"], A=s["A"], gelu=case["gelu"])
        return {"Y": s["Y"], "A": s["A"]}
    if op == "grouped_dx":
        layers.grouped_dx(s["dY"], s["W"], s["offsets"], s["dX"], A=s["A"])
        return s["dX"]
    if op == "grouped_dw":
        layers.grouped_dw(s["X"], s["dY"], s["offsets"], s["dW"])
        return s["dW"]
    if op == "combine_fwd":
        layers.combine_fwd(s["Z"], s["slots"], s["weights"], s["Y"])
        return s["Y"]
    if op == "combine_bwd":
        layers.combine_bwd(s["dY"], s["Z"], s["slots"], s["weights"], s["dZ"], s["dweights"])
        return {"dZ": s["dZ"], "dweights": s["dweights"]}
    if op == "adapters_fwd":
        layers.adapters_fwd(s["X"], s["A"], s["B"], s["offsets"], s["ids"], s["scales"], s["Y"], s["work"], Y0=s["Y0"], U=s["U"])
        return {"Y": s["Y"], "U": s["U"]}
    layers.adapters_bwd(s["X"], s["dY"], s["U"], s["A"], s["B"], s["offsets"], s["ids"], s["scales"], s["dA"], s["dB"],
                        s["work"], dX=s["dX"], dX0=s["dX0"])
    return {"dX": s["dX"], "dA": s["dA"], "dB": s["dB"]}


def _gelu(a):
    return 0.5 * a * (1.0 + torch.erf(a * math.sqrt(0.5)))


def _gelu_grad(a):
    return 0.5 * (1.0 + torch.erf(a * math.sqrt(0.5))) + a * torch.exp(-0.5 * a * a) / math.sqrt(2.0 * math.pi)


def _spread(s):
    """[T, N]: the scale of the adapter of each row in that adapter's column, zero elsewhere."""
    case = s["case"]
    row = torch.arange(case["T"], device="cuda")
    at = s["ids"][torch.searchsorted(s["offsets"], row, right=True, out_int32=True).sub_(1).clamp_(0, case["S"] - 1).long()]
    return (at[:, None] == torch.arange(case["N"], device="cuda")) * s["scales"]


def _hidden(s, X):
    """[r, T]: each row of X times its adapter's A, zero for rows without one."""
    case = s["case"]
    u = (X.float() @ s["A"].float().view(-1, case["K"]).t()).view(case["T"], case["N"], case["r"])
    return (u * (_spread(s) != 0)[:, :, None]).sum(1).t().contiguous()


def run(s):
    if own:
        return _run_own(s)
    case = s["case"]
    op = case["op"]
    if op == "route_fwd":
        T, E, k = case["T"], case["E"], case["k"]
        logits = s["logits"].float()
        ids = _top(logits, k)
        chosen = ids >= 0
        e = (logits - logits.amax(1, keepdim=True)).exp()
        w = torch.where(chosen, e.gather(1, ids.clamp(min=0)), 0.0)
        total = (w if case["norm"] else e).sum(1, keepdim=True)
        weights = torch.where(chosen, w / total, 0.0)
        # the (token, choice) pairs by expert, pairs without one last
        key, order = torch.sort(torch.where(chosen, ids, E).flatten(), stable=True)
        offsets = torch.searchsorted(key, torch.arange(E + 1, device="cuda"), out_int32=True)
        rows = torch.where(key < E, order // k, -1).int()
        at = torch.where(key < E, torch.arange(T * k, device="cuda"), -1).int()
        slots = torch.empty_like(at).scatter_(0, order, at).view(T, k)
        return {"ids": ids.int(), "weights": weights, "offsets": offsets, "rows": rows, "slots": slots}
    if op == "route_bwd":
        ids, logits = s["ids"].long(), s["logits"].float()
        g = torch.zeros_like(logits).scatter_(1, ids.clamp(min=0), torch.where(ids >= 0, s["dweights"], 0.0))
        if case["norm"]:
            p = torch.zeros_like(logits).scatter_(1, ids.clamp(min=0), torch.where(ids >= 0, s["weights"], 0.0))
        else:
            p = (logits - logits.amax(1, keepdim=True)).exp()
            p = torch.where(ids[:, :1] >= 0, p / p.sum(1, keepdim=True), 0.0)
        return (p * (g - (p * g).sum(1, keepdim=True))).to(s["logits"].dtype)
    if op == "grouped_fwd":
        acc = torch.cat([s["X"][a:b].float() @ w.float().t() for a, b, w in zip(s["at"], s["at"][1:], s["W"]) if b > a])
        A = acc.to(s["X"].dtype) if case["keep"] else None
        return {"Y": (_gelu(acc) if case["gelu"] else acc).to(s["Y"].dtype), "A": A}
    if op == "grouped_dx":
        acc = torch.cat([s["dY"][a:b].float() @ w.float() for a, b, w in zip(s["at"], s["at"][1:], s["W"]) if b > a])
        return (acc * _gelu_grad(s["A"].float()) if case["gelu"] else acc).to(s["dX"].dtype)
    if op == "grouped_dw":
        X, dY = s["X"].float(), s["dY"].float()
        return torch.stack([(dY[a:b].t() @ X[a:b]).to(s["dW"].dtype) for a, b in zip(s["at"], s["at"][1:])])
    if op in ("combine_fwd", "combine_bwd"):
        slots = s["slots"].long()
        w = torch.where(slots >= 0, s["weights"], 0.0)
        Z = s["Z"][slots.clamp(min=0)].float()
        if op == "combine_fwd":
            return (Z * w[:, :, None]).sum(1).to(s["Y"].dtype)
        dY = s["dY"].float()
        live = slots.flatten() >= 0
        dZ = torch.empty_like(s["Z"])
        dZ[slots.flatten()[live]] = (w[:, :, None] * dY[:, None]).to(dZ.dtype).flatten(0, 1)[live]
        return {"dZ": dZ, "dweights": torch.where(slots >= 0, (Z * dY[:, None]).sum(2), 0.0)}
    # adapters: all of them side by side in one product, with the scale of each row's own (zero for the others)
    T, r, N = case["T"], case["r"], case["N"]
    scale = _spread(s)
    A, B = s["A"].float().view(N * r, -1), s["B"].float().view(N * r, -1)
    if op == "adapters_fwd":
        U = _hidden(s, s["X"])
        y = (U.t()[:, None] * scale[:, :, None]).reshape(T, N * r) @ B
        return {"Y": (s["Y0"].float() + y).to(s["Y"].dtype), "U": U}
    dY = s["dY"].float()
    dU = ((dY @ B.t()).view(T, N, r) * scale[:, :, None]).view(T, N * r)
    U = (s["U"].t()[:, None] * scale[:, :, None]).reshape(T, N * r)
    return {"dX": (s["dX0"].float() + dU @ A).to(s["dX"].dtype), "dA": (dU.t() @ s["X"].float()).view(N, r, -1),
            "dB": (U.t() @ dY).view(N, r, -1)}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("route_fwd", "route_bwd"):
        z = s["logits"].double()
        if op == "route_fwd":
            val = torch.topk(z, case["k"], dim=1).values
            w = torch.exp(val - (torch.logsumexp(val, 1, keepdim=True) if case["norm"] else torch.logsumexp(z, 1, keepdim=True)))
            return {"ids": None, "weights": torch.where(val > -math.inf, w, 0.0), "offsets": None, "rows": None, "slots": None}
        # by the Jacobian of the softmax over the experts that count
        keep = torch.zeros_like(z, dtype=torch.bool)
        g = torch.zeros_like(z)
        for j in range(case["k"]):
            live = torch.nonzero(s["ids"][:, j] >= 0).squeeze(1)
            keep[live, s["ids"][live, j].long()] = True
            g[live, s["ids"][live, j].long()] = s["dweights"][live, j].double()
        if case["norm"]:  # the weights are inputs, as the forward stored them
            p = torch.zeros_like(z)
            for j in range(case["k"]):
                live = torch.nonzero(s["ids"][:, j] >= 0).squeeze(1)
                p[live, s["ids"][live, j].long()] = s["weights"][live, j].double()
        else:
            p = torch.softmax(z, 1).nan_to_num(0.0)
        return p * g - p * torch.linalg.vecdot(p, g).unsqueeze(1)
    if op == "grouped_fwd":
        A = torch.empty((case["R"], case["M"]), dtype=torch.float64, device="cuda")
        for n in range(case["E"]):
            a, b = s["at"][n], s["at"][n + 1]
            if b > a:
                A[a:b] = torch.mm(s["X"][a:b].double(), s["W"][n].double().t())
        Y = A * torch.special.ndtr(A) if case["gelu"] else A
        return {"Y": Y, "A": A if case["keep"] else None}
    if op == "grouped_dx":
        D = torch.empty((case["R"], case["K"]), dtype=torch.float64, device="cuda")
        for n in range(case["E"]):
            a, b = s["at"][n], s["at"][n + 1]
            if b > a:
                D[a:b] = torch.mm(s["dY"][a:b].double(), s["W"][n].double())
        if case["gelu"]:
            h = s["A"].double()
            D *= torch.special.ndtr(h) + h * torch.exp(-h.square() / 2 - 0.5 * math.log(2 * math.pi))
        return D
    if op == "grouped_dw":
        D = torch.zeros((case["E"], case["M"], case["K"]), dtype=torch.float64, device="cuda")
        for n in range(case["E"]):
            a, b = s["at"][n], s["at"][n + 1]
            if b > a:
                torch.mm(s["dY"][a:b].double().t(), s["X"][a:b].double(), out=D[n])
        return D
    if op in ("combine_fwd", "combine_bwd"):
        T, k, D = case["T"], case["k"], case["D"]
        Y = torch.zeros((T, D), dtype=torch.float64, device="cuda")
        dZ = torch.zeros((s["Z"].shape[0], D), dtype=torch.float64, device="cuda") if op == "combine_bwd" else None
        dw = torch.zeros((T, k), dtype=torch.float64, device="cuda")
        for j in range(k):
            live = torch.nonzero(s["slots"][:, j] >= 0).squeeze(1)
            at, w = s["slots"][live, j].long(), s["weights"][live, j].double().unsqueeze(1)
            z = s["Z"].index_select(0, at).double()
            if op == "combine_fwd":
                Y[live] += w * z
            else:
                d = s["dY"].index_select(0, live).double()
                dZ[at] = w * d
                dw[live, j] = torch.linalg.vecdot(z, d)
        return Y if op == "combine_fwd" else {"dZ": dZ, "dweights": dw}
    # adapters, request by request
    at, ids, scales = s["offsets"].tolist(), s["ids"].tolist(), s["scales"].double()
    if op == "adapters_fwd":
        Y, U = s["Y0"].double(), torch.zeros((case["r"], case["T"]), dtype=torch.float64, device="cuda")
        for n, a, b in zip(ids, at, at[1:]):
            if 0 <= n and b > a:
                u = torch.mm(s["X"][a:b].double(), s["A"][n].double().t())
                U[:, a:b] = u.t()
                Y[a:b] += scales[n] * torch.mm(u, s["B"][n].double())
        return {"Y": Y, "U": U}
    dX, dA, dB = s["dX0"].double(), torch.zeros_like(s["dA"], dtype=torch.float64), torch.zeros_like(s["dB"], dtype=torch.float64)
    for n, a, b in zip(ids, at, at[1:]):
        if 0 <= n and b > a:
            d, x = s["dY"][a:b].double(), s["X"][a:b].double()
            du = torch.mm(d, s["B"][n].double().t()) * scales[n]
            dX[a:b] += torch.mm(du, s["A"][n].double())
            dA[n] += torch.mm(du.t(), x)
            dB[n] += torch.mm(s["U"][:, a:b].double(), d) * scales[n]
    return {"dX": dX, "dA": dA, "dB": dB}


def _used(rows, groups):
    """About how many of `groups` uneven groups have one of `rows` rows."""
    return min(groups, rows) if rows < groups // 2 else groups * -math.expm1(-rows / groups)


def work(case):
    op = case["op"]
    if op in ("route_fwd", "route_bwd"):
        T, E, k, l = case["T"], case["E"], case["k"], SIZE[case["l"]]
        if op == "route_fwd":
            return {"bytes": T * E * l + T * k * 16 + 4 * (E + 1), "flops": 4 * T * E}
        return {"bytes": T * E * l * (1 if case["norm"] else 2) + T * k * (12 if case["norm"] else 8), "flops": 6 * T * E}
    if op in ("combine_fwd", "combine_bwd"):
        T, k, D, x = case["T"], case["k"], case["D"], SIZE[case["x"]]
        if op == "combine_fwd":
            return {"bytes": T * D * (k + 1) * x + T * k * 8, "flops": 2 * T * k * D}
        return {"bytes": T * D * (2 * k + 1) * x + T * k * 12, "flops": 3 * T * k * D}
    if op in ("adapters_fwd", "adapters_bwd"):
        T, S, N, r, K, M, x, y = (case[n] for n in ("T", "S", "N", "r", "K", "M", "x", "y"))
        ab = min(N, S) * r * (K + M)
        if op == "adapters_fwd":
            return {"bytes": T * K * SIZE[x] + 2 * T * M * SIZE[y] + ab * SIZE[x] + 4 * r * T, "flops": 2 * T * r * (K + M)}
        return {"bytes": T * (K + M) * SIZE[x] + 2 * T * K * SIZE[y] + ab * SIZE[x] + N * r * (K + M) * 4 + 4 * r * T,
                "flops": 4 * T * r * (K + M)}
    R, E, K, M, x, y = (case[n] for n in ("R", "E", "K", "M", "x", "y"))
    flops = 2 * R * K * M
    if op == "grouped_dw":
        return {"bytes": R * (K + M) * SIZE[x] + E * K * M * SIZE[y], "flops": flops}
    w = _used(R, E) * K * M * SIZE[x]
    if op == "grouped_fwd":
        return {"bytes": R * K * SIZE[x] + R * M * (SIZE[y] + (SIZE[x] if case["keep"] else 0)) + w, "flops": flops}
    return {"bytes": R * M * SIZE[x] + R * K * (SIZE[y] + (SIZE[x] if case["gelu"] else 0)) + w, "flops": flops}
