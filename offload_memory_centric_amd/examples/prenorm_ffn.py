"""A pre-norm feed-forward network trained on synthetic tokens.

    X = scale E[ids]                         token embedding
    Z = W2 GeLU(W1 norm(X))                  the tiled block, its weights in pinned host memory
    P = norm(X + Z)                          prediction of a target row for every token

W1 and W2 are staged tile by tile, forward and backward; their gradients land in
host memory, and their update is orthogonalised on the device.  The embedding
and the norms live on the device.  Everything between two updates is enqueued on
the context's product stream, without waiting for the host.

Run:  python -m offload_memory_centric_amd.examples.prenorm_ffn [--steps N]
"""
from __future__ import annotations

import argparse
import math

import torch

from .. import layers, tiling


class PrenormFFN:
    def __init__(self, tokens=512, vocab=2000, width=512, hidden=2048, tiles=4, dtype="bf16", seed=0):
        T, V, D, F = tokens, vocab, width, hidden
        self.T, self.V, self.D, self.F, self.dtype = T, V, D, F, dtype
        lp = self.lp = tiling.inputs_dtype(dtype)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.scale = math.sqrt(D)

        def randn(*shape, std=1.0):
            return torch.randn(shape, generator=g, device="cuda") * std

        # on the device: the embedding and the norms (fp32 masters; the table also in 16 bits)
        self.E = randn(V, D, std=1 / math.sqrt(D))
        self.E16 = self.E.to(lp)
        self.norm = [(torch.ones(D, device="cuda"), torch.zeros(D, device="cuda")) for _ in range(2)]
        # in host memory: the block's weights, out-major, and their gradients
        self.master = [randn(F, D, std=1 / math.sqrt(D)), randn(D, F, std=1 / math.sqrt(F))]
        self.W = [tiling.host_tensor(tuple(w.shape), lp) for w in self.master]
        self.dW = [tiling.host_tensor(tuple(w.shape), lp) for w in self.master]
        for w, m in zip(self.W, self.master):
            w.copy_(m)
        self.plans = [tiling.Plan(T, D, F, tiles, 2, dtype, self.W[0], self.dW[0]),
                      tiling.Plan(T, F, D, tiles, 2, dtype, self.W[1], self.dW[1])]
        ring = max((p.info.ring_bytes, i) for i, p in enumerate(self.plans))[1]
        self.ctx = tiling.Context(self.plans[ring])
        self.stream = torch.cuda.ExternalStream(self.ctx.streams[0])

        def lo(*shape):
            return torch.empty(shape, dtype=lp, device="cuda")

        def hi(*shape):
            return torch.empty(shape, device="cuda")

        self.X, self.Y, self.A, self.H, self.Z, self.S, self.P = (lo(T, n) for n in (D, D, F, F, D, D, D))
        self.dS, self.dA, self.dX = lo(T, D), lo(T, F), lo(T, D)
        self.dH, self.dY = hi(T, F), hi(T, D)
        self.stats = [(hi(T), hi(T)) for _ in range(2)]
        self.dnorm = [(hi(D), hi(D)) for _ in range(2)]
        self.dE = hi(V, D)
        self.momentum = [torch.zeros_like(m) for m in self.master]
        self.update = [torch.empty_like(m, dtype=torch.bfloat16) for m in self.master]
        self.norm_work = layers.workspace(layers.layer_norm_bwd_bytes(T, D))
        self.embed_work = layers.workspace(layers.embedding_bwd_bytes(T, V, D))
        self.orth_work = layers.workspace(max(layers.orthogonalize_bytes(*m.shape) for m in self.master))
        torch.cuda.synchronize()

    def forward(self, ids):
        """Enqueues the forward pass; P is ready when the product stream is."""
        p1, p2 = self.plans
        layers.embedding_fwd(ids, self.E16, self.X, scale=self.scale)
        layers.layer_norm_fwd(self.X, *self.norm[0], self.Y, *self.stats[0])
        self.ctx.fwd_gelu(p1, self.Y, self.A, self.H)
        self.ctx.fwd(p2, self.H, self.Z)
        layers.layer_norm_fwd(self.X, *self.norm[1], self.P, *self.stats[1], R=self.Z, S=self.S)
        return self.P

    def backward(self, ids, dP):
        """Enqueues the backward pass of the last forward."""
        p1, p2 = self.plans
        (g1, _), (g2, _) = self.norm
        layers.layer_norm_bwd(dP, self.S, g2, *self.stats[1], self.dS, *self.dnorm[1], self.norm_work)
        self.ctx.bwd(p2, self.H, self.dS, self.dH)
        self.ctx.gelu_bwd(self.dtype, self.dH, self.A, self.dA, self.A.numel())
        self.ctx.bwd(p1, self.Y, self.dA, self.dY)
        layers.layer_norm_bwd(self.dY, self.X, g1, *self.stats[0], self.dX, *self.dnorm[0], self.norm_work, dS=self.dS)
        layers.embedding_bwd(ids, self.dX, self.dE, self.embed_work, scale=self.scale)

    def loss_and_gradients(self, ids, target):
        """Half the mean squared distance from P to target; its gradients in dW, dnorm and dE."""
        self.stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(self.stream):
            d = self.forward(ids).float() - target
            loss = 0.5 * d.square().sum() / self.T
            self.backward(ids, (d / self.T).to(self.lp))
        self.ctx.sync()
        return float(loss)

    def step(self, ids, target, lr=0.02, momentum=0.9, lr_rows=0.3):
        """One training step: the block's weights by their orthogonalised momentum, the rest by its gradient."""
        loss = self.loss_and_gradients(ids, target)
        with torch.cuda.stream(self.stream):
            for W, dW, master, m, u in zip(self.W, self.dW, self.master, self.momentum, self.update):
                m.mul_(momentum).add_(dW.to("cuda", non_blocking=True))
                layers.orthogonalize(m, u, self.orth_work)
                master.sub_(u, alpha=lr * math.sqrt(max(1.0, master.shape[0] / master.shape[1])))
                W.copy_(master)
            for (g, b), (dg, db) in zip(self.norm, self.dnorm):
                g.sub_(dg, alpha=lr_rows)
                b.sub_(db, alpha=lr_rows)
            self.E.sub_(self.dE, alpha=lr_rows / self.D)
            self.E16.copy_(self.E)
        self.stream.synchronize()
        return loss

    def close(self):
        self.ctx.close()
        for p in self.plans:
            p.close()


def task(tokens, vocab, width, seed=1):
    """Token ids (some positions padding) and the rows that a model has to predict from them."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    ids = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    ids[torch.rand(tokens, generator=g, device="cuda") < 0.05] = -1
    return ids, torch.randn((tokens, width), generator=g, device="cuda")


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=30)
    a = ap.parse_args()
    net = PrenormFFN()
    ids, target = task(net.T, net.V, net.D)
    for k in range(a.steps):
        loss = net.step(ids, target)
        if k % 5 == 0 or k + 1 == a.steps:
            print("step %d  loss %.4f" % (k, loss), flush=True)
    net.close()


if __name__ == "__main__":
    main()
