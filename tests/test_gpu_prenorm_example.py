"""The operators together, as the example uses them: the gradients of a pre-norm
feed-forward network against torch's in fp32 on the CPU, and its loss falling."""
import math

import pytest
import torch

from zi_testlib import say

pytestmark = pytest.mark.gpu

# Every tensor between the operators is rounded to bf16, by half a step (2^-8)
# at most, and a gradient passes at most sixteen of them (X, Y, A, H, Z, S, P, dP,
# dS, dA, dX, dW, E, W1, W2, and H's slope): relative to its norm.
TOL = 16 * 2.0 ** -8


def reference(net, ids, target):
    E, g1, b1, g2, b2, W1, W2 = [t.detach().cpu().float().requires_grad_() for t in (
        net.E16, *net.norm[0], *net.norm[1], net.W[0], net.W[1])]
    i = ids.cpu()
    X = torch.where((i >= 0)[:, None], E[i.clamp(min=0)] * net.scale, 0.0)
    Y = torch.nn.functional.layer_norm(X, (net.D,), g1, b1)
    Z = torch.nn.functional.gelu(Y @ W1.t()) @ W2.t()
    P = torch.nn.functional.layer_norm(X + Z, (net.D,), g2, b2)
    loss = 0.5 * (P - target.cpu()).square().sum() / net.T
    loss.backward()
    return float(loss.detach()), P.detach(), {"dE": E.grad, "dg1": g1.grad, "db1": b1.grad, "dg2": g2.grad, "db2": b2.grad,
                                     "dW1": W1.grad, "dW2": W2.grad}


def test_gradients_match_autograd():
    from offload_memory_centric_amd.examples import prenorm_ffn
    net = prenorm_ffn.PrenormFFN(tokens=200, vocab=300, width=128, hidden=512, tiles=2)
    ids, target = prenorm_ffn.task(net.T, net.V, net.D)
    loss = net.loss_and_gradients(ids, target)
    want_loss, P, grads = reference(net, ids, target)
    assert abs(loss - want_loss) <= TOL * want_loss
    got = {"dE": net.dE, "dg1": net.dnorm[0][0], "db1": net.dnorm[0][1], "dg2": net.dnorm[1][0], "db2": net.dnorm[1][1],
           "dW1": net.dW[0], "dW2": net.dW[1]}
    live = ids.cpu() >= 0  # a padding row's norm divides by sqrt(eps): its P is compared, its share of a gradient is small
    off = float((net.P.cpu().float() - P)[live].norm() / P[live].norm())
    assert off <= TOL, off
    for name, want in grads.items():
        off = float((got[name].cpu().float() - want).norm() / want.norm())
        say(name, "relative difference %.2g" % off)
        assert off <= TOL, (name, off)
    net.close()


def test_training_lowers_the_loss():
    from offload_memory_centric_amd.examples import prenorm_ffn
    net = prenorm_ffn.PrenormFFN(tokens=256, vocab=500, width=256, hidden=1024, tiles=4)
    ids, target = prenorm_ffn.task(net.T, net.V, net.D)
    losses = [net.step(ids, target) for _ in range(20)]
    say("losses", ["%.3f" % v for v in losses])
    assert all(math.isfinite(v) for v in losses)
    assert losses[-1] < 0.7 * losses[0]
    net.close()
