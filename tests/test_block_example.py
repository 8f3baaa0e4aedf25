"""The block operators together: the example's transformer against the same
network in float64, gradients of every weight, and its training loop with the
optimizer."""

import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu


def plain(net, x, cond):
    """The example's network, float64, from the same (bf16) weights."""
    w = {k: t.detach().double().requires_grad_(True) for k, t in zip(net.names, net.leaf)}
    x, cond = x.double(), cond.double()
    b, n, d = x.shape

    def norm(x, scale=None, shift=None):
        y = torch.nn.functional.layer_norm(x, (d,), eps=1e-6)
        return y if scale is None else y * (1 + scale[:, None]) + shift[:, None]
    for i in range(net.blocks):
        sh1, sc1, g1, sh2, sc2, g2 = (cond @ w[i, "ada"].T).chunk(6, dim=1)
        qkv = (norm(x, sc1, sh1) @ w[i, "qkv"].T).view(b, n, 3, net.heads, d // net.heads)
        q, k, v = (t.transpose(1, 2) for t in qkv.unbind(2))
        p = torch.softmax(q @ k.transpose(2, 3) * (d // net.heads) ** -0.5, dim=-1)
        x = x + g1[:, None] * ((p @ v).transpose(1, 2).reshape(b, n, d) @ w[i, "proj"].T)
        y = norm(x, sc2, sh2)
        h = torch.nn.functional.silu(y @ w[i, "gate"].T) * (y @ w[i, "up"].T)
        x = x + g2[:, None] * (h @ w[i, "down"].T)
    return norm(x) @ w[net.blocks, "out"].T, list(w.values())


def test_gradients_of_the_whole_network():
    """Each of the about ten roundings to bf16 on a path is off by 2^-8 / sqrt(3)
    of a value at random: 3% of a gradient's norm covers ten of them twice
    over (2 sqrt(10) 2^-8 / sqrt(3) = 1.4%)."""
    import train_dit
    net = train_dit.Dit(128, 2, 344, 2, seed=3)
    x, cond, want = train_dit.batch(3, 50, 128, 0)
    got = torch.autograd.grad((net(x, cond).float() - want).square().mean(), net.leaf)
    y, weights = plain(net, x, cond)
    ref = torch.autograd.grad((y - want.double()).square().mean(), weights)
    for name, g, r in zip(net.names, got, ref):
        assert float((g.double() - r).norm() / r.norm()) < 0.03, name


def test_training_reduces_the_loss():
    import train_dit
    losses = train_dit.train(dim=128, heads=2, hidden=344, blocks=2, samples=4, tokens=64, steps=24, report=None)
    assert all(x == x and x < 1e3 for x in losses)
    assert sum(losses[-4:]) < 0.8 * sum(losses[:4]), losses
