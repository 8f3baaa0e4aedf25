"""Linear, rotary and dropout together with the other block operators: the
example's transformer with rotated queries and keys, biases and dropout against
the same network in float64, gradients of every weight, and its training loop."""

import os
import sys

import pytest
import torch

from block_reference import act
from block_reference_linear import drop, rotary

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu


def plain(net, x, cond, step):
    """The network, float64, from the same weights and masks."""
    w = {k: t.detach().double().requires_grad_(True) for k, t in zip(net.names, net.leaf)}
    x, cond = x.double(), cond.double()
    b, n, d = x.shape
    turns = net.turns(n)

    def norm(x, scale=None, shift=None):
        y = torch.nn.functional.layer_norm(x, (d,), eps=1e-6)
        return y if scale is None else y * (1 + scale[:, None]) + shift[:, None]
    for i in range(net.blocks):
        masks = [(net.seed, 2 * (step * net.blocks + i) + j) for j in range(2)]
        sh1, sc1, g1, sh2, sc2, g2 = (cond @ w[i, "ada"].T).chunk(6, dim=1)
        q, k, v = (norm(x, sc1, sh1) @ w[i, "qkv"].T).view(b, n, 3, net.heads, d // net.heads).unbind(2)
        if turns is not None:
            q, k = (rotary(t, turns["freqs"], turns["positions"][None]) for t in (q, k))
        q, k, v = (t.transpose(1, 2) for t in (q, k, v))
        p = torch.softmax(q @ k.transpose(2, 3) * (d // net.heads) ** -0.5, dim=-1)
        h = (p @ v).transpose(1, 2).reshape(b, n, d) @ w[i, "proj"].T
        x = x + g1[:, None] * drop(h, net.p, masks[0])
        y = norm(x, sc2, sh2)
        if net.mlp == "gated":
            h = (torch.nn.functional.silu(y @ w[i, "gate"].T) * (y @ w[i, "up"].T)) @ w[i, "down"].T
        else:
            h = act(y @ w[i, "fc1"].T + w[i, "b1"], "gelu") @ w[i, "fc2"].T + w[i, "b2"]
        x = x + g2[:, None] * drop(h, net.p, masks[1])
    return norm(x) @ w[net.blocks, "out"].T, list(w.values())


KINDS = [dict(rotary=True), dict(mlp="gelu"), dict(mlp="gelu", rotary=True, dropout=0.2), dict(rotary=True, dropout=0.1)]


@pytest.mark.parametrize("kind", KINDS)
def test_gradients_of_the_whole_network(kind):
    """Each of the about twelve roundings to bf16 on a path is off by 2^-8 /
    sqrt(3) of a value at random: 3% of a gradient's norm covers them nearly twice
    over (2 sqrt(12) 2^-8 / sqrt(3) = 1.6%)."""
    import train_dit
    net = train_dit.Dit(128, 2, 344, 2, seed=3, **kind)
    x, cond, want = train_dit.batch(3, 50, 128, 0)
    got = torch.autograd.grad((net(x, cond, 7).float() - want).square().mean(), net.leaf)
    y, weights = plain(net, x, cond, 7)
    ref = torch.autograd.grad((y - want.double()).square().mean(), weights)
    for name, g, r in zip(net.names, got, ref):
        assert float((g.double() - r).norm() / r.norm()) < 0.03, name


@pytest.mark.parametrize("kind", KINDS)
def test_training_runs(kind):
    import train_dit
    losses = train_dit.train(dim=128, heads=2, hidden=344, blocks=2, samples=4, tokens=64, steps=8, report=None, **kind)
    assert len(losses) == 8 and all(x == x and abs(x) < 1e3 for x in losses)


def test_dropout_differs_by_step():
    import train_dit
    net = train_dit.Dit(128, 2, 344, 2, seed=3, dropout=0.2)
    x, cond, _ = train_dit.batch(3, 50, 128, 0)
    assert torch.equal(net(x, cond, 1), net(x, cond, 1)) and not torch.equal(net(x, cond, 1), net(x, cond, 2))


@pytest.mark.parametrize("kind", KINDS)
def test_training_moves_every_weight(kind, monkeypatch):
    """Every weight and bias goes somewhere in each of the first steps (refresh and
    between), and the leaves are what the optimizer's weights round to."""
    import train_dit
    nets, seen = [], []

    class Kept(train_dit.Dit):
        def __init__(self, *args, **how):
            super().__init__(*args, **how)
            nets.append(self)

        def __call__(self, *args):
            seen.append([t.detach().clone() for t in self.leaf])
            return super().__call__(*args)
    monkeypatch.setattr(train_dit, "Dit", Kept)
    train_dit.train(dim=128, heads=2, hidden=344, blocks=2, samples=4, tokens=64, steps=4, report=None, **kind)
    net, = nets
    seen.append([t.detach() for t in net.leaf])
    assert len(seen) == 5 and ({"b1", "b2"} <= {n for _, n in net.names}) == (kind.get("mlp") == "gelu")
    for step, (before, after) in enumerate(zip(seen, seen[1:])):
        for name, p, q in zip(net.names, before, after):
            assert not torch.equal(p, q) and bool(torch.isfinite(q).all()), (step, name)
    for name, leaf, master in zip(net.names, net.leaf, net.master):
        assert torch.equal(leaf, master.to(leaf.dtype)), name
