"""Trains a small Diffusion-Transformer stack on the GPU with this package's
block operators and optimizer: what computes the gradients, and what consumes
them.

Per block (x the fp32 residual stream, modulation from the sample's condition):

    y = LayerNorm(x) (1 + scale_1) + shift_1            residual_norm
    h = proj(attention(qkv(y)))                         attention_qkv
    x = x + gate_1 h;  y = LayerNorm(x) (1 + scale_2) + shift_2
    h = (silu(y Wg^T) * (y Wu^T)) Wd^T                  gated_ffn
    x = x + gate_2 h;  y = the next block's norm

Each residual_norm call ends one sub-block and begins the next.  Weights are
fp32, used through bf16 copies; the gradients of the copies go to MuonSession
(Newton-Schulz refresh on every third step, RowNorm between).

    python examples/train_dit.py --dim 512 --blocks 4 --steps 30
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import matrix_aware_optimizer_periodic_amd as mm  # noqa: E402

BF16 = torch.bfloat16


class Dit:
    """Blocks of width `dim`; weights in `master` (fp32), their bf16 copies
    (the leaves of autograd) in `leaf`."""

    def __init__(self, dim: int, heads: int, hidden: int, blocks: int, seed: int = 0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        shapes = {"ada": (6 * dim, dim), "qkv": (3 * dim, dim), "proj": (dim, dim), "gate": (hidden, dim),
                  "up": (hidden, dim), "down": (dim, hidden)}
        self.dim, self.heads, self.blocks = dim, heads, blocks
        self.names = [(i, n) for i in range(blocks) for n in shapes] + [(blocks, "out")]
        self.master = [torch.randn(shapes.get(n, (dim, dim)), generator=gen, device="cuda") * dim ** -0.5
                       for _, n in self.names]
        self.leaf = [w.to(BF16).requires_grad_(True) for w in self.master]

    def weight(self, i: int, name: str):
        return self.leaf[self.names.index((i, name))]

    def __call__(self, x, cond):
        """x (samples, tokens, dim) fp32, cond (samples, dim) bf16 -> prediction, bf16."""
        linear = torch.nn.functional.linear
        b, n, d = x.shape
        # shift_1, scale_1, gate_1, shift_2, scale_2, gate_2 of every block
        mod = [linear(cond, self.weight(i, "ada")).float().chunk(6, dim=1) for i in range(self.blocks)]
        x, y = mm.residual_norm(x, scale=mod[0][1], shift=mod[0][0], y_dtype=BF16)
        for i in range(self.blocks):
            qkv = linear(y, self.weight(i, "qkv")).view(b, n, 3, self.heads, d // self.heads)
            h = linear(mm.attention_qkv(qkv).reshape(b, n, d), self.weight(i, "proj"))
            x, y = mm.residual_norm(x, h, gate=mod[i][2], scale=mod[i][4], shift=mod[i][3])
            h = mm.gated_ffn(y, self.weight(i, "gate"), self.weight(i, "up"), self.weight(i, "down"))
            nxt = {"scale": mod[i + 1][1], "shift": mod[i + 1][0]} if i + 1 < self.blocks else {}
            x, y = mm.residual_norm(x, h, gate=mod[i][5], **nxt)
        return linear(y, self.weight(self.blocks, "out"))


def batch(samples: int, tokens: int, dim: int, step: int):
    """A synthetic denoising pair: clean signals of a few fixed directions,
    mixed with noise by the sample's time, and the velocity to predict."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    basis = torch.randn(8, dim, generator=gen, device="cuda")
    gen.manual_seed(1000 + step)
    clean = torch.randn(samples, tokens, 8, generator=gen, device="cuda") @ basis * 8 ** -0.5
    noise = torch.randn(samples, tokens, dim, generator=gen, device="cuda")
    t = torch.rand(samples, 1, 1, generator=gen, device="cuda")
    freq = torch.exp(torch.linspace(0, 5, dim // 2, device="cuda"))
    cond = torch.cat([torch.sin(t[:, :, 0] * freq), torch.cos(t[:, :, 0] * freq)], dim=1).to(BF16)
    return (1 - t) * noise + t * clean, cond, clean - noise


def train(dim=512, heads=8, hidden=1376, blocks=4, samples=8, tokens=256, steps=30, lr=0.02, report=print):
    """Losses of `steps` optimizer steps."""
    net = Dit(dim, heads, hidden, blocks)
    opt = mm.MuonSession(net.master, [torch.zeros_like(w) for w in net.leaf], lr=lr)
    losses = []
    for t in range(steps):
        x, cond, want = batch(samples, tokens, dim, t)
        loss = (net(x, cond).float() - want).square().mean()
        grads = torch.autograd.grad(loss, net.leaf)
        opt.step(t, grads=grads)
        with torch.no_grad():
            for w, leaf in zip(net.master, net.leaf):
                leaf.copy_(w)
        losses.append(float(loss.detach()))
        if report is not None and (t % 5 == 0 or t == steps - 1):
            report(f"step {t}: loss {losses[-1]:.4f}")
    opt.sync()
    opt.close()
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("dim", 512), ("heads", 8), ("hidden", 1376), ("blocks", 4), ("samples", 8), ("tokens", 256),
                        ("steps", 30)):
        ap.add_argument(f"--{name}", type=int, default=value)
    ap.add_argument("--lr", type=float, default=0.02)
    train(**vars(ap.parse_args()))
