"""What the autograd functions of linear, rotary and dropout take, save and form, on
the CPU with stand-ins for the library's calls."""

import pytest
import torch

from test_block_linear_boundary import b, leaves, stand_ins  # noqa: F401

BF16 = torch.bfloat16


def test_learned_frequencies_are_refused(stand_ins):  # noqa: F811
    """They would stay as they are, without a word."""
    q, k, f = leaves((2, 3, 2, 8), (2, 3, 1, 8), (1, 4))
    qkv, = leaves((2, 3, 3, 2, 8))
    calls = (lambda f: b.rotary(q, k, f)[0], lambda f: b.attention_qkv(qkv, rotary={"freqs": f}))
    for call in calls:
        with pytest.raises(ValueError, match="freqs"):
            call(f)
        call(f.detach()).sum().backward()
        with torch.no_grad():
            call(f)


def test_rotary_turns_only_the_gradients_that_are_wanted(stand_ins, monkeypatch):  # noqa: F811
    q, k, f = leaves((2, 3, 2, 8), (2, 3, 1, 8), (1, 4))
    f = f.detach()
    turned = []
    call = b.rotary_bwd
    monkeypatch.setattr(b, "rotary_bwd", lambda d_q, d_k, *a, **h: (turned.append((d_q, d_k)), call(d_q, d_k, *a, **h))[1])

    def shapes(q, k):
        turned.clear()
        torch.cat(b.rotary(q, k, f), 2).sum().backward()
        (d_q, d_k), = turned
        return d_q.shape, None if d_k is None else d_k.shape
    assert shapes(q, k) == (q.shape, k.shape)
    assert shapes(q, k.detach()) == (q.shape, None)
    k.grad = None
    assert shapes(q.detach(), k) == (k.shape, None)         # (one tensor is turned in q's place)
    assert torch.equal(k.grad, torch.full_like(k, 3.0))


def test_rotary_reads_gradients_where_they_lie(stand_ins, monkeypatch):  # noqa: F811
    """Heads before positions, slices of a packed gradient and sums over samples as
    they are; a last dimension that is not contiguous is copied."""
    q, k, f = leaves((2, 3, 2, 8), (2, 3, 1, 8), (1, 4))
    f = f.detach()
    seen = []
    call = b.rotary_bwd
    monkeypatch.setattr(b, "rotary_bwd", lambda d_q, d_k, *a, **h: (seen.append((d_q.stride(), d_k.stride())), call(d_q, d_k, *a, **h))[1])
    gen = torch.Generator().manual_seed(1)
    w = torch.randn(2, 3, 2, 8, generator=gen, dtype=torch.float64)
    ways = {"heads first": (w.transpose(1, 2).contiguous().transpose(1, 2), (48, 8, 24, 1)),
            "packed": (torch.stack([w, w], 2)[:, :, 1], (96, 32, 8, 1)),
            "one sample's": (w[:1].expand_as(w), (0, 16, 8, 1)),
            "dim first": (w.transpose(2, 3).contiguous().transpose(2, 3), (48, 16, 8, 1)),
            "one value": (w[:1, :1, :1, :1].expand_as(w), (48, 16, 8, 1))}
    for name, (d, stride) in ways.items():
        seen.clear()
        q.grad = None
        torch.autograd.backward(b.rotary(q, k, f), (d, torch.ones_like(k)))
        assert seen[0][0] == stride, name
        assert torch.equal(q.grad, d * 3), name


@pytest.mark.gpu
def test_rotary_gradients_of_any_strides():
    gen = torch.Generator(device="cuda").manual_seed(2)
    q, k, w = (torch.randn(2, 9, h, 64, generator=gen, device="cuda").to(BF16) for h in (4, 2, 4))
    f = b.rotary_freqs(40)
    want = b.rotary_bwd(w, None, f)[0]
    for d in (w.transpose(1, 2).contiguous().transpose(1, 2), torch.stack([w, w], 2)[:, :, 1],
              torch.cat([w.new_zeros(1), w.flatten()])[1:].view(w.shape), w.transpose(2, 3).contiguous().transpose(2, 3)):
        leaf, other = q.clone().requires_grad_(True), k.clone().requires_grad_(True)
        turned = b.rotary(leaf, other, f)
        torch.autograd.backward(turned, (d, torch.ones_like(k)))
        assert torch.equal(leaf.grad, want) and torch.equal(other.grad, b.rotary_bwd(torch.ones_like(k), None, f)[0])
    leaf = q.clone().requires_grad_(True)
    b.rotary(leaf, None, f)[0].backward(w[:1].expand_as(w))
    assert torch.equal(leaf.grad, want[:1].expand_as(w))
