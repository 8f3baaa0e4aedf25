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
