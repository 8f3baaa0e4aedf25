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
