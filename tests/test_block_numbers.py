"""Numbers that rotary, linear and dropout take, on the CPU: whole ones, of 64 bits,
of any type that stands for one; others raise as other arguments do."""

import numpy as np
import pytest
import torch

from test_block_linear_boundary import b, m, packed  # noqa: F401

BF16 = torch.bfloat16


def test_numbers_that_are_not_whole_or_too_large(packed):  # noqa: F811
    q, f = torch.zeros(2, 5, 4, 16), torch.zeros(1, 8, dtype=torch.float64)
    x, w = torch.zeros(6, 64, dtype=BF16), torch.zeros(96, 64, dtype=BF16)
    for rng in ((1.5, 2), (1, 2.0), (1, None), ("1", 2)):
        for call in (lambda: m.linear_fwd(x, w, p=0.5, rng=rng), lambda: m.linear_bwd(x[:, :8], x, w[:8], p=0.5, rng=rng),
                     lambda: m.dropout_fwd(x, 0.5, rng), lambda: m.dropout_bwd(x, 0.5, rng)):
            with pytest.raises(TypeError):
                call()
    for offset, error in ((1 << 63, ValueError), (-(1 << 63) - 1, ValueError), (1.5, TypeError)):
        for call in (m.rotary_fwd, m.rotary_bwd):
            with pytest.raises(error):
                call(q, None, f, offset=offset)
    assert not packed
    for one in (7, np.int64(7), torch.tensor(7)):
        packed.clear()
        m.dropout_fwd(x, 0.5, (one, one))
        m.rotary_fwd(q, None, f, offset=one)
        assert b.DROPOUT_ARGS.unpack(packed[0][1])[3:5] == (7, 7) and b.ROTARY_ARGS.unpack(packed[1][1])[12] == 7
