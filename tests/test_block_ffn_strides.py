"""The gated feed-forward block with weights whose rows lie differently far
apart: every result equals the one of contiguous weights, bit for bit."""

import pytest
import torch

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def wide(t, extra):
    """t as columns of a buffer `extra` wider, NaN beside them."""
    if extra == 0:
        return t
    buf = torch.full((t.shape[0], t.shape[1] + extra), float("nan"), dtype=t.dtype, device="cuda")
    view = buf[:, 8:8 + t.shape[1]]
    view.copy_(t)
    return view


# few rows, one stage and several per matrix, 128- and 256-tiles, sums over k
# in ranges that begin in the first and in the second matrix
@pytest.mark.parametrize("t,d,f", [(4, 64, 128), (200, 64, 128), (130, 136, 8), (130, 136, 72), (300, 264, 392),
                                   (70, 64, 2048), (200, 128, 4096), (2049, 1032, 1288)])
@pytest.mark.parametrize("gate,up,down", [(0, 32, 0), (32, 0, 0), (512, 16, 48), (8, 264, 0)])
def test_rows_of_gate_up_and_down_apart(t, d, f, gate, up, down):
    from matrix_aware_optimizer_periodic_amd import block as b
    gen = torch.Generator(device="cuda").manual_seed(t + d + f)

    def r(*shape, s=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * s).to(BF16)
    x, dy, wg, wu, wd = r(t, d), r(t, d), r(f, d, s=d ** -0.5), r(f, d, s=d ** -0.5), r(d, f, s=f ** -0.5)
    y, gu = b.ffn_fwd(x, wg, wu, wd)
    want = b.ffn_bwd(dy, x, wg, wu, wd, gu)
    apart = wide(wg, gate), wide(wu, up), wide(wd, down)
    y2, gu2 = b.ffn_fwd(x, *apart)
    assert torch.equal(y, y2) and torch.equal(gu, gu2)
    for name, p, q in zip(("d_x", "d_w_gate", "d_w_up", "d_w_down"), want, b.ffn_bwd(dy, x, *apart, gu)):
        assert torch.equal(p, q), name
