"""linear_bwd's one rounding within: dz to bf16, as the products' operand.  Against
fp64 products of that rounded dz the gradients are off by their own sums and
rounding alone, whatever was dropped and whatever the slopes."""

import pytest
import torch

from block_reference_linear import acted, drop

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
RNG = (0x0123456789ABCDEF, 1 << 40)


# up to 16 rows of a large weight, tiles, tiles of several rounds, a divided gradient of
# either kind, widths that are no multiple of a tile
SIZES = [(6, 5120, 20480), (150, 200, 264), (777, 1000, 2728), (4096, 512, 1536), (9000, 256, 32), (200, 4096, 136),
         (300, 64, 8192), (130, 8, 8)]


@pytest.mark.parametrize("grad_dtype", [F32, BF16])
@pytest.mark.parametrize("kind,p", [("none", 0.3), ("silu", 0.0), ("gelu", 0.2)])
@pytest.mark.parametrize("t,d,n", SIZES)
def test_gradients_are_those_of_the_rounded_dz(t, d, n, kind, p, grad_dtype):
    """dz in fp32 is off by 2^-21 at most (a slope's exponential), so that one in 2^12
    falls on the other side of a border between two bf16 values, by a step of 2^-7
    at most: 2^-6 x 2^-7 = 1.2e-4 of a gradient's norm, and twice that is allowed.
    On top of it come the results' own roundings: of bf16 what rounding the fp64
    gradient does (a thirtieth more, for values that cross a border by the former)."""
    from matrix_aware_optimizer_periodic_amd import block as b
    gen = torch.Generator(device="cuda").manual_seed(t + d + n)

    def r(*shape, s=1.0, dtype=BF16):
        return (torch.randn(shape, generator=gen, device="cuda") * s).to(dtype)
    x, w, z, dy = r(t, d), r(n, d, s=d ** -0.5), r(t, n), r(t, n, dtype=F32)
    got = b.linear_bwd(dy, x, w, None, None if kind == "none" else z, act=kind, p=p, rng=RNG if p else None, grad_dtype=grad_dtype)
    dz = drop(dy.double(), p, RNG)
    if kind != "none":
        leaf = z.double().requires_grad_(True)
        dz, = torch.autograd.grad(acted(leaf, kind), leaf, dz)
    rounded = dz.to(BF16).double()
    for name, g, want in (("d_x", got[0], rounded @ w.double()), ("d_weight", got[1], rounded.T @ x.double())):
        own = 0.0 if g.dtype == F32 else float((want.to(BF16).double() - want).norm() / want.norm())
        off = float((g.double() - want).norm() / want.norm())
        assert off <= own * (1 + 1 / 30) + 2.4e-4, (name, off, own)
    exact = dz.T @ x.double()
    if grad_dtype == F32:
        # what the rounding itself does: up to half a step of 2^-8 of every term, at random
        assert float((got[1].double() - exact).norm() / exact.norm()) <= 2.0 ** -8 / 3 ** 0.5
