"""d_bias to the rounding of its own sums, however the rows are shared out."""

import pytest
import torch

from block_reference import close

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def deviations(t, n):
    """The sums' error in deviations of a standard normal, in the order in which a
    call of t rows and n columns adds: a thread down its rows, the threads of a
    workgroup, the shares.  A partial sum of k rows is sqrt(k) large, its rounding
    2^-24 / sqrt(3) of that at random."""
    chunks, width = n // 8, 1
    while width < 64 and width < chunks:
        width *= 2
    blocks, turn = -(-chunks // width), 256 // width
    turns = -(-t // turn)
    shares = max(1, min(turns, 256, 1024 // blocks))
    deep = -(-turns // shares)
    shares = -(-t // (deep * turn))
    # sums of the partial sums' squares: i rows, i threads of `deep` rows, i shares
    thread = shares * turn * deep * (deep + 1) / 2
    group = shares * deep * turn * (turn + 1) / 2
    joined = deep * turn * shares * (shares + 1) / 2
    return 2.0 ** -24 * ((thread + group + joined) / 3) ** 0.5


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("t,n", [(1, 8), (64, 256), (65, 520), (300, 136), (1000, 1000), (4097, 2048), (5000, 24), (9000, 520),
                                 (20000, 3208), (70_000, 8)])
def test_sums_to_their_own_rounding(t, n, act, dtype):
    """Within eight deviations of the largest sum that t rows come to, sqrt(t): for
    70000 rows of 8 columns 4e-6 of it (and, with an activation, 2^-22 of each term
    for its slope, at random: 2^-22 of the sum)."""
    from matrix_aware_optimizer_periodic_amd import block as b
    gen = torch.Generator(device="cuda").manual_seed(t + n)
    x, w = (torch.randn(s, 64, generator=gen, device="cuda").to(BF16) for s in (t, n))
    dy, z = torch.randn(t, n, generator=gen, device="cuda").to(dtype), torch.randn(t, n, generator=gen, device="cuda").to(BF16)
    bias = torch.zeros(n, device="cuda")
    dz = dy.double()
    if act == "gelu":
        leaf = z.double().requires_grad_(True)
        dz, = torch.autograd.grad(torch.nn.functional.gelu(leaf, approximate="tanh"), leaf, dz)
    want = dz.sum(0)
    tol = 8 * deviations(t, n) + (4 * 2.0 ** -22 * t ** 0.5 if act == "gelu" else 0.0)
    for which in (dict(need_x=False, need_weight=False), {}):
        got = b.linear_bwd(dy, x, w, bias, z if act == "gelu" else None, act=act, **which)[2]
        off = (got.double() - want).abs() - 2.0 ** -24 * want.abs()
        assert float(off.max()) <= tol, (float(off.max()), tol)
    close(got, want, "d_bias:f32")
