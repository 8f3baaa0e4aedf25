"""Linear layers with their epilogue against the definition in float64: forward
and gradients, row counts from one to several tiles, widths that are no multiple
of a tile or stage, every type, strided operands, dropout, graphs, streams."""

import pytest
import torch

from block_reference import close, name_of
from block_reference_linear import acted, drop, kept, linear

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
# dz is rounded to bf16 before the products: 2^-8 of each term at most, of
# random sign, so of a gradient's largest value.
ROUND = 2.0 ** -8
RNG = (0x1234567890ABCDEF, 0xFEDCBA9876543210)


def block():
    from matrix_aware_optimizer_periodic_amd import block as b
    return b


def make(t, d, n, seed=0, std=1.0, bias=F32, resid=None):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def r(*shape, s=1.0, dtype=BF16):
        return (torch.randn(shape, generator=gen, device="cuda") * s).to(dtype)
    x, w = r(t, d, s=std), r(n, d, s=d ** -0.5)
    b = None if bias is None else r(n, s=0.5, dtype=bias)
    res = None if resid is None else r(t, n, s=2.0, dtype=resid)
    return x, w, b, res, r(t, n, dtype=BF16 if resid is None else resid)


def wide(t):
    return None if t is None else t.double()


def small(x, w):
    """Whether the backward call keeps dz in fp32."""
    t, (n, d) = x.shape[0], w.shape
    return t <= 128 and n <= 128 and t * d * n <= 20_000_000


def check(x, w, bias, res, dy, kind="none", p=0.0, rng=None, grads=True, grad_dtype=BF16):
    b = block()
    y, z = b.linear_fwd(x, w, bias, res, act=kind, p=p, rng=rng)
    y64, z64 = linear(wide(x), wide(w), wide(bias), wide(res), kind, p, rng)
    assert y.dtype == (BF16 if res is None else res.dtype) and (z is None) == (kind == "none")
    close(y, y64, "y:" + name_of(y))
    if z is not None:
        close(z, z64, "z:bf16")
    y2, none = b.linear_fwd(x, w, bias, res, act=kind, p=p, rng=rng, save=False)
    assert torch.equal(y, y2) and none is None
    if not grads:
        return
    how = dict(act=kind, p=p, rng=rng, grad_dtype=grad_dtype)
    got = b.linear_bwd(dy, x, w, bias, z, **how)
    again = b.linear_bwd(dy, x, w, bias, z, **how)
    assert all((p is None and q is None) or torch.equal(p, q) for p, q in zip(got, again))
    # from the z that was kept
    dz = drop(wide(dy), p, rng)
    if kind != "none":
        leaf = wide(z).requires_grad_(True)
        dz, = torch.autograd.grad(acted(leaf, kind), leaf, dz)
    exact = kind == "none" and p == 0.0 and dy.dtype == BF16 or small(x, w)
    inner = 0.0 if exact else ROUND
    close(got[0], dz @ wide(w), "d_x:bf16", inner=inner)
    close(got[1], dz.T @ wide(x), "d_weight:" + name_of(got[1]), inner=inner)
    assert (got[2] is None) == (bias is None)
    if bias is not None:
        assert got[2].dtype == bias.dtype
        close(got[2], dz.sum(0), "d_bias:" + name_of(got[2]))


@pytest.mark.parametrize("t", [1, 2, 7, 8, 9, 16, 17, 32, 33, 64, 65, 127, 128, 129, 300])
def test_row_counts(t):
    check(*make(t, 320, 712, seed=t))
    check(*make(t, 320, 712, seed=t, resid=F32), kind="gelu", p=0.3, rng=RNG)


@pytest.mark.parametrize("d,n", [(8, 8), (8, 264), (264, 8), (56, 72), (64, 64), (120, 136), (128, 128), (136, 120),
                                 (200, 1000), (1000, 200), (256, 256), (512, 520), (8, 520), (24, 528), (72, 584),
                                 (120, 640), (136, 1032), (520, 8), (2056, 24)])
@pytest.mark.parametrize("t", [3, 150, 600])
def test_widths(t, d, n):
    check(*make(t, d, n, seed=d + n, resid=BF16), kind="silu", p=0.1, rng=RNG)


@pytest.mark.parametrize("kind", ["none", "silu", "gelu"])
@pytest.mark.parametrize("bias", [None, F32, BF16])
@pytest.mark.parametrize("resid", [None, F32, BF16])
@pytest.mark.parametrize("t", [5, 40, 200])
def test_types(t, kind, bias, resid):
    check(*make(t, 128, 136, bias=bias, resid=resid), kind=kind)
    check(*make(t, 128, 136, bias=bias, resid=resid), kind=kind, p=0.25, rng=RNG, grad_dtype=F32)


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_far_activations(kind):
    """Projections far out, where the activation is 0 or the value."""
    check(*make(90, 256, 384, std=30.0), kind=kind)


@pytest.mark.parametrize("t,d,n", [(4096, 1280, 2576), (3000, 2048, 5000), (2049, 2056, 4104)])
def test_large_tiles(t, d, n):
    check(*make(t, d, n, seed=t, resid=F32), kind="gelu", p=0.1, rng=RNG)
    check(*make(t, d, n, seed=t), grad_dtype=F32)


@pytest.mark.parametrize("t,d,n", [(200, 4096, 128), (70, 2048, 64), (4096, 4096, 256), (300, 64, 8192)])
def test_few_tiles_and_long_sums(t, d, n):
    """Sums over k divided over several workgroups, in every product."""
    check(*make(t, d, n, seed=d + t, resid=BF16), kind="gelu", p=0.5, rng=RNG)


@pytest.mark.parametrize("t,d,n", [(20000, 256, 32), (3000, 24, 16), (16400, 136, 4096), (40, 16, 16384), (9000, 8, 8),
                                   (5000, 1152, 32)])
def test_one_product_with_few_tiles(t, d, n):
    """The weight's gradient, the input's or both have few tiles of long sums:
    divided first, second or in launches of their own.  fp32 sums of 20000 terms,
    32 at a time: 625 additions of 2^-24 of random sign, within 1e-5."""
    check(*make(t, d, n, seed=d + t), grad_dtype=F32)
    check(*make(t, d, n, seed=d + t, resid=F32), kind="silu")


@pytest.mark.parametrize("t", [1, 8, 9, 33])
@pytest.mark.parametrize("d,n", [(4072, 136), (4104, 72), (136, 4072), (72, 4104), (2048, 12288)])
def test_few_rows_and_many_columns(t, d, n):
    check(*make(t, d, n, seed=d + t, resid=F32), kind="silu")


@pytest.mark.parametrize("t,n", [(1, 8), (70_000, 8), (5000, 24), (9000, 520), (1000, 1000), (4097, 2048)])
def test_bias_sums(t, n):
    """d_bias alone and with the others, over one and many shares of the rows.
    A share's thread adds up to 9000 / 8 values in turn: within 2^-24 x 1125 of
    the sums' size, 1e-4 of the largest at worst."""
    b = block()
    x, w, bias, _, dy = make(t, 64, n)
    for which in (dict(need_x=False, need_weight=False), dict(need_x=False), dict(need_weight=False)):
        got = b.linear_bwd(dy, x, w, bias, **which)
        assert (got[0] is None) == (which.get("need_x") is False) and (got[1] is None) == (which.get("need_weight") is False)
        close(got[2], dy.double().sum(0), "d_bias:f32", f32_tol=1e-4)
    assert b.linear_bwd(dy, x, w, None)[2] is None
    got = b.linear_bwd(dy, None, w, None, need_weight=False)
    # (alone, a product's sum may be divided otherwise than beside the other)
    assert got[1] is None
    close(got[0], dy.double() @ w.double(), "d_x:bf16")


@pytest.mark.parametrize("t", [4, 50, 300])
def test_strided_operands(t):
    b = block()
    x, w, bias, res, dy = make(t, 264, 392, resid=F32)
    z = b.linear_fwd(x, w, bias, res, act="silu", p=0.2, rng=RNG)[1]

    def apart(v, before, after):
        o = torch.full((v.shape[0], before + v.shape[1] + after), float("nan"), dtype=v.dtype, device="cuda")
        o[:, before:before + v.shape[1]] = v
        return o[:, before:before + v.shape[1]]
    xs, ws, rs, dys, zs = apart(x, 64, 8), apart(w, 8, 16), apart(res, 4, 4), apart(dy, 8, 0), apart(z, 8, 8)
    bs = torch.cat([bias[:3], bias])[3:]          # off every boundary but its type's
    for p, q in zip(b.linear_fwd(xs, ws, bs, rs, act="silu", p=0.2, rng=RNG),
                    b.linear_fwd(x, w, bias, res, act="silu", p=0.2, rng=RNG)):
        assert torch.equal(p, q)
    for p, q in zip(b.linear_bwd(dys, xs, ws, bs, zs, act="silu", p=0.2, rng=RNG),
                    b.linear_bwd(dy, x, w, bias, z, act="silu", p=0.2, rng=RNG)):
        assert torch.equal(p, q)


def test_shapes_and_empty():
    b = block()
    x, w, bias, res, dy = make(30, 64, 128, resid=BF16)
    y, z = b.linear_fwd(x.view(2, 15, 64), w, bias, res.view(2, 15, 128), act="gelu")
    assert y.shape == (2, 15, 128) and z.shape == (30, 128)
    d = b.linear_bwd(dy.view(2, 15, 128), x.view(2, 15, 64), w, bias, z, act="gelu")
    assert d[0].shape == (2, 15, 64) and d[1].shape == w.shape and d[2].shape == bias.shape
    assert b.linear_fwd(x[0], w, bias)[0].shape == (128,)
    y, z = b.linear_fwd(x[:0], w, bias, res[:0], act="gelu")
    d = b.linear_bwd(dy[:0], x[:0], w, bias, z, act="gelu")
    assert y.shape == (0, 128) and d[0].shape == (0, 64) and all(bool((t == 0).all()) for t in d[1:])
    assert b.linear_fwd(x, w, y_dtype=F32)[0].dtype == F32


@pytest.mark.parametrize("t", [6, 40, 500])
def test_dropout_is_the_operator(t):
    """The same elements as dropout drops of the same shape, dropped ones exactly
    the residual; all of them with p = 1."""
    b = block()
    x, w, bias, res, dy = make(t, 128, 264, resid=F32)
    mask = kept((t, 264), 0.4, RNG)
    y, _ = b.linear_fwd(x, w, bias, res, p=0.4, rng=RNG)
    assert torch.equal(y[~mask], res[~mask])
    plain = b.linear_fwd(x, w, bias, y_dtype=F32)[0]
    assert torch.equal(y, b.dropout_fwd(plain, 0.4, RNG, res))
    state = torch.tensor([RNG[0], RNG[1] - 2 ** 64], device="cuda")
    assert torch.equal(y, b.linear_fwd(x, w, bias, res, p=0.4, rng=state)[0])
    assert torch.equal(b.linear_fwd(x, w, bias, res, p=1.0, rng=RNG)[0], res)
    for g in b.linear_bwd(dy, x, w, bias, p=1.0, rng=RNG):
        assert bool((g == 0).all())
    assert all(torch.equal(p, q) for p, q in zip(b.linear_bwd(dy, x, w, bias, p=0.4, rng=RNG),
                                                 b.linear_bwd(dy, x, w, bias, p=0.4, rng=state)))


@pytest.mark.parametrize("t", [3, 40, 300])
def test_values_that_are_not_finite(t):
    """A row of NaN or infinities reaches its own row of y, and d_x and no other."""
    b = block()
    x, w, bias, res, dy = make(t, 128, 136, resid=F32)
    y, _ = b.linear_fwd(x, w, bias, res, act="gelu")
    bad = x.clone()
    bad[1] = float("nan")
    y2, _ = b.linear_fwd(bad, w, bias, res, act="gelu")
    others = torch.arange(t, device="cuda") != 1
    assert bool(torch.isnan(y2[1]).all()) and torch.equal(y2[others], y[others])
    bad = dy.clone()
    bad[1, 5] = float("inf")
    d, d2 = b.linear_bwd(dy, x, w, bias), b.linear_bwd(bad, x, w, bias)
    assert not bool(torch.isfinite(d2[0][1]).any()) and torch.equal(d2[0][others], d[0][others])
    cols = torch.arange(136, device="cuda") != 5
    assert torch.equal(d2[1][cols], d[1][cols]) and torch.equal(d2[2][cols], d[2][cols]) and d2[2][5] == float("inf")


def test_gradient_against_differences():
    """Differences of the forward pass along the gradient, in fp32 (y_dtype),
    where y = act(...) is rounded once by 2^-24: the step is small against the
    curvature; the slope is held to 2%, over the 2^-8 of dz's rounding."""
    b = block()
    x, w, bias, _, _ = make(40, 128, 256, seed=3)
    weight = torch.randn(40, 256, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    how = dict(act="gelu", p=0.2, rng=RNG)
    z = b.linear_fwd(x, w, bias, **how)[1]
    for i, d in enumerate(b.linear_bwd(weight, x, w, bias, z, **how)):
        u = d.float() / d.float().norm()
        f, moved = [], []
        for s in (0.5, -0.5):
            a = [x, w, bias]
            a[i] = (a[i].float() + s * u).to(a[i].dtype)
            moved.append(a[i].double())
            f.append(float((b.linear_fwd(*a, y_dtype=F32, **how)[0].double() * weight.double()).sum()))
        want = float(((moved[0] - moved[1]) * d.double()).sum())
        assert abs(f[0] - f[1] - want) <= 0.02 * abs(want), (i, f, want)


def test_autograd():
    b = block()
    x, w, bias, res, dy = make(50, 128, 256, resid=F32)
    how = dict(act="gelu", p=0.1, rng=RNG)
    leaves = [t.clone().requires_grad_(True) for t in (x, w, bias, res)]
    b.linear(*leaves, **how).backward(dy)
    z = b.linear_fwd(x, w, bias, res, **how)[1]
    for t, g in zip(leaves, (*b.linear_bwd(dy, x, w, bias, z, **how), dy)):
        assert torch.equal(t.grad, g)
    # an expanded gradient, frozen weights
    x2 = x.clone().requires_grad_(True)
    b.linear(x2, w, bias, act="silu").sum().backward()
    z = b.linear_fwd(x, w, bias, act="silu")[1]
    assert torch.equal(x2.grad, b.linear_bwd(torch.ones(50, 256, dtype=BF16, device="cuda"), x, w, None, z, act="silu")[0])


@pytest.mark.parametrize("t", [1, 40, 300])
def test_graph_replays(t):
    """Each replay with another mask, by the offset in device memory."""
    b = block()
    x, w, bias, res, dy = make(t, 256, 512, resid=F32)
    state = torch.tensor([7, 0], device="cuda")
    how = dict(act="silu", p=0.3, rng=state)
    b.linear_fwd(x, w, bias, res, **how)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, z = b.linear_fwd(x, w, bias, res, **how)
        d = b.linear_bwd(dy, x, w, bias, z, **how)
    seen = []
    for i in range(3):
        x.normal_()
        state[1] = i
        graph.replay()
        torch.cuda.synchronize()
        y2, z2 = b.linear_fwd(x, w, bias, res, act="silu", p=0.3, rng=(7, i))
        d2 = b.linear_bwd(dy, x, w, bias, z2, act="silu", p=0.3, rng=(7, i))
        assert torch.equal(y, y2) and torch.equal(z, z2) and all(torch.equal(p, q) for p, q in zip(d, d2))
        seen.append(y == res)
    assert not torch.equal(seen[0], seen[1]) and not torch.equal(seen[1], seen[2])


def test_another_stream():
    b = block()
    x, w, bias, res, dy = make(700, 256, 512, resid=F32)
    how = dict(act="gelu", p=0.1, rng=RNG)
    y, z = b.linear_fwd(x, w, bias, res, **how)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y2, z2 = b.linear_fwd(x, w, bias, res, **how)
        d2 = b.linear_bwd(dy, x, w, bias, z2, **how)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, y2)
    assert all(torch.equal(p, q) for p, q in zip(d2, b.linear_bwd(dy, x, w, bias, z, **how)))


def test_offsets_past_32_bits():
    """Rows 2^15 values apart, more than 2^31 values in all, on every side."""
    b = block()
    t = 70_000
    x1, w, bias, res1, dy1 = make(t, 64, 128, resid=BF16)

    def far(v):
        o = torch.empty(t * 32768, dtype=v.dtype, device="cuda").view(t, 32768)[:, 64:64 + v.shape[1]]
        o.copy_(v)
        return o
    how = dict(act="silu", p=0.1, rng=RNG)
    x, res = far(x1), far(res1)
    y, z = b.linear_fwd(x, w, bias, res, **how)
    y1, z1 = b.linear_fwd(x1, w, bias, res1, **how)
    assert torch.equal(y, y1) and torch.equal(z, z1)
    del res
    dy, z = far(dy1), far(z1)
    for p, q in zip(b.linear_bwd(dy, x, w, bias, z, **how), b.linear_bwd(dy1, x1, w, bias, z1, **how)):
        assert torch.equal(p, q)


def test_numbers_of_dropped_elements_past_32_bits():
    """2^32 elements and some: the mask of the last rows."""
    b = block()
    t, n = (1 << 29) + 40, 8
    x = torch.zeros(t, 8, dtype=BF16, device="cuda")
    bias = torch.ones(n, device="cuda")
    w = torch.zeros(n, 8, dtype=BF16, device="cuda")
    y = b.linear_fwd(x, w, bias, p=0.5, rng=RNG)[0]
    for first in (0, 1 << 29, (1 << 29) + 32):
        part = min(40, t - first)
        assert torch.equal(y[first:first + part] != 0, kept((part, n), 0.5, RNG, first=first * n))


@pytest.mark.parametrize("t", [1, 3, 4, 5, 8, 9, 13, 16, 17])
@pytest.mark.parametrize("d,n", [(4096, 24504), (16392, 6104), (5128, 19504), (104, 1048568), (1048568, 104)])
@pytest.mark.parametrize("exact", [False, True])
def test_large_gradients_from_few_rows(t, d, n, exact):
    """On both sides of the limits of the weight's gradient from few rows, last
    columns cut both ways, with dz formed and as it comes."""
    x, w, bias, _, dy = make(t, d, n, seed=t, resid=None if exact else F32)
    how = dict(grad_dtype=F32) if exact else dict(kind="silu")
    check(x, w, bias, None, dy, **how)
    if t == 5:
        b = block()
        got = b.linear_bwd(dy, x, w, bias, torch.zeros(t, n, dtype=BF16, device="cuda"), act="silu", need_x=False)
        # act'(0) = 1/2, which every type holds
        close(got[1], (dy.double() / 2).T @ x.double(), "d_weight:bf16", inner=0.0 if exact else ROUND)
        close(got[2], dy.double().sum(0) / 2, "d_bias:f32")


@pytest.mark.parametrize("t", [1, 31, 32, 33, 128, 129])
@pytest.mark.parametrize("d,n", [(8, 8), (40, 24), (1216, 128), (1224, 128), (144, 136), (4096, 32)])
@pytest.mark.parametrize("kind,p", [("none", 0.0), ("gelu", 0.0), ("silu", 0.3)])
def test_small_gradients(t, d, n, kind, p):
    """On both sides of the small form's limits, its blocks of 32 cut every way,
    each gradient alone and together."""
    x, w, bias, _, dy = make(t, d, n, seed=t + n, resid=F32 if p else None)
    rng = RNG if p else None
    check(x, w, bias, None, dy, kind=kind, p=p, rng=rng, grad_dtype=F32)
    if not small(x, w):
        return
    b = block()
    z = b.linear_fwd(x, w, bias, act=kind, p=p, rng=rng)[1]
    how = dict(act=kind, p=p, rng=rng)
    every = b.linear_bwd(dy, x, w, bias, z, **how)
    assert torch.equal(b.linear_bwd(dy, None, w, None, z, need_weight=False, **how)[0], every[0])
    assert torch.equal(b.linear_bwd(dy, x, w, None, z, need_x=False, **how)[1], every[1])
    assert torch.equal(b.linear_bwd(dy, x, w, bias, z, need_x=False, need_weight=False, **how)[2], every[2])
