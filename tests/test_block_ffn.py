"""The gated feed-forward block against its definition in float64: forward and
gradients, row counts from one to several tiles, widths that are no multiple
of a tile or stage, strided operands, both gradient types."""

import pytest
import torch

from block_reference import act, close

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
# h, dg and du are rounded to bf16 before the next product: 2^-8 of each term
# at most, so of an output's largest value.
ROUND = 2.0 ** -8


def block():
    from matrix_aware_optimizer_periodic_amd import block as b
    return b


def make(t, d, f, seed=0, std=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def r(*shape, s=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * s).to(BF16)
    return r(t, d, s=std), r(f, d, s=d ** -0.5), r(f, d, s=d ** -0.5), r(d, f, s=f ** -0.5), r(t, d)


def check(x, wg, wu, wd, dy, kind="silu", grads=True, grad_dtype=BF16):
    b = block()
    f = wg.shape[0]
    y, gu = b.ffn_fwd(x, wg, wu, wd, act=kind)
    x2 = x.reshape(-1, x.shape[-1]).double()
    g64, u64 = x2 @ wg.double().T, x2 @ wu.double().T
    close(gu, torch.cat([g64, u64], 1), "gu:bf16")
    close(y.reshape(x2.shape), (act(g64, kind) * u64) @ wd.double().T, "y:bf16", inner=ROUND)
    y2, none = b.ffn_fwd(x, wg, wu, wd, act=kind, save=False)
    assert torch.equal(y, y2) and none is None
    if not grads:
        return
    got = b.ffn_bwd(dy, x, wg, wu, wd, gu, act=kind, grad_dtype=grad_dtype)
    again = b.ffn_bwd(dy, x, wg, wu, wd, gu, act=kind, grad_dtype=grad_dtype)
    assert all(torch.equal(p, q) for p, q in zip(got, again))
    leaf = gu.double().requires_grad_(True)
    h = act(leaf[:, :f], kind) * leaf[:, f:]
    dy2 = dy.reshape(x2.shape).double()
    h.backward(dy2 @ wd.double())
    dg, du = leaf.grad[:, :f], leaf.grad[:, f:]
    want = (dg @ wg.double() + du @ wu.double(), dg.T @ x2, du.T @ x2, dy2.T @ h.detach())
    kinds = ("bf16",) + ("bf16" if grad_dtype == BF16 else "f32",) * 3
    for name, p, q, k in zip(("d_x", "d_w_gate", "d_w_up", "d_w_down"), got, want, kinds):
        close(p.reshape(q.shape), q, f"{name}:{k}", inner=ROUND)


@pytest.mark.parametrize("t", [1, 2, 7, 16, 17, 32, 33, 64, 65, 127, 128, 129, 300])
def test_row_counts(t):
    check(*make(t, 320, 712, seed=t))


@pytest.mark.parametrize("d,f", [(8, 8), (8, 264), (264, 8), (56, 72), (64, 64), (120, 136), (128, 128), (136, 120),
                                 (200, 1000), (1000, 200), (256, 256), (512, 520)])
@pytest.mark.parametrize("t", [3, 150])
def test_widths(t, d, f):
    check(*make(t, d, f, seed=d + f))


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("std", [1.0, 30.0])
def test_activations(kind, std):
    """std 30: projections far out, where the activation is 0 or the value."""
    check(*make(90, 256, 384, std=std), kind=kind)


@pytest.mark.parametrize("t,d,f", [(4096, 1280, 2576), (3000, 2048, 5000), (2049, 2056, 4104)])
def test_large_tiles(t, d, f):
    check(*make(t, d, f, seed=t), grad_dtype=torch.float32)


@pytest.mark.parametrize("t", [4, 200])
def test_fp32_gradients_and_strided_operands(t):
    b = block()
    x, wg, wu, wd, dy = make(t, 264, 392)
    check(x, wg, wu, wd, dy, grad_dtype=torch.float32)
    both = torch.cat([wg, wu], 1)                 # weights side by side in one buffer
    wide = torch.full((t, 400), float("nan"), device="cuda").to(BF16)
    wide[:, 64:328] = x
    y, gu = b.ffn_fwd(wide[:, 64:328], both[:, :264], both[:, 264:], wd)
    y2, gu2 = b.ffn_fwd(x, wg, wu, wd)
    assert torch.equal(y, y2) and torch.equal(gu, gu2)
    for p, q in zip(b.ffn_bwd(dy, wide[:, 64:328], both[:, :264], both[:, 264:], wd, gu),
                    b.ffn_bwd(dy, x, wg, wu, wd, gu)):
        assert torch.equal(p, q)


def test_shapes_and_empty():
    b = block()
    x, wg, wu, wd, dy = make(30, 64, 128)
    y, gu = b.ffn_fwd(x.view(2, 15, 64), wg, wu, wd)
    assert y.shape == (2, 15, 64) and gu.shape == (30, 256)
    y, gu = b.ffn_fwd(x[:0], wg, wu, wd)
    d = b.ffn_bwd(dy[:0], x[:0], wg, wu, wd, gu)
    assert y.shape == (0, 64) and all(bool((t == 0).all()) for t in d[1:])


def test_gradient_against_differences():
    """Differences of the forward pass along the gradient.  y is rounded to
    bf16 (2^-8 of each value, random sign): the step is large against that and
    small against the curvature; the slope is held to 10%."""
    b = block()
    args = list(make(40, 128, 256, seed=3))
    w = args.pop().float()
    y, gu = b.ffn_fwd(*args)
    for i, d in enumerate(b.ffn_bwd(w.to(BF16), *args, gu)):
        u = d.float() / d.float().norm()
        f, moved = [], []
        for s in (1.0, -1.0):
            a = list(args)
            a[i] = (a[i].float() + s * u).to(BF16)
            moved.append(a[i].double())
            f.append(float((b.ffn_fwd(*a)[0].double() * w.to(BF16).double()).sum()))
        want = float(((moved[0] - moved[1]) * d.double()).sum())
        assert abs(f[0] - f[1] - want) <= 0.1 * abs(want), (i, f, want)


def test_autograd():
    b = block()
    x, wg, wu, wd, dy = make(50, 128, 256)
    leaves = [t.clone().requires_grad_(True) for t in (x, wg, wu, wd)]
    b.gated_ffn(*leaves, act="gelu").backward(dy)
    _, gu = b.ffn_fwd(x, wg, wu, wd, act="gelu")
    for t, g in zip(leaves, b.ffn_bwd(dy, x, wg, wu, wd, gu, act="gelu")):
        assert torch.equal(t.grad, g)


@pytest.mark.parametrize("t", [1, 200])
def test_graph_replays(t):
    b = block()
    x, wg, wu, wd, dy = make(t, 256, 512)
    b.ffn_fwd(x, wg, wu, wd)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, gu = b.ffn_fwd(x, wg, wu, wd)
        d = b.ffn_bwd(dy, x, wg, wu, wd, gu)
    for _ in range(3):
        x.normal_()
        graph.replay()
        torch.cuda.synchronize()
        y2, gu2 = b.ffn_fwd(x, wg, wu, wd)
        d2 = b.ffn_bwd(dy, x, wg, wu, wd, gu2)
        assert torch.equal(y, y2) and all(torch.equal(p, q) for p, q in zip(d, d2))


@pytest.mark.parametrize("t", [70_000])
def test_offsets_past_32_bits(t):
    """Rows 2^15 values apart, more than 2^31 values in all, on every side."""
    b = block()
    x1, wg, wu, wd, dy1 = make(t, 64, 128)
    x, dy = (torch.empty(t * 32768, dtype=BF16, device="cuda").view(t, 32768)[:, 64:128] for _ in range(2))
    x.copy_(x1)
    dy.copy_(dy1)
    y, gu = b.ffn_fwd(x, wg, wu, wd)
    y1, gu1 = b.ffn_fwd(x1, wg, wu, wd)
    assert torch.equal(y, y1) and torch.equal(gu, gu1)
    wide = torch.empty(t * 32768, dtype=BF16, device="cuda").view(t, 32768)[:, 8:264]
    wide.copy_(gu)
    for p, q in zip(b.ffn_bwd(dy, x, wg, wu, wd, wide), b.ffn_bwd(dy1, x1, wg, wu, wd, gu)):
        assert torch.equal(p, q)


def test_another_stream():
    b = block()
    x, wg, wu, wd, dy = make(700, 256, 512)
    y, gu = b.ffn_fwd(x, wg, wu, wd)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y2, gu2 = b.ffn_fwd(x, wg, wu, wd)
        d2 = b.ffn_bwd(dy, x, wg, wu, wd, gu2)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, y2)
    assert all(torch.equal(p, q) for p, q in zip(d2, b.ffn_bwd(dy, x, wg, wu, wd, gu)))


@pytest.mark.parametrize("t,d,f", [(200, 4096, 128), (70, 2048, 64), (4096, 2048, 4096)])
def test_few_tiles_and_long_sums(t, d, f):
    """Sums over k divided over several workgroups, in every kind of product."""
    check(*make(t, d, f, seed=d + t), kind="gelu")


@pytest.mark.parametrize("t", [1, 8, 9, 33])
@pytest.mark.parametrize("d,f", [(4072, 136), (4104, 72), (136, 4072), (72, 4104), (5128, 20488)])
def test_few_rows_and_many_columns(t, d, f):
    """Each form of the few-row products on both sides of the limits of its
    rows and columns, where the last group of columns is cut."""
    check(*make(t, d, f, seed=d + t), grads=False)
