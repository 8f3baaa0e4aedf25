"""The fused residual norm against its definition in float64: forward,
gradients (autograd of the definition, and differences of the kernel itself),
types, widths that are no multiple of eight, strided operands, absent parts,
rows of zeros and streams."""

import pytest
import torch

from block_reference import close, name_of, norm_block

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def block():
    from matrix_aware_optimizer_periodic_amd import block as b
    return b


def make(samples, rows, cols, rt, ht, pt, vectors=True, weights=True, seed=0, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def r(*shape, dt=F32, s=1.0, add=0.0):
        return (torch.randn(shape, generator=g, device="cuda") * s + add).to(dt)
    t = {"resid": r(samples, rows, cols, dt=rt, s=2.0), "h": r(samples, rows, cols, dt=ht, s=std, add=0.5),
         "gate": None, "scale": None, "shift": None, "post_weight": None, "pre_weight": None}
    if vectors:
        t["shift"], t["scale"], t["gate"] = r(samples, 3 * cols, dt=pt, s=0.4).chunk(3, dim=1)
    if weights:
        t["post_weight"], t["pre_weight"] = r(cols, dt=pt, s=0.1, add=1.0), r(cols, dt=pt, s=0.1, add=1.0)
    return t


NAMES = ("resid", "h", "gate", "post_weight", "pre_weight", "scale", "shift")


def check(t, post, pre, alpha, seed=1):
    b = block()
    how = {"post": post, "pre": pre, "alpha": alpha}
    args = [t[n] for n in NAMES]
    out, y, stats = b.norm_fwd(*args, **how)
    ref = {n: None if t[n] is None else t[n].double().requires_grad_(True) for n in NAMES}
    r64, y64 = norm_block(*[ref[n] for n in NAMES], post, pre, alpha)
    close(out, r64, "resid_out:" + name_of(out))
    if y is not None:
        close(y, y64, "y:" + name_of(y))
    g = torch.Generator(device="cuda").manual_seed(seed)
    d_out = torch.randn(out.shape, generator=g, device="cuda").to(out.dtype)
    d_y = None if y is None else torch.randn(y.shape, generator=g, device="cuda").to(y.dtype)
    # the backward pass is defined from the stored (rounded) resid_out: the
    # definition there is the branch into it plus the norm out of it
    got = b.norm_bwd(d_out, d_y, out, t["h"], stats, *args[2:], **how)
    again = b.norm_bwd(d_out, d_y, out, t["h"], stats, *args[2:], **how)
    for n in NAMES:
        if got[n] is not None:
            assert torch.equal(got[n], again[n]), f"{n}: two runs differ"
    leaf = {n: None if t[n] is None else t[n].double().requires_grad_(True) for n in NAMES}
    x = out.detach().double().requires_grad_(True)
    total = d_out.double()
    if y is not None:
        _, yy = norm_block(x, None, None, None, leaf["pre_weight"], leaf["scale"], leaf["shift"], post, pre, alpha)
        yy.backward(d_y.double())
        total = total + x.grad
    zero = torch.zeros_like(x)
    rr, _ = norm_block(zero, leaf["h"], leaf["gate"], leaf["post_weight"], None, None, None, post, "none", alpha)
    if leaf["h"] is not None:
        rr.backward(total)
    # stats come from the unrounded resid_out, x from the stored one: with a
    # bf16 stream each x is off by up to 2^-8, which averages out in the
    # statistics to 2^-8 / sqrt(cols) of a deviation
    inner = 2.0 ** -8 * 4 / x.shape[-1] ** 0.5 if out.dtype == BF16 and y is not None else 0.0
    close(got["resid"], total, "d_resid:" + name_of(got["resid"]), inner=inner)
    for n in NAMES[1:]:
        if t[n] is not None:
            close(got[n], leaf[n].grad, f"d_{n}:" + name_of(got[n]), inner=inner)


@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("pre", ["rms", "layer"])
@pytest.mark.parametrize("rt,ht,pt", [(F32, BF16, F32), (F32, F32, BF16), (BF16, BF16, BF16), (BF16, F32, F32)])
def test_kinds_and_types(post, pre, rt, ht, pt):
    check(make(3, 21, 520, rt, ht, pt), post, pre, 0.5)


@pytest.mark.parametrize("cols", [1, 7, 8, 64, 257, 512, 520, 1001, 2048, 4104, 5120, 8192, 8200, 10001, 16384])
def test_widths(cols):
    check(make(2, 11, cols, F32, BF16, F32, seed=cols), "layer" if cols > 1 else "none", "rms", 1.0)


@pytest.mark.parametrize("samples,rows", [(1, 1), (1, 700), (700, 1), (5, 129), (2, 4099)])
def test_row_counts(samples, rows):
    check(make(samples, rows, 264, F32, F32, F32), "rms", "layer", 1.0)


@pytest.mark.parametrize("vectors,weights", [(False, False), (True, False), (False, True)])
def test_absent_parts(vectors, weights):
    check(make(2, 40, 768, F32, BF16, F32, vectors, weights), "rms", "layer", 0.25)


def test_no_branch_and_no_output_norm():
    b = block()
    t = make(2, 10, 96, F32, BF16, F32)
    t["h"] = t["gate"] = t["post_weight"] = None
    check(t, "none", "layer", 1.0)
    t = make(2, 10, 96, F32, BF16, F32)
    t["pre_weight"] = t["scale"] = t["shift"] = None
    check(t, "rms", "none", 0.5)
    x = torch.randn(4, 96, device="cuda")
    out, y, _ = b.norm_fwd(x, pre="rms")
    assert out is x and y.dtype == F32


def test_rows_of_zeros_and_large_offsets():
    """A constant row has no deviation (its LayerNorm is 0, not NaN), and a
    mean far above the deviation keeps its digits (the squares are centred)."""
    t = make(1, 6, 640, F32, F32, F32, vectors=False, weights=False)
    t["resid"][0, 0] = 0
    t["h"][0, 0] = 0
    t["h"][0, 1] = 7.0
    t["resid"][0, 2] += 1000.0
    out, y, _ = block().norm_fwd(*[t[n] for n in NAMES], post="layer", pre="layer")
    r64, y64 = norm_block(*[None if t[n] is None else t[n].double() for n in NAMES], "layer", "layer", 1.0)
    assert torch.isfinite(y).all()
    # resid + 1000 carries 2^-24 * 1000 = 6e-5 of the row's deviation 2
    close(y, y64, "y:f32", f32_tol=1e-4)


def test_strided_rows():
    """Rows inside a wider buffer, aligned (eight columns at once) and not."""
    for off in (8, 3):
        t = make(1, 33, 400, F32, BF16, F32)
        for n in ("resid", "h"):
            wide = torch.full((1, 33, 448), float("nan"), dtype=t[n].dtype, device="cuda")
            wide[..., off:off + 400] = t[n]
            t[n] = wide[..., off:off + 400]
        check(t, "rms", "layer", 1.0)


def test_empty():
    b = block()
    x = torch.empty(2, 0, 64, device="cuda")
    g = torch.ones(2, 64, device="cuda")
    out, y, st = b.norm_fwd(x, x, g)
    assert y.shape == (2, 0, 64) and st.shape == (0, 4)
    d = b.norm_bwd(x, x, out, x, st, g)
    assert torch.equal(d["gate"], torch.zeros_like(g))


def test_gradient_against_differences():
    """Central differences of the kernel's own forward pass along random
    directions.  fp32, step 1e-2: the cubic term is O(1e-4) of the value and
    the rounding 2^-24 * sqrt(n) / 1e-2."""
    b = block()
    t = make(2, 5, 72, F32, F32, F32, seed=3)
    how = {"post": "rms", "pre": "layer", "alpha": 0.5}
    args = {n: t[n].contiguous().clone() for n in NAMES}
    out, y, st = b.norm_fwd(*args.values(), **how)
    g = torch.Generator(device="cuda").manual_seed(9)
    co, cy = torch.randn(out.shape, generator=g, device="cuda"), torch.randn(y.shape, generator=g, device="cuda")
    d = b.norm_bwd(co, cy, out, args["h"], st, *list(args.values())[2:], **how)
    for n in NAMES:
        v = torch.randn(args[n].shape, generator=g, device="cuda")
        v /= v.norm()
        f = []
        for s in (1e-2, -1e-2):
            moved = dict(args, **{n: args[n] + s * v})
            o, yy, _ = b.norm_fwd(*moved.values(), **how)
            f.append(float((o.double() * co).sum() + (yy.double() * cy).sum()))
        slope = (f[0] - f[1]) / 2e-2
        want = float((d[n].double() * v).sum())
        assert abs(slope - want) <= 2e-3 * max(1.0, abs(want)), (n, slope, want)


def test_autograd_matches_and_reaches_every_input():
    b = block()
    t = {n: v.contiguous().requires_grad_(True) for n, v in make(2, 9, 256, F32, BF16, F32).items()}
    out, y = b.residual_norm(*[t[n] for n in NAMES], post="rms", pre="layer", alpha=0.5)
    (out.sum() + (y.float() ** 2).sum()).backward()
    o, yy, st = b.norm_fwd(*[t[n].detach() for n in NAMES], post="rms", pre="layer", alpha=0.5)
    d = b.norm_bwd(torch.ones_like(o), (2 * yy.float()).to(yy.dtype), o, t["h"].detach(), st,
                   *[t[n].detach() for n in NAMES[2:]], post="rms", pre="layer", alpha=0.5)
    for n in NAMES:
        assert torch.equal(t[n].grad, d[n]), n


def test_side_stream_and_graph_replays():
    b = block()
    t = make(2, 64, 512, F32, BF16, F32)
    args = [t[n] for n in NAMES]
    eager = b.norm_fwd(*args)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = b.norm_fwd(*args)
        gr = b.norm_bwd(eager[0], eager[1], eager[0], t["h"], other[2], *args[2:])
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(x, y) for x, y in zip(eager, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, y, st = b.norm_fwd(*args)
        d = b.norm_bwd(o, y, o, t["h"], st, *args[2:])
    for k in range(3):
        t["resid"].normal_()
        t["h"].normal_()
        graph.replay()
        torch.cuda.synchronize()
        eo, ey, est = b.norm_fwd(*args)
        ed = b.norm_bwd(eo, ey, eo, t["h"], est, *args[2:])
        assert torch.equal(o, eo) and torch.equal(y, ey)
        assert all(torch.equal(d[n], ed[n]) for n in NAMES), k
    assert gr["resid"].shape == o.shape


def test_offsets_past_32_bits():
    """A row more than 2^31 values into its tensor."""
    b = block()
    rows, cols = 280_000, 8192
    x = torch.zeros(rows, cols, dtype=BF16, device="cuda")
    x[-3:] = torch.randn(3, cols, generator=torch.Generator(device="cuda").manual_seed(0), device="cuda").to(BF16)
    out, y, _ = b.norm_fwd(x, pre="rms")
    want = b.norm_fwd(x[-3:].clone(), pre="rms")[1]
    assert torch.equal(y[-3:], want) and bool((y[:5] == 0).all())
