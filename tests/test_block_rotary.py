"""Rotary positions against the definition in float64: layouts, parts of a head,
several axes, far positions, types, strides, in place, gradients, and attention
over rotated queries and keys."""

import math

import pytest
import torch

from block_reference import close, name_of
from block_reference import attention as attention64
from block_reference_linear import rotary as rotary64

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def block():
    from matrix_aware_optimizer_periodic_amd import block as b
    return b


def heads(b, n, h, d, dtype=BF16, seed=0):
    return torch.randn(b, n, h, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)).to(dtype)


def own_freqs(axes, pairs):
    f = torch.zeros((axes, pairs), dtype=F64)
    for p in range(pairs):
        f[p % axes, p] = 0.9 ** p
    return f.cuda()


def check(q, k, freqs, positions=None, offset=0, interleaved=False, scale=1.0):
    """Forward and gradient, fp32 sines: 2^-24 of an angle of at most half a turn
    in turns and a few 2^-24 of their own, within 1e-6 of a pair's size, which is
    below 1e-5 of the largest value."""
    b = block()
    n = q.shape[1]
    where = torch.arange(n, device="cuda")[:, None] + offset if positions is None else positions.long()
    if positions is not None and freqs.shape[0] == 1:
        where = where[..., None]
    where = where if where.dim() == 3 else where[None]
    how = dict(offset=offset, interleaved=interleaved, scale=scale)
    for call, inverse in ((b.rotary_fwd, False), (b.rotary_bwd, True)):
        got = call(q, k, freqs, positions, **how)
        for name, x, y in zip(("q", "k"), (q, k), got):
            assert (x is None) == (y is None)
            if x is None:
                continue
            assert y.dtype == x.dtype and y.shape == x.shape and y.is_contiguous()
            close(y, rotary64(x.double(), freqs, where, interleaved, scale, inverse), f"{name}:{name_of(x)}")
            rot = 2 * freqs.shape[1]
            assert torch.equal(y[..., rot:], x[..., rot:])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot", [(2, 2), (8, 8), (16, 16), (64, 64), (72, 72), (72, 36), (80, 32), (128, 128), (128, 64),
                                     (128, 2), (96, 94), (6, 4), (40, 40), (24, 8), (256, 256), (1024, 1024), (1024, 512)])
def test_heads_and_parts(dim, rot, interleaved, dtype):
    check(heads(2, 5, 3, dim, dtype), heads(2, 5, 1, dim, dtype, 1), own_freqs(1, rot // 2), interleaved=interleaved,
          scale=1.25, offset=3)


@pytest.mark.gpu
@pytest.mark.parametrize("batch,n,h,g", [(1, 1, 1, 1), (4, 1, 32, 8), (1, 7, 1, 3), (3, 1000, 5, 5), (2, 333, 40, 8),
                                         (1, 4099, 2, 2), (70, 3, 16, 0), (1, 2, 300, 200)])
def test_lengths_and_head_counts(batch, n, h, g):
    k = heads(batch, n, g, 64, seed=1) if g else None
    check(heads(batch, n, h, 64), k, own_freqs(1, 32), interleaved=bool(n % 2))


@pytest.mark.gpu
@pytest.mark.parametrize("axes", [1, 2, 3, 8])
@pytest.mark.parametrize("per_sample", [False, True])
def test_positions(axes, per_sample):
    b, n = 3, 50
    gen = torch.Generator(device="cuda").manual_seed(axes)
    shape = (*((b,) if per_sample else ()), n, *((axes,) if axes > 1 else ()))
    pos = torch.randint(-1000, 1000, shape, generator=gen, device="cuda", dtype=torch.int32)
    check(heads(b, n, 4, 64), heads(b, n, 4, 64, seed=1), own_freqs(axes, 24), pos)


@pytest.mark.gpu
@pytest.mark.parametrize("first", [1_000_000, 2 ** 31 - 9, -5, 2 ** 40])
def test_far_positions_keep_their_digits(first):
    """Next to 64 bits: 2^40 positions of up to one radian each leave 2^-13 of a
    turn to fp64's 2^-53, so 2^-10 of a value there, and 2^-20 at 2^31."""
    q = heads(2, 9, 2, 64, F32)
    f = own_freqs(1, 32)
    got, _ = block().rotary_fwd(q, None, f, offset=first)
    where = torch.arange(9, device="cuda")[None, :, None].double() + first
    bound = 1e-5 + abs(first) * 2.0 ** -52
    off = (got.double() - rotary64(q.double(), f, where)).abs().max()
    assert float(off) <= bound * float(q.abs().max()) * 2
    if abs(first) < 2 ** 31 - 9:
        pos = torch.arange(first, first + 9, device="cuda", dtype=torch.int32)
        assert torch.equal(block().rotary_fwd(q, None, f, pos)[0], got)


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_strides_and_in_place(interleaved):
    b = block()
    f = own_freqs(1, 20)
    how = dict(interleaved=interleaved, scale=0.5)
    qkv = torch.randn(3, 11, 3, 4, 64, device="cuda").to(BF16)
    q, k, v = qkv.unbind(2)
    want = b.rotary_fwd(q.contiguous(), k.contiguous(), f, **how)
    got = b.rotary_fwd(q, k, f, **how)
    assert all(torch.equal(p, w) for p, w in zip(got, want))
    # batch and heads the other way round, heads shared by samples, off every boundary but the type's
    swapped = q.permute(1, 0, 2, 3).contiguous().permute(1, 0, 2, 3)
    assert torch.equal(b.rotary_fwd(swapped, None, f, **how)[0], want[0])
    flat = torch.empty(q.numel() + 1, dtype=BF16, device="cuda")[1:].view(q.shape)
    flat.copy_(q)
    assert torch.equal(b.rotary_fwd(flat, None, f, **how)[0], want[0])
    heads_first = q.transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(b.rotary_fwd(heads_first, k, f, **how)[0], want[0])
    one = q[:1].expand(3, -1, -1, -1)
    assert torch.equal(b.rotary_fwd(one, None, f, **how)[0], b.rotary_fwd(one.contiguous(), None, f, **how)[0])
    # in place, and into slices of another buffer
    before = qkv.clone()
    out = b.rotary_fwd(q, k, f, out=(q, k), **how)
    assert out[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, before[:, :, 2])
    b.rotary_fwd(before[:, :, 0], before[:, :, 1], f, out=(qkv[:, :, 1], qkv[:, :, 0]), **how)
    assert torch.equal(qkv[:, :, 1], want[0]) and torch.equal(qkv[:, :, 0], want[1])
    odd = torch.zeros(3, 11, 4, 65, dtype=BF16, device="cuda")
    b.rotary_fwd(before[:, :, 0], None, f, out=(odd[..., :64], None), **how)
    assert torch.equal(odd[..., :64], want[0]) and bool((odd[..., 64] == 0).all())


@pytest.mark.gpu
def test_empty_and_not_finite():
    b = block()
    f = own_freqs(1, 4)
    q = heads(2, 5, 2, 16)
    assert b.rotary_fwd(q[:0], None, f)[0].shape == (0, 5, 2, 16) and b.rotary_fwd(q[:, :0], q[:, :0], f)[1].shape == (2, 0, 2, 16)
    q[1, 2, 1, 0] = float("nan")              # its pair, and nothing else
    y = b.rotary_fwd(q, None, f)[0]
    bad = torch.isnan(y).nonzero().tolist()
    assert bad == [[1, 2, 1, 0], [1, 2, 1, 4]]


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient_against_differences(interleaved):
    """y is linear in q: a difference of any size is the gradient's, to fp32's
    rounding of sums of 640 terms."""
    b = block()
    f = own_freqs(2, 12)
    q, k, w = (heads(2, 5, 2, 32, F32, s) for s in range(3))
    pos = torch.randint(0, 99, (5, 2), device="cuda", dtype=torch.int32)
    d, _ = b.rotary_bwd(w, None, f, pos, interleaved=interleaved, scale=1.5)
    moved = b.rotary_fwd(q + k, None, f, pos, interleaved=interleaved, scale=1.5)[0].double() \
        - b.rotary_fwd(q - k, None, f, pos, interleaved=interleaved, scale=1.5)[0].double()
    got, want = float((moved * w.double()).sum()), float((2 * k.double() * d.double()).sum())
    assert abs(got - want) <= 1e-5 * float((moved * w.double()).abs().sum())


@pytest.mark.gpu
def test_autograd():
    b = block()
    f = own_freqs(1, 32)
    q, k = (heads(2, 9, h, 64, seed=h).requires_grad_(True) for h in (4, 2))
    wq, wk = heads(2, 9, 4, 64, seed=7), heads(2, 9, 2, 64, seed=8)
    torch.autograd.backward(b.rotary(q, k, f, offset=4), (wq, wk))
    want = b.rotary_bwd(wq, wk, f, offset=4)
    assert torch.equal(q.grad, want[0]) and torch.equal(k.grad, want[1])
    q.grad = k.grad = None
    b.rotary(q, k, f)[1].backward(wk)
    assert q.grad is None and torch.equal(k.grad, b.rotary_bwd(wk, None, f)[0])
    q.grad = None
    b.rotary(q, None, f)[0].sum().backward()
    assert torch.equal(q.grad, b.rotary_bwd(torch.ones_like(q), None, f)[0])


@pytest.mark.gpu
def test_graph_replays_and_streams():
    b = block()
    f = own_freqs(1, 64)
    q, k = heads(4, 1, 32, 128), heads(4, 1, 8, 128, seed=1)
    pos = torch.tensor([[5], [0], [77], [3]], dtype=torch.int32, device="cuda")
    b.rotary_fwd(q, k, f, pos)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = b.rotary_fwd(q, k, f, pos)
        pos.add_(1)
    for _ in range(3):
        q.normal_()
        want = b.rotary_fwd(q, k, f, pos)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, w) for p, w in zip(out, want))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = b.rotary_fwd(q, k, f, pos)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(p, w) for p, w in zip(again, b.rotary_fwd(q, k, f, pos)))


@pytest.mark.gpu
def test_offsets_past_32_bits():
    b = block()
    f = own_freqs(1, 32)
    base = torch.empty(3 << 30, dtype=BF16, device="cuda")
    far = torch.as_strided(base, (3, 4, 2, 64), (1 << 30, 1 << 28, 64, 1))
    q = heads(3, 4, 2, 64)
    far.copy_(q)
    want = b.rotary_fwd(q, None, f)[0]
    assert torch.equal(b.rotary_fwd(far, None, f)[0], want)
    b.rotary_fwd(far, None, f, out=(far, None))
    assert torch.equal(far, want)


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,h", [(20_000_000, 1), (1_100_000, 512)])
def test_many_tokens(tokens, h):
    """Many tokens to a workgroup, and more workgroups than go out at once."""
    b = block()
    q = torch.ones(1, tokens, h, 2, dtype=BF16, device="cuda")
    f = torch.tensor([[0.001]], dtype=F64, device="cuda")
    y = b.rotary_fwd(q, None, f)[0].view(-1, h, 2)
    i = torch.arange(0, tokens, 9973, device="cuda")
    t = i.double()[:, None].expand(-1, h) * 0.001
    close(y[i], torch.stack([torch.cos(t) - torch.sin(t), torch.cos(t) + torch.sin(t)], 2), "y:bf16")
    assert torch.equal(y[-1], y[-1, :1].expand(h, 2))


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [False, True])
def test_attention_over_rotated(causal):
    """attention_qkv(rotary=...) is rotary and then attention, with the packed
    gradient."""
    b = block()
    qkv = torch.randn(2, 60, 3, 4, 64, device="cuda", generator=torch.Generator(device="cuda").manual_seed(0)).to(BF16)
    pos = torch.stack(torch.meshgrid(torch.arange(6), torch.arange(10), indexing="ij"), -1).view(60, 2).int().cuda()
    f = b.rotary_freqs((32, 32))
    lens = torch.tensor([60, 33], dtype=torch.int32, device="cuda")
    w = heads(2, 60, 4, 64, seed=5)
    packed = qkv.clone().requires_grad_(True)
    o = b.attention_qkv(packed, causal=causal, k_lens=lens, q_lens=lens,
                        rotary={"freqs": f, "positions": pos, "interleaved": True})
    o.backward(w)
    parts = [t.contiguous().requires_grad_(True) for t in qkv.unbind(2)]
    q, k = b.rotary(parts[0], parts[1], f, pos, interleaved=True)
    o2 = b.attention(q, k, parts[2], causal=causal, k_lens=lens, q_lens=lens)
    o2.backward(w)
    assert torch.equal(o, o2)
    for i, t in enumerate(parts):
        # (d_q and d_k are rotated in place there, from the same bf16 values)
        assert torch.equal(packed.grad[:, :, i], t.grad)
    q64, k64 = (rotary64(t.detach().double(), f, pos[None], True) for t in parts[:2])
    want, _ = attention64(q64, k64, parts[2].detach().double(), causal, 0, lens, lens)
    # q and k rounded to bf16 after the rotation: scores off by 2 x 2^-8 of
    # |q||k| / sqrt(64), sqrt(64) x 2^-8 at random of about one: 3%; probabilities
    # then too, and their products' sums
    assert float((o.detach().double() - want).norm() / want.norm()) < 0.03


def test_frequencies():
    b = block()
    f = b.rotary_freqs(8, device="cpu")
    assert f.shape == (1, 4) and f.dtype == F64
    assert torch.allclose(f[0], torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=F64))
    g = b.rotary_freqs((8, 4), base=100.0, device="cpu")
    assert g.shape == (2, 6) and bool((g[0, 4:] == 0).all()) and bool((g[1, :4] == 0).all())
    assert math.isclose(g[0, 3], 100 ** -0.75) and math.isclose(g[1, 5], 100 ** -0.5)
    assert torch.equal(b.rotary_freqs(8, stretch="linear", factor=4.0, device="cpu"), f / 4)
    n = b.rotary_freqs(8, stretch="ntk", factor=4.0, device="cpu")
    assert n[0, 0] == 1.0 and math.isclose(n[0, 3], f[0, 3] / 4)
    y = b.rotary_freqs(128, stretch="yarn", factor=8.0, length=4096, device="cpu")
    plain = b.rotary_freqs(128, device="cpu")
    turns = 4096 * plain / (2 * math.pi)
    assert torch.equal(y[turns >= 32], plain[turns >= 32]) and torch.allclose(y[turns <= 1], plain[turns <= 1] / 8)
    between = (turns > 1) & (turns < 32)
    assert bool(((y < plain) & (y > plain / 8))[between].all()) and bool(between.any())
    for bad in (dict(dim=7), dict(dim=()), dict(dim=8, stretch="other"), dict(dim=8, factor=0.0), dict(dim=8, stretch="yarn")):
        with pytest.raises(ValueError):
            b.rotary_freqs(**bad, device="cpu")
