"""What the autograd functions of the block operators take, save and form, on the CPU
with stand-ins for the library's calls, and on the GPU where strides decide."""

import pytest
import torch

from test_block_autograd import stand_ins as block_stand_ins  # noqa: F401
from test_block_autograd import through_attention, through_ffn, through_packed_attention
from test_block_linear_boundary import b, leaves, stand_ins, through_linear  # noqa: F401

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


def test_rotary_reads_gradients_where_they_lie(stand_ins, monkeypatch):  # noqa: F811
    """Heads before positions, slices of a packed gradient and sums over samples as
    they are; a last dimension that is not contiguous is copied."""
    q, k, f = leaves((2, 3, 2, 8), (2, 3, 1, 8), (1, 4))
    f = f.detach()
    seen = []
    call = b.rotary_bwd
    monkeypatch.setattr(b, "rotary_bwd", lambda d_q, d_k, *a, **h: (seen.append((d_q.stride(), d_k.stride())), call(d_q, d_k, *a, **h))[1])
    gen = torch.Generator().manual_seed(1)
    w = torch.randn(2, 3, 2, 8, generator=gen, dtype=torch.float64)
    ways = {"heads first": (w.transpose(1, 2).contiguous().transpose(1, 2), (48, 8, 24, 1)),
            "packed": (torch.stack([w, w], 2)[:, :, 1], (96, 32, 8, 1)),
            "one sample's": (w[:1].expand_as(w), (0, 16, 8, 1)),
            "dim first": (w.transpose(2, 3).contiguous().transpose(2, 3), (48, 16, 8, 1)),
            "one value": (w[:1, :1, :1, :1].expand_as(w), (48, 16, 8, 1))}
    for name, (d, stride) in ways.items():
        seen.clear()
        q.grad = None
        torch.autograd.backward(b.rotary(q, k, f), (d, torch.ones_like(k)))
        assert seen[0][0] == stride, name
        assert torch.equal(q.grad, d * 3), name


@pytest.mark.gpu
def test_rotary_gradients_of_any_strides():
    gen = torch.Generator(device="cuda").manual_seed(2)
    q, k, w = (torch.randn(2, 9, h, 64, generator=gen, device="cuda").to(BF16) for h in (4, 2, 4))
    f = b.rotary_freqs(40)
    want = b.rotary_bwd(w, None, f)[0]
    for d in (w.transpose(1, 2).contiguous().transpose(1, 2), torch.stack([w, w], 2)[:, :, 1],
              torch.cat([w.new_zeros(1), w.flatten()])[1:].view(w.shape), w.transpose(2, 3).contiguous().transpose(2, 3)):
        leaf, other = q.clone().requires_grad_(True), k.clone().requires_grad_(True)
        turned = b.rotary(leaf, other, f)
        torch.autograd.backward(turned, (d, torch.ones_like(k)))
        assert torch.equal(leaf.grad, want) and torch.equal(other.grad, b.rotary_bwd(torch.ones_like(k), None, f)[0])
    leaf = q.clone().requires_grad_(True)
    b.rotary(leaf, None, f)[0].backward(w[:1].expand_as(w))
    assert torch.equal(leaf.grad, want[:1].expand_as(w))


def test_what_no_backward_pass_reads_may_be_written(stand_ins):  # noqa: F811
    """Weights and biases of an optimizer step between the passes, and random
    numbers that nothing was dropped by."""
    x, w, bias, res = leaves((3, 8), (16, 8), (16,), (3, 16))
    state = torch.tensor([1, 2])

    def write(*tensors):
        with torch.no_grad():
            for t in tensors:
                t.add_(1)
    y = b.linear(x.detach(), w, bias, res, act="gelu", rng=state)      # weight and bias: from x, z and d_y
    write(w, bias, res, state)
    y.sum().backward()
    assert torch.equal(w.grad, x.detach().sum(0).expand(16, 8)) and torch.equal(bias.grad, torch.full_like(bias, 3.0))
    y = b.linear(x, w.detach().clone(), bias, p=0.5, rng=(1, 2))       # x: from the weight
    write(x, bias)
    y.sum().backward()
    y = b.linear(x, w, bias.detach().clone(), res)
    write(bias, res)
    y.sum().backward()
    y = b.dropout(x, 0.0, state)
    write(state)
    y.sum().backward()
    y = b.dropout(x.detach(), 0.5, state, x) + b.linear(x.detach(), w.detach()[:8], None, x, p=0.5, rng=state)
    write(state)
    y.sum().backward()
    # what is read is still noticed
    for write_to, call in ((w, lambda: b.linear(x, w)), (x, lambda: b.linear(x, w)), (state, lambda: b.dropout(x, 0.5, state)),
                           (state, lambda: b.linear(x, w, p=0.5, rng=state))):
        y = call()
        write(write_to)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.sum().backward()


def off_the_boundary(y):
    """y beside one other value, whose gradient has y's begin one value further on."""
    return torch.cat([torch.ones(1, dtype=y.dtype, device=y.device, requires_grad=True), y.flatten()]).square().sum()


@pytest.mark.parametrize("call,through", [("linear_bwd", through_linear), ("attn_bwd", through_attention),
                                          ("attn_bwd", through_packed_attention), ("ffn_bwd", through_ffn)])
def test_gradients_come_on_their_boundary(stand_ins, block_stand_ins, monkeypatch, call, through):  # noqa: F811
    """A run out of a larger gradient is contiguous, and may begin at any value: the
    library takes rows on 16 bytes only."""
    got = []
    plain = getattr(b, call)
    monkeypatch.setattr(b, call, lambda d, *a, **how: (got.append(d), plain(d, *a, **how))[1])
    _, y = through()
    off_the_boundary(y).backward()
    assert got[0].is_contiguous() and got[0].data_ptr() % 16 == 0
    assert torch.equal(got[0], 2 * y)
    got.clear()
    _, y = through()
    mine = torch.randn(y.shape, dtype=y.dtype)
    assert mine.data_ptr() % 16 == 0
    y.backward(mine)
    assert got[0].data_ptr() == mine.data_ptr()                 # (and is not copied for nothing)


@pytest.mark.gpu
def test_gradients_off_their_boundary():
    gen = torch.Generator(device="cuda").manual_seed(3)

    def r(*shape):
        return (0.3 * torch.randn(shape, generator=gen, device="cuda")).to(BF16).requires_grad_(True)
    ways = {"linear": lambda: (b.linear, (r(20, 64), r(72, 64), r(72)), {"act": "gelu"}),
            "attention": lambda: (b.attention, (r(2, 9, 2, 64), r(2, 11, 2, 64), r(2, 11, 2, 64)), {}),
            "packed": lambda: (b.attention_qkv, (r(2, 9, 3, 2, 64),), {}),
            "ffn": lambda: (b.gated_ffn, (r(20, 64), r(72, 64), r(72, 64), r(64, 72)), {})}
    for name, way in ways.items():
        call, given, how = way()
        got = torch.autograd.grad(off_the_boundary(call(*given, **how)), given)
        want = torch.autograd.grad(call(*given, **how).square().sum(), given)
        assert all(torch.equal(p, q) for p, q in zip(got, want)), name
