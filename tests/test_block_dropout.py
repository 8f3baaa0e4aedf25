"""Dropout from a counter-based generator: the generator's published answers,
masks by an element's number, types, strides, gradients, graphs, streams."""

import numpy as np
import pytest
import torch

from block_reference import close, name_of
from block_reference_linear import drop, kept, philox_words

BF16, F32 = torch.bfloat16, torch.float32
RNG = (0xA0761D6478BD642F, 0xE7037ED1A0B428DB)


def block():
    from matrix_aware_optimizer_periodic_amd import block as b
    return b


def test_generator_gives_the_published_answers():
    """The generator's known-answer vectors (counter, key, words)."""
    for index, offset, seed, want in (
            (0, 0, 0, "6627e8d5 e169c58d bc57ac4c 9b00dbd8"),
            (2 ** 64 - 1, 2 ** 64 - 1, 2 ** 64 - 1, "408f276d 41c83b0e a20bc7c6 6d5451fd"),
            (0x85a308d3243f6a88, 0x0370734413198a2e, 0x299f31d0a4093822, "d16cfe09 94fdcceb 5001e420 24126ea1")):
        got = philox_words(np.array([index], dtype=np.uint64), seed, offset)[0]
        assert " ".join(f"{int(w):08x}" for w in got) == want


@pytest.mark.gpu
@pytest.mark.parametrize("resid", [None, F32, BF16])
@pytest.mark.parametrize("act", [F32, BF16])
@pytest.mark.parametrize("shape", [(1, 1), (1, 7), (3, 8), (7, 1001), (129, 264), (2, 5, 24), (1000,), (4099,), (65, 1)])
def test_values(shape, act, resid):
    b = block()
    gen = torch.Generator(device="cuda").manual_seed(sum(shape))
    x = torch.randn(shape, generator=gen, device="cuda").to(act)
    r = None if resid is None else torch.randn(shape, generator=gen, device="cuda").to(resid)
    for p in (0.0, 0.1, 0.5, 0.93, 1.0):
        y = b.dropout_fwd(x, p, RNG, r)
        want = drop(x.double(), p, RNG)
        want = want if r is None else r.double() + want
        assert y.dtype == (resid or act) and y.shape == x.shape
        close(y, want, "y:" + name_of(y))
        if 0.0 < p < 1.0 and r is None:
            assert torch.equal(y != 0, kept(shape, p, RNG) & (x != 0))
        d = b.dropout_bwd(x, p, RNG, dtype=resid)
        close(d, drop(x.double(), p, RNG), "d:" + name_of(d))


@pytest.mark.gpu
@pytest.mark.parametrize("cols", [8, 24, 1001, 1024])
@pytest.mark.parametrize("pad", [1, 3, 8, 40])
def test_strides_do_not_move_the_mask(cols, pad):
    b = block()
    base = torch.randn(37, cols + pad, device="cuda")
    x, r = base[:, :cols], torch.randn(37, cols + 2 * pad, device="cuda")[:, pad:pad + cols]
    y = b.dropout_fwd(x.contiguous(), 0.3, RNG, r.contiguous())
    assert torch.equal(b.dropout_fwd(x, 0.3, RNG, r), y)
    assert torch.equal(b.dropout_fwd(x, 0.3, RNG, r.contiguous()), y)
    one = torch.randn(37 * cols + 1, device="cuda").to(BF16)
    assert torch.equal(b.dropout_fwd(one[1:], 0.3, RNG), b.dropout_fwd(one[1:].clone(), 0.3, RNG))


@pytest.mark.gpu
def test_dropped_elements_may_hold_anything():
    b = block()
    x = torch.randn(50, 64, device="cuda")
    keep = kept((50, 64), 0.5, RNG)
    y = b.dropout_fwd(x, 0.5, RNG)
    bad = torch.where(keep, x, float("nan"))
    assert torch.equal(b.dropout_fwd(bad, 0.5, RNG), y)
    x[3] = float("inf")
    assert torch.equal(torch.isinf(b.dropout_fwd(x, 0.5, RNG)[3]), keep[3])


@pytest.mark.gpu
def test_share_that_is_dropped():
    """2^22 elements: the share's deviation is sqrt(p (1 - p)) 2^-11; five of them."""
    b = block()
    x = torch.ones(1 << 22, device="cuda")
    for p in (0.1, 0.5, 0.9):
        for offset in (0, 1, 2):
            share = float((b.dropout_fwd(x, p, (1, offset)) == 0).double().mean())
            assert abs(share - p) < 5 * (p * (1 - p)) ** 0.5 * 2 ** -11
    a, c = (b.dropout_fwd(x, 0.5, (1, o)) == 0 for o in (0, 1))
    assert abs(float((a & c).double().mean()) - 0.25) < 5 * (3 / 16) ** 0.5 * 2 ** -11


@pytest.mark.gpu
def test_numbers_past_32_bits():
    b = block()
    n = (1 << 32) + 4096
    x = torch.ones(n, dtype=BF16, device="cuda")
    y = b.dropout_fwd(x, 0.5, RNG)
    for first in (0, (1 << 32) - 512, 1 << 32, n - 1024):
        assert torch.equal(y[first:first + 1024] != 0, kept((1024,), 0.5, RNG, first=first))


@pytest.mark.gpu
def test_autograd_and_empty():
    b = block()
    x = torch.randn(20, 40, device="cuda").to(BF16).requires_grad_(True)
    r = torch.randn(20, 40, device="cuda").requires_grad_(True)
    w = torch.randn(20, 40, device="cuda")
    b.dropout(x, 0.3, RNG, r).backward(w)
    assert x.grad.dtype == BF16 and torch.equal(x.grad, b.dropout_bwd(w, 0.3, RNG, dtype=BF16)) and torch.equal(r.grad, w)
    x2 = torch.randn(20, 40, device="cuda").requires_grad_(True)
    b.dropout(x2, 0.3, RNG).sum().backward()
    assert torch.equal(x2.grad != 0, kept((20, 40), 0.3, RNG))
    assert b.dropout_fwd(x[:0], 0.3, RNG).shape == (0, 40) and b.dropout_fwd(x[:, :0], 0.3, RNG).shape == (20, 0)


@pytest.mark.gpu
def test_graph_replays_and_streams():
    b = block()
    x = torch.randn(300, 520, device="cuda").to(BF16)
    state = torch.tensor([3, 0], device="cuda")
    b.dropout_fwd(x, 0.4, state)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = b.dropout_fwd(x, 0.4, state)
        state[1:].add_(1)
    for i in range(3):
        x.normal_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, b.dropout_fwd(x, 0.4, (3, i))) and int(state[1]) == i + 1
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        z = b.dropout_fwd(x, 0.4, (3, 2))
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, z)
