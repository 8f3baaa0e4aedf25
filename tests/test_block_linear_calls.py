"""How linear, rotary and dropout may be called: at once on two streams, in a graph
for every form of the backward pass, in inference mode, under checkpointing, and
with the same tensor in several places."""

import pytest
import torch

from block_reference import close
from block_reference_linear import linear as linear64

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
RNG = (77, 5)


def block():
    from matrix_aware_optimizer_periodic_amd import block as b
    return b


def make(t, d, n, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    return r(t, d).to(BF16), (r(n, d) * d ** -0.5).to(BF16), r(n), r(t, n), r(t, n)


# small calls, few rows with a large weight, tiles, a divided weight's gradient
FORMS = [(40, 64, 96), (6, 5120, 20480), (300, 512, 1024), (9000, 256, 32)]


@pytest.mark.parametrize("t,d,n", FORMS)
def test_replays(t, d, n):
    b = block()
    x, w, bias, res, dy = make(t, d, n)
    state = torch.tensor([7, 0], device="cuda")

    def both(rng):
        y, z = b.linear_fwd(x, w, bias, res, act="gelu", p=0.2, rng=rng)
        return (y, z, *b.linear_bwd(dy, x, w, bias, z, act="gelu", p=0.2, rng=rng))
    both(state)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both(state)
    for i in range(3):
        x.normal_()
        dy.normal_()
        state[1] = i
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, both((7, i)))), i


@pytest.mark.parametrize("t,d,n", FORMS)
def test_two_streams_at_once(t, d, n):
    b = block()
    data = [make(t, d, n, s) for s in range(2)]

    def both(x, w, bias, res, dy):
        y, z = b.linear_fwd(x, w, bias, res, act="silu", p=0.1, rng=RNG)
        return (y, *b.linear_bwd(dy, x, w, bias, z, act="silu", p=0.1, rng=RNG))
    want = [both(*v) for v in data]
    streams = [torch.cuda.Stream() for _ in data]
    got = [[], []]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(both(*data[i]))
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    for runs, ref in zip(got, want):
        assert all(torch.equal(p, q) for run in runs for p, q in zip(run, ref))


def test_inference_mode():
    b = block()
    x, w, bias, res, _ = make(50, 64, 128)
    f = b.rotary_freqs(32)
    want = b.linear(x, w, bias, res, act="gelu", p=0.1, rng=RNG)
    q = want.view(1, 50, 4, 32)
    turned, _ = b.rotary(q, None, f)
    dropped = b.dropout(want, 0.3, RNG)
    qkv = torch.randn(2, 9, 3, 2, 32, device="cuda").to(BF16)
    o = b.attention_qkv(qkv, rotary={"freqs": f})
    with torch.inference_mode():
        y = b.linear(x, w, bias, res, act="gelu", p=0.1, rng=RNG)
        assert torch.equal(y, want) and torch.equal(b.dropout(y, 0.3, RNG), dropped)
        assert torch.equal(b.rotary(y.view(1, 50, 4, 32), None, f)[0], turned)
        z = y.clone().view(1, 50, 4, 32)
        b.rotary_fwd(z, None, f, out=(z, None))
        assert torch.equal(z, turned) and torch.equal(b.attention_qkv(qkv, rotary={"freqs": f}), o)


@pytest.mark.parametrize("state", [False, True])
def test_checkpointing_forms_the_same_mask(state):
    from torch.utils.checkpoint import checkpoint
    b = block()
    x, w, bias, res, dy = make(200, 64, 128)
    rng = torch.tensor(RNG, device="cuda") if state else RNG

    def f(x, w, bias, res):
        return b.dropout(b.linear(x, w, bias, res, act="silu", p=0.2, rng=rng), 0.4, rng)
    grads = []
    for run in (f, lambda *a: checkpoint(f, *a, use_reentrant=False)):
        leaves = [t.clone().requires_grad_(True) for t in (x, w, bias, res)]
        run(*leaves).backward(dy)
        grads.append([t.grad for t in leaves])
    assert all(torch.equal(p, q) for p, q in zip(*grads))


def test_the_same_tensor_in_several_places():
    """x as weight and as residual, q as k, x as dy: read only, so each counts."""
    b = block()
    x = torch.randn(128, 128, device="cuda").to(BF16)
    y, z = b.linear_fwd(x, x, None, x, act="gelu")
    y64, _ = linear64(x.double(), x.double(), None, x.double(), "gelu", 0.0, None)
    close(y, y64, "y:bf16")
    leaf = x.clone().requires_grad_(True)
    b.linear(leaf, leaf, None, leaf).backward(x)
    d = b.linear_bwd(x, x, x)
    want = d[0].double() + d[1].double() + x.double()
    # (autograd adds the three in bf16: two roundings of 2^-8 of what is added)
    assert float((leaf.grad.double() - want).abs().max()) <= 2 ** -7 * float(want.abs().max())
    q = torch.randn(2, 7, 3, 64, device="cuda").to(BF16)
    f = b.rotary_freqs(64)
    one, two = b.rotary_fwd(q, q, f)
    assert one.data_ptr() != two.data_ptr() and torch.equal(one, two)
    assert torch.equal(b.dropout_fwd(x, 0.5, RNG, x), b.dropout_fwd(x.clone(), 0.5, RNG, x))
