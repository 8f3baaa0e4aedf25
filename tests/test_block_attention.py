"""Attention against its definition in float64: forward and gradients, head
sizes and groups, lengths around the tile edges, causal borders that leave
rows empty, per-sample lengths with anything in the padding, packed and
transposed layouts, few queries over long caches."""

import pytest
import torch

from block_reference import attention, close

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16

# Probabilities and their gradients are rounded to bf16 before the second
# product: each term is off by at most 2^-8 of itself (half a step), so a sum
# of n terms of random sign by about 2^-8 / sqrt(3) of its typical size; at an
# element that is 2^-8 of the output's largest value at most.
ROUND = 2.0 ** -8


def block():
    from matrix_aware_optimizer_periodic_amd import block as b
    return b


def make(b, m, n, h, g, d, seed=0, std=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def r(*shape):
        return (torch.randn(shape, generator=gen, device="cuda") * std).to(BF16)
    return r(b, m, h, d), r(b, n, g, d), r(b, n, g, d), r(b, m, h, d)


def lens(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def check(q, k, v, d_o, grads=True, **how):
    b = block()
    o, lse = b.attn_fwd(q, k, v, **how)
    qn, kn = how.get("q_lens"), how.get("k_lens")

    def there(t, n):
        """float64 leaf with zeros past the lengths (which may hold NaN)."""
        t = t.double()
        if n is not None:
            t = torch.where((torch.arange(t.shape[1], device="cuda") < n[:, None])[:, :, None, None], t, 0.0)
        return t.detach().requires_grad_(True)
    q64, k64, v64 = there(q, qn), there(k, kn), there(v, kn)
    o64, lse64 = attention(q64, k64, v64, **how)
    close(o, o64, "o:bf16", inner=ROUND)
    close(lse, lse64, "lse:f32")
    o2, lse2 = b.attn_fwd(q, k, v, **how)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    if not grads:
        return
    o64.backward(there(d_o, qn).detach())
    got = b.attn_bwd(d_o, q, k, v, o, lse, **how)
    again = b.attn_bwd(d_o, q, k, v, o, lse, **how)
    for x, y, ref, name in zip(got, again, (q64, k64, v64), ("d_q", "d_k", "d_v")):
        assert torch.equal(x, y), f"{name}: two runs differ"
        # delta is formed from the rounded o: off by 2^-8 |do . o|, at most the
        # size of the dp it is taken from
        close(x, ref.grad, f"{name}:bf16", inner=2 * ROUND)


@pytest.mark.parametrize("d", [8, 16, 32, 40, 64, 72, 96, 104, 128])
def test_head_sizes(d):
    check(*make(2, 150, 170, 4, 2, d, seed=d))


@pytest.mark.parametrize("h,g", [(1, 1), (3, 3), (4, 1), (6, 2), (5, 1)])
@pytest.mark.parametrize("causal", [False, True])
def test_groups(h, g, causal):
    check(*make(2, 90, 90, h, g, 64), causal=causal)


@pytest.mark.parametrize("m,n", [(1, 1), (1, 64), (31, 33), (63, 65), (64, 64), (65, 63), (127, 129), (128, 128),
                                 (129, 127), (200, 1), (1, 300), (257, 513)])
@pytest.mark.parametrize("causal", [False, True])
def test_lengths(m, n, causal):
    check(*make(1, m, n, 2, 2, 128, seed=m + n), causal=causal, offset=n - m)


@pytest.mark.parametrize("offset", [-300, -100, -33, -1, 0, 5, 64, 1000])
def test_causal_borders(offset):
    """A negative offset leaves the first rows without a key, a very negative
    one all of them, and keys that no query sees get zero gradients."""
    check(*make(1, 140, 130, 2, 1, 64), causal=True, offset=offset)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_ragged_with_padding_of_anything(d, causal):
    q, k, v, g = make(5, 130, 200, 4, 2, d)
    qn, kn = lens([130, 64, 0, 1, 100]), lens([0, 200, 50, 65, 128])
    for i in range(5):
        q[i, int(qn[i]):] = float("nan")
        g[i, int(qn[i]):] = float("inf")
        k[i, int(kn[i]):] = float("inf")
        v[i, int(kn[i]):] = float("nan")
    check(q, k, v, g, q_lens=qn, k_lens=kn, causal=causal, offset=70)


def test_lengths_outside_are_clamped():
    q, k, v, g = make(2, 40, 50, 2, 2, 32)
    check(q, k, v, g, q_lens=lens([99, -3]), k_lens=lens([1000, 20]))


def test_no_keys_and_no_queries():
    b = block()
    q, k, v, g = make(2, 5, 0, 2, 2, 64)
    o, lse = b.attn_fwd(q, k, v)
    assert torch.equal(o, torch.zeros_like(o)) and bool((lse == float("-inf")).all())
    d_q, d_k, _ = b.attn_bwd(g, q, k, v, o, lse)
    assert torch.equal(d_q, torch.zeros_like(d_q)) and d_k.shape == k.shape
    q, k, v, g = make(2, 0, 70, 2, 1, 64)
    o, lse = b.attn_fwd(q, k, v)
    d_q, d_k, d_v = b.attn_bwd(g, q, k, v, o, lse)
    assert torch.equal(d_k, torch.zeros_like(d_k)) and torch.equal(d_v, torch.zeros_like(d_v))


def test_layouts():
    """Slices of one packed projection, heads before length, and keys shared
    by the batch (stride 0)."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    qkv = torch.randn(2, 100, 3, 4, 72, generator=gen, device="cuda").to(BF16)
    q, k, v = qkv.unbind(2)
    g = torch.randn(2, 4, 100, 72, generator=gen, device="cuda").to(BF16).transpose(1, 2)
    check(q, k, v, g)
    q, k, v, g = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in make(2, 70, 90, 4, 2, 64))
    check(q, k, v, g)
    b = block()
    q, k, v, g = make(3, 70, 90, 4, 2, 64)
    k1, v1 = k[:1].expand(3, -1, -1, -1), v[:1].expand(3, -1, -1, -1)
    o, lse = b.attn_fwd(q, k1, v1)
    o2, lse2 = b.attn_fwd(q, k1.contiguous(), v1.contiguous())
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    for x, y in zip(b.attn_bwd(g, q, k1, v1, o, lse), b.attn_bwd(g, q, k1.contiguous(), v1.contiguous(), o, lse)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("b,m,n,h,g,d", [(1, 1, 5000, 8, 2, 128), (3, 2, 1999, 4, 4, 64), (1, 33, 4100, 2, 1, 72),
                                         (2, 1, 255, 3, 1, 128), (1, 1, 8191, 1, 1, 128)])
def test_few_queries_over_long_keys(b, m, n, h, g, d):
    check(*make(b, m, n, h, g, d), causal=True, offset=n - m)
    q, k, v, _ = make(b, m, n, h, g, d, seed=2)
    kn = lens([n // 3 + 1] + [0] * (b - 1))
    check(q, k, v, None, grads=False, k_lens=kn)


def test_large_scores():
    """Scores of hundreds: the running maximum keeps the exponents in range;
    one key takes nearly all of the weight."""
    q, k, v, g = make(1, 100, 300, 2, 2, 128, std=8.0)
    check(q, k, v, g, grads=False)


def test_rising_scores():
    """Keys whose scores rise steadily, so that every tile raises the maximum."""
    b, n, d = 1, 640, 64
    q = torch.ones(b, 50, 1, d, device="cuda").to(BF16)
    k = (torch.arange(n, device="cuda")[None, :, None, None] * 0.05).expand(b, n, 1, d).to(BF16).contiguous()
    v = torch.randn(b, n, 1, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(4)).to(BF16)
    check(q, k, v, None, grads=False)


def test_long():
    check(*make(1, 2100, 2300, 2, 1, 128), causal=True, offset=200)


def test_gradient_against_differences():
    """Differences of the kernel's forward pass along the gradient itself.  o
    is rounded to bf16, so each of the 2 sums over n values is off by about
    2^-8 sqrt(n) |o| / sqrt(3) at random: the step is taken large (the change
    of f is then 30 times that) and the slope held to 10%."""
    b = block()
    q, k, v, _ = make(1, 64, 64, 2, 2, 64, seed=5)
    gen = torch.Generator(device="cuda").manual_seed(6)
    w = torch.randn(q.shape, generator=gen, device="cuda").to(BF16)
    o, lse = b.attn_fwd(q, k, v)
    for i, d in enumerate(b.attn_bwd(w, q, k, v, o, lse)):
        u = d.float() / d.float().norm()
        f, h = [], 4.0
        moved = []
        for s in (h, -h):
            args = [q, k, v]
            args[i] = (args[i].float() + s * u).to(BF16)
            moved.append(args[i].double())
            f.append(float((b.attn_fwd(*args)[0].double() * w.double()).sum()))
        want = float(((moved[0] - moved[1]) * d.double()).sum())
        assert abs(f[0] - f[1] - want) <= 0.1 * abs(want), (i, f, want)


def test_autograd():
    b = block()
    q, k, v, g = (t.requires_grad_(True) for t in make(2, 50, 60, 4, 2, 64))
    b.attention(q, k, v, causal=True, offset=10).backward(g.detach())
    o, lse = b.attn_fwd(q.detach(), k.detach(), v.detach(), causal=True, offset=10)
    for x, t in zip(b.attn_bwd(g.detach(), q.detach(), k.detach(), v.detach(), o, lse, causal=True, offset=10), (q, k, v)):
        assert torch.equal(t.grad, x)


def test_graph_replays():
    b = block()
    q, k, v, g = make(1, 3, 1500, 4, 2, 128)
    kn = lens([1200])
    b.attn_fwd(q, k, v, k_lens=kn)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = b.attn_fwd(q, k, v, k_lens=kn)
        grads = b.attn_bwd(g, q, k, v, o, lse, k_lens=kn)
    for n in (1200, 7, 0, 1500):
        q.normal_()
        kn.fill_(n)
        graph.replay()
        torch.cuda.synchronize()
        o2, lse2 = b.attn_fwd(q, k, v, k_lens=kn)
        g2 = b.attn_bwd(g, q, k, v, o2, lse2, k_lens=kn)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        assert all(torch.equal(x, y) for x, y in zip(grads, g2)), n


def test_offsets_past_32_bits():
    """Keys whose rows lie 2^15 values apart, more than 2^31 values in all."""
    b = block()
    n = 70_000
    cache = torch.empty(n * 32768, dtype=BF16, device="cuda").view(1, n, 32768)
    gen = torch.Generator(device="cuda").manual_seed(0)
    k1, v1 = (torch.randn(1, n, 1, 64, generator=gen, device="cuda").to(BF16) for _ in range(2))
    k, v = cache[:, :, 64:128].unflatten(2, (1, 64)), cache[:, :, 128:192].unflatten(2, (1, 64))
    k.copy_(k1)
    v.copy_(v1)
    q, g = (torch.randn(1, 3, 2, 64, generator=gen, device="cuda").to(BF16) for _ in range(2))
    o, lse = b.attn_fwd(q, k, v)
    o1, lse1 = b.attn_fwd(q, k1, v1)
    assert torch.equal(o, o1) and torch.equal(lse, lse1)
    for x, y in zip(b.attn_bwd(g, q, k, v, o, lse), b.attn_bwd(g, q, k1, v1, o, lse)):
        assert torch.equal(x, y)


def test_gradients_into_given_tensors():
    b = block()
    qkv = make(2, 77, 77, 2, 2, 64)[0].repeat(1, 1, 3, 1).view(2, 77, 3, 2, 64)
    q, k, v = qkv.unbind(2)
    o, lse = b.attn_fwd(q, k, v, causal=True)
    g = make(2, 77, 77, 2, 2, 64, seed=1)[3]
    packed = torch.full_like(qkv, float("nan"))
    b.attn_bwd(g, q, k, v, o, lse, causal=True, out=packed.unbind(2))
    for x, y in zip(packed.unbind(2), b.attn_bwd(g, q, k, v, o, lse, causal=True)):
        assert torch.equal(x, y)
    leaf = qkv.clone().requires_grad_(True)
    b.attention_qkv(leaf, causal=True).backward(g)
    assert torch.equal(leaf.grad, packed)
    with pytest.raises(ValueError):
        b.attn_bwd(g, q, k, v, o, lse, out=(q, k, v[:1]))


def test_another_stream():
    b = block()
    q, k, v, g = make(1, 2, 6000, 4, 2, 128)       # few queries: takes a workspace
    o, lse = b.attn_fwd(q, k, v)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o2, lse2 = b.attn_fwd(q, k, v)
        grads = b.attn_bwd(g, q, k, v, o2, lse2)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert all(torch.equal(x, y) for x, y in zip(grads, b.attn_bwd(g, q, k, v, o, lse)))


@pytest.mark.parametrize("b,m,n,h,g,d", [(9, 600, 65, 16, 16, 64), (9, 600, 128, 16, 16, 128), (33, 130, 190, 16, 8, 64),
                                         (10, 500, 257, 14, 14, 72), (3, 2000, 320, 12, 12, 32)])
def test_more_row_blocks_than_fit_at_once(b, m, n, h, g, d):
    """More workgroups than the card holds, with two, three, five key tiles,
    whole and not."""
    check(*make(b, m, n, h, g, d, seed=n))
