"""Attention with NaN and infinities among what a query sees: they come out
where the formulas put them, and nowhere else.  The definition here is written
pair by pair, so that a pair that is not there adds nothing."""

import pytest
import torch

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
NAN, INF = float("nan"), float("inf")


def block():
    from matrix_aware_optimizer_periodic_amd import block as b
    return b


def make(b, m, n, h, g, d, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def r(*shape):
        return torch.randn(shape, generator=gen, device="cuda").to(BF16)
    return r(b, m, h, d), r(b, n, g, d), r(b, n, g, d), r(b, m, h, d)


def seen(b, m, n, causal, offset, q_lens, k_lens):
    i, j = torch.arange(m, device="cuda")[:, None], torch.arange(n, device="cuda")[None, :]
    see = ((j <= i + offset) if causal else torch.ones((m, n), dtype=torch.bool, device="cuda")).expand(b, m, n)
    if q_lens is not None:
        see = see & (i < q_lens[:, None, None])
    if k_lens is not None:
        see = see & (j < k_lens[:, None, None])
    return see


def by_pairs(q, k, v, d_o, causal=False, offset=0, q_lens=None, k_lens=None):
    """o, lse, dq, dk, dv in float64 (dq, dk, dv from the exact o)."""
    b, m, h, d = q.shape
    n, g, a = k.shape[1], k.shape[2], d ** -0.5
    see_all = seen(b, m, n, causal, offset, q_lens, k_lens)
    o, lse = torch.zeros_like(q, dtype=torch.float64), torch.full((b, h, m), -INF, dtype=torch.float64, device="cuda")
    dq = torch.zeros_like(o)
    dk, dv = torch.zeros_like(k, dtype=torch.float64), torch.zeros_like(v, dtype=torch.float64)
    for i in range(b):
        see = see_all[i]
        some = see.any(1)
        for j in range(h):
            kj = j * g // h
            qi, gi, ki, vi = q[i, :, j].double(), d_o[i, :, j].double(), k[i, :, kj].double(), v[i, :, kj].double()
            s = torch.where(see, (qi[:, None] * ki[None]).sum(-1) * a, -INF)
            top = torch.where(some, s.amax(1), 0.0)
            e = torch.where(see, (s - top[:, None]).exp(), 0.0)
            total = torch.where(some, e.sum(1), 1.0)
            p = e / total[:, None]
            lse[i, j] = torch.where(some, top + total.log(), -INF)
            oi = torch.where(see[..., None], p[..., None] * vi[None], 0.0).sum(1)
            o[i, :, j] = oi
            dp = (gi[:, None] * vi[None]).sum(-1)
            ds = torch.where(see, p * (dp - (gi * oi).sum(-1)[:, None]) * a, 0.0)
            dq[i, :, j] = torch.where(see[..., None], ds[..., None] * ki[None], 0.0).sum(1)
            dk[i, :, kj] += torch.where(see[..., None], ds[..., None] * qi[:, None], 0.0).sum(0)
            dv[i, :, kj] += torch.where(see[..., None], p[..., None] * gi[:, None], 0.0).sum(0)
    return o, lse, dq, dk, dv


def close(got, ref, where, tol):
    """NaN and infinities in the same places; the others off by half a bf16
    step of the value (lse: fp32 sums) and `tol` of the largest value, for the
    operands' roundings to bf16, 2^-8 of a term each."""
    got, ref = got.double(), ref.double()
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{where}: NaN in other places"
    inf = torch.isinf(ref)
    assert torch.equal(torch.isinf(got), inf) and torch.equal(got[inf], ref[inf]), f"{where}: infinities differ"
    fin = torch.isfinite(ref)
    if not bool(fin.any()):
        return
    off = (got[fin] - ref[fin]).abs()
    bound = (2.0 ** -8 if where != "lse" else 2.0 ** -24) * ref[fin].abs() + tol * ref[fin].abs().max()
    assert bool((off <= bound).all()), (where, float((off - bound).max()))


def check(q, k, v, d_o, **how):
    b = block()
    o, lse = b.attn_fwd(q, k, v, **how)
    want = by_pairs(q, k, v, d_o, **how)
    close(o, want[0], "o", 2.0 ** -8)
    close(lse, want[1], "lse", 1e-5)
    for name, x, y in zip(("d_q", "d_k", "d_v"), b.attn_bwd(d_o, q, k, v, o, lse, **how), want[2:]):
        close(x, y, name, 2.0 ** -7)


# keys in one range, and divided into several whose results are joined
@pytest.mark.parametrize("b,m,n,h,g,d", [(1, 5, 60, 2, 1, 64), (1, 5, 3000, 2, 1, 64), (2, 3, 1500, 4, 2, 128),
                                         (40, 130, 70, 2, 2, 72)])
@pytest.mark.parametrize("value", [NAN, INF, -INF])
def test_queries_that_are_not_finite(b, m, n, h, g, d, value):
    q, k, v, d_o = make(b, m, n, h, g, d, seed=n)
    q[0, 1, 0, 3] = value
    q[b - 1, m - 1, h - 1, :] = value
    check(q, k, v, d_o)


@pytest.mark.parametrize("n", [60, 3000])
def test_keys_and_values_that_are_not_finite(n):
    for what in range(2):
        q, k, v, d_o = make(2, 5, n, 4, 2, 64, seed=n)
        (k, v)[what][1, n // 2, 1, 7] = NAN
        check(q, k, v, d_o)
        check(q, k, v, d_o, k_lens=torch.tensor([n, n // 2], dtype=torch.int32, device="cuda"))


# A cache whose end holds anything, bounded by the causal border alone: whole
# and part tiles past it, few queries and many, heads in groups.
@pytest.mark.parametrize("b,m,n,h,g,d", [(1, 1, 90, 4, 2, 64), (2, 3, 2500, 4, 1, 128), (2, 70, 200, 2, 2, 128),
                                         (3, 260, 700, 2, 1, 40), (40, 130, 300, 2, 1, 72)])
@pytest.mark.parametrize("value", [NAN, INF])
def test_keys_that_no_query_sees_hold_anything(b, m, n, h, g, d, value):
    for past in (1, 29, 64, n - m):
        q, k, v, d_o = make(b, m, n, h, g, d, seed=n + past)
        offset = n - m - past                       # the last query sees all keys but `past`
        k[:, n - past:] = value
        v[:, n - past:] = -value
        check(q, k, v, d_o, causal=True, offset=offset)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("m,n,offset", [(140, 130, -33), (140, 130, -64), (300, 90, -280), (5, 900, -3), (70, 70, -200)])
def test_queries_that_see_no_key_hold_anything(m, n, offset, d):
    q, k, v, d_o = make(2, m, n, 4, 2, d, seed=m)
    q[:, :-offset] = NAN
    d_o[:, :-offset] = INF
    check(q, k, v, d_o, causal=True, offset=offset)
    v[0, 1, 0, 2] = INF                             # nor does what they do not see reach them
    k[1, 0, 1, 2] = NAN
    b = block()
    o, lse = b.attn_fwd(q, k, v, causal=True, offset=offset)
    dq = b.attn_bwd(d_o, q, k, v, o, lse, causal=True, offset=offset)[0]
    empty = slice(0, min(m, -offset))
    assert bool((o[:, empty] == 0).all()) and bool((lse[:, :, empty] == -INF).all()) and bool((dq[:, empty] == 0).all())


def test_rows_and_keys_that_are_there_do_not_reach_the_others():
    """A value of infinity within a sample's lengths, beside queries and keys
    past them and a range of keys that a row does not see."""
    q, k, v, d_o = make(3, 150, 200, 2, 2, 64, seed=8)
    v[:, 5, 0, 9] = INF
    kn, qn = torch.tensor([200, 80, 6], dtype=torch.int32, device="cuda"), torch.tensor([150, 0, 3], dtype=torch.int32, device="cuda")
    check(q, k, v, d_o, q_lens=qn, k_lens=kn)
    q, k, v, d_o = make(1, 3, 4000, 2, 1, 128, seed=9)
    k[0, 3000:], v[0, 3000:] = NAN, NAN
    check(q, k, v, d_o, causal=True, offset=1000)
    check(q, k, v, d_o, k_lens=torch.tensor([2999], dtype=torch.int32, device="cuda"))


def test_how_far_a_key_reaches_over_the_border():
    """A key and value that are not finite, and a d_o, may reach rows (keys)
    on the border's other side that are less than 128 positions away."""
    m, at = 700, 400
    b = block()
    q, k, v, d_o = make(1, m, m, 2, 2, 64, seed=3)
    o, lse = b.attn_fwd(q, k, v, causal=True)
    want = b.attn_bwd(d_o, q, k, v, o, lse, causal=True)
    k1, v1 = k.clone(), v.clone()
    k1[0, at], v1[0, at] = NAN, NAN
    o1, lse1 = b.attn_fwd(q, k1, v1, causal=True)
    assert bool(torch.isnan(o1[:, at:]).all()) and torch.equal(lse1[:, :, :at], lse[:, :, :at])
    assert torch.equal(o1[:, :at - 127], o[:, :at - 127])
    got = b.attn_bwd(d_o, q, k1, v1, o1, lse1, causal=True)
    assert torch.equal(got[0][:, :at - 127], want[0][:, :at - 127])
    g1 = d_o.clone()
    g1[0, at] = NAN
    got = b.attn_bwd(g1, q, k, v, o, lse, causal=True)
    assert torch.equal(got[0][:, :at], want[0][:, :at])
    for x, y in zip(got[1:], want[1:]):
        assert bool(torch.isnan(x[:, :at + 1]).all()) and torch.equal(x[:, at + 128:], y[:, at + 128:])
