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
