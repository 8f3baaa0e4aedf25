"""fp64 definitions of the transformer-block operators, and the comparison the
GPU tests use.  Plain torch in float64, one formula after the other; gradients
by autograd."""

import torch

EPS = 1e-6


def close(got, ref, where, f32_tol=1e-5, inner=0.0):
    """|got - ref| elementwise: half a step of got's type, relative to the
    value, plus f32_tol of the largest reference value (fp32 sums: under 64
    additions of 2^-24 deep at a few times the output's size), plus `inner`
    of the reference's largest value (roundings of bf16 operands, derived by
    the caller).  Infinities and NaN must agree in place."""
    got, ref = got.detach().double(), ref.detach().double().to(got.device)
    assert got.shape == ref.shape, (where, got.shape, ref.shape)
    fin = torch.isfinite(ref)
    assert torch.equal(torch.isfinite(got), fin), f"{where}: non-finite values differ"
    assert torch.equal(got[~fin], ref[~fin]), where
    if not fin.any():
        return
    g, r = got[fin], ref[fin]
    step = 2.0 ** -8 if where.endswith(":bf16") else 2.0 ** -24
    bound = step * r.abs() + (f32_tol + inner) * r.abs().max()
    off = (g - r).abs()
    worst = int((off - bound).argmax())
    assert bool((off <= bound).all()), (
        f"{where}: off {off[worst].item():.3e} at value {r[worst].item():.3e}, bound {bound[worst].item():.3e}")


def name_of(t):
    return "bf16" if t.dtype == torch.bfloat16 else "f32"


def norm_rows(x, kind, eps=EPS):
    if kind == "none":
        return x
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    return x / (x.square().mean(-1, keepdim=True) + eps).sqrt()


def norm_block(resid, h, gate, post_weight, pre_weight, scale, shift, post, pre, alpha, eps=EPS):
    """(resid_out, y) for (samples, rows, cols) tensors in float64."""
    def vec(t):
        return t[:, None, :]
    r = resid
    if h is not None:
        p = norm_rows(h, post, eps)
        if post_weight is not None:
            p = p * post_weight
        if gate is not None:
            p = p * vec(gate)
        r = resid + alpha * p
    y = norm_rows(r, pre, eps)
    if pre_weight is not None:
        y = y * pre_weight
    if scale is not None:
        y = y * (1 + vec(scale))
    if shift is not None:
        y = y + vec(shift)
    return r, y


def attention(q, k, v, causal=False, offset=0, q_lens=None, k_lens=None, scale=None):
    """(o, lse) of (batch, len, heads, dim) tensors, float64, one sample and
    head at a time over what is there."""
    b, m, h, d = q.shape
    n, g = k.shape[1], k.shape[2]
    scale = d ** -0.5 if scale is None else scale
    o = torch.zeros((b, m, h, d), dtype=torch.float64, device=q.device)
    lse = torch.full((b, h, m), float("-inf"), dtype=torch.float64, device=q.device)
    for i in range(b):
        mi = m if q_lens is None else min(max(int(q_lens[i]), 0), m)
        ni = n if k_lens is None else min(max(int(k_lens[i]), 0), n)
        if mi == 0 or ni == 0:
            continue
        see = torch.ones((mi, ni), dtype=torch.bool, device=q.device)
        if causal:
            rows = torch.arange(mi, device=q.device)[:, None]
            see = torch.arange(ni, device=q.device)[None, :] <= rows + offset
        some = see.any(1)
        for j in range(h):
            kj = j * g // h
            s = (q[i, :mi, j] @ k[i, :ni, kj].T * scale).masked_fill(~see, -1e300)
            p = torch.softmax(s, dim=1) * some[:, None]
            o[i, :mi, j] = p @ v[i, :ni, kj]
            lse[i, j, :mi] = torch.where(some, torch.logsumexp(s, dim=1), float("-inf"))
    return o, lse


def act(g, kind):
    if kind == "silu":
        return torch.nn.functional.silu(g)
    return torch.nn.functional.gelu(g, approximate="tanh")
