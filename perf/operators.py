"""Cases of the transformer-block operators: what is run, on which inputs,
and what it has to read, write and compute.

Three operators, forward and backward apart, as a training loop calls them:

  norm   r' = r + alpha gate_b post_norm(h) w_post and
         y = pre_norm(r') w_pre (1 + scale_b) + shift_b, b the sample
  attn   softmax attention with grouped heads, a causal border, and query and
         key lengths per sample; the backward pass recomputes the probabilities
  ffn    y = (act(x Wg^T) * (x Wu^T)) Wd^T

``own`` false computes the plain form in torch operations (fp32, rounded once
at the end), ``own`` true calls this package.
"""

from __future__ import annotations

import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
TYPES = {"bf16": BF16, "f32": F32}


# ------------------------------------------------------------------- cases
def _norm(do, samples, rows, cols, resid="f32", act="bf16", param="f32", post="none", pre="layer", modulated=True,
          weights=False, alpha=1.0):
    return {"op": "norm", "do": do, "samples": samples, "rows": rows, "cols": cols, "resid": resid, "act": act,
            "param": param, "post": post, "pre": pre, "modulated": modulated, "weights": weights, "alpha": alpha}


def _attn(do, batch, q_len, k_len, heads, kv_heads, dim, causal=False, ragged=False, packed=False):
    return {"op": "attn", "do": do, "batch": batch, "q_len": q_len, "k_len": k_len, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "causal": causal, "ragged": ragged, "packed": packed}


def _ffn(do, rows, cols, hidden, act="silu"):
    return {"op": "ffn", "do": do, "rows": rows, "cols": cols, "hidden": hidden, "act": act}


def listed():
    return [
        # a few tokens of an odd width with both norms' weights: a call whose launch counts
        dict(_norm("fwd", 1, 7, 1001, act="f32", post="rms", pre="rms", modulated=False, weights=True),
             name="norm-fwd-few-odd"),
        # DiT-1.3B block at 512 x 512 pixels (1024 latent tokens): gate, residual, modulated LayerNorm
        dict(_norm("fwd", 16, 1024, 2048), name="norm-fwd-dit-1.3b"),
        # DiT-15B block's backward, sandwich norms with weights, and every gradient of modulation and weights
        dict(_norm("bwd", 8, 1024, 5120, post="rms", weights=True), name="norm-bwd-dit-15b"),
        # one new token of each of four sequences against long caches with grouped heads
        dict(_attn("fwd", 4, 1, 8191, 32, 8, 128), name="attn-fwd-one-token"),
        # DiT-1.3B self-attention, q, k and v inside one projection's output
        dict(_attn("fwd", 16, 1024, 1024, 16, 16, 128, packed=True), name="attn-fwd-dit-1.3b"),
        # image tokens over padded captions of uneven lengths (one sample has none), head size 72
        dict(_attn("fwd", 5, 1000, 333, 16, 16, 72, ragged=True), name="attn-fwd-cross-ragged"),
        # DiT-15B self-attention's gradients
        dict(_attn("bwd", 4, 1024, 1024, 40, 40, 128, packed=True), name="attn-bwd-dit-15b"),
        # gradients of a long causal sequence with four query heads to a key head
        dict(_attn("bwd", 1, 8192, 8192, 16, 4, 128, causal=True), name="attn-bwd-long-causal"),
        # one token through a feed-forward block of DiT-1.3B's sizes: bound by the weights
        dict(_ffn("fwd", 1, 2048, 8192), name="ffn-fwd-one-token"),
        # DiT-1.3B feed-forward on four 512 x 512 images
        dict(_ffn("fwd", 4096, 2048, 8192), name="ffn-fwd-dit-1.3b"),
        # sizes that are no multiple of a tile
        dict(_ffn("bwd", 777, 1000, 2728, "gelu"), name="ffn-bwd-ragged"),
        # DiT-15B feed-forward's gradients on four images: the largest case
        dict(_ffn("bwd", 4096, 5120, 20480), name="ffn-bwd-dit-15b"),
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], even over its logarithm."""
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high + 0.5))))))


def draw(rng):
    op = rng.choice(["norm", "attn", "ffn"])
    do = rng.choice(["fwd", "bwd"])
    if op == "norm":
        samples = rng.randint(1, 9)
        cols = _spread(rng, 33, 5200)
        if rng.random() < 0.5:
            cols = max(40, cols // 8 * 8)
        rows = _spread(rng, 1, max(1, min(4096, 40_000_000 // (samples * cols))))
        post = rng.choice(["none", "rms", "layer"])
        return _norm(do, samples, rows, cols, rng.choice(["f32", "bf16"]), rng.choice(["f32", "bf16"]),
                     rng.choice(["f32", "bf16"]), post, rng.choice(["rms", "layer"]),
                     rng.random() < 0.7, rng.random() < 0.5, rng.choice([1.0, 0.5, 0.125]))
    if op == "attn":
        kv_heads = rng.randint(1, 8)
        heads = kv_heads * rng.choice([1, 1, 2, 4])
        dim = rng.choice([8, 32, 40, 64, 64, 72, 96, 128, 128, 128])
        batch = rng.randint(1, 8)
        q_len = _spread(rng, 1, 5000)
        k_len = q_len if rng.random() < 0.5 else _spread(rng, 1, 8200)
        while batch * heads * q_len * k_len > 500_000_000:
            batch, q_len, k_len = max(1, batch // 2), (q_len + 1) // 2, (k_len + 1) // 2
        return _attn(do, batch, q_len, k_len, heads, kv_heads, dim, rng.random() < 0.5, rng.random() < 0.4,
                     q_len == k_len and heads == kv_heads and rng.random() < 0.5)
    cols, hidden = 8 * _spread(rng, 8, 512), 8 * _spread(rng, 8, 1300)
    rows = _spread(rng, 1, 6000)
    while rows * cols * hidden > 1.5e11:
        rows = (rows + 1) // 2
    return _ffn(do, rows, cols, hidden, rng.choice(["silu", "gelu"]))


# ------------------------------------------------------------------ inputs
def _rand(gen, shape, dtype=F32, std=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return {"norm": _prepare_norm, "attn": _prepare_attn, "ffn": _prepare_ffn}[case["op"]](case, gen)


def _prepare_norm(c, gen):
    b, n, d = c["samples"], c["rows"], c["cols"]
    rt, ht, pt = TYPES[c["resid"]], TYPES[c["act"]], TYPES[c["param"]]
    s = {"case": c, "resid": _rand(gen, (b, n, d), rt, 2.0), "h": _rand(gen, (b, n, d), ht),
         "gate": None, "scale": None, "shift": None, "post_weight": None, "pre_weight": None}
    if c["modulated"]:
        # shift, scale and gate are slices of one projection's output, as adaLN gives them
        s["shift"], s["scale"], s["gate"] = _rand(gen, (b, 3 * d), pt, 0.3).chunk(3, dim=1)
    if c["weights"]:
        s["pre_weight"] = (1 + _rand(gen, (d,), F32, 0.1)).to(pt)
        if c["post"] != "none":
            s["post_weight"] = (1 + _rand(gen, (d,), F32, 0.1)).to(pt)
    if c["do"] == "bwd":
        # what the forward pass left: the new residual stream and the rows' statistics
        s["resid_out"] = s.pop("resid")
        s["stats"] = torch.cat([_stats(s["h"], c["post"]), _stats(s["resid_out"], c["pre"])], dim=-1).reshape(b * n, 4)
        s["d_resid"] = _rand(gen, (b, n, d), rt, 1e-2)
        s["d_y"] = _rand(gen, (b, n, d), ht, 1e-2)
    return s


def _prepare_attn(c, gen):
    b, m, n, h, g, d = c["batch"], c["q_len"], c["k_len"], c["heads"], c["kv_heads"], c["dim"]
    if c["packed"]:
        q, k, v = _rand(gen, (b, m, 3, h, d), BF16).unbind(2)
    else:
        q, k, v = _rand(gen, (b, m, h, d), BF16), _rand(gen, (b, n, g, d), BF16), _rand(gen, (b, n, g, d), BF16)
    s = {"case": c, "q": q, "k": k, "v": v, "qn": None, "kn": None}
    if c["ragged"]:
        # uneven lengths, one of the samples (of more than one) without a key; padding holds what it may
        s["qn"] = torch.randint(m // 2, m + 1, (b,), generator=gen, device="cuda", dtype=torch.int32)
        s["kn"] = torch.randint(0, n + 1, (b,), generator=gen, device="cuda", dtype=torch.int32)
        if b > 1:
            s["kn"][b // 2] = 0
        k.masked_fill_((torch.arange(n, device="cuda") >= s["kn"][:, None])[:, :, None, None], float("nan"))
        v.masked_fill_((torch.arange(n, device="cuda") >= s["kn"][:, None])[:, :, None, None], float("inf"))
    if c["do"] == "bwd":
        s["o"], s["lse"] = _attn_fwd(s)
        s["do"] = _rand(gen, (b, m, h, d), BF16, 1e-1)
    return s


def _prepare_ffn(c, gen):
    t, d, f = c["rows"], c["cols"], c["hidden"]
    s = {"case": c, "x": _rand(gen, (t, d), BF16), "wg": _rand(gen, (f, d), BF16, d ** -0.5),
         "wu": _rand(gen, (f, d), BF16, d ** -0.5), "wd": _rand(gen, (d, f), BF16, f ** -0.5)}
    if c["do"] == "bwd":
        # the projections that the forward pass kept, gate then up
        s["gu"] = torch.cat([s["x"].float() @ s["wg"].float().T, s["x"].float() @ s["wu"].float().T], dim=1).to(BF16)
        s["dy"] = _rand(gen, (t, d), BF16, 1e-1)
    return s


# ------------------------------------------------------------ a pass through
def run(state):
    c = state["case"]
    if own:
        return _own(c, state)
    return {"normfwd": _norm_fwd, "normbwd": _norm_bwd, "attnfwd": _attn_fwd, "attnbwd": _attn_bwd,
            "ffnfwd": _ffn_fwd, "ffnbwd": _ffn_bwd}[c["op"] + c["do"]](state)


def _own(c, s):
    import matrix_aware_optimizer_periodic_amd as mm

    if c["op"] == "norm":
        params = (s["gate"], s["post_weight"], s["pre_weight"], s["scale"], s["shift"])
        how = {"post": c["post"], "pre": c["pre"], "alpha": c["alpha"]}
        if c["do"] == "fwd":
            return mm.norm_fwd(s["resid"], s["h"], *params, **how)
        return mm.norm_bwd(s["d_resid"], s["d_y"], s["resid_out"], s["h"], s["stats"], *params, **how)
    if c["op"] == "attn":
        how = {"causal": c["causal"], "offset": c["k_len"] - c["q_len"], "q_lens": s["qn"], "k_lens": s["kn"]}
        if c["do"] == "fwd":
            return mm.attn_fwd(s["q"], s["k"], s["v"], **how)
        return mm.attn_bwd(s["do"], s["q"], s["k"], s["v"], s["o"], s["lse"], **how)
    if c["do"] == "fwd":
        return mm.ffn_fwd(s["x"], s["wg"], s["wu"], s["wd"], act=c["act"])
    return mm.ffn_bwd(s["dy"], s["x"], s["wg"], s["wu"], s["wd"], s["gu"], act=c["act"])


# ------------------------------------------------------------- plain forms
EPS = 1e-6


def _stats(x, kind):
    """Mean and reciprocal deviation of each row, fp32."""
    x = x.double()
    mean = x.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(x[..., :1])
    rstd = torch.rsqrt((x - mean).square().mean(-1, keepdim=True) + EPS) if kind != "none" else torch.ones_like(mean)
    return torch.cat([mean, rstd], dim=-1).float()


def _norm_rows(x, kind):
    mean = x.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(x[..., :1])
    rstd = torch.rsqrt((x - mean).square().mean(-1, keepdim=True) + EPS) if kind != "none" else torch.ones_like(mean)
    return (x - mean) * rstd, torch.cat([mean, rstd], dim=-1)


def _row(t):
    """A per-sample vector (samples, cols) next to (samples, rows, cols), or the number 0."""
    return 0.0 if t is None else t.float()[:, None, :]


def _one(t):
    return 1.0 if t is None else t.float()


def _norm_fwd(s):
    c = s["case"]
    p, sh = _norm_rows(s["h"].float(), c["post"])
    gate = 1.0 if s["gate"] is None else _row(s["gate"])
    r = s["resid"].float() + c["alpha"] * gate * (p * _one(s["post_weight"]))
    x, sr = _norm_rows(r, c["pre"])
    y = x * _one(s["pre_weight"]) * (1.0 + _row(s["scale"])) + _row(s["shift"])
    return r.to(s["resid"].dtype), y.to(s["h"].dtype), torch.cat([sh, sr], dim=-1).reshape(-1, 4)


def _norm_rows_bwd(g, xhat, rstd, kind):
    """The gradient of a row's normalisation."""
    if kind == "none":
        return g
    g = g - g.mean(-1, keepdim=True) - xhat * (g * xhat).mean(-1, keepdim=True) if kind == "layer" else \
        g - xhat * (g * xhat).mean(-1, keepdim=True)
    return g * rstd


def _norm_bwd(s):
    c = s["case"]
    b, n, d = s["h"].shape
    st = s["stats"].view(b, n, 4)
    hhat = (s["h"].float() - st[..., 0:1]) * st[..., 1:2]
    xhat = (s["resid_out"].float() - st[..., 2:3]) * st[..., 3:4]
    dy = s["d_y"].float()
    gate = 1.0 if s["gate"] is None else _row(s["gate"])
    g = dy * _one(s["pre_weight"]) * (1.0 + _row(s["scale"]))
    dr = s["d_resid"].float() + _norm_rows_bwd(g, xhat, st[..., 3:4], c["pre"])
    dh = _norm_rows_bwd(c["alpha"] * gate * _one(s["post_weight"]) * dr, hhat, st[..., 1:2], c["post"])
    mod, w_post, w_pre = s["gate"], s["post_weight"], s["pre_weight"]
    return {
        "resid": dr.to(s["resid_out"].dtype), "h": dh.to(s["h"].dtype),
        "gate": None if mod is None else (c["alpha"] * dr * (hhat * _one(w_post))).sum(1).to(mod.dtype),
        "post_weight": None if w_post is None else (c["alpha"] * gate * dr * hhat).sum((0, 1)).to(w_post.dtype),
        "pre_weight": None if w_pre is None else (dy * (1.0 + _row(s["scale"])) * xhat).sum((0, 1)).to(w_pre.dtype),
        "scale": None if mod is None else (dy * xhat * _one(w_pre)).sum(1).to(mod.dtype),
        "shift": None if mod is None else dy.sum(1).to(mod.dtype),
    }


def _visible(c, s):
    """Which key each query of a sample sees: (batch, q_len, k_len), and which queries and keys are there."""
    i = torch.arange(c["q_len"], device="cuda")[None, :, None]
    j = torch.arange(c["k_len"], device="cuda")[None, None, :]
    there_q = i < (c["q_len"] if s["qn"] is None else s["qn"][:, None, None])
    there_k = j < (c["k_len"] if s["kn"] is None else s["kn"][:, None, None])
    see = there_q & there_k
    if c["causal"]:
        see = see & (j <= i + (c["k_len"] - c["q_len"]))
    return see.expand(c["batch"], -1, -1), there_q[:, :, 0], there_k[:, 0, :]


def _heads_first(t, there, times):
    """(batch, len, heads, dim) -> (batch, heads * times, len, dim) in fp32, what lies past a length as zeros."""
    t = torch.where(there[:, :, None, None], t.float(), 0.0).transpose(1, 2)
    return t.repeat_interleave(times, dim=1).contiguous()


def _attn_fwd(s):
    c = s["case"]
    see, tq, tk = _visible(c, s)
    times = c["heads"] // c["kv_heads"]
    q, k, v = _heads_first(s["q"], tq, 1), _heads_first(s["k"], tk, times), _heads_first(s["v"], tk, times)
    x = (q @ k.transpose(2, 3).contiguous()).mul_(c["dim"] ** -0.5)
    x = x.masked_fill_(~see[:, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), 0.0, top)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = (x @ v) / torch.where(total == 0, 1.0, total)
    return o.transpose(1, 2).to(BF16).contiguous(), (top + total.log()).squeeze(-1)


def _attn_bwd(s):
    c = s["case"]
    see, tq, tk = _visible(c, s)
    times, a = c["heads"] // c["kv_heads"], c["dim"] ** -0.5
    q, k, v = _heads_first(s["q"], tq, 1), _heads_first(s["k"], tk, times), _heads_first(s["v"], tk, times)
    do, o = _heads_first(s["do"], tq, 1), _heads_first(s["o"], tq, 1)
    lse = torch.where(s["lse"] == float("-inf"), 0.0, s["lse"])
    p = (q @ k.transpose(2, 3).contiguous()).mul_(a)
    p = p.sub_(lse[..., None]).exp_().masked_fill_(~see[:, None], 0.0)
    dv = p.transpose(2, 3).contiguous() @ do
    ds = (do @ v.transpose(2, 3).contiguous()).sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(a)
    dq, dk = ds @ k, ds.transpose(2, 3).contiguous() @ q
    shape = (c["batch"], c["kv_heads"], times, c["k_len"], c["dim"])
    dk, dv = dk.view(shape).sum(2), dv.view(shape).sum(2)
    return tuple(t.transpose(1, 2).to(BF16).contiguous() for t in (dq, dk, dv))


def _act(g, kind):
    """The activation and its derivative; gelu in its tanh form."""
    if kind == "silu":
        e = 1.0 / (1.0 + torch.exp(-g))
        return g * e, e * (1.0 + g * (1.0 - e))
    a, b = math.sqrt(2.0 / math.pi), 0.044715
    t = torch.tanh(a * (g + b * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * a * (1.0 + 3.0 * b * g * g)


def _ffn_fwd(s):
    x = s["x"].float()
    g, u = x @ s["wg"].float().T, x @ s["wu"].float().T
    y = (_act(g, s["case"]["act"])[0] * u) @ s["wd"].float().T
    return y.to(BF16), torch.cat([g, u], dim=1).to(BF16)


def _ffn_bwd(s):
    f = s["case"]["hidden"]
    x, dy = s["x"].float(), s["dy"].float()
    g, u = s["gu"][:, :f].float(), s["gu"][:, f:].float()
    a, da = _act(g, s["case"]["act"])
    dh = dy @ s["wd"].float()
    dg, du = dh * u * da, dh * a
    dx = dg @ s["wg"].float() + du @ s["wu"].float()
    return tuple(t.to(BF16) for t in (dx, dg.T @ x, du.T @ x, dy.T @ (a * u)))


# -------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "norm":
        e = c["samples"] * c["rows"] * c["cols"]
        rb, hb, pb = (4 if c[k] == "f32" else 2 for k in ("resid", "act", "param"))
        vectors = c["cols"] * pb * ((3 * c["samples"] if c["modulated"] else 0) + (2 if c["weights"] else 0))
        if c["do"] == "fwd":
            return {"bytes": e * 2 * (rb + hb) + vectors, "flops": 12 * e}
        return {"bytes": e * 3 * (rb + hb) + 2 * vectors, "flops": 26 * e}
    if c["op"] == "attn":
        q = c["batch"] * c["q_len"] * c["heads"] * c["dim"]
        kv = c["batch"] * c["k_len"] * c["kv_heads"] * c["dim"]
        pairs = _pairs(c["q_len"], c["k_len"]) if c["causal"] else c["q_len"] * c["k_len"]
        if c["ragged"]:
            pairs = pairs * 3 // 8      # lengths of 3/4 and 1/2 on average
        flops = c["batch"] * c["heads"] * pairs * c["dim"] * (4 if c["do"] == "fwd" else 10)
        return {"bytes": 2 * (q * 2 + kv * 2) if c["do"] == "fwd" else 2 * (q * 4 + kv * 4), "flops": max(flops, 1)}
    t, d, f = c["rows"], c["cols"], c["hidden"]
    if c["do"] == "fwd":
        return {"bytes": 2 * (2 * t * d + 3 * d * f + 2 * t * f), "flops": 6 * t * d * f}
    return {"bytes": 2 * (3 * t * d + 6 * d * f + 2 * t * f), "flops": 12 * t * d * f}


def _pairs(m, n):
    """Pairs below a causal border that ends at the last query and key."""
    first = n - m + 1                 # keys that the first query sees
    if first >= 1:
        return m * first + m * (m - 1) // 2
    return n * (n + 1) // 2


# --------------------------------------------------------- 64-bit definition
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "attn": _exact_attn, "ffn": _exact_ffn}[case["op"]](case, s)


def _exact_norm(c, s):
    def leaf(t):
        return None if t is None else t.detach().double().requires_grad_(True)

    def normed(x, kind):
        """x with each row normalised."""
        if kind == "none":
            return x
        if kind == "layer":
            return torch.nn.functional.layer_norm(x, x.shape[-1:], eps=EPS)
        return x / (x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()

    def moments(x, kind):
        x = x.detach()
        m = x.mean(-1) if kind == "layer" else x.new_zeros(x.shape[:-1])
        second = (x.square().mean(-1) if kind == "rms" else x.var(-1, correction=0)) + EPS
        return [m.reshape(-1), (x.new_ones(m.shape) if kind == "none" else second ** -0.5).reshape(-1)]

    names = ("gate", "post_weight", "pre_weight", "scale", "shift")
    par = {n: leaf(s[n]) for n in names}
    h = leaf(s["h"])

    def through(t, per_sample):
        return t.unsqueeze(1) if per_sample else t

    def branch(h):
        p = normed(h, c["post"])
        for n, per in (("post_weight", False), ("gate", True)):
            if par[n] is not None:
                p = p * through(par[n], per)
        return c["alpha"] * p

    def out(r):
        y = normed(r, c["pre"])
        if par["pre_weight"] is not None:
            y = y * par["pre_weight"]
        if par["scale"] is not None:
            y = torch.addcmul(through(par["shift"], True), y, 1 + through(par["scale"], True))
        return y

    if c["do"] == "fwd":
        with torch.no_grad():
            r = s["resid"].double() + branch(h)
            return r, out(r), torch.stack(moments(h, c["post"]) + moments(r, c["pre"]), dim=1)
    r = leaf(s["resid_out"])
    out(r).backward(s["d_y"].double())
    total = r.grad + s["d_resid"].double()
    branch(h).backward(total)
    return {"resid": total, "h": h.grad, **{n: None if par[n] is None else par[n].grad for n in names}}


def _exact_attn(c, s):
    b, m, n, h, g, d = c["batch"], c["q_len"], c["k_len"], c["heads"], c["kv_heads"], c["dim"]
    bwd = c["do"] == "bwd"
    shapes = {"q": (b, m, h, d), "k": (b, n, g, d), "v": (b, n, g, d)}
    grads = {t: torch.zeros(shapes[t], dtype=torch.float64, device="cuda") for t in shapes}
    o = torch.zeros((b, m, h, d), dtype=torch.float64, device="cuda")
    lse = torch.full((b, h, m), float("-inf"), dtype=torch.float64, device="cuda")
    qn = [m] * b if s["qn"] is None else s["qn"].tolist()
    kn = [n] * b if s["kn"] is None else s["kn"].tolist()
    for i in range(b):
        qi, ki = qn[i], kn[i]
        if qi == 0 or ki == 0:
            continue
        allowed = torch.ones((qi, ki), dtype=torch.bool, device="cuda")
        if c["causal"]:
            allowed = allowed.tril(n - m)
        some = allowed.any(1, keepdim=True)
        for j in range(h):
            kv = j * g // h
            q = s["q"][i, :qi, j].double().requires_grad_(bwd)
            k = s["k"][i, :ki, kv].double().requires_grad_(bwd)
            v = s["v"][i, :ki, kv].double().requires_grad_(bwd)
            score = torch.where(allowed, torch.mm(q, k.t()) / math.sqrt(d), -1e300)
            out = torch.where(some, torch.mm(torch.softmax(score, dim=1), v), 0.0)
            if bwd:
                out.backward(s["do"][i, :qi, j].double())
                grads["q"][i, :qi, j] = q.grad
                grads["k"][i, :ki, kv] += k.grad
                grads["v"][i, :ki, kv] += v.grad
            else:
                o[i, :qi, j] = out
                lse[i, j, :qi] = torch.where(some[:, 0], torch.logsumexp(score, dim=1), float("-inf"))
    return (grads["q"], grads["k"], grads["v"]) if bwd else (o, lse)


def _exact_ffn(c, s):
    f = c["hidden"]
    x, wg, wu, wd = (s[k].double() for k in ("x", "wg", "wu", "wd"))

    def gated(g, u):
        if c["act"] == "silu":
            return torch.nn.functional.silu(g) * u
        return torch.nn.functional.gelu(g, approximate="tanh") * u

    if c["do"] == "fwd":
        gu = torch.mm(x, torch.cat([wg, wu]).t())
        return torch.mm(gated(gu[:, :f], gu[:, f:]), wd.t()), gu
    gu = s["gu"].double().requires_grad_(True)
    hidden = gated(gu[:, :f], gu[:, f:])
    dy = s["dy"].double()
    hidden.backward(torch.mm(dy, wd))
    dgu = gu.grad
    dw = torch.mm(dgu.t(), x)
    return torch.mm(dgu, torch.cat([wg, wu])), dw[:f], dw[f:], torch.mm(dy.t(), hidden.detach())
