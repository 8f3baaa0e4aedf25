"""Cases of the operators between a transformer block's norms and its
attention: what is run, on which inputs, and what it has to read, write and
compute.

  linear   y = residual + drop(act(x W^T + bias)), and its gradients
  rotary   queries and keys rotated by their positions, and back
  dropout  y = residual + keep x / (1 - p), the mask from a counter-based
           generator (Philox4x32-10), and its gradient

``own`` false computes the plain form in torch operations (fp32, rounded once
at the end; angles in fp64), ``own`` true calls this package.
"""

from __future__ import annotations

import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
TYPES = {"bf16": BF16, "f32": F32}


# ------------------------------------------------------------------- cases
def _linear(do, rows, cols, out, act="none", bias="f32", resid="none", p=0.0, save=True, grad="bf16"):
    return {"op": "linear", "do": do, "rows": rows, "cols": cols, "out": out, "act": act, "bias": bias, "resid": resid,
            "p": p, "save": save, "grad": grad}


def _rotary(do, batch, length, heads, kv_heads, dim, rot, interleaved=False, axes=1, per_sample=False, first=0,
            scale=1.0, packed=False, dtype="bf16"):
    return {"op": "rotary", "do": do, "batch": batch, "len": length, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "rot": rot, "interleaved": interleaved, "axes": axes, "per_sample": per_sample, "first": first,
            "scale": scale, "packed": packed, "dtype": dtype}


def _dropout(do, rows, cols, p, act="bf16", resid="none", pad=0):
    return {"op": "dropout", "do": do, "rows": rows, "cols": cols, "p": p, "act": act, "resid": resid, "pad": pad}


def listed():
    return [
        # one sample's condition through a time embedding's layer: a call whose launch counts
        dict(_linear("fwd", 1, 256, 2048, act="silu", save=False), name="linear-fwd-one-row"),
        # the modulation vectors of sixteen samples (DiT-1.3B): bound by reading the weights
        dict(_linear("fwd", 16, 2048, 12288), name="linear-fwd-modulation"),
        # DiT-1.3B, first feed-forward product on four 512 x 512 images, keeping what the backward pass reads
        dict(_linear("fwd", 4096, 2048, 8192, act="gelu", bias="bf16"), name="linear-fwd-fc1"),
        # the second one, with dropout and the fp32 residual stream in its epilogue
        dict(_linear("fwd", 4096, 8192, 2048, resid="f32", p=0.1), name="linear-fwd-fc2-residual"),
        # gradients of sizes that are no multiple of a tile, through dropout and an activation
        dict(_linear("bwd", 777, 1000, 2728, act="silu", resid="f32", p=0.2), name="linear-bwd-ragged"),
        # DiT-15B's modulation of eight samples: the gradients of a large matrix from few rows
        dict(_linear("bwd", 8, 5120, 30720), name="linear-bwd-modulation"),
        # DiT-15B's first feed-forward product, every gradient: the largest case
        dict(_linear("bwd", 4096, 5120, 20480, act="gelu"), name="linear-bwd-fc1"),
        # one new token of each of four sequences, far into a stretched context, grouped heads
        dict(_rotary("fwd", 4, 1, 32, 8, 128, 128, per_sample=True, first=1_000_000, scale=1.1386),
             name="rotary-fwd-one-token"),
        # DiT-1.3B self-attention: rows and columns of the image's grid, q and k inside one projection's output
        dict(_rotary("fwd", 16, 1024, 16, 16, 128, 128, axes=2, packed=True), name="rotary-fwd-grid"),
        # gradients of a part of each head of 72, interleaved pairs, odd length, positions of packed documents
        dict(_rotary("bwd", 5, 1001, 16, 16, 72, 36, interleaved=True, per_sample=True), name="rotary-bwd-part"),
        # a few rows of an odd width, rows apart as a slice leaves them
        dict(_dropout("fwd", 7, 1001, 0.5, act="f32", pad=7), name="dropout-fwd-few-odd"),
        # a DiT-1.3B branch dropped onto the fp32 residual stream
        dict(_dropout("fwd", 16384, 2048, 0.1, resid="f32"), name="dropout-fwd-residual"),
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], even over its logarithm."""
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high + 0.5))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "rotary", "dropout"])
    do = rng.choice(["fwd", "bwd"])
    if op == "linear":
        rows = _spread(rng, 1, 64) if rng.random() < 0.3 else _spread(rng, 1, 6000)
        cols, out = 8 * _spread(rng, 2, 1000), 8 * _spread(rng, 1, 2000)
        while rows * cols * out > 2e11:
            rows = (rows + 1) // 2
        act, bias = rng.choice(["none", "silu", "gelu"]), rng.choice(["none", "f32", "bf16"])
        resid, p = rng.choice(["none", "f32", "bf16"]), rng.choice([0.0, 0.0, 0.1, 0.37])
        # (the weights' gradient in fp32 where dz is dy itself, in bf16: elsewhere it is a product of rounded operands)
        same = act == "none" and p == 0.0 and resid != "f32"
        return _linear(do, rows, cols, out, act, bias, resid, p, rng.random() < 0.7, "f32" if same else "bf16")
    if op == "rotary":
        kv_heads = rng.randint(1, 9)
        heads = kv_heads * rng.choice([1, 1, 2, 4])
        dim = rng.choice([8, 32, 40, 64, 64, 72, 80, 96, 128, 128, 128])
        axes = rng.choice([1, 1, 2, 3])
        rot = dim if rng.random() < 0.6 else 2 * rng.randint(1, dim // 2)
        batch = rng.randint(1, 9)
        length = _spread(rng, 1, max(1, min(9000, 40_000_000 // (batch * heads * dim))))
        return _rotary(do, batch, length, heads, kv_heads, dim, rot, rng.random() < 0.5, axes, rng.random() < 0.4,
                       rng.choice([0, 0, 5, 100_000]), rng.choice([1.0, 1.0, 1.2]),
                       heads == kv_heads and rng.random() < 0.5, rng.choice(["bf16", "bf16", "f32"]))
    cols = _spread(rng, 1, 9000)
    if rng.random() < 0.5:
        cols = max(8, cols // 8 * 8)
    rows = _spread(rng, 1, max(1, min(20_000, 30_000_000 // cols)))
    return _dropout(do, rows, cols, rng.choice([0.05, 0.1, 0.25, 0.5, 0.9]), rng.choice(["f32", "bf16"]),
                    rng.choice(["none", "f32", "bf16"]), rng.choice([0, 0, 0, 8, 3]))


# ------------------------------------------------------------------ inputs
def _rand(gen, shape, dtype=F32, std=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return {"linear": _prepare_linear, "rotary": _prepare_rotary, "dropout": _prepare_dropout}[case["op"]](case, gen, seed)


def _prepare_linear(c, gen, seed):
    t, d, n = c["rows"], c["cols"], c["out"]
    s = {"case": c, "x": _rand(gen, (t, d), BF16), "w": _rand(gen, (n, d), BF16, d ** -0.5), "bias": None, "resid": None,
         "z": None, "rng": (seed * 0x9E3779B1 + 17, seed + (1 << 33))}
    if c["bias"] != "none":
        s["bias"] = _rand(gen, (n,), TYPES[c["bias"]], 0.5)
    if c["do"] == "fwd":
        if c["resid"] != "none":
            s["resid"] = _rand(gen, (t, n), TYPES[c["resid"]], 2.0)
        return s
    if c["act"] != "none":
        # what the forward pass kept
        s["z"] = (s["x"].float() @ s["w"].float().T + (0.0 if s["bias"] is None else s["bias"].float())).to(BF16)
    s["dy"] = _rand(gen, (t, n), BF16 if c["resid"] == "none" else TYPES[c["resid"]], 1e-1)
    return s


def _prepare_rotary(c, gen, seed):
    b, n, h, g, d, axes, pairs = c["batch"], c["len"], c["heads"], c["kv_heads"], c["dim"], c["axes"], c["rot"] // 2
    dt = TYPES[c["dtype"]]
    if c["packed"]:
        q, k, _ = _rand(gen, (b, n, 3, h, d), dt).unbind(2)
    else:
        q, k = _rand(gen, (b, n, h, d), dt), _rand(gen, (b, n, g, d), dt)
    # each axis turns a run of the pairs, the frequencies falling off geometrically within the run
    freqs = torch.zeros((axes, pairs), dtype=F64)
    for a in range(axes):
        low, high = a * pairs // axes, (a + 1) * pairs // axes
        if high > low:
            freqs[a, low:high] = 10000.0 ** (-torch.arange(high - low, dtype=F64) / (high - low))
    s = {"case": c, "q": q, "k": k, "freqs": freqs.cuda(), "pos": None}
    if axes == 1 and not c["per_sample"]:
        return s                                   # the token's number, from `first` on
    shape = (b, n) if c["per_sample"] else (n,)
    i = torch.arange(n, device="cuda").expand(shape)
    if c["per_sample"]:
        # every sample begins elsewhere, and again from 0 at a document's end inside it
        begin = torch.randint(0, 100, (b, 1), generator=gen, device="cuda")
        cut = torch.randint(0, n + 1, (b, 1), generator=gen, device="cuda")
        i = torch.where(i < cut, i + begin, i - cut)
    i = i + c["first"]
    if axes > 1:
        side = max(1, math.isqrt(n))
        parts = [i // side, i % side, i % 7][:axes]
        i = torch.stack(parts, dim=-1)
    s["pos"] = i.to(torch.int32).contiguous()
    return s


def _prepare_dropout(c, gen, seed):
    t, d = c["rows"], c["cols"]

    def rows_of(dt, std):
        return _rand(gen, (t, d + c["pad"]), dt, std)[:, :d]
    s = {"case": c, "resid": None, "rng": (seed * 0x9E3779B1 + 5, seed)}
    if c["do"] == "fwd":
        s["x"] = rows_of(TYPES[c["act"]], 1.0)
        if c["resid"] != "none":
            s["resid"] = rows_of(TYPES[c["resid"]], 2.0)
    else:
        s["dy"] = rows_of(TYPES[c["act"] if c["resid"] == "none" else c["resid"]], 1e-1)
    return s


# ------------------------------------------------------------ a pass through
def run(state):
    c = state["case"]
    if own:
        return _own(c, state)
    return {"linearfwd": _linear_fwd, "linearbwd": _linear_bwd, "rotaryfwd": _rotate, "rotarybwd": _rotate,
            "dropoutfwd": _dropout_fwd, "dropoutbwd": _dropout_bwd}[c["op"] + c["do"]](state)


def _own(c, s):
    import matrix_aware_optimizer_periodic_amd as mm

    if c["op"] == "linear":
        how = {"act": c["act"], "p": c["p"], "rng": s["rng"] if c["p"] else None}
        if c["do"] == "fwd":
            return mm.linear_fwd(s["x"], s["w"], s["bias"], s["resid"], save=c["save"], **how)
        return mm.linear_bwd(s["dy"], s["x"], s["w"], s["bias"], s["z"], grad_dtype=TYPES[c["grad"]], **how)
    if c["op"] == "rotary":
        call = mm.rotary_fwd if c["do"] == "fwd" else mm.rotary_bwd
        return call(s["q"], s["k"], s["freqs"], s["pos"], offset=0 if s["pos"] is not None else c["first"],
                    interleaved=c["interleaved"], scale=c["scale"])
    if c["do"] == "fwd":
        return mm.dropout_fwd(s["x"], c["p"], s["rng"], s["resid"])
    return mm.dropout_bwd(s["dy"], c["p"], s["rng"], dtype=TYPES[c["act"]])


# ------------------------------------------------------------- plain forms
LOW = 0xFFFFFFFF


def _words(n, rng):
    """n 32-bit words of Philox4x32-10 as int64: word i % 4 of counter (i / 4, offset) under key seed."""
    seed, offset = rng
    i = torch.arange((n + 3) // 4, device="cuda", dtype=torch.int64)
    c0, c1 = i & LOW, i >> 32
    c2, c3 = torch.full_like(i, offset & LOW), torch.full_like(i, offset >> 32 & LOW)
    k0, k1 = seed & LOW, seed >> 32 & LOW
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57           # low 64 bits, as the words are below 2^32
        c0, c1, c2, c3 = (b >> 32 & LOW) ^ c1 ^ k0, b & LOW, (a >> 32 & LOW) ^ c3 ^ k1, a & LOW
        k0, k1 = k0 + 0x9E3779B9 & LOW, k1 + 0xBB67AE85 & LOW
    return torch.stack([c0, c1, c2, c3], dim=1).reshape(-1)[:n]


def _drop(x, p, rng):
    """x with dropped elements as zeros and the others over 1 - p."""
    if p == 0.0:
        return x
    keep = (_words(x.numel(), rng) >= round(p * 2 ** 32)).view(x.shape)
    return torch.where(keep, x * (1.0 / (1.0 - p)), 0.0)


def _act(z, kind):
    """The activation and its derivative; gelu in its tanh form."""
    if kind == "none":
        return z, torch.ones_like(z)
    if kind == "silu":
        e = 1.0 / (1.0 + torch.exp(-z))
        return z * e, e * (1.0 + z * (1.0 - e))
    a, b = math.sqrt(2.0 / math.pi), 0.044715
    t = torch.tanh(a * (z + b * z * z * z))
    return 0.5 * z * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * a * (1.0 + 3.0 * b * z * z)


def _linear_fwd(s):
    c = s["case"]
    z = s["x"].float() @ s["w"].float().T
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = z if c["act"] == "none" else _act(z, c["act"])[0]
    y = _drop(y, c["p"], s["rng"])
    if s["resid"] is not None:
        y = s["resid"].float() + y
    kept = z.to(BF16) if c["save"] and c["act"] != "none" else None
    return y.to(BF16 if s["resid"] is None else s["resid"].dtype), kept


def _linear_bwd(s):
    c = s["case"]
    dz = _drop(s["dy"].float(), c["p"], s["rng"])
    if s["z"] is not None:
        dz = dz * _act(s["z"].float(), c["act"])[1]
    db = None if s["bias"] is None else dz.sum(0).to(s["bias"].dtype)
    return (dz @ s["w"].float()).to(BF16), (dz.T @ s["x"].float()).to(TYPES[c["grad"]]), db


def _turned(x, cos, sin, c):
    """x (batch, len, heads, dim) with its first `rot` values rotated."""
    pairs = c["rot"] // 2
    x = x.float()
    out = x.clone()
    a, b = (slice(0, c["rot"], 2), slice(1, c["rot"], 2)) if c["interleaved"] else (slice(0, pairs), slice(pairs, c["rot"]))
    u, v = x[..., a], x[..., b]
    out[..., a] = u * cos - v * sin
    out[..., b] = v * cos + u * sin
    return out


def _rotate(s):
    c = s["case"]
    pos = s["pos"]
    if pos is None:
        pos = torch.arange(c["len"], device="cuda") + c["first"]
    pos = pos.to(F64)
    angle = pos[..., None] * s["freqs"][0] if c["axes"] == 1 else pos @ s["freqs"]
    if c["do"] == "bwd":
        angle = -angle
    cos, sin = ((f(angle).float() * c["scale"])[..., None, :] for f in (torch.cos, torch.sin))
    return tuple(_turned(t, cos, sin, c).to(t.dtype) for t in (s["q"], s["k"]))


def _dropout_fwd(s):
    x = s["x"]
    y = _drop(x.float(), s["case"]["p"], s["rng"])
    if s["resid"] is None:
        return y.to(x.dtype)
    return (s["resid"].float() + y).to(s["resid"].dtype)


def _dropout_bwd(s):
    c = s["case"]
    return _drop(s["dy"].float(), c["p"], s["rng"]).to(TYPES[c["act"]])


# -------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    width = {"none": 0, "bf16": 2, "f32": 4}
    if c["op"] == "linear":
        t, d, n = c["rows"], c["cols"], c["out"]
        stream = 2 if c["resid"] == "none" else width[c["resid"]]
        kept = 2 if c["act"] != "none" else 0
        if c["do"] == "fwd":
            kept = kept if c["save"] else 0
            return {"bytes": 2 * t * d + 2 * n * d + n * width[c["bias"]] + t * n * (stream + kept + width[c["resid"]]),
                    "flops": 2 * t * d * n}
        return {"bytes": 4 * t * d + (2 + width[c["grad"]]) * n * d + n * width[c["bias"]] + t * n * (stream + kept),
                "flops": 4 * t * d * n}
    if c["op"] == "rotary":
        e = c["batch"] * c["len"] * (c["heads"] + c["kv_heads"]) * c["dim"]
        places = 0 if c["axes"] == 1 and not c["per_sample"] else c["len"] * c["axes"] * (c["batch"] if c["per_sample"] else 1)
        return {"bytes": e * 2 * width[c["dtype"]] + 4 * places + 4 * c["axes"] * c["rot"], "flops": 3 * e}
    e = c["rows"] * c["cols"]
    out = width[c["act"] if c["resid"] == "none" else c["resid"]]
    return {"bytes": e * (width[c["act"]] + out + (width[c["resid"]] if c["do"] == "fwd" else 0)), "flops": 20 * e}


# --------------------------------------------------------- 64-bit definition
def exact(case, seed):
    s = prepare(case, seed)
    return {"linear": _exact_linear, "rotary": _exact_rotary, "dropout": _exact_dropout}[case["op"]](case, s)


def _mulhilo(x, m):
    """High and low words of x m from products of 16-bit halves."""
    x0, x1, m0, m1 = x % 65536, x // 65536, m % 65536, m // 65536
    low, mid = x0 * m0, x1 * m0 + x0 * m1
    total = low + mid % 65536 * 65536
    return (x1 * m1 + mid // 65536 + total // 2 ** 32) % 2 ** 32, total % 2 ** 32


def _kept(shape, p, rng):
    """Which elements stay, a round of the generator after the other on all counters."""
    n = math.prod(shape)
    blocks = -(-n // 4)
    first = torch.arange(blocks, device="cuda", dtype=torch.int64)
    ctr = [first % 2 ** 32, first // 2 ** 32] + [torch.full((blocks,), rng[1] // 2 ** (32 * j) % 2 ** 32, device="cuda")
                                                 for j in range(2)]
    key = [rng[0] // 2 ** (32 * j) % 2 ** 32 for j in range(2)]
    for turn in range(10):
        hi0, lo0 = _mulhilo(ctr[0], 0xD2511F53)
        hi1, lo1 = _mulhilo(ctr[2], 0xCD9E8D57)
        ctr = [hi1.bitwise_xor(ctr[1]).bitwise_xor((key[0] + turn * 0x9E3779B9) % 2 ** 32), lo1,
               hi0.bitwise_xor(ctr[3]).bitwise_xor((key[1] + turn * 0xBB67AE85) % 2 ** 32), lo0]
    word = torch.empty(blocks, 4, dtype=torch.int64, device="cuda")
    for j in range(4):
        word[:, j] = ctr[j]
    return ~(word.flatten()[:n] < round(p * 4294967296)).reshape(shape)


def _masked(x, c, rng):
    if c["p"] == 0:
        return x
    return (x / (1 - c["p"])).masked_fill(~_kept(x.shape, c["p"], rng), 0)


def _exact_linear(c, s):
    def acted(z):
        if c["act"] == "none":
            return z
        if c["act"] == "silu":
            return torch.nn.functional.silu(z)
        return torch.nn.functional.gelu(z, approximate="tanh")

    x, w = s["x"].double(), s["w"].double()
    if c["do"] == "fwd":
        z = torch.mm(x, w.t())
        if s["bias"] is not None:
            z += s["bias"].double()[None]
        y = _masked(acted(z), c, s["rng"])
        if s["resid"] is not None:
            y = y + s["resid"].double()
        return y, z if c["save"] and c["act"] != "none" else None
    dz = _masked(s["dy"].double(), c, s["rng"])
    if c["act"] != "none":
        leaf = s["z"].double().requires_grad_(True)
        dz, = torch.autograd.grad(acted(leaf), leaf, dz)
    return torch.mm(dz, w), torch.mm(dz.t(), x), None if s["bias"] is None else dz.sum(dim=0)


def _exact_rotary(c, s):
    b, n = c["batch"], c["len"]
    places = torch.zeros((b, n, c["axes"]), dtype=F64, device="cuda")
    if s["pos"] is None:
        places += torch.arange(c["first"], c["first"] + n, device="cuda")[None, :, None]
    else:
        places += s["pos"].double().reshape((b if c["per_sample"] else 1), n, c["axes"])
    phase = sum(places[:, :, a, None] * s["freqs"][a] for a in range(c["axes"]))
    turn = torch.polar(torch.full_like(phase, c["scale"]), phase if c["do"] == "fwd" else -phase)[:, :, None, :]
    out = []
    for t in (s["q"], s["k"]):
        t = t.double()
        head, rest = t[..., :c["rot"]], t[..., c["rot"]:]
        if c["interleaved"]:
            z = torch.view_as_complex(head.unflatten(-1, (-1, 2)).contiguous()) * turn
            head = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(*head.chunk(2, dim=-1)) * turn
            head = torch.cat([z.real, z.imag], dim=-1)
        out.append(torch.cat([head, rest], dim=-1))
    return tuple(out)


def _exact_dropout(c, s):
    if c["do"] == "bwd":
        return _masked(s["dy"].double(), c, s["rng"])
    y = _masked(s["x"].double(), c, s["rng"])
    return y if s["resid"] is None else y + s["resid"].double()
