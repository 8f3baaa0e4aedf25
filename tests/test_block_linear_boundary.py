"""The linear, rotary and dropout operators' C ABI and bindings on the CPU: packed
structures against the header, every bad argument's status before anything is
enqueued, workspace sizes, sizes at the limits, and the Python calls' checks and
autograd functions with stand-ins for the library.  Nothing here launches a
kernel."""

import ctypes
import os
import shutil
import subprocess

import pytest
import torch

m = pytest.importorskip("matrix_aware_optimizer_periodic_amd")
from matrix_aware_optimizer_periodic_amd import binding as bd  # noqa: E402
from matrix_aware_optimizer_periodic_amd import block as b  # noqa: E402
from test_block_boundary import FAKE, NONE, ROOT, heads, mat, need, needs_lib  # noqa: E402

E = bd


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_packed_structures_match_the_header(tmp_path):
    src = tmp_path / "s.cpp"
    fields = {"muon_linear_args": ("act", "p", "rng", "x", "bias", "z", "d_bias"),
              "muon_dropout_args": ("p", "rng", "x", "y"),
              "muon_rotary_args": ("heads", "dtype", "scale", "offset", "freqs", "positions_batch", "q", "k_out")}
    say = "".join(f'printf("%zu ", sizeof({s}));' + "".join(f'printf("%zu ", offsetof({s}, {f}));' for f in names)
                  for s, names in fields.items())
    src.write_text('#include "muon_block.h"\n#include <cstdio>\nint main() { ' + say + " }\n")
    exe = tmp_path / "s"
    subprocess.run(["g++", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    size = {"linear": b.LINEAR_ARGS.size, "dropout": b.DROPOUT_ARGS.size, "rotary": b.ROTARY_ARGS.size}
    mats = 64
    assert got == [size["linear"], 24, 32, 40, mats, mats + 80, mats + 200, mats + 360,
                   size["dropout"], 16, 24, 48, 128,
                   size["rotary"], 16, 44, 48, 56, 64, 80, 88, 184]


# ------------------------------------------------------------------- linear
def linear_args(**over):
    """Arguments of a valid backward call (which hold the forward's too)."""
    v = dict(rows=40, cols=64, out=96, act=1, reserved=0, p=0.1, seed=1, offset=2, state=0, x=mat(40, 64), weight=mat(96, 64),
             bias=mat(1, 96, 0), residual=mat(40, 96, 0), y=mat(40, 96, 0), z=mat(40, 96), d_y=mat(40, 96, 0),
             d_x=mat(40, 64), d_weight=mat(96, 64, 0), d_bias=mat(1, 96, 0))
    v.update(over)
    order = ("x", "weight", "bias", "residual", "y", "z", "d_y", "d_x", "d_weight", "d_bias")
    return b.LINEAR_ARGS.pack(*(v[k] for k in ("rows", "cols", "out", "act", "reserved", "p", "seed", "offset", "state")),
                              *sum((v[k] for k in order), []))


@needs_lib
@pytest.mark.parametrize("over,status", [
    (dict(rows=-1), E.MUON_E_SHAPE), (dict(rows=(1 << 30) + 1), E.MUON_E_SHAPE), (dict(cols=60), E.MUON_E_SHAPE),
    (dict(out=0), E.MUON_E_SHAPE), (dict(out=(1 << 20) + 8), E.MUON_E_SHAPE), (dict(act=3), E.MUON_E_ARG),
    (dict(act=-1), E.MUON_E_ARG), (dict(reserved=1), E.MUON_E_ARG), (dict(p=-0.1), E.MUON_E_ARG), (dict(p=1.1), E.MUON_E_ARG),
    (dict(p=float("nan")), E.MUON_E_ARG), (dict(state=FAKE + 4), E.MUON_E_ALIGN),
    (dict(x=NONE), E.MUON_E_ARG), (dict(x=mat(41, 64)), E.MUON_E_SHAPE), (dict(x=mat(40, 64, 0)), E.MUON_E_DTYPE),
    (dict(x=mat(40, 64, ld=66)), E.MUON_E_ALIGN), (dict(x=mat(40, 64, ptr=FAKE + 8)), E.MUON_E_ALIGN),
    (dict(x=mat(40, 64, ld=(1 << 22) + 8)), E.MUON_E_ALIGN), (dict(weight=mat(64, 96)), E.MUON_E_SHAPE),
    (dict(weight=NONE), E.MUON_E_ARG), (dict(z=mat(40, 96, 0)), E.MUON_E_DTYPE), (dict(z=mat(40, 64)), E.MUON_E_SHAPE),
])
def test_linear_refuses_both_ways(over, status):
    args = linear_args(**over)
    assert b._lib().muon_linear_fwd(args, FAKE, 1 << 40, None) == status
    assert b._lib().muon_linear_bwd(args, FAKE, 1 << 40, None) == status
    assert b._lib().muon_block_last_error()


@needs_lib
@pytest.mark.parametrize("over,status", [
    (dict(bias=mat(1, 97, 0)), E.MUON_E_SHAPE), (dict(bias=mat(1, 96, 2)), E.MUON_E_DTYPE),
    (dict(bias=mat(1, 96, 0, ptr=FAKE + 2)), E.MUON_E_ALIGN), (dict(residual=mat(40, 96, 1)), E.MUON_E_DTYPE),
    (dict(residual=mat(40, 96, 0, ptr=FAKE + 4)), E.MUON_E_ALIGN), (dict(residual=mat(40, 95, 0)), E.MUON_E_SHAPE),
    (dict(y=NONE), E.MUON_E_ARG), (dict(y=mat(40, 96, 0, ld=98)), E.MUON_E_ALIGN), (dict(y=mat(40, 96, 3)), E.MUON_E_DTYPE),
])
def test_linear_fwd_refuses(over, status):
    assert b._lib().muon_linear_fwd(linear_args(**over), FAKE, 1 << 40, None) == status


@needs_lib
@pytest.mark.parametrize("over,status", [
    (dict(rows=0), E.MUON_E_SHAPE), (dict(d_y=NONE), E.MUON_E_ARG), (dict(d_y=mat(40, 96, 0, ld=97)), E.MUON_E_ALIGN),
    (dict(z=NONE), E.MUON_E_ARG), (dict(d_x=mat(40, 64, 0)), E.MUON_E_DTYPE), (dict(d_weight=mat(64, 96)), E.MUON_E_SHAPE),
    (dict(d_weight=mat(96, 64, 0, ptr=FAKE + 4)), E.MUON_E_ALIGN), (dict(d_bias=mat(1, 64)), E.MUON_E_SHAPE),
    (dict(d_bias=mat(1, 96, 5)), E.MUON_E_DTYPE),
])
def test_linear_bwd_refuses(over, status):
    assert b._lib().muon_linear_bwd(linear_args(**over), FAKE, 1 << 40, None) == status


@needs_lib
def test_linear_workspace():
    L = b._lib()
    big = dict(rows=700, x=mat(700, 64), z=mat(700, 96), d_y=mat(700, 96, 0), d_x=mat(700, 64))
    st, n = need("muon_linear_bwd", linear_args(**big))
    assert st == E.MUON_OK and n >= 700 * 96 * 2
    assert L.muon_linear_bwd(linear_args(**big), FAKE, n - 1, None) == E.MUON_E_WORKSPACE
    assert L.muon_linear_bwd(linear_args(**big), None, n, None) == E.MUON_E_WORKSPACE
    assert L.muon_linear_bwd(linear_args(**big), FAKE + 16, n, None) == E.MUON_E_ALIGN
    assert need("muon_linear_bwd", linear_args()) == (E.MUON_OK, 0)      # a small call forms dz where it is used
    # dz is dy itself: bf16, no activation, no dropout
    same = dict(act=2, p=0.0, d_y=mat(700, 96), d_bias=NONE, d_weight=NONE, d_x=NONE)
    assert need("muon_linear_bwd", linear_args(**dict(big, **same))) == (E.MUON_OK, 0)
    assert L.muon_linear_bwd(linear_args(**same), None, 0, None) == E.MUON_OK       # nothing is wanted
    assert L.muon_linear_fwd(linear_args(rows=0), None, 0, None) == E.MUON_OK
    assert L.muon_linear_bwd(linear_args(rows=0, d_weight=NONE, d_bias=NONE), None, 0, None) == E.MUON_OK
    # one row tile over a long sum is divided and needs room
    st, n = need("muon_linear_fwd", linear_args(rows=100, cols=8192, out=128))
    assert st == E.MUON_OK and n > 0
    for name in ("muon_linear_fwd", "muon_linear_bwd"):
        assert getattr(L, name + "_workspace")(linear_args(), None) == E.MUON_E_ARG


@needs_lib
@pytest.mark.parametrize("rows,cols,out,fits", [
    (1 << 30, 8, 8, True), (1 << 30, 128, 128, True), (1 << 30, 256, 8, False), (1 << 30, 8, 256, False),
    (128, 1 << 20, 1 << 17, True), (128, 1 << 20, 1 << 18, False), (128, 1 << 20, 1 << 20, False),
])
def test_linear_limits(rows, cols, out, fits):
    for name in ("muon_linear_fwd", "muon_linear_bwd"):
        st, n = need(name, linear_args(rows=rows, cols=cols, out=out))
        assert st == (E.MUON_OK if fits else E.MUON_E_SHAPE), name


# ------------------------------------------------------------------ dropout
def dropout_args(**over):
    v = dict(rows=10, cols=33, p=0.5, seed=1, offset=0, state=0, x=mat(10, 33), residual=mat(10, 33, 0), y=mat(10, 33, 0))
    v.update(over)
    return b.DROPOUT_ARGS.pack(*(v[k] for k in ("rows", "cols", "p", "seed", "offset", "state")), *v["x"], *v["residual"],
                               *v["y"])


@needs_lib
@pytest.mark.parametrize("over,status", [
    (dict(rows=-1), E.MUON_E_SHAPE), (dict(cols=-1), E.MUON_E_SHAPE), (dict(cols=(1 << 40) + 1), E.MUON_E_SHAPE),
    (dict(rows=1 << 30, cols=1 << 30), E.MUON_E_SHAPE), (dict(p=-1e-9), E.MUON_E_ARG), (dict(p=1.0001), E.MUON_E_ARG),
    (dict(p=float("nan")), E.MUON_E_ARG), (dict(state=FAKE + 1), E.MUON_E_ALIGN), (dict(x=NONE), E.MUON_E_ARG),
    (dict(x=mat(10, 32)), E.MUON_E_SHAPE), (dict(x=mat(10, 33, 2)), E.MUON_E_DTYPE), (dict(x=mat(10, 33, ld=32)), E.MUON_E_ALIGN),
    (dict(x=mat(10, 33, ptr=FAKE + 1)), E.MUON_E_ALIGN), (dict(y=NONE), E.MUON_E_ARG),
    (dict(residual=mat(10, 33, 1)), E.MUON_E_DTYPE), (dict(residual=mat(9, 33, 0)), E.MUON_E_SHAPE),
    (dict(rows=0), E.MUON_OK), (dict(cols=0), E.MUON_OK),
])
def test_dropout_refuses(over, status):
    assert b._lib().muon_dropout(dropout_args(**over), None) == status


# ------------------------------------------------------------------- rotary
def rotary_args(**over):
    v = dict(batch=2, len=10, heads=4, kv_heads=2, dim=64, pairs=32, axes=1, interleaved=0, inverse=0, dtype=1, scale=1.0,
             reserved=0, offset=0, freqs=FAKE, positions=FAKE, between=0, q=heads(), k=heads(), q_out=heads(), k_out=heads(ptr=2 * FAKE))
    v.update(over)
    return b.ROTARY_ARGS.pack(*(v[k] for k in ("batch", "len", "heads", "kv_heads", "dim", "pairs", "axes", "interleaved",
                                               "inverse", "dtype", "scale", "reserved", "offset", "freqs", "positions",
                                               "between")), *v["q"], *v["k"], *v["q_out"], *v["k_out"])


@needs_lib
@pytest.mark.parametrize("over,status", [
    (dict(batch=-1), E.MUON_E_SHAPE), (dict(len=-1), E.MUON_E_SHAPE), (dict(batch=1 << 16, len=1 << 15), E.MUON_E_SHAPE),
    (dict(batch=1 << 62, len=4), E.MUON_E_SHAPE), (dict(heads=0), E.MUON_E_SHAPE), (dict(kv_heads=-1), E.MUON_E_SHAPE),
    (dict(heads=1 << 16), E.MUON_E_SHAPE), (dict(dim=63), E.MUON_E_SHAPE), (dict(dim=1026), E.MUON_E_SHAPE),
    (dict(dim=0), E.MUON_E_SHAPE), (dict(pairs=0), E.MUON_E_SHAPE), (dict(pairs=33), E.MUON_E_SHAPE),
    (dict(axes=0), E.MUON_E_ARG), (dict(axes=9), E.MUON_E_ARG), (dict(axes=2, positions=0), E.MUON_E_ARG),
    (dict(interleaved=2), E.MUON_E_ARG), (dict(inverse=-1), E.MUON_E_ARG), (dict(dtype=2), E.MUON_E_DTYPE),
    (dict(scale=float("inf")), E.MUON_E_ARG), (dict(reserved=1), E.MUON_E_ARG), (dict(offset=1 << 53), E.MUON_E_ARG),
    (dict(freqs=0), E.MUON_E_ARG), (dict(freqs=FAKE + 4), E.MUON_E_ALIGN), (dict(positions=FAKE + 2), E.MUON_E_ALIGN),
    (dict(between=-1), E.MUON_E_SHAPE), (dict(q=heads(ptr=0)), E.MUON_E_ARG), (dict(k=heads(ptr=0)), E.MUON_E_ARG),
    (dict(q_out=heads(ptr=0)), E.MUON_E_ARG), (dict(k_out=heads(ptr=0)), E.MUON_E_ARG),
    (dict(q=heads(ptr=FAKE + 1)), E.MUON_E_ALIGN), (dict(k=heads(sl=-8)), E.MUON_E_SHAPE),
    (dict(q_out=heads(sb=(1 << 40) + 8)), E.MUON_E_SHAPE), (dict(k_out=heads()), E.MUON_E_ARG), (dict(batch=0), E.MUON_OK), (dict(len=0), E.MUON_OK),
])
def test_rotary_refuses(over, status):
    assert b._lib().muon_rotary(rotary_args(**over), None) == status


# ------------------------------------------------------------- Python checks
def test_cpu_tensors_are_refused():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        m.linear_fwd(x, x)
    with pytest.raises(ValueError, match="GPU"):
        m.linear_bwd(x, x, x)
    with pytest.raises(ValueError, match="GPU"):
        m.dropout_fwd(x, 0.5, (1, 2))
    with pytest.raises(ValueError, match="GPU"):
        m.rotary_fwd(x.view(1, 4, 1, 64), None, m.rotary_freqs(64, device="cpu"))


@pytest.fixture
def packed(monkeypatch):
    """The calls' structures, taken in place of the library's call, from tensors
    on the CPU."""
    calls = []
    monkeypatch.setattr(b, "_device", lambda first, *others: first.device)
    monkeypatch.setattr(b, "_call", lambda name, args, dev, workspace=True: calls.append((name, args)))
    return calls


BF16, F32 = torch.bfloat16, torch.float32


def test_linear_checks_its_arguments(packed):
    x, w = torch.zeros(6, 64, dtype=BF16), torch.zeros(96, 64, dtype=BF16)
    bias, res, dy, z = torch.zeros(96), torch.zeros(6, 96), torch.zeros(6, 96), torch.zeros(6, 96, dtype=BF16)
    bad = [lambda: m.linear_fwd(x, w, act="relu"), lambda: m.linear_fwd(x, w.T), lambda: m.linear_fwd(x.float(), w),
           lambda: m.linear_fwd(x, w.float()), lambda: m.linear_fwd(x, w, bias[:95]), lambda: m.linear_fwd(x, w, bias[None]),
           lambda: m.linear_fwd(x, w, None, res[:5]), lambda: m.linear_fwd(x, w, None, res, y_dtype=BF16),
           lambda: m.linear_fwd(x, w, None, res.expand(2, 6, 96)), lambda: m.linear_fwd(x, w, y_dtype=torch.float16),
           lambda: m.linear_fwd(x, w, p=0.5), lambda: m.linear_fwd(x, w, p=1.5, rng=(1, 2)),
           lambda: m.linear_fwd(x, w, p=0.5, rng=(1, -2)), lambda: m.linear_fwd(x, w, p=0.5, rng=(1 << 64, 0)),
           lambda: m.linear_fwd(x, w, p=0.5, rng=torch.zeros(3, dtype=torch.int64)),
           lambda: m.linear_fwd(x, w, p=0.5, rng=torch.zeros(2, dtype=torch.int32)),
           lambda: m.linear_fwd(x.T, w), lambda: m.linear_fwd(x, w[0]), lambda: m.linear_fwd(x[0, 0], w),
           lambda: m.linear_fwd(x, w, bias.half()), lambda: m.linear_fwd(x, w, None, res.half()),
           lambda: m.linear_bwd(dy[:5], x, w), lambda: m.linear_bwd(dy, None, w), lambda: m.linear_bwd(dy, x, w, act="silu"),
           lambda: m.linear_bwd(dy, x, w, grad_dtype=torch.float16), lambda: m.linear_bwd(dy, x, w, None, z[:5], act="gelu"),
           lambda: m.linear_bwd(dy[:, :95], x, w), lambda: m.linear_bwd(dy, x, w, p=0.5)]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            call()
        assert not packed, i
    y, kept = m.linear_fwd(x, w, bias, res, act="gelu", p=0.5, rng=(3, 4))
    assert y.dtype == F32 and kept.shape == (6, 96) and packed[0][0] == "muon_linear_fwd"
    got = b.LINEAR_ARGS.unpack(packed[0][1])
    assert got[:9] == (6, 64, 96, 1, 0, 0.5, 3, 4, 0)
    assert got[9] == x.data_ptr() and got[15] == w.data_ptr() and got[21] == bias.data_ptr() and got[27] == res.data_ptr()
    assert got[33] == y.data_ptr() and got[39] == kept.data_ptr() and not any(got[45:])
    state = torch.tensor([5, 6])
    m.linear_bwd(dy, None, w, None, z, act="silu", p=0.25, rng=state, need_weight=False)
    got = b.LINEAR_ARGS.unpack(packed[1][1])
    assert got[3:9] == (0, 0, 0.25, 0, 0, state.data_ptr()) and got[9] == 0 and got[39] == z.data_ptr() and got[57] == 0


def test_dropout_checks_its_arguments(packed):
    x = torch.zeros(6, 40)
    for call in (lambda: m.dropout_fwd(x, 0.5), lambda: m.dropout_fwd(x, 2.0, (1, 2)), lambda: m.dropout_fwd(x, 0.5, (1, 2), x[:5]),
                 lambda: m.dropout_fwd(x.half(), 0.5, (1, 2)), lambda: m.dropout_fwd(x.T, 0.5, (1, 2)),
                 lambda: m.dropout_fwd(x[0, 0], 0.5, (1, 2)), lambda: m.dropout_bwd(x, 0.5, (1, 2), dtype=torch.float16),
                 lambda: m.dropout_fwd(x, float("nan"), (1, 2))):
        with pytest.raises((ValueError, TypeError)):
            call()
    assert not packed
    y = m.dropout_fwd(x[:, :20], 0.5, (2 ** 64 - 1, 7), x[:, 20:].to(BF16))
    assert y.dtype == BF16 and b.DROPOUT_ARGS.unpack(packed[0][1])[:10] == (6, 20, 0.5, 2 ** 64 - 1, 7, 0, x.data_ptr(), 6, 20, 40)


def test_rotary_checks_its_arguments(packed):
    q, k = torch.zeros(2, 5, 4, 16), torch.zeros(2, 5, 2, 16)
    f, f2 = torch.zeros(1, 8, dtype=torch.float64), torch.zeros(2, 8, dtype=torch.float64)
    pos = torch.zeros(2, 5, dtype=torch.int32)
    bad = [lambda: m.rotary_fwd(q[0], None, f), lambda: m.rotary_fwd(q, k[:1], f), lambda: m.rotary_fwd(q, k[..., :8], f),
           lambda: m.rotary_fwd(q, k.to(BF16), f), lambda: m.rotary_fwd(q.half(), None, f), lambda: m.rotary_fwd(q, k, f.float()),
           lambda: m.rotary_fwd(q, k, f[0]), lambda: m.rotary_fwd(q, k, f, pos.long()), lambda: m.rotary_fwd(q, k, f, pos[:1]),
           lambda: m.rotary_fwd(q, k, f2, pos), lambda: m.rotary_fwd(q, k, f, pos, offset=1),
           lambda: m.rotary_fwd(q, k, f, pos.T.contiguous().T), lambda: m.rotary_fwd(q, k, f, out=(q,)),
           lambda: m.rotary_fwd(q, k, f, out=(q, q)), lambda: m.rotary_fwd(q, k, f, out=(q, None)),
           lambda: m.rotary_fwd(q, k, f, out=(q.to(BF16), k)), lambda: m.rotary_fwd(q.transpose(2, 3), None, f),
           lambda: m.rotary_fwd(q, k, f, out=(q, k[:, :, :1].expand(-1, -1, 2, -1))),
           lambda: m.rotary_fwd(q, q, f, out=(q, q)),
           lambda: m.attention_qkv(torch.zeros(2, 5, 3, 4, 16), rotary={"freqs": f, "out": (q, q)})]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            call()
        assert not packed, i
    saved = (q.clone().requires_grad_(True) * q).sum()
    m.rotary_fwd(q, None, f, out=(q, None))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        saved.backward()
    packed.clear()
    m.rotary_fwd(q, k, f, pos, interleaved=True, scale=0.5)
    m.rotary_bwd(q, None, f2, torch.zeros(5, 2, dtype=torch.int32))
    first, second = (b.ROTARY_ARGS.unpack(a) for _, a in packed)
    assert first[:13] == (2, 5, 4, 2, 16, 8, 1, 1, 0, 0, 0.5, 0, 0) and first[15] == 5 and first[16:20] == (q.data_ptr(), 320, 64, 16)
    assert second[:13] == (2, 5, 4, 0, 16, 8, 2, 0, 1, 0, 1.0, 0, 0) and second[15] == 0 and second[20:24] == (0,) * 4


# ---------------------------------------------------------- autograd functions
@pytest.fixture
def stand_ins(monkeypatch):
    """The plain formulas, outside autograd as the library's results are."""
    calls = []

    def outside(name, f):
        def call(*args, **how):
            calls.append((name, how))
            with torch.no_grad():
                return f(*args, **how)
        monkeypatch.setattr(b, name, call)

    def linear_fwd(x, w, bias=None, residual=None, act="none", p=0.0, rng=None, save=True, y_dtype=None):
        z = x @ w.T + (0 if bias is None else bias)
        return z + (0 if residual is None else residual), z if save and act != "none" else None

    def linear_bwd(dy, x, w, bias=None, z=None, act="none", p=0.0, rng=None, need_x=True, need_weight=True):
        return dy @ w if need_x else None, dy.T @ x if need_weight else None, None if bias is None else dy.sum(0)
    outside("linear_fwd", linear_fwd)
    outside("linear_bwd", linear_bwd)
    outside("dropout_fwd", lambda x, p, rng, residual=None: x * 2 + (0 if residual is None else residual))
    outside("dropout_bwd", lambda d, p, rng, dtype=None: d * 2)
    outside("rotary_fwd", lambda q, k, freqs=None, positions=None, **how: (q * 3, None if k is None else k * 3))

    def rotary_bwd(q, k, f, pos=None, out=None, **how):
        got = (q * 3, None if k is None else k * 3)
        for t, g in zip(out or (), got):
            t.copy_(g)
        return out or got
    outside("rotary_bwd", rotary_bwd)

    def soft(q, k, v):
        return torch.einsum("bhmn,bnhd->bmhd", torch.softmax(torch.einsum("bmhd,bnhd->bhmn", q, k), -1), v)

    def attn_bwd(d_o, q, k, v, o, lse, out=None, **how):
        with torch.enable_grad():
            leaves = [t.detach().clone().requires_grad_(True) for t in (q, k, v)]
            for t, g in zip(out, torch.autograd.grad(soft(*leaves), leaves, d_o)):
                t.copy_(g)
        return out
    outside("attn_fwd", lambda q, k, v, **how: (soft(q, k, v), torch.zeros(1)))
    outside("attn_bwd", attn_bwd)
    return calls


def leaves(*shapes):
    gen = torch.Generator().manual_seed(0)
    return [torch.randn(s, generator=gen, dtype=torch.float64).requires_grad_(True) for s in shapes]


def through_linear():
    t = leaves((3, 8), (16, 8), (16,), (3, 16))
    return t, b.linear(*t, act="silu", p=0.5, rng=(1, 2))


def through_dropout():
    t = leaves((3, 8), (3, 8))
    return t, b.dropout(t[0], 0.5, (1, 2), t[1])


def through_rotary():
    t = leaves((2, 3, 2, 8), (2, 3, 1, 8))
    q, k = b.rotary(*t, torch.zeros(1, 4))
    return t, torch.cat([q, k], 2)


@pytest.mark.parametrize("through", [through_linear, through_dropout, through_rotary])
def test_gradients_once(stand_ins, through):
    inputs, y = through()
    first = torch.autograd.grad(y.square().sum(), inputs, create_graph=True)
    assert all(bool((g != 0).any()) for g in first)
    penalty = sum(g.square().sum() for g in first) + sum(t.square().sum() for t in inputs)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        penalty.backward()


def test_only_what_is_needed_is_asked_for(stand_ins):
    x, w, bias, res = leaves((3, 8), (16, 8), (16,), (3, 16))

    def asked(*given):
        stand_ins.clear()
        y = b.linear(*given, act="gelu")
        y.sum().backward()
        return [h for n, h in stand_ins if n == "linear_bwd"]
    how, = asked(x, w.detach(), bias.detach(), None)
    assert how["need_x"] and not how["need_weight"]
    how, = asked(x.detach(), w, bias, None)
    assert not how["need_x"] and how["need_weight"]
    assert asked(x.detach(), w.detach(), None, res) == []
    assert torch.equal(res.grad, torch.ones(3, 16, dtype=torch.float64))
    for off in (torch.no_grad, torch.inference_mode):
        with off():
            stand_ins.clear()
            b.linear(x, w, act="gelu")
            assert stand_ins[0][1]["save"] is False


@pytest.mark.parametrize("which", ["linear", "dropout", "rotary", "positions", "packed"])
def test_what_is_written_between_the_passes_is_noticed(stand_ins, which):
    """Numbers, positions or frequencies refilled for the next batch before the
    backward pass would give gradients of another mask or rotation."""
    state, f, pos = torch.tensor([1, 2]), torch.zeros(1, 4), torch.zeros(3, dtype=torch.int32)

    def forward():
        if which == "linear":
            return b.linear(*leaves((3, 8), (16, 8)), p=0.5, rng=state)
        if which == "dropout":
            return b.dropout(*leaves((3, 8)), 0.5, state)
        if which == "packed":
            return b.attention_qkv(*leaves((2, 3, 3, 2, 8)), rotary={"freqs": f, "positions": pos})
        return b.rotary(*leaves((2, 3, 2, 8)), None, f, pos)[0]
    y = forward()
    {"linear": state, "dropout": state, "rotary": f}.get(which, pos).add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    forward().sum().backward()


def test_packed_attention_over_rotated(stand_ins):
    """The packed gradient is what rotary and attention apart give; rotary's
    arguments reach both of its calls."""
    qkv, = leaves((2, 4, 3, 2, 8))
    w = torch.randn(2, 4, 2, 8, dtype=torch.float64)
    f, pos = torch.zeros(1, 4), torch.zeros(4, dtype=torch.int32)
    how = {"offset": 0, "interleaved": True, "scale": 1.5}
    b.attention_qkv(qkv, rotary={"freqs": f, "positions": pos, **how}).backward(w)
    assert [h for n, h in stand_ins if n == "rotary_fwd"] == [{"freqs": f, "positions": pos, **how}]
    back, = [h for n, h in stand_ins if n == "rotary_bwd"]
    assert {n: back[n] for n in how} == how
    q, k, v = (t.detach().clone().requires_grad_(True) for t in qkv.unbind(2))
    s = torch.softmax(torch.einsum("bmhd,bnhd->bhmn", q * 3, k * 3), -1)
    torch.einsum("bhmn,bnhd->bmhd", s, v).backward(w)
    for i, t in enumerate((q, k, v)):
        assert torch.allclose(qkv.grad[:, :, i], t.grad)


def test_names_are_reached_through_the_package():
    for n in ("linear_fwd", "linear_bwd", "linear", "rotary_freqs", "rotary_fwd", "rotary_bwd", "rotary", "dropout_fwd",
              "dropout_bwd", "dropout"):
        assert callable(getattr(m, n))
