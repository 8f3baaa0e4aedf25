"""PyTorch entry points of the transformer-block operators declared in
include/muon_block.h: the fused residual norm, softmax attention, the gated
feed-forward block, linear layers with their epilogue, rotary positions and
dropout.

``norm_fwd`` / ``norm_bwd``, ``attn_fwd`` / ``attn_bwd``, ``ffn_fwd`` /
``ffn_bwd``, ``linear_fwd`` / ``linear_bwd``, ``rotary_fwd`` / ``rotary_bwd`` and
``dropout_fwd`` / ``dropout_bwd`` are one call of the library each: they check devices, types and
shapes, take outputs and workspace from PyTorch's allocator and enqueue the
kernels on the current stream of the tensors' device.  Nothing is copied or
made contiguous behind the caller's back: a layout that the kernels cannot
read raises.  Tensors made on another stream need the caller's wait (and
``record_stream``), as with PyTorch's own operators.  All of them may be
captured into a HIP graph.

``residual_norm``, ``attention``, ``gated_ffn``, ``linear``, ``rotary`` and
``dropout`` wrap them for autograd, once:
gradients of their gradients raise.  To capture a training step into a graph,
call the forward and backward functions themselves: an autograd graph that
shares leaves with a captured backward pass must not be alive during the
capture.
"""

from __future__ import annotations

import ctypes
import operator
import struct

import torch
from torch.autograd.function import once_differentiable

from .binding import MUON_OK, MuonError, lib

NORM_KINDS = {"none": 0, "rms": 1, "layer": 2}
ACTS = {"silu": 0, "gelu": 1}
LINEAR_ACTS = {**ACTS, "none": 2}
BLOCK_EXPORTED = ("muon_block_last_error", "muon_norm_fwd", "muon_norm_bwd_workspace", "muon_norm_bwd",
                  "muon_attn_fwd_workspace", "muon_attn_fwd", "muon_attn_bwd_workspace", "muon_attn_bwd",
                  "muon_ffn_fwd_workspace", "muon_ffn_fwd", "muon_ffn_bwd_workspace", "muon_ffn_bwd",
                  "muon_linear_fwd_workspace", "muon_linear_fwd", "muon_linear_bwd_workspace", "muon_linear_bwd",
                  "muon_rotary", "muon_dropout")
_NO_WORKSPACE = ("muon_norm_fwd", "muon_rotary", "muon_dropout")

_TYPES = {torch.float32: 0, torch.bfloat16: 1}
# The argument structures of muon_block.h, packed field by field (a few
# microseconds where a ctypes.Structure of some 120 fields takes ten times that).
_MAT, _HEADS, _RNG = "Pqqqii", "Pqqq", "QQP"
NORM_ARGS = struct.Struct("@qqqiiff" + 9 * _MAT + "P" + 9 * _MAT)
ATTN_ARGS = struct.Struct("@qqqiiiiqfiPP" + 4 * _HEADS + "P" + 4 * _HEADS)
FFN_ARGS = struct.Struct("@qqqii" + 11 * _MAT)
LINEAR_ARGS = struct.Struct("@qqqiid" + _RNG + 10 * _MAT)
LINEAR_FWD_ARGS = struct.Struct("@qqqiid" + _RNG + 6 * _MAT)      # what comes before the backward call's own
_NO_LINEAR_BWD = bytes(LINEAR_ARGS.size - LINEAR_FWD_ARGS.size)
DROPOUT_ARGS = struct.Struct("@qqd" + _RNG + 3 * _MAT)
ROTARY_ARGS = struct.Struct("@qqiiiiiiiifiqPPq" + 4 * _HEADS)
_NO_MAT, _NO_HEADS, _NO_RNG = (0,) * 6, (0,) * 4, (0,) * 3

_READY = None


def _lib():
    global _READY
    if _READY is None:
        L = lib()
        L.muon_block_last_error.restype = ctypes.c_char_p
        void, size = ctypes.c_void_p, ctypes.c_size_t
        for name in BLOCK_EXPORTED[1:]:
            f = getattr(L, name)
            f.restype = ctypes.c_int
            if name.endswith("_workspace"):
                f.argtypes = [ctypes.c_char_p, ctypes.POINTER(size)]
            elif name in _NO_WORKSPACE:
                f.argtypes = [ctypes.c_char_p, void]
            else:
                f.argtypes = [ctypes.c_char_p, void, size, void]
        _READY = L
    return _READY


def _check(status: int) -> None:
    if status != MUON_OK:
        raise MuonError(status, _lib().muon_block_last_error().decode())


def _stream(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


# The handle of the current stream without the Python object around it (2 us
# of a call's 15), where this torch has it.
_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call(name: str, args: bytes, device, workspace: bool = True) -> None:
    L = _READY or _lib()
    index = device.index
    if index != _current_device():
        with torch.cuda.device(device):
            return _call(name, args, device, workspace)
    if not workspace:
        status = getattr(L, name)(args, _stream(index))
    else:
        need = ctypes.c_size_t(0)
        _check(getattr(L, name + "_workspace")(args, need))
        if need.value:
            ws = torch.empty(need.value, dtype=torch.uint8, device=device)
            status = getattr(L, name)(args, ws.data_ptr(), need.value, _stream(index))
        else:
            status = getattr(L, name)(args, None, 0, _stream(index))
    if status != MUON_OK:
        _check(status)


def _device(first, *others):
    """The device that all the tensors are on; they may be None."""
    d = first.device
    if d.type != "cuda":
        raise ValueError("tensors must be on a GPU")
    for t in others:
        if t is not None and t.device != d:
            raise ValueError(f"tensors on {d} and {t.device}")
    return d


def _out(t):
    """A contiguous tensor of t's shape, type and device."""
    return torch.empty_like(t) if t.is_contiguous() else torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _mat(t, rows: int, cols: int):
    """Descriptor of a tensor as rows x cols: its last dimension contiguous,
    the others one run of evenly spaced rows."""
    if t is None:
        return _NO_MAT
    dt = _TYPES.get(t.dtype)
    if dt is None:
        raise TypeError(f"unsupported dtype {t.dtype}")
    if t.is_contiguous():
        if t.numel() != rows * cols or t.shape[-1] != cols:
            raise ValueError(f"shape {tuple(t.shape)} where {rows} x {cols} is wanted")
        return t.data_ptr(), rows, cols, cols, dt, 0
    shape, stride = t.shape, t.stride()
    if t.numel() != rows * cols or shape[-1] != cols:
        raise ValueError(f"shape {tuple(shape)} where {rows} x {cols} is wanted")
    if cols > 1 and stride[-1] != 1:
        raise ValueError("the last dimension must be contiguous")
    ld, span = None, 0
    for n, s in zip(reversed(shape[:-1]), reversed(stride[:-1])):
        if n == 1:
            continue
        if ld is None:
            ld, span = s, s * n
        elif s != span:
            raise ValueError(f"rows are not evenly spaced: shape {tuple(shape)}, strides {tuple(stride)}")
        else:
            span = s * n
    if ld is None:
        ld = cols
    if ld < cols:
        raise ValueError("rows overlap")
    return t.data_ptr(), rows, cols, ld, dt, 0


# ------------------------------------------------------------ residual norm
def _norm_shape(x):
    """(rows, cols, rows of one sample) of (samples, rows, cols) or (rows, cols)."""
    if x.dim() not in (2, 3):
        raise ValueError(f"(rows, cols) or (samples, rows, cols) is wanted: got {tuple(x.shape)}")
    rows = x.shape[:-1].numel()
    return rows, x.shape[-1], x.shape[-2]


def _norm_kinds(post: str, pre: str):
    if post not in NORM_KINDS or pre not in NORM_KINDS:
        raise ValueError(f"norm kinds are {sorted(NORM_KINDS)}: got {post!r}, {pre!r}")
    return NORM_KINDS[post], NORM_KINDS[pre]


def norm_fwd(resid, h=None, gate=None, post_weight=None, pre_weight=None, scale=None, shift=None, *,
             post: str = "none", pre: str = "layer", alpha: float = 1.0, eps: float = 1e-6, y_dtype=None):
    """resid_out = resid + alpha gate N_post(h) post_weight;
    y = N_pre(resid_out) pre_weight (1 + scale) + shift.

    resid, h: (samples, rows, cols) or (rows, cols), fp32 or bf16 each; gate,
    scale, shift: (samples, cols); weights: (cols).  post, pre: "none", "rms"
    or "layer".  Returns (resid_out, y, stats): resid_out is resid where h is
    None; y has h's type (resid's where h is None) and is None where pre is
    "none" and nothing modulates it; stats (rows, 4) is what norm_bwd reads."""
    dev = _device(resid, h, gate, post_weight, pre_weight, scale, shift)
    rows, cols, group = _norm_shape(resid)
    k_post, k_pre = _norm_kinds(post, pre)
    if h is not None and (h.shape != resid.shape or y_dtype not in (None, h.dtype)):
        raise ValueError(f"h {tuple(h.shape)} {h.dtype}, resid {tuple(resid.shape)}, y_dtype {y_dtype}")
    want_y = k_pre != 0 or pre_weight is not None or scale is not None or shift is not None
    out = resid if h is None else _out(resid)
    y = None
    if want_y:
        y = _out(h) if h is not None else _out(resid) if y_dtype in (None, resid.dtype) else \
            torch.empty(resid.shape, dtype=y_dtype, device=dev)
    stats = torch.empty((rows, 4), dtype=torch.float32, device=dev)
    if rows == 0 or cols == 0:
        return out, y, stats
    groups = rows // group
    args = NORM_ARGS.pack(
        rows, cols, group, k_post, k_pre, alpha, eps,
        *_mat(resid, rows, cols), *_mat(h, rows, cols), *(_mat(out, rows, cols) if h is not None else _NO_MAT),
        *_mat(y, rows, cols), *_mat(gate, groups, cols), *_mat(scale, groups, cols), *_mat(shift, groups, cols),
        *_mat(post_weight, 1, cols), *_mat(pre_weight, 1, cols), stats.data_ptr(), *(9 * _NO_MAT))
    _call("muon_norm_fwd", args, dev, workspace=False)
    return out, y, stats


def norm_bwd(d_resid_out, d_y, resid_out, h, stats, gate=None, post_weight=None, pre_weight=None, scale=None,
             shift=None, *, post: str = "none", pre: str = "layer", alpha: float = 1.0, eps: float = 1e-6):
    """Gradients of norm_fwd's inputs, as a dict with the keys resid, h, gate,
    post_weight, pre_weight, scale and shift (None for what was None).

    d_resid_out, d_y: gradients of norm_fwd's first two results (either may be
    None: zero); resid_out and stats are its results, the rest its arguments."""
    x = resid_out
    dev = _device(x, d_resid_out, d_y, h, stats, gate, post_weight, pre_weight, scale, shift)
    rows, cols, group = _norm_shape(x)
    k_post, k_pre = _norm_kinds(post, pre)
    if stats.dtype != torch.float32 or not stats.is_contiguous() or stats.shape != (rows, 4):
        raise ValueError("stats is norm_fwd's third result")
    # (a missing d_y is taken as zeros of h's type)
    if d_y is None and (k_pre != 0 or pre_weight is not None or scale is not None or shift is not None):
        d_y = torch.zeros(x.shape, dtype=(x if h is None else h).dtype, device=dev)
    d_h = None if h is None else _out(h)
    d_resid = _out(x)
    vectors = [None if t is None else _out(t)
               for t in (gate, scale, shift, post_weight, pre_weight)]
    if rows == 0 or cols == 0:
        for t in vectors:
            if t is not None:
                t.zero_()
    else:
        groups = rows // group
        m = [_mat(t, groups if i < 3 else 1, cols) for i, t in enumerate((gate, scale, shift, post_weight, pre_weight))]
        dm = [_mat(t, groups if i < 3 else 1, cols) for i, t in enumerate(vectors)]
        args = NORM_ARGS.pack(
            rows, cols, group, k_post, k_pre, alpha, eps,
            *_NO_MAT, *_mat(h, rows, cols), *_mat(x, rows, cols), *_NO_MAT, *m[0], *m[1], *m[2], *m[3], *m[4],
            stats.data_ptr(), *_mat(d_resid_out, rows, cols), *_mat(d_y, rows, cols), *_mat(d_resid, rows, cols),
            *_mat(d_h, rows, cols), *dm[0], *dm[1], *dm[2], *dm[3], *dm[4])
        _call("muon_norm_bwd", args, dev)
    return {"resid": d_resid, "h": d_h, "gate": vectors[0], "post_weight": vectors[3], "pre_weight": vectors[4],
            "scale": vectors[1], "shift": vectors[2]}


class _ResidualNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, resid, h, gate, post_weight, pre_weight, scale, shift, how, y_dtype):
        out, y, stats = norm_fwd(resid, h, gate, post_weight, pre_weight, scale, shift, y_dtype=y_dtype, **how)
        if h is None:
            out = resid.view_as(resid)
        ctx.how = how
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(out, h, stats, gate, post_weight, pre_weight, scale, shift)
        return out, y

    @staticmethod
    @once_differentiable
    def backward(ctx, d_out, d_y):
        out, h, stats, gate, post_weight, pre_weight, scale, shift = ctx.saved_tensors
        if d_out is None and d_y is None:
            return (None,) * 9
        d_out = None if d_out is None else d_out.contiguous()
        d_y = None if d_y is None else d_y.contiguous()
        g = norm_bwd(d_out, d_y, out, h, stats, gate, post_weight, pre_weight, scale, shift, **ctx.how)
        return (g["resid"], g["h"], g["gate"], g["post_weight"], g["pre_weight"], g["scale"], g["shift"], None, None)


def residual_norm(resid, h=None, gate=None, post_weight=None, pre_weight=None, scale=None, shift=None, *,
                  post: str = "none", pre: str = "layer", alpha: float = 1.0, eps: float = 1e-6, y_dtype=None):
    """norm_fwd for autograd; returns (resid_out, y)."""
    return _ResidualNorm.apply(resid, h, gate, post_weight, pre_weight, scale, shift,
                               {"post": post, "pre": pre, "alpha": alpha, "eps": eps}, y_dtype)


# ---------------------------------------------------------------- attention
def _heads(t, name: str):
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name}: bf16 is wanted, got {t.dtype}")
    b, n, h, d = t.shape
    sb, sl, sh, sd = t.stride()
    if sd != 1 and d > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    # the stride of a dimension of one says nothing
    return t.data_ptr(), sb if b > 1 else 0, sl if n > 1 else 0, sh if h > 1 else 0


def _attn_dims(q, k, v, q_lens, k_lens, scale):
    if q.dim() != 4 or k.dim() != 4 or v.shape != k.shape or q.shape[0] != k.shape[0] or q.shape[3] != k.shape[3]:
        raise ValueError(f"(batch, len, heads, dim) each: q {tuple(q.shape)}, k {tuple(k.shape)}, v {tuple(v.shape)}")
    for name, t in (("q_lens", q_lens), ("k_lens", k_lens)):
        if t is None:
            continue
        if t.dtype != torch.int32:
            raise TypeError(f"{name}: int32 is wanted, got {t.dtype}")
        if t.shape != (q.shape[0],) or not t.is_contiguous():
            raise ValueError(f"{name}: one length per sample is wanted")
    b, m, h, d = q.shape
    return b, m, k.shape[1], h, k.shape[2], d, float(d) ** -0.5 if scale is None else float(scale)


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def attn_fwd(q, k, v, *, causal: bool = False, offset: int = 0, q_lens=None, k_lens=None, scale: float | None = None):
    """Softmax attention: q (batch, q_len, heads, dim), k and v (batch, k_len,
    kv_heads, dim), bf16, any strides that are multiples of eight with the last
    dimension contiguous (slices of a packed projection are fine); dim a
    multiple of 8 up to 128; kv_heads divides heads.

    q_lens, k_lens: int32 (batch,) on the GPU, how many of a sample's queries
    and keys are there.  causal: query i sees key j for j <= i + offset.
    scale: above 0, dim ** -0.5 where None.  Returns o (batch, q_len, heads, dim) bf16
    and lse (batch, heads, q_len) fp32; a query that sees no key has o = 0 and
    lse = -inf.  What lies past a length, and keys that no query sees, may hold
    anything."""
    dev = _device(q, k, v, q_lens, k_lens)
    b, m, n, h, g, d, scale = _attn_dims(q, k, v, q_lens, k_lens, scale)
    o = _out(q)                              # q's type is checked by _heads
    lse = torch.empty((b, h, m), dtype=torch.float32, device=dev)
    args = ATTN_ARGS.pack(b, m, n, h, g, d, int(causal), offset, scale, 0, _ptr(q_lens), _ptr(k_lens),
                          *_heads(q, "q"), *_heads(k, "k"), *_heads(v, "v"), *_heads(o, "o"), lse.data_ptr(),
                          *(4 * _NO_HEADS))
    _call("muon_attn_fwd", args, dev)
    return o, lse


def attn_bwd(d_o, q, k, v, o, lse, *, causal: bool = False, offset: int = 0, q_lens=None, k_lens=None,
             scale: float | None = None, out=None):
    """Gradients (d_q, d_k, d_v) of attn_fwd's o, from d_o and what attn_fwd
    took and gave, zero past the lengths.  They are written to `out`, three
    tensors of q's, k's and v's shapes (slices of a packed projection's
    gradient, say), or to new contiguous ones."""
    dev = _device(q, d_o, k, v, o, lse, q_lens, k_lens)
    b, m, n, h, g, d, scale = _attn_dims(q, k, v, q_lens, k_lens, scale)
    if d_o.shape != q.shape or o.shape != q.shape or lse.shape != (b, h, m):
        raise ValueError(f"d_o {tuple(d_o.shape)}, o {tuple(o.shape)}, lse {tuple(lse.shape)} for q {tuple(q.shape)}")
    if lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse is attn_fwd's second result")
    if out is None:
        out = _out(q), _out(k), _out(v)
    else:
        _device(q, *out)
        if tuple(t.shape for t in out) != (q.shape, k.shape, v.shape):
            raise ValueError(f"out: shapes {[tuple(t.shape) for t in out]}")
    d_q, d_k, d_v = out
    args = ATTN_ARGS.pack(b, m, n, h, g, d, int(causal), offset, scale, 0, _ptr(q_lens), _ptr(k_lens),
                          *_heads(q, "q"), *_heads(k, "k"), *_heads(v, "v"), *_heads(o, "o"), lse.data_ptr(),
                          *_heads(d_o, "d_o"), *_heads(d_q, "d_q"), *_heads(d_k, "d_k"), *_heads(d_v, "d_v"))
    _call("muon_attn_bwd", args, dev)
    return d_q, d_k, d_v


def _gradient(t):
    """t contiguous and on the 16-byte boundary that matrix operands need: autograd
    may pass a run out of a larger gradient, from any value on."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _keep(ctx, how, *tensors):
    """Saves what the backward pass reads, the lengths with it: written again
    before that pass, they then raise as any saved tensor does."""
    ctx.how = {name: value for name, value in how.items() if name not in ("q_lens", "k_lens")}
    ctx.save_for_backward(*tensors, how["q_lens"], how["k_lens"])


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, how):
        o, lse = attn_fwd(q, k, v, **how)
        _keep(ctx, how, q, k, v, o, lse)
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, d_o):
        q, k, v, o, lse, q_lens, k_lens = ctx.saved_tensors
        return (*attn_bwd(_gradient(d_o), q, k, v, o, lse, q_lens=q_lens, k_lens=k_lens, **ctx.how), None)


class _PackedAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, qkv, how, turn):
        q, k, v = qkv.unbind(2)
        if turn is None:
            o, lse = attn_fwd(q, k, v, **how)
            _keep(ctx, how, qkv, o, lse)
            return o
        q, k = rotary_fwd(q, k, **turn)
        o, lse = attn_fwd(q, k, v, **how)
        ctx.turn = {name: value for name, value in turn.items() if name not in ("freqs", "positions")}
        _keep(ctx, how, qkv, o, lse, q, k, turn["freqs"], turn.get("positions"))
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, d_o):
        qkv, o, lse, *rotated, q_lens, k_lens = ctx.saved_tensors
        q, k, v = qkv.unbind(2)
        d_qkv = torch.empty_like(qkv, memory_format=torch.contiguous_format)
        d_q, d_k, d_v = d_qkv.unbind(2)
        if rotated:
            q, k, freqs, positions = rotated
        attn_bwd(_gradient(d_o), q, k, v, o, lse, q_lens=q_lens, k_lens=k_lens, out=(d_q, d_k, d_v), **ctx.how)
        if rotated:
            rotary_bwd(d_q, d_k, freqs, positions, out=(d_q, d_k), **ctx.turn)
        return d_qkv, None, None


def attention_qkv(qkv, *, causal: bool = False, offset: int = 0, q_lens=None, k_lens=None,
                  scale: float | None = None, rotary: dict | None = None):
    """attention of a packed projection's output (batch, len, 3, heads, dim),
    whose gradient comes out packed alike; returns o.  rotary: rotary_fwd's
    arguments from freqs on, by name, where queries and keys are to be rotated
    first."""
    if rotary is not None and "out" in rotary:
        raise ValueError("rotary: queries and keys are rotated into tensors of their own")
    if rotary is not None:
        _no_learned(rotary.get("freqs"))
    return _PackedAttention.apply(qkv, {"causal": causal, "offset": offset, "q_lens": q_lens, "k_lens": k_lens,
                                        "scale": scale}, rotary)


def attention(q, k, v, *, causal: bool = False, offset: int = 0, q_lens=None, k_lens=None,
              scale: float | None = None):
    """attn_fwd for autograd; returns o."""
    return _Attention.apply(q, k, v, {"causal": causal, "offset": offset, "q_lens": q_lens, "k_lens": k_lens,
                                      "scale": scale})


# ------------------------------------------------------- gated feed-forward
def _ffn_dims(x, w_gate, w_up, w_down, act: str):
    if act not in ACTS:
        raise ValueError(f"act is one of {sorted(ACTS)}: got {act!r}")
    for name, t in (("x", x), ("w_gate", w_gate), ("w_up", w_up), ("w_down", w_down)):
        if t.dtype != torch.bfloat16:
            raise TypeError(f"{name}: bf16 is wanted, got {t.dtype}")
    if w_gate.dim() != 2 or x.dim() < 1:
        raise ValueError("x is (..., cols), the weights are matrices")
    hidden, cols = w_gate.shape
    if x.shape[-1] != cols or w_up.shape != (hidden, cols) or w_down.shape != (cols, hidden):
        raise ValueError(f"x {tuple(x.shape)}, w_gate {tuple(w_gate.shape)}, w_up {tuple(w_up.shape)}, "
                         f"w_down {tuple(w_down.shape)}")
    return x.shape[:-1].numel(), cols, hidden


def ffn_fwd(x, w_gate, w_up, w_down, *, act: str = "silu", save: bool = True):
    """y = (act(x w_gate^T) * (x w_up^T)) w_down^T, bf16 with fp32 sums.

    x (..., cols); w_gate, w_up (hidden, cols); w_down (cols, hidden); cols and
    hidden multiples of 8.  act: "silu", or "gelu" in its tanh form.  Returns
    (y, gu): gu (rows, 2 hidden) holds both projections for ffn_bwd, None where
    save is false."""
    dev = _device(x, w_gate, w_up, w_down)
    rows, cols, hidden = _ffn_dims(x, w_gate, w_up, w_down, act)
    y = _out(x)
    gu = torch.empty((rows, 2 * hidden), dtype=x.dtype, device=dev) if save else None
    if rows == 0:
        return y, gu
    args = FFN_ARGS.pack(rows, cols, hidden, ACTS[act], 0, *_mat(x, rows, cols), *_mat(y, rows, cols),
                         *_mat(w_gate, hidden, cols), *_mat(w_up, hidden, cols), *_mat(w_down, cols, hidden),
                         *_mat(gu, rows, 2 * hidden), *(5 * _NO_MAT))
    _call("muon_ffn_fwd", args, dev)
    return y, gu


def ffn_bwd(d_y, x, w_gate, w_up, w_down, gu, *, act: str = "silu", grad_dtype=torch.bfloat16):
    """Gradients (d_x, d_w_gate, d_w_up, d_w_down) of ffn_fwd's y; the weights'
    are contiguous, of grad_dtype (bf16 or fp32): what muon_step reads."""
    dev = _device(x, d_y, w_gate, w_up, w_down, gu)
    rows, cols, hidden = _ffn_dims(x, w_gate, w_up, w_down, act)
    if d_y.shape != x.shape:
        raise ValueError(f"d_y {tuple(d_y.shape)} for x {tuple(x.shape)}")
    if grad_dtype not in _TYPES:
        raise TypeError(f"unsupported grad_dtype {grad_dtype}")
    d_x = _out(x)
    grads = [torch.empty(w.shape, dtype=grad_dtype, device=dev) for w in (w_gate, w_up, w_down)]
    if rows == 0:
        return (d_x, *(w.zero_() for w in grads))
    args = FFN_ARGS.pack(rows, cols, hidden, ACTS[act], 0, *_mat(x, rows, cols), *_NO_MAT,
                         *_mat(w_gate, hidden, cols), *_mat(w_up, hidden, cols), *_mat(w_down, cols, hidden),
                         *_mat(gu, rows, 2 * hidden), *_mat(d_y, rows, cols), *_mat(d_x, rows, cols),
                         *_mat(grads[0], hidden, cols), *_mat(grads[1], hidden, cols), *_mat(grads[2], cols, hidden))
    _call("muon_ffn_bwd", args, dev)
    return (d_x, *grads)


class _GatedFfn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_gate, w_up, w_down, act, save):
        y, gu = ffn_fwd(x, w_gate, w_up, w_down, act=act, save=save)
        ctx.act = act
        ctx.save_for_backward(x, w_gate, w_up, w_down, gu)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, d_y):
        return (*ffn_bwd(_gradient(d_y), *ctx.saved_tensors, act=ctx.act), None, None)


def gated_ffn(x, w_gate, w_up, w_down, *, act: str = "silu"):
    """ffn_fwd for autograd; returns y."""
    # (inside forward the grad mode is off, and needs_input_grad does not know it)
    save = torch.is_grad_enabled() and any(t.requires_grad for t in (x, w_gate, w_up, w_down))
    return _GatedFfn.apply(x, w_gate, w_up, w_down, act, save)


# -------------------------------------------------------------------- dropout
def _rng(p, rng, device):
    """(seed, offset, address of both): two numbers, or a tensor that holds them."""
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"p is in 0 .. 1: got {p}")
    if p == 0.0:
        return _NO_RNG
    if rng is None:
        raise ValueError("dropout needs rng: (seed, offset), or an int64 tensor of both")
    if isinstance(rng, torch.Tensor):
        if rng.dtype != torch.int64 or rng.shape != (2,) or not rng.is_contiguous() or rng.device != device:
            raise ValueError(f"rng: two contiguous int64 on {device} are wanted, got {tuple(rng.shape)} {rng.dtype} on {rng.device}")
        return 0, 0, rng.data_ptr()
    seed, offset = map(operator.index, rng)
    if not (0 <= seed < 1 << 64 and 0 <= offset < 1 << 64):
        raise ValueError(f"rng: seed and offset are 64-bit numbers, got {rng}")
    return seed, offset, 0


def _dropout(x, p, rng, residual, dtype):
    dev = _device(x, residual)
    if residual is not None and residual.shape != x.shape:
        raise ValueError(f"residual {tuple(residual.shape)} for x {tuple(x.shape)}")
    if x.dim() == 0:
        raise ValueError("(..., cols) is wanted")
    if dtype not in _TYPES:
        raise TypeError(f"unsupported dtype {dtype}")
    seed, offset, state = _rng(p, rng, dev)
    y = _out(x) if dtype == x.dtype else torch.empty(x.shape, dtype=dtype, device=dev)
    if x.numel() == 0:
        return y
    rows, cols = x.shape[:-1].numel(), x.shape[-1]
    args = DROPOUT_ARGS.pack(rows, cols, p, seed, offset, state, *_mat(x, rows, cols),
                             *(_NO_MAT if residual is None else _mat(residual, rows, cols)),
                             y.data_ptr(), rows, cols, cols, _TYPES[dtype], 0)
    _call("muon_dropout", args, dev, workspace=False)
    return y


def dropout_fwd(x, p: float, rng=None, residual=None):
    """y = residual + keep x / (1 - p), the mask formed from rng and never
    stored.

    x, residual: (..., cols), fp32 or bf16 each; y has the residual's type (x's
    where there is none).  rng: (seed, offset), or an int64 tensor of the two on
    the GPU that is read when the kernel runs, so that a captured graph's replays
    differ by what is written there.  Calls whose masks are to differ take
    different offsets; the same seed and offset give the same mask, by an
    element's number in x.  Dropped elements count as 0 whatever they hold."""
    return _dropout(x, p, rng, residual, x.dtype if residual is None else residual.dtype)


def dropout_bwd(d_y, p: float, rng=None, *, dtype=None):
    """Gradient of dropout_fwd's x, of `dtype` (x's type; d_y's where None).
    The residual's is d_y."""
    return _dropout(d_y, p, rng, None, d_y.dtype if dtype is None else dtype)


def _keep_rng(ctx, rng, *tensors):
    """Saves what the backward pass reads, numbers in a tensor with it: written
    again before that pass, they then raise as any saved tensor does."""
    held = isinstance(rng, torch.Tensor)
    ctx.rng = None if held else rng
    ctx.save_for_backward(*tensors, rng if held else None)


class _Dropout(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, p, rng):
        ctx.p, ctx.dtype = p, x.dtype
        _keep_rng(ctx, rng if p != 0.0 and ctx.needs_input_grad[0] else None)
        return dropout_fwd(x, p, rng, residual)

    @staticmethod
    @once_differentiable
    def backward(ctx, d_y):
        held, = ctx.saved_tensors
        d_x = None
        if ctx.needs_input_grad[0]:
            d_x = dropout_bwd(d_y.contiguous(), ctx.p, ctx.rng if held is None else held, dtype=ctx.dtype)
        return d_x, d_y if ctx.needs_input_grad[1] else None, None, None


def dropout(x, p: float, rng=None, residual=None):
    """dropout_fwd for autograd; returns y."""
    return _Dropout.apply(x, residual, p, rng)


# --------------------------------------------------------------------- linear
def _linear_dims(weight, act: str):
    if act not in LINEAR_ACTS:
        raise ValueError(f"act is one of {sorted(LINEAR_ACTS)}: got {act!r}")
    if weight.dim() != 2:
        raise ValueError("the weight is a matrix")
    if weight.dtype != torch.bfloat16:
        raise TypeError(f"weight: bf16 is wanted, got {weight.dtype}")
    return weight.shape


def _vec(t, n: int):
    if t.shape != (n,):
        raise ValueError(f"bias: shape {tuple(t.shape)} where ({n},) is wanted")
    return _mat(t, 1, n)


def linear_fwd(x, weight, bias=None, residual=None, *, act: str = "none", p: float = 0.0, rng=None, save: bool = True,
               y_dtype=None):
    """z = x weight^T + bias; y = residual + drop(act(z)), with fp32 sums and
    epilogue.

    x (..., cols) and weight (out, cols) bf16, cols and out multiples of 8; bias
    (out,) fp32 or bf16; residual (..., out) fp32 or bf16, whose type y has (else
    y_dtype, bf16 where None).  act: "none", "silu", or "gelu" in its tanh form.
    p, rng: dropout as in dropout_fwd, the same mask as it gives for y's shape.
    Returns (y, z): z (rows, out) bf16 is what linear_bwd reads, None where act is
    "none" or save is false."""
    dev = _device(x, weight, bias, residual)
    out, cols = _linear_dims(weight, act)
    if x.dtype != torch.bfloat16:
        raise TypeError(f"x: bf16 is wanted, got {x.dtype}")
    if x.dim() < 1 or x.shape[-1] != cols:
        raise ValueError(f"x {tuple(x.shape)} for a weight {tuple(weight.shape)}")
    shape = (*x.shape[:-1], out)
    if residual is not None and (residual.shape != shape or y_dtype not in (None, residual.dtype)):
        raise ValueError(f"residual {tuple(residual.shape)} {residual.dtype} for {shape}, y_dtype {y_dtype}")
    dtype = residual.dtype if residual is not None else y_dtype or torch.bfloat16
    if dtype not in _TYPES:
        raise TypeError(f"unsupported dtype {dtype}")
    rows = x.shape[:-1].numel()
    rng = _rng(p, rng, dev) if p != 0.0 else _NO_RNG
    y = x.new_empty(shape) if dtype == torch.bfloat16 else torch.empty(shape, dtype=dtype, device=dev)
    z = x.new_empty((rows, out)) if save and act != "none" else None
    b = _NO_MAT if bias is None else _vec(bias, out)
    if rows == 0:
        return y, z
    args = LINEAR_FWD_ARGS.pack(rows, cols, out, LINEAR_ACTS[act], 0, p, *rng, *_mat(x, rows, cols),
                                *_mat(weight, out, cols), *b, *(_NO_MAT if residual is None else _mat(residual, rows, out)),
                                y.data_ptr(), rows, out, out, _TYPES[dtype], 0,
                                *(_NO_MAT if z is None else (z.data_ptr(), rows, out, out, 1, 0))) + _NO_LINEAR_BWD
    _call("muon_linear_fwd", args, dev)
    return y, z


def linear_bwd(d_y, x, weight, bias=None, z=None, *, act: str = "none", p: float = 0.0, rng=None,
               grad_dtype=torch.bfloat16, need_x: bool = True, need_weight: bool = True):
    """Gradients (d_x, d_weight, d_bias) of linear_fwd's y.

    z is linear_fwd's second result, the rest its arguments (x may be None where
    need_weight is false); d_y is fp32 or bf16.  d_weight is contiguous, of
    grad_dtype (bf16 or fp32), d_bias of the bias's type: what muon_step reads.
    None stands for what is not needed, d_bias where bias is None.  The
    residual's gradient is d_y.

    drop(d_y) act'(z) is rounded to bf16 as an operand of both products, unless it
    is a bf16 d_y itself: d_x and d_weight are off by some 1.7e-3 of their norm for
    that, in fp32 too.  Calls of at most 128 rows and 128 outputs (and rows x cols x
    out of 2e7) keep it in fp32; d_bias is summed from fp32 always."""
    dev = _device(d_y, x, weight, bias, z)
    out, cols = _linear_dims(weight, act)
    if d_y.dim() < 1 or d_y.shape[-1] != out:
        raise ValueError(f"d_y {tuple(d_y.shape)} for a weight {tuple(weight.shape)}")
    shape = (*d_y.shape[:-1], cols)
    if (need_weight or x is not None) and (x is None or x.shape != shape):
        raise ValueError(f"x {None if x is None else tuple(x.shape)} where {shape} is wanted")
    if act != "none" and z is None:
        raise ValueError("z is linear_fwd's second result")
    if grad_dtype not in _TYPES:
        raise TypeError(f"unsupported grad_dtype {grad_dtype}")
    rows = d_y.shape[:-1].numel()
    rng = _rng(p, rng, dev) if p != 0.0 else _NO_RNG
    b = _NO_MAT if bias is None else _vec(bias, out)
    d_x = weight.new_empty(shape) if need_x else None
    d_w = None
    if need_weight:
        d_w = weight.new_empty((out, cols)) if grad_dtype == torch.bfloat16 else \
            torch.empty((out, cols), dtype=grad_dtype, device=dev)
    d_b = None if bias is None else _out(bias)
    if rows == 0:
        for t in (d_w, d_b):
            if t is not None:
                t.zero_()
        return d_x, d_w, d_b
    args = LINEAR_ARGS.pack(rows, cols, out, LINEAR_ACTS[act], 0, p, *rng,
                            *(_NO_MAT if x is None else _mat(x, rows, cols)), *_mat(weight, out, cols), *b, *_NO_MAT, *_NO_MAT,
                            *(_NO_MAT if z is None else _mat(z, rows, out)), *_mat(d_y, rows, out),
                            *((d_x.data_ptr(), rows, cols, cols, 1, 0) if need_x else _NO_MAT),
                            *((d_w.data_ptr(), out, cols, cols, _TYPES[grad_dtype], 0) if need_weight else _NO_MAT),
                            *(_NO_MAT if d_b is None else (d_b.data_ptr(), 1, out, out, _TYPES[d_b.dtype], 0)))
    _call("muon_linear_bwd", args, dev)
    return d_x, d_w, d_b


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, residual, act, p, rng, y_dtype, save):
        y, z = linear_fwd(x, weight, bias, residual, act=act, p=p, rng=rng, save=save, y_dtype=y_dtype)
        ctx.act, ctx.p = act, p
        need_x, need_w, need_b = ctx.needs_input_grad[:3]
        # What the backward pass reads, and no more: anything else may be written
        # before it.  Of a weight without d_x, and of the bias, shape and type count.
        ctx.shapes = None if need_x else weight.detach(), bias.detach() if need_b else None
        _keep_rng(ctx, rng if p != 0.0 and (need_x or need_w or need_b) else None, x if need_w else None,
                  weight if need_x else None, z)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, d_y):
        x, weight, z, held = ctx.saved_tensors
        shape, bias = ctx.shapes
        need_x, need_w, need_b, need_r = ctx.needs_input_grad[:4]
        d = (None,) * 3
        if need_x or need_w or need_b:
            d = linear_bwd(_gradient(d_y), x, shape if weight is None else weight, bias, z, act=ctx.act, p=ctx.p,
                           rng=ctx.rng if held is None else held, need_x=need_x, need_weight=need_w)
        return (*d, d_y if need_r else None, None, None, None, None, None)


def linear(x, weight, bias=None, residual=None, *, act: str = "none", p: float = 0.0, rng=None, y_dtype=None):
    """linear_fwd for autograd; returns y."""
    # (inside forward the grad mode is off, and needs_input_grad does not know it)
    save = torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (x, weight, bias))
    return _Linear.apply(x, weight, bias, residual, act, p, rng, y_dtype, save)


# ----------------------------------------------------------- rotary positions
STRETCHES = ("none", "linear", "ntk", "yarn")


def rotary_freqs(dim, *, base: float = 10000.0, stretch: str = "none", factor: float = 1.0, length: int | None = None,
                 device="cuda"):
    """Frequencies for rotary_fwd, float64 (axes, pairs): base ** (-2 i / d) for
    the i-th pair of the d values that an axis turns.

    dim: the values that are rotated, or a sequence of them, one per axis, which
    take consecutive pairs (an image's rows and columns: (dim // 2, dim // 2)).
    stretch, for contexts `factor` times the one trained on: "linear" divides the
    frequencies (positions are interpolated), "ntk" raises the base by
    factor ** (d / (d - 2)), which leaves the fastest pair and divides the slowest,
    "yarn" divides those that turn less than once over `length` trained tokens,
    leaves those that turn more than 32 times and goes between by their turns, as the
    paper has it (Peng et al., "YaRN", which also scales queries and keys, rotary_fwd's
    scale, by 0.1 log(factor) + 1).  Programs that go between by a pair's number
    instead give other frequencies there: weights trained with those need them as
    they are, in a tensor of one's own."""
    dims = (dim,) if isinstance(dim, int) else tuple(dim)
    if not dims or any(d < 2 or d % 2 for d in dims):
        raise ValueError(f"each axis turns an even number of values: got {dim}")
    if stretch not in STRETCHES or not factor > 0.0 or not base > 0.0:
        raise ValueError(f"stretch is one of {STRETCHES}, factor and base above 0: got {stretch!r}, {factor}, {base}")
    if stretch == "yarn" and (length is None or length < 1):
        raise ValueError("yarn needs the length trained on")
    out = torch.zeros((len(dims), sum(dims) // 2), dtype=torch.float64)
    at = 0
    for axis, d in enumerate(dims):
        b = base * factor ** (d / (d - 2)) if stretch == "ntk" and d > 2 else base
        f = b ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
        if stretch == "linear":
            f = f / factor
        elif stretch == "yarn":
            kept = ((length * f / (2 * torch.pi) - 1) / 31).clamp(0, 1)
            f = f * (kept + (1 - kept) / factor)
        out[axis, at:at + d // 2] = f
        at += d // 2
    return out.to(device)


def _turned_heads(t, name: str, dtype):
    """Descriptor of (batch, len, heads, dim), any strides."""
    if t is None:
        return _NO_HEADS
    if t.dtype != dtype:
        raise TypeError(f"{name}: {dtype} is wanted, got {t.dtype}")
    b, n, h, _ = t.shape
    sb, sl, sh, sd = t.stride()
    if sd != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return t.data_ptr(), sb if b > 1 else 0, sl if n > 1 else 0, sh if h > 1 else 0


def _new_heads(t):
    """A contiguous tensor of t's shape and its descriptor."""
    if t is None:
        return None, _NO_HEADS
    o = _out(t)
    _, n, h, d = t.shape
    return o, (o.data_ptr(), n * h * d, h * d, d)


def _rotary(q, k, freqs, positions, offset, interleaved, scale, out, inverse):
    dev = _device(q, k, freqs, positions)
    if q.dim() != 4 or (k is not None and (k.dim() != 4 or k.shape[:2] != q.shape[:2] or k.shape[3] != q.shape[3])):
        raise ValueError(f"(batch, len, heads, dim) each: q {tuple(q.shape)}, k {None if k is None else tuple(k.shape)}")
    dtype = q.dtype
    if dtype not in _TYPES:
        raise TypeError(f"unsupported dtype {dtype}")
    b, n, h, d = q.shape
    if freqs.dtype != torch.float64 or freqs.dim() != 2 or not freqs.is_contiguous():
        raise ValueError("freqs: contiguous float64 (axes, pairs) is wanted")
    axes, pairs = freqs.shape
    between = 0
    if positions is not None:
        if positions.dtype != torch.int32 or not positions.is_contiguous():
            raise TypeError("positions: contiguous int32 is wanted")
        one = (n,) if axes == 1 else (n, axes)
        if positions.shape not in (one, (b, *one)):
            raise ValueError(f"positions {tuple(positions.shape)} where {one} or {(b, *one)} is wanted")
        if offset:
            raise ValueError("offset is for tokens without positions")
        between = n * axes if len(positions.shape) > len(one) else 0
    if not -1 << 63 <= operator.index(offset) < 1 << 63:
        raise ValueError(f"offset is a 64-bit number, got {offset}")
    hq, hk = _turned_heads(q, "q", dtype), _turned_heads(k, "k", dtype)
    if out is None:
        (oq, to_q), (ok, to_k) = _new_heads(q), _new_heads(k)
    else:
        _device(q, *out)
        if len(out) != 2 or tuple(None if t is None else t.shape for t in out) != (q.shape, None if k is None else k.shape):
            raise ValueError(f"out: shapes {[None if t is None else tuple(t.shape) for t in out]}")
        oq, ok = out
        for t in out:
            if t is not None and any(n > 1 and s == 0 for n, s in zip(t.shape, t.stride())):
                raise ValueError("out: values on top of each other")
        if ok is not None and oq.numel() and oq.data_ptr() == ok.data_ptr():
            raise ValueError("out: both in one place")
        to_q, to_k = _turned_heads(oq, "out", dtype), _turned_heads(ok, "out", dtype)
    args = ROTARY_ARGS.pack(
        b, n, h, 0 if k is None else k.shape[2], d, pairs, axes, int(interleaved), inverse, _TYPES[dtype], scale, 0, offset,
        freqs.data_ptr(), _ptr(positions), between, *hq, *hk, *to_q, *to_k)
    _call("muon_rotary", args, dev, workspace=False)
    if out is not None:
        # autograd is told, so that a backward pass that saved them raises
        for t in out:
            if t is not None and not t.is_inference():
                torch.autograd.graph.increment_version(t)
    return oq, ok


def rotary_fwd(q, k, freqs, positions=None, *, offset: int = 0, interleaved: bool = False, scale: float = 1.0, out=None):
    """Rotates queries and keys by their positions: pair p of a head turns by
    t = sum_a positions[..., a] freqs[a, p], (u, v) -> scale (u cos t - v sin t,
    v cos t + u sin t).

    q (batch, len, heads, dim) and k (batch, len, kv_heads, dim) or None, fp32 or
    bf16, any strides with the last dimension contiguous (slices of a packed
    projection are fine); dim even, up to 1024.  freqs: float64 (axes, pairs),
    rotary_freqs gives some; 2 pairs values of each head are rotated, the rest is
    copied.  interleaved: pairs of neighbours (2 p, 2 p + 1), else of halves
    (p, p + pairs).  positions: int32, (len,) or (batch, len), with several axes
    (len, axes) or (batch, len, axes); None: a token's number plus offset.

    Returns both, written to `out`, two tensors of q's and k's shapes, or to new
    contiguous ones.  out may be (q, k) themselves; one that holds a value of q or
    k in any other way, or two values in one place, raises."""
    return _rotary(q, k, freqs, positions, offset, interleaved, scale, out, 0)


def rotary_bwd(d_q, d_k, freqs, positions=None, *, offset: int = 0, interleaved: bool = False, scale: float = 1.0, out=None):
    """Gradients of rotary_fwd's q and k from those of its results: the inverse
    rotation, with the same scale."""
    return _rotary(d_q, d_k, freqs, positions, offset, interleaved, scale, out, 1)


def _no_learned(freqs):
    if isinstance(freqs, torch.Tensor) and freqs.requires_grad and torch.is_grad_enabled():
        raise ValueError("freqs: no gradient is formed for frequencies (detach them)")


class _Rotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, freqs, positions, how):
        ctx.how = how
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(freqs, positions)
        return rotary_fwd(q, k, freqs, positions, **how)

    @staticmethod
    @once_differentiable
    def backward(ctx, d_q, d_k):
        freqs, positions = ctx.saved_tensors
        # (any strides will do, but for an expanded last dimension)
        d = [None if t is None or not need else t if t.stride(-1) == 1 else t.contiguous()
             for t, need in zip((d_q, d_k), ctx.needs_input_grad)]
        if d[0] is None:
            d[1] = None if d[1] is None else rotary_bwd(d[1], None, freqs, positions, **ctx.how)[0]
        else:
            d = rotary_bwd(*d, freqs, positions, **ctx.how)
        return (*d, None, None, None)


def rotary(q, k, freqs, positions=None, *, offset: int = 0, interleaved: bool = False, scale: float = 1.0):
    """rotary_fwd for autograd; returns both rotated (None for a k that is None).
    Frequencies get no gradient: those that want one raise."""
    _no_learned(freqs)
    return _Rotary.apply(q, k, freqs, positions, {"offset": offset, "interleaved": interleaved, "scale": scale})
