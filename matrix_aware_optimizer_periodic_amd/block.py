"""PyTorch entry points of the transformer-block operators declared in
include/muon_block.h: the fused residual norm, softmax attention and the gated
feed-forward block.

``norm_fwd`` / ``norm_bwd``, ``attn_fwd`` / ``attn_bwd`` and ``ffn_fwd`` /
``ffn_bwd`` are one call of the library each: they check devices, types and
shapes, take outputs and workspace from PyTorch's allocator and enqueue the
kernels on the current stream of the tensors' device.  Nothing is copied or
made contiguous behind the caller's back: a layout that the kernels cannot
read raises.  Tensors made on another stream need the caller's wait (and
``record_stream``), as with PyTorch's own operators.  All six may be captured
into a HIP graph.

``residual_norm``, ``attention`` and ``gated_ffn`` wrap them for autograd, once:
gradients of their gradients raise.  To capture a training step into a graph,
call the forward and backward functions themselves: an autograd graph that
shares leaves with a captured backward pass must not be alive during the
capture.
"""

from __future__ import annotations

import ctypes
import struct

import torch
from torch.autograd.function import once_differentiable

from .binding import MUON_OK, MuonError, lib

NORM_KINDS = {"none": 0, "rms": 1, "layer": 2}
ACTS = {"silu": 0, "gelu": 1}
BLOCK_EXPORTED = ("muon_block_last_error", "muon_norm_fwd", "muon_norm_bwd_workspace", "muon_norm_bwd",
                  "muon_attn_fwd_workspace", "muon_attn_fwd", "muon_attn_bwd_workspace", "muon_attn_bwd",
                  "muon_ffn_fwd_workspace", "muon_ffn_fwd", "muon_ffn_bwd_workspace", "muon_ffn_bwd")

_TYPES = {torch.float32: 0, torch.bfloat16: 1}
# The argument structures of muon_block.h, packed field by field (a few
# microseconds where a ctypes.Structure of some 120 fields takes ten times that).
_MAT, _HEADS = "Pqqqii", "Pqqq"
NORM_ARGS = struct.Struct("@qqqiiff" + 9 * _MAT + "P" + 9 * _MAT)
ATTN_ARGS = struct.Struct("@qqqiiiiqfiPP" + 4 * _HEADS + "P" + 4 * _HEADS)
FFN_ARGS = struct.Struct("@qqqii" + 11 * _MAT)
_NO_MAT, _NO_HEADS = (0,) * 6, (0,) * 4

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
            elif name == "muon_norm_fwd":
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


def _call(name: str, args: bytes, device, workspace: bool = True) -> None:
    L = _READY or _lib()
    index = device.index
    if index != torch.cuda.current_device():
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
        return (*attn_bwd(d_o.contiguous(), q, k, v, o, lse, q_lens=q_lens, k_lens=k_lens, **ctx.how), None)


class _PackedAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, qkv, how):
        q, k, v = qkv.unbind(2)
        o, lse = attn_fwd(q, k, v, **how)
        _keep(ctx, how, qkv, o, lse)
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, d_o):
        qkv, o, lse, q_lens, k_lens = ctx.saved_tensors
        d_qkv = torch.empty_like(qkv, memory_format=torch.contiguous_format)
        attn_bwd(d_o.contiguous(), *qkv.unbind(2), o, lse, q_lens=q_lens, k_lens=k_lens, out=d_qkv.unbind(2), **ctx.how)
        return d_qkv, None


def attention_qkv(qkv, *, causal: bool = False, offset: int = 0, q_lens=None, k_lens=None,
                  scale: float | None = None):
    """attention of a packed projection's output (batch, len, 3, heads, dim),
    whose gradient comes out packed alike; returns o."""
    return _PackedAttention.apply(qkv, {"causal": causal, "offset": offset, "q_lens": q_lens, "k_lens": k_lens,
                                        "scale": scale})


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
        return (*ffn_bwd(d_y.contiguous(), *ctx.saved_tensors, act=ctx.act), None, None)


def gated_ffn(x, w_gate, w_up, w_down, *, act: str = "silu"):
    """ffn_fwd for autograd; returns y."""
    # (inside forward the grad mode is off, and needs_input_grad does not know it)
    save = torch.is_grad_enabled() and any(t.requires_grad for t in (x, w_gate, w_up, w_down))
    return _GatedFfn.apply(x, w_gate, w_up, w_down, act, save)
