// Host side of the transformer-block operators (muon_block.h): argument
// checks, workspace sizes and the launch of each call.  No device memory is
// allocated and nothing is synchronised.  No function here throws: the only
// state is a fixed buffer of error text per thread.
#include "../../include/muon_block.h"
#include "block_internal.h"
#include "block_overlap.h"

#include <cmath>
#include <cstdarg>
#include <cstdio>

using namespace muon;

namespace {

thread_local char g_text[256] = "";

muon_status fail(muon_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_text, sizeof g_text, fmt, ap);
  va_end(ap);
  return st;
}

#define CHECK(x)                              \
  do {                                        \
    const muon_status st_ = (x);              \
    if (st_ != MUON_OK) return st_;           \
  } while (0)

constexpr int64_t kMaxRows = int64_t(1) << 40;
// Row strides stay below 2^22 values so that the rows of one tile can be
// addressed with 32-bit byte offsets.
constexpr int64_t kMaxLd = int64_t(1) << 22;

size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

size_t type_size(int32_t dt) { return dt == MUON_F32 ? 4 : 2; }

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// A present matrix: shape, type (dt < 0: F32 or BF16), stride, alignment.
muon_status check_mat(const char* name, const muon_tensor& t, int64_t rows, int64_t cols, int32_t dt,
                      int64_t max_ld = kMaxLd) {
  if (!t.ptr) return fail(MUON_E_ARG, "%s is missing", name);
  if (t.rows != rows || t.cols != cols || t.reserved != 0)
    return fail(MUON_E_SHAPE, "%s: %lld x %lld where %lld x %lld is wanted", name, (long long)t.rows,
                (long long)t.cols, (long long)rows, (long long)cols);
  if ((t.dtype != MUON_F32 && t.dtype != MUON_BF16) || (dt >= 0 && t.dtype != dt))
    return fail(MUON_E_DTYPE, "%s: dtype %d", name, t.dtype);
  if (t.ld < cols || t.ld > max_ld)
    return fail(MUON_E_ALIGN, "%s: ld %lld for %lld columns", name, (long long)t.ld, (long long)cols);
  if (!aligned(t.ptr, type_size(t.dtype))) return fail(MUON_E_ALIGN, "%s: pointer not aligned to its type", name);
  return MUON_OK;
}

muon_status check_opt(const char* name, const muon_tensor& t, int64_t rows, int64_t cols, int32_t dt) {
  return t.ptr ? check_mat(name, t, rows, cols, dt) : MUON_OK;
}

muon_status check_workspace(void* ws, size_t have, size_t need) {
  if (need == 0) return MUON_OK;
  if (!ws || have < need) return fail(MUON_E_WORKSPACE, "workspace of %zu bytes where %zu are needed", ws ? have : 0, need);
  if (!aligned(ws, 256)) return fail(MUON_E_ALIGN, "workspace not 256-byte aligned");
  return MUON_OK;
}

muon_status launched(const char* what, hipError_t e) {
  if (e == hipSuccess) return MUON_OK;
  return fail(MUON_E_HIP, "%s: %s", what, hipGetErrorString(e));
}

// ---- residual norm ----------------------------------------------------------
muon_status norm_dims(const muon_norm_args* a) {
  if (!a) return fail(MUON_E_ARG, "args is NULL");
  if (a->rows < 0 || a->rows > kMaxRows || a->cols < 1 || a->cols > kNormMaxCols)
    return fail(MUON_E_SHAPE, "rows %lld, cols %lld (1 .. %d)", (long long)a->rows, (long long)a->cols, kNormMaxCols);
  if (a->group_rows < 1 || a->rows % a->group_rows)
    return fail(MUON_E_SHAPE, "group_rows %lld does not divide rows %lld", (long long)a->group_rows, (long long)a->rows);
  if (a->post_kind < 0 || a->post_kind > 2 || a->pre_kind < 0 || a->pre_kind > 2)
    return fail(MUON_E_ARG, "unknown norm kind");
  if (!std::isfinite(a->alpha) || !(a->eps >= 0.f) || !std::isfinite(a->eps))
    return fail(MUON_E_ARG, "alpha and eps must be finite, eps >= 0");
  // 32-bit numbers of workgroups, one per 64 columns and group in the sums'
  // launch, per row in the forward's
  if (a->rows / a->group_rows * ((a->cols + 63) / 64) > 0x7fffffff || a->rows > 0x7fffffff)
    return fail(MUON_E_SHAPE, "too many rows for one call");
  return MUON_OK;
}

muon_status norm_vectors(const muon_norm_args* a) {
  const int64_t g = a->rows / a->group_rows;
  CHECK(check_opt("gate", a->gate, g, a->cols, -1));
  CHECK(check_opt("scale", a->scale, g, a->cols, -1));
  CHECK(check_opt("shift", a->shift, g, a->cols, -1));
  CHECK(check_opt("post_weight", a->post_weight, 1, a->cols, -1));
  CHECK(check_opt("pre_weight", a->pre_weight, 1, a->cols, -1));
  if (!a->h.ptr && (a->gate.ptr || a->post_weight.ptr || a->post_kind != MUON_NORM_NONE))
    return fail(MUON_E_ARG, "gate, post_weight and a post norm need h");
  if (a->rows > 0 && (!a->stats || !aligned(a->stats, 16))) return fail(a->stats ? MUON_E_ALIGN : MUON_E_ARG, "stats is missing or not 16-byte aligned");
  return MUON_OK;
}

NormMat norm_mat(const muon_tensor& t) { return NormMat{t.ptr, t.ld, t.dtype, 0}; }

// Whether eight columns can move at once: whole groups of eight, 16-byte
// aligned rows of every matrix and vector that the kernels read that way.
bool norm_vec(const muon_norm_args* a) {
  if (a->cols % 8) return false;
  const muon_tensor* all[] = {&a->resid, &a->h, &a->resid_out, &a->y, &a->gate, &a->scale, &a->shift, &a->post_weight,
                              &a->pre_weight, &a->d_resid_out, &a->d_y, &a->d_resid, &a->d_h};
  for (const muon_tensor* t : all)
    if (t->ptr && (t->ld % 8 || !aligned(t->ptr, 16))) return false;
  return true;
}

NormDev norm_dev(const muon_norm_args* a) {
  NormDev d{};
  d.rows = a->rows; d.group_rows = a->group_rows; d.cols = int32_t(a->cols);
  d.post_kind = a->post_kind; d.pre_kind = a->pre_kind; d.alpha = a->alpha; d.eps = a->eps;
  d.resid = norm_mat(a->resid); d.h = norm_mat(a->h); d.resid_out = norm_mat(a->resid_out); d.y = norm_mat(a->y);
  d.gate = norm_mat(a->gate); d.scale = norm_mat(a->scale); d.shift = norm_mat(a->shift);
  d.post_weight = norm_mat(a->post_weight); d.pre_weight = norm_mat(a->pre_weight);
  d.stats = a->stats;
  d.d_resid_out = norm_mat(a->d_resid_out); d.d_y = norm_mat(a->d_y);
  d.d_resid = norm_mat(a->d_resid); d.d_h = norm_mat(a->d_h);
  d.d_gate = norm_mat(a->d_gate); d.d_scale = norm_mat(a->d_scale); d.d_shift = norm_mat(a->d_shift);
  d.d_post_weight = norm_mat(a->d_post_weight); d.d_pre_weight = norm_mat(a->d_pre_weight);
  d.splits = 1;
  return d;
}

bool norm_sums(const muon_norm_args* a) {
  return a->d_gate.ptr || a->d_scale.ptr || a->d_shift.ptr || a->d_post_weight.ptr || a->d_pre_weight.ptr;
}

size_t norm_bwd_bytes(const muon_norm_args* a) {
  if (!norm_sums(a) || a->rows == 0) return 0;
  const int64_t g = a->rows / a->group_rows;
  const size_t part = align_up(size_t(g) * norm_splits(g, a->group_rows, int(a->cols)) * kNormSums * size_t(a->cols) * 4);
  const bool weights = g > 1 && (a->d_post_weight.ptr || a->d_pre_weight.ptr);
  return part + (weights ? align_up(size_t(g) * 2 * size_t(a->cols) * 4) : 0);
}

// ---- attention ----------------------------------------------------------------
muon_status attn_dims(const muon_attn_args* a, bool backward) {
  if (!a) return fail(MUON_E_ARG, "args is NULL");
  if (a->batch < 0 || a->q_len < 0 || a->k_len < 0 || a->heads < 1 || a->kv_heads < 1 || a->heads % a->kv_heads)
    return fail(MUON_E_SHAPE, "batch %lld, lengths %lld and %lld, heads %d over %d", (long long)a->batch,
                (long long)a->q_len, (long long)a->k_len, a->heads, a->kv_heads);
  if (a->dim < 8 || a->dim > 128 || a->dim % 8) return fail(MUON_E_SHAPE, "dim %d: a multiple of 8 up to 128", a->dim);
  if ((a->causal != 0 && a->causal != 1) || a->reserved != 0) return fail(MUON_E_ARG, "causal is 0 or 1, reserved 0");
  if (!std::isfinite(a->scale) || !(a->scale > 0.f)) return fail(MUON_E_ARG, "scale must be positive and finite");
  // 32-bit row and key numbers, and fewer than 2^32 threads to a launch: 256 per
  // 128 rows, backward 512 per 256 keys.  (Launches whose keys or key blocks are
  // divided have far fewer.)
  const int64_t group = a->heads / a->kv_heads, top = 1 << 30, most = 1 << 24;
  const int64_t pairs = a->batch > 1 << 20 ? most : a->batch * a->kv_heads;
  if (pairs >= most || a->q_len > top || a->k_len > top || a->q_len * group > top ||
      (a->q_len * group + 127) / 128 * pairs >= most || (backward && (a->k_len + 255) / 256 * pairs >= most / 2))
    return fail(MUON_E_SHAPE, "too many rows for one call");
  return MUON_OK;
}

muon_status attn_heads(const char* name, const muon_heads& t) {
  if (!t.ptr) return fail(MUON_E_ARG, "%s is missing", name);
  if (!aligned(t.ptr, 16)) return fail(MUON_E_ALIGN, "%s: pointer not 16-byte aligned", name);
  if (t.stride_batch % 8 || t.stride_len % 8 || t.stride_head % 8)
    return fail(MUON_E_ALIGN, "%s: strides must be multiples of 8 values", name);
  if (t.stride_batch < 0 || t.stride_len < 0 || t.stride_head < 0 || t.stride_len > kMaxLd)
    return fail(MUON_E_SHAPE, "%s: stride out of range", name);
  return MUON_OK;
}

HeadsDev heads_dev(const muon_heads& t) { return HeadsDev{t.ptr, t.stride_batch, t.stride_len, t.stride_head}; }

AttnDev attn_dev(const muon_attn_args* a) {
  AttnDev d{};
  d.batch = int32_t(a->batch); d.q_len = int32_t(a->q_len); d.k_len = int32_t(a->k_len);
  d.heads = a->heads; d.kv_heads = a->kv_heads; d.dim = a->dim; d.causal = a->causal; d.scale = a->scale;
  const int64_t far = int64_t(1) << 31;      // beyond every length
  d.offset = a->offset > far ? far : a->offset < -far ? -far : a->offset;
  d.q_lens = a->q_lens; d.k_lens = a->k_lens;
  d.q = heads_dev(a->q); d.k = heads_dev(a->k); d.v = heads_dev(a->v); d.o = heads_dev(a->o);
  d.lse = a->lse;
  d.d_o = heads_dev(a->d_o); d.d_q = heads_dev(a->d_q); d.d_k = heads_dev(a->d_k); d.d_v = heads_dev(a->d_v);
  attn_plan(d);
  return d;
}

size_t attn_lines(const AttnDev& d) { return size_t(d.batch) * d.heads * d.q_len; }

size_t attn_fwd_bytes(const AttnDev& d) {
  if (d.splits <= 1 || attn_lines(d) == 0) return 0;
  return align_up(attn_lines(d) * d.splits * d.dim * 4) + align_up(attn_lines(d) * d.splits * 4);
}

size_t attn_bwd_bytes(const AttnDev& d) {
  const size_t sums = size_t(d.batch) * d.kv_heads * d.k_len * 2 * d.dim * 4;
  return 2 * align_up(attn_lines(d) * 4) + (d.parts > 1 ? d.parts * sums : 0);
}

// ---- gated feed-forward ---------------------------------------------------------
muon_status ffn_dims(const muon_ffn_args* a) {
  if (!a) return fail(MUON_E_ARG, "args is NULL");
  const int64_t most = 1 << 20;    // 2 hidden and a column tile stay within kMaxLd
  if (a->rows < 0 || a->rows > (1 << 30) || a->cols < 8 || a->hidden < 8 || a->cols % 8 || a->hidden % 8 ||
      a->cols > most || a->hidden > most)
    return fail(MUON_E_SHAPE, "rows %lld, cols %lld, hidden %lld: cols and hidden are multiples of 8 up to 2^20",
                (long long)a->rows, (long long)a->cols, (long long)a->hidden);
  // fewer than 2^32 threads to a launch: 256 per tile, of 128 x 128 results at
  // least (64 hidden columns of g and u); divided tiles add 2^20 at most
  const int64_t tiles = 15 << 20, rb = (a->rows + 127) / 128, cb = (a->cols + 127) / 128, hb = (a->hidden + 63) / 64;
  if (rb * hb >= tiles || rb * cb + 2 * hb * cb >= tiles)
    return fail(MUON_E_SHAPE, "too many rows or columns for one call: %lld x %lld x %lld", (long long)a->rows,
                (long long)a->cols, (long long)a->hidden);
  if ((a->act != MUON_ACT_SILU && a->act != MUON_ACT_GELU_TANH) || a->reserved != 0)
    return fail(MUON_E_ARG, "unknown act, or reserved is not 0");
  return MUON_OK;
}

// As check_mat, and rows whose 16-byte groups are aligned.
muon_status ffn_mat(const char* name, const muon_tensor& t, int64_t rows, int64_t cols, int32_t dt) {
  CHECK(check_mat(name, t, rows, cols, dt));
  if (!aligned(t.ptr, 16) || t.ld % (t.dtype == MUON_F32 ? 4 : 8))
    return fail(MUON_E_ALIGN, "%s: rows must be 16-byte aligned", name);
  return MUON_OK;
}

muon_status ffn_weights(const muon_ffn_args* a) {
  CHECK(ffn_mat("w_gate", a->w_gate, a->hidden, a->cols, MUON_BF16));
  CHECK(ffn_mat("w_up", a->w_up, a->hidden, a->cols, MUON_BF16));
  return ffn_mat("w_down", a->w_down, a->cols, a->hidden, MUON_BF16);
}

FfnDev ffn_dev(const muon_ffn_args* a) {
  FfnDev d{};
  d.rows = a->rows; d.cols = a->cols; d.hidden = a->hidden; d.act = a->act;
  d.x = a->x.ptr; d.ld_x = a->x.ld;
  d.w_gate = a->w_gate.ptr; d.ld_wg = a->w_gate.ld;
  d.w_up = a->w_up.ptr; d.ld_wu = a->w_up.ld;
  d.w_down = a->w_down.ptr; d.ld_wd = a->w_down.ld;
  d.y = a->y.ptr; d.ld_y = a->y.ld;
  d.gu = a->gu.ptr; d.ld_gu = a->gu.ld;
  d.d_y = a->d_y.ptr; d.ld_dy = a->d_y.ld;
  d.d_x = a->d_x.ptr; d.ld_dx = a->d_x.ld;
  d.d_wg = a->d_w_gate.ptr; d.ld_dwg = a->d_w_gate.ld;
  d.d_wu = a->d_w_up.ptr; d.ld_dwu = a->d_w_up.ld;
  d.d_wd = a->d_w_down.ptr; d.ld_dwd = a->d_w_down.ld;
  d.grad_bf16 = a->d_w_gate.dtype == MUON_BF16;
  return d;
}

size_t ffn_hid_bytes(const muon_ffn_args* a) { return align_up(size_t(a->rows) * size_t(a->hidden) * 2); }
size_t ffn_fwd_bytes(const muon_ffn_args* a) {
  return ffn_hid_bytes(a) + align_up(ffn_fwd_part_bytes(a->rows, a->cols, a->hidden));
}
size_t ffn_bwd_bytes(const muon_ffn_args* a) {
  return 3 * ffn_hid_bytes(a) + align_up(ffn_bwd_part_bytes(a->rows, a->cols, a->hidden));
}

// ---- dropout ----------------------------------------------------------------
// p as the last word that drops its element.
muon_status drop_dev(double p, const muon_rng& rng, DropDev* d) {
  *d = DropDev{};
  if (!(p >= 0.0) || !(p <= 1.0)) return fail(MUON_E_ARG, "p must be in 0 .. 1");
  const double words = std::nearbyint(p * 4294967296.0);
  if (words < 1.0) return MUON_OK;
  if (!aligned(rng.state, 8)) return fail(MUON_E_ALIGN, "rng.state not aligned");
  d->seed = rng.seed; d->offset = rng.offset; d->state = rng.state;
  d->last = uint32_t(uint64_t(words) - 1);
  d->on = 1;
  d->scale = p < 1.0 ? float(1.0 / (1.0 - p)) : 0.f;
  return MUON_OK;
}

// ---- linear -----------------------------------------------------------------
muon_status linear_dims(const muon_linear_args* a, DropDev* d) {
  if (!a) return fail(MUON_E_ARG, "args is NULL");
  const int64_t most = 1 << 20;
  if (a->rows < 0 || a->rows > (1 << 30) || a->cols < 8 || a->out < 8 || a->cols % 8 || a->out % 8 || a->cols > most ||
      a->out > most)
    return fail(MUON_E_SHAPE, "rows %lld, cols %lld, out %lld: cols and out are multiples of 8 up to 2^20",
                (long long)a->rows, (long long)a->cols, (long long)a->out);
  // fewer than 2^32 threads to a launch, 256 per tile; divided tiles add 2^20 at most
  const int64_t tiles = 15 << 20, rb = (a->rows + 127) / 128, cb = (a->cols + 127) / 128, ob = (a->out + 127) / 128;
  if (rb * ob >= tiles || rb * cb + ob * cb >= tiles)
    return fail(MUON_E_SHAPE, "too many rows or columns for one call: %lld x %lld x %lld", (long long)a->rows,
                (long long)a->cols, (long long)a->out);
  if ((a->act != MUON_ACT_SILU && a->act != MUON_ACT_GELU_TANH && a->act != MUON_ACT_NONE) || a->reserved != 0)
    return fail(MUON_E_ARG, "unknown act, or reserved is not 0");
  return drop_dev(a->p, a->rng, d);
}

LinearDev linear_dev(const muon_linear_args* a, const DropDev& drop) {
  LinearDev d{};
  d.rows = a->rows; d.cols = a->cols; d.out = a->out; d.act = a->act; d.drop = drop;
  d.x = norm_mat(a->x); d.w = norm_mat(a->weight); d.bias = norm_mat(a->bias); d.resid = norm_mat(a->residual);
  d.y = norm_mat(a->y); d.z = norm_mat(a->z); d.d_y = norm_mat(a->d_y); d.d_x = norm_mat(a->d_x);
  d.d_w = norm_mat(a->d_weight); d.d_bias = norm_mat(a->d_bias);
  return d;
}

// Whether the backward products' operand is formed apart from d_y.
bool linear_forms_dz(const muon_linear_args* a, const DropDev& drop) {
  return (a->d_x.ptr || a->d_weight.ptr) && (a->act != MUON_ACT_NONE || drop.on || a->d_y.dtype != MUON_BF16);
}
size_t linear_dz_bytes(const muon_linear_args* a, const DropDev& drop) {
  return linear_forms_dz(a, drop) ? align_up(size_t(a->rows) * size_t(a->out) * 2) : 0;
}
size_t linear_sums_bytes(const muon_linear_args* a) {
  if (!a->d_bias.ptr || a->rows == 0) return 0;
  const int splits = linear_sum_splits(a->rows, a->out);
  return splits > 1 ? align_up(size_t(splits) * size_t(a->out) * 4) : 0;
}
size_t linear_fwd_bytes(const muon_linear_args* a) { return align_up(linear_fwd_part_bytes(a->rows, a->cols, a->out)); }
size_t linear_bwd_bytes(const muon_linear_args* a, const DropDev& drop) {
  if (linear_small_grads(a->rows, a->cols, a->out)) return 0;
  return linear_dz_bytes(a, drop) + linear_sums_bytes(a) +
         align_up(linear_bwd_part_bytes(a->rows, a->cols, a->out, a->d_x.ptr, a->d_weight.ptr));
}

// ---- rotary positions ---------------------------------------------------------
muon_status rotary_heads(const char* name, const muon_heads& t, int32_t dtype) {
  if (!t.ptr) return fail(MUON_E_ARG, "%s is missing", name);
  if (!aligned(t.ptr, type_size(dtype))) return fail(MUON_E_ALIGN, "%s: pointer not aligned to its type", name);
  const int64_t far = int64_t(1) << 40;
  if (t.stride_batch < 0 || t.stride_len < 0 || t.stride_head < 0 || t.stride_batch > far || t.stride_len > far ||
      t.stride_head > far)
    return fail(MUON_E_SHAPE, "%s: stride out of range", name);
  return MUON_OK;
}

// Whether runs of v values of every head of t lie on the boundary their access
// needs (16 bytes at most).
bool rotary_runs(const muon_heads& t, int32_t dtype, int v) {
  const size_t size = type_size(dtype), need = v * size > 16 ? 16 : v * size;
  return aligned(t.ptr, need) && t.stride_batch * size % need == 0 && t.stride_len * size % need == 0 &&
         t.stride_head * size % need == 0;
}

Places rotary_places(const muon_rotary_args* a, const muon_heads& t, int32_t heads) {
  return Places{t.ptr, {t.stride_batch, t.stride_len, t.stride_head, 1}, {a->batch, a->len, heads, a->dim}};
}

}  // namespace

extern "C" {

const char* muon_block_last_error(void) { return g_text; }

muon_status muon_norm_fwd(const muon_norm_args* a, void* hip_stream) {
  CHECK(norm_dims(a));
  CHECK(norm_vectors(a));
  if (a->rows == 0) return MUON_OK;
  const int64_t n = a->rows, d = a->cols;
  CHECK(check_mat("resid", a->resid, n, d, -1));
  if (a->h.ptr) {
    CHECK(check_mat("h", a->h, n, d, -1));
    CHECK(check_mat("resid_out", a->resid_out, n, d, a->resid.dtype));
  }
  if (a->pre_kind != MUON_NORM_NONE || a->y.ptr) CHECK(check_mat("y", a->y, n, d, a->h.ptr ? a->h.dtype : -1));
  if (!a->y.ptr && (a->scale.ptr || a->shift.ptr || a->pre_weight.ptr)) return fail(MUON_E_ARG, "scale, shift and pre_weight need y");
  NormDev dev = norm_dev(a);
  if (!a->h.ptr) dev.resid_out = dev.resid;
  return launched("muon_norm_fwd", launch_norm_fwd(static_cast<hipStream_t>(hip_stream), dev, norm_vec(a)));
}

muon_status muon_norm_bwd_workspace(const muon_norm_args* a, size_t* bytes) {
  if (!bytes) return fail(MUON_E_ARG, "bytes is NULL");
  CHECK(norm_dims(a));
  *bytes = norm_bwd_bytes(a);
  return MUON_OK;
}

muon_status muon_norm_bwd(const muon_norm_args* a, void* ws, size_t ws_bytes, void* hip_stream) {
  CHECK(norm_dims(a));
  CHECK(norm_vectors(a));
  const int64_t n = a->rows, d = a->cols, g = n / a->group_rows;
  const bool sums = norm_sums(a);
  CHECK(check_opt("d_gate", a->d_gate, g, d, a->gate.ptr ? a->gate.dtype : -1));
  CHECK(check_opt("d_scale", a->d_scale, g, d, a->scale.ptr ? a->scale.dtype : -1));
  CHECK(check_opt("d_shift", a->d_shift, g, d, a->shift.ptr ? a->shift.dtype : -1));
  CHECK(check_opt("d_post_weight", a->d_post_weight, 1, d, a->post_weight.ptr ? a->post_weight.dtype : -1));
  CHECK(check_opt("d_pre_weight", a->d_pre_weight, 1, d, a->pre_weight.ptr ? a->pre_weight.dtype : -1));
  if ((a->d_gate.ptr || a->d_post_weight.ptr) && !a->h.ptr) return fail(MUON_E_ARG, "d_gate and d_post_weight need h");
  if (n == 0 && sums) return fail(MUON_E_SHAPE, "no rows: the vectors' gradients have none to be summed over");
  if (n == 0) return MUON_OK;
  CHECK(check_mat("d_resid", a->d_resid, n, d, -1));
  const int32_t rt = a->d_resid.dtype;
  CHECK(check_opt("d_resid_out", a->d_resid_out, n, d, rt));
  if (a->h.ptr) {
    CHECK(check_mat("h", a->h, n, d, -1));
    CHECK(check_mat("d_h", a->d_h, n, d, a->h.dtype));
  }
  if (a->d_y.ptr) {
    CHECK(check_mat("d_y", a->d_y, n, d, a->h.ptr ? a->h.dtype : -1));
    CHECK(check_mat("resid_out", a->resid_out, n, d, rt));
  } else if (a->pre_kind != MUON_NORM_NONE || a->d_scale.ptr || a->d_shift.ptr || a->d_pre_weight.ptr) {
    return fail(MUON_E_ARG, "d_y is missing");
  }
  const size_t need = norm_bwd_bytes(a);
  CHECK(check_workspace(ws, ws_bytes, need));
  NormDev dev = norm_dev(a);
  dev.resid_out.dt = rt;
  dev.splits = norm_splits(g, a->group_rows, int(a->cols));
  dev.split_rows = int32_t((a->group_rows + dev.splits - 1) / dev.splits);
  if (sums) {
    dev.part = static_cast<float*>(ws);
    if (g > 1 && (a->d_post_weight.ptr || a->d_pre_weight.ptr))
      dev.gsum = reinterpret_cast<float*>(static_cast<char*>(ws) +
                                          align_up(size_t(g) * dev.splits * kNormSums * size_t(d) * 4));
  }
  return launched("muon_norm_bwd", launch_norm_bwd(static_cast<hipStream_t>(hip_stream), dev, norm_vec(a), sums));
}

muon_status muon_attn_fwd_workspace(const muon_attn_args* a, size_t* bytes) {
  if (!bytes) return fail(MUON_E_ARG, "bytes is NULL");
  CHECK(attn_dims(a, false));
  *bytes = attn_fwd_bytes(attn_dev(a));
  return MUON_OK;
}

muon_status muon_attn_fwd(const muon_attn_args* a, void* ws, size_t ws_bytes, void* hip_stream) {
  CHECK(attn_dims(a, false));
  if (a->batch == 0 || a->q_len == 0) return MUON_OK;
  CHECK(attn_heads("q", a->q));
  if (a->k_len > 0) {
    CHECK(attn_heads("k", a->k));
    CHECK(attn_heads("v", a->v));
  }
  CHECK(attn_heads("o", a->o));
  if (!a->lse || !aligned(a->lse, 4)) return fail(MUON_E_ARG, "lse is missing or not aligned");
  AttnDev d = attn_dev(a);
  CHECK(check_workspace(ws, ws_bytes, attn_fwd_bytes(d)));
  if (d.splits > 1) {
    d.part_o = static_cast<float*>(ws);
    d.part_lse = reinterpret_cast<float*>(static_cast<char*>(ws) + align_up(attn_lines(d) * d.splits * d.dim * 4));
  }
  return launched("muon_attn_fwd", launch_attn_fwd(static_cast<hipStream_t>(hip_stream), d));
}

muon_status muon_attn_bwd_workspace(const muon_attn_args* a, size_t* bytes) {
  if (!bytes) return fail(MUON_E_ARG, "bytes is NULL");
  CHECK(attn_dims(a, true));
  *bytes = attn_bwd_bytes(attn_dev(a));
  return MUON_OK;
}

muon_status muon_attn_bwd(const muon_attn_args* a, void* ws, size_t ws_bytes, void* hip_stream) {
  CHECK(attn_dims(a, true));
  if (a->batch == 0 || (a->q_len == 0 && a->k_len == 0)) return MUON_OK;
  if (a->q_len > 0) {
    CHECK(attn_heads("q", a->q));
    CHECK(attn_heads("o", a->o));
    CHECK(attn_heads("d_o", a->d_o));
    CHECK(attn_heads("d_q", a->d_q));
    if (!a->lse || !aligned(a->lse, 4)) return fail(MUON_E_ARG, "lse is missing or not aligned");
  }
  if (a->k_len > 0) {
    CHECK(attn_heads("k", a->k));
    CHECK(attn_heads("v", a->v));
    CHECK(attn_heads("d_k", a->d_k));
    CHECK(attn_heads("d_v", a->d_v));
  }
  AttnDev d = attn_dev(a);
  CHECK(check_workspace(ws, ws_bytes, attn_bwd_bytes(d)));
  d.part_lse = static_cast<float*>(ws);
  d.delta = reinterpret_cast<float*>(static_cast<char*>(ws) + align_up(attn_lines(d) * 4));
  d.part_kv = reinterpret_cast<float*>(static_cast<char*>(ws) + 2 * align_up(attn_lines(d) * 4));
  return launched("muon_attn_bwd", launch_attn_bwd(static_cast<hipStream_t>(hip_stream), d));
}

muon_status muon_ffn_fwd_workspace(const muon_ffn_args* a, size_t* bytes) {
  if (!bytes) return fail(MUON_E_ARG, "bytes is NULL");
  CHECK(ffn_dims(a));
  *bytes = ffn_fwd_bytes(a);
  return MUON_OK;
}

muon_status muon_ffn_fwd(const muon_ffn_args* a, void* ws, size_t ws_bytes, void* hip_stream) {
  CHECK(ffn_dims(a));
  CHECK(ffn_weights(a));
  if (a->rows == 0) return MUON_OK;
  CHECK(ffn_mat("x", a->x, a->rows, a->cols, MUON_BF16));
  CHECK(ffn_mat("y", a->y, a->rows, a->cols, MUON_BF16));
  if (a->gu.ptr) CHECK(ffn_mat("gu", a->gu, a->rows, 2 * a->hidden, MUON_BF16));
  CHECK(check_workspace(ws, ws_bytes, ffn_fwd_bytes(a)));
  FfnDev d = ffn_dev(a);
  d.hid = ws;
  d.part = reinterpret_cast<float*>(static_cast<char*>(ws) + ffn_hid_bytes(a));
  return launched("muon_ffn_fwd", launch_ffn_fwd(static_cast<hipStream_t>(hip_stream), d));
}

muon_status muon_ffn_bwd_workspace(const muon_ffn_args* a, size_t* bytes) {
  if (!bytes) return fail(MUON_E_ARG, "bytes is NULL");
  CHECK(ffn_dims(a));
  *bytes = ffn_bwd_bytes(a);
  return MUON_OK;
}

muon_status muon_ffn_bwd(const muon_ffn_args* a, void* ws, size_t ws_bytes, void* hip_stream) {
  CHECK(ffn_dims(a));
  CHECK(ffn_weights(a));
  if (a->rows == 0) return fail(MUON_E_SHAPE, "no rows: the weights' gradients have none to be summed over");
  CHECK(ffn_mat("x", a->x, a->rows, a->cols, MUON_BF16));
  CHECK(ffn_mat("gu", a->gu, a->rows, 2 * a->hidden, MUON_BF16));
  CHECK(ffn_mat("d_y", a->d_y, a->rows, a->cols, MUON_BF16));
  CHECK(ffn_mat("d_x", a->d_x, a->rows, a->cols, MUON_BF16));
  CHECK(ffn_mat("d_w_gate", a->d_w_gate, a->hidden, a->cols, -1));
  CHECK(ffn_mat("d_w_up", a->d_w_up, a->hidden, a->cols, a->d_w_gate.dtype));
  CHECK(ffn_mat("d_w_down", a->d_w_down, a->cols, a->hidden, a->d_w_gate.dtype));
  CHECK(check_workspace(ws, ws_bytes, ffn_bwd_bytes(a)));
  FfnDev d = ffn_dev(a);
  d.hid = ws;
  d.dgu = static_cast<char*>(ws) + ffn_hid_bytes(a);
  d.part = reinterpret_cast<float*>(static_cast<char*>(ws) + 3 * ffn_hid_bytes(a));
  return launched("muon_ffn_bwd", launch_ffn_bwd(static_cast<hipStream_t>(hip_stream), d));
}

muon_status muon_dropout(const muon_dropout_args* a, void* hip_stream) {
  if (!a) return fail(MUON_E_ARG, "args is NULL");
  const int64_t top = int64_t(1) << 56, far = int64_t(1) << 40;
  if (a->rows < 0 || a->cols < 0 || a->cols > far || (a->cols > 0 && a->rows > top / a->cols))
    return fail(MUON_E_SHAPE, "rows %lld, cols %lld", (long long)a->rows, (long long)a->cols);
  DropoutDev d{};
  CHECK(drop_dev(a->p, a->rng, &d.drop));
  if (a->rows == 0 || a->cols == 0) return MUON_OK;
  CHECK(check_mat("x", a->x, a->rows, a->cols, -1, far));
  CHECK(check_mat("y", a->y, a->rows, a->cols, -1, far));
  if (a->residual.ptr) CHECK(check_mat("residual", a->residual, a->rows, a->cols, a->y.dtype, far));
  d.rows = a->rows; d.cols = a->cols;
  d.x = norm_mat(a->x); d.resid = norm_mat(a->residual); d.y = norm_mat(a->y);
  // Rows beside each other everywhere are one row.
  bool one = true, vec = true;
  for (const muon_tensor* t : {&a->x, &a->residual, &a->y})
    if (t->ptr && t->ld != a->cols) one = false;
  if (one) { d.cols *= d.rows; d.rows = 1; }
  for (const muon_tensor* t : {&a->x, &a->residual, &a->y})
    if (t->ptr && (!aligned(t->ptr, 16) || (d.rows > 1 && t->ld % 8))) vec = false;
  if (d.rows > 1 && a->cols % 8) vec = false;
  return launched("muon_dropout", launch_dropout(static_cast<hipStream_t>(hip_stream), d, vec));
}

muon_status muon_linear_fwd_workspace(const muon_linear_args* a, size_t* bytes) {
  if (!bytes) return fail(MUON_E_ARG, "bytes is NULL");
  DropDev drop;
  CHECK(linear_dims(a, &drop));
  *bytes = linear_fwd_bytes(a);
  return MUON_OK;
}

muon_status muon_linear_fwd(const muon_linear_args* a, void* ws, size_t ws_bytes, void* hip_stream) {
  DropDev drop;
  CHECK(linear_dims(a, &drop));
  CHECK(ffn_mat("weight", a->weight, a->out, a->cols, MUON_BF16));
  CHECK(check_opt("bias", a->bias, 1, a->out, -1));
  if (a->rows == 0) return MUON_OK;
  CHECK(ffn_mat("x", a->x, a->rows, a->cols, MUON_BF16));
  CHECK(ffn_mat("y", a->y, a->rows, a->out, -1));
  if (a->residual.ptr) CHECK(ffn_mat("residual", a->residual, a->rows, a->out, a->y.dtype));
  if (a->z.ptr) CHECK(ffn_mat("z", a->z, a->rows, a->out, MUON_BF16));
  CHECK(check_workspace(ws, ws_bytes, linear_fwd_bytes(a)));
  LinearDev d = linear_dev(a, drop);
  d.part = static_cast<float*>(ws);
  return launched("muon_linear_fwd", launch_linear_fwd(static_cast<hipStream_t>(hip_stream), d));
}

muon_status muon_linear_bwd_workspace(const muon_linear_args* a, size_t* bytes) {
  if (!bytes) return fail(MUON_E_ARG, "bytes is NULL");
  DropDev drop;
  CHECK(linear_dims(a, &drop));
  *bytes = linear_bwd_bytes(a, drop);
  return MUON_OK;
}

muon_status muon_linear_bwd(const muon_linear_args* a, void* ws, size_t ws_bytes, void* hip_stream) {
  DropDev drop;
  CHECK(linear_dims(a, &drop));
  if (!a->d_x.ptr && !a->d_weight.ptr && !a->d_bias.ptr) return MUON_OK;
  if (a->rows == 0 && (a->d_weight.ptr || a->d_bias.ptr))
    return fail(MUON_E_SHAPE, "no rows: the weights' gradients have none to be summed over");
  if (a->rows == 0) return MUON_OK;
  CHECK(ffn_mat("d_y", a->d_y, a->rows, a->out, -1));
  if (a->act != MUON_ACT_NONE) CHECK(ffn_mat("z", a->z, a->rows, a->out, MUON_BF16));
  if (a->d_x.ptr) {
    CHECK(ffn_mat("weight", a->weight, a->out, a->cols, MUON_BF16));
    CHECK(ffn_mat("d_x", a->d_x, a->rows, a->cols, MUON_BF16));
  }
  if (a->d_weight.ptr) {
    CHECK(ffn_mat("x", a->x, a->rows, a->cols, MUON_BF16));
    CHECK(ffn_mat("d_weight", a->d_weight, a->out, a->cols, -1));
  }
  CHECK(check_opt("d_bias", a->d_bias, 1, a->out, -1));
  const size_t need = linear_bwd_bytes(a, drop);
  CHECK(check_workspace(ws, ws_bytes, need));
  LinearDev d = linear_dev(a, drop);
  char* at = static_cast<char*>(ws);
  if (need > 0 && linear_forms_dz(a, drop)) d.dz = at;
  at += linear_dz_bytes(a, drop);
  d.sums = reinterpret_cast<float*>(at);
  d.part = reinterpret_cast<float*>(at + linear_sums_bytes(a));
  return launched("muon_linear_bwd", launch_linear_bwd(static_cast<hipStream_t>(hip_stream), d));
}

muon_status muon_rotary(const muon_rotary_args* a, void* hip_stream) {
  if (!a) return fail(MUON_E_ARG, "args is NULL");
  const int64_t top = 0x7fffffff;
  if (a->batch < 0 || a->len < 0 || a->batch > top || a->len > top || a->batch * a->len > top || a->heads < 1 ||
      a->kv_heads < 0 || int64_t(a->heads) + a->kv_heads > 1 << 16)
    return fail(MUON_E_SHAPE, "batch %lld, len %lld, heads %d and %d", (long long)a->batch, (long long)a->len, a->heads,
                a->kv_heads);
  if (a->dim < 2 || a->dim > 1024 || a->dim % 2 || a->pairs < 1 || a->pairs > a->dim / 2)
    return fail(MUON_E_SHAPE, "dim %d (even, up to 1024), pairs %d (up to half of that)", a->dim, a->pairs);
  if (a->axes < 1 || a->axes > 8 || (a->axes > 1 && !a->positions))
    return fail(MUON_E_ARG, "axes %d: 1 .. 8, and 1 without positions", a->axes);
  if ((a->interleaved | a->inverse) & ~1 || a->reserved != 0) return fail(MUON_E_ARG, "interleaved and inverse are 0 or 1, reserved 0");
  if (a->dtype != MUON_F32 && a->dtype != MUON_BF16) return fail(MUON_E_DTYPE, "dtype %d", a->dtype);
  if (!std::isfinite(a->scale)) return fail(MUON_E_ARG, "scale must be finite");
  const int64_t far = int64_t(1) << 52;
  if (a->offset > far || a->offset < -far) return fail(MUON_E_ARG, "offset beyond 2^52");
  if (a->batch == 0 || a->len == 0) return MUON_OK;
  if (!a->freqs || !aligned(a->freqs, 8)) return fail(a->freqs ? MUON_E_ALIGN : MUON_E_ARG, "freqs is missing or not aligned");
  if (!aligned(a->positions, 4)) return fail(MUON_E_ALIGN, "positions not aligned");
  if (a->positions_batch < 0 || a->positions_batch > int64_t(1) << 40) return fail(MUON_E_SHAPE, "positions_batch out of range");
  CHECK(rotary_heads("q", a->q, a->dtype));
  CHECK(rotary_heads("q_out", a->q_out, a->dtype));
  if (a->kv_heads > 0) {
    CHECK(rotary_heads("k", a->k, a->dtype));
    CHECK(rotary_heads("k_out", a->k_out, a->dtype));
  }
  // Workgroups turn the tokens in any order, so that a value that is written is
  // read by its own thread alone, which reads it first, or by none.
  const Places q = rotary_places(a, a->q, a->heads), q_out = rotary_places(a, a->q_out, a->heads);
  const Places k = rotary_places(a, a->k, a->kv_heads), k_out = rotary_places(a, a->k_out, a->kv_heads);
  const int64_t size = int64_t(type_size(a->dtype));
  const bool q_same = same_places(q, q_out), k_same = same_places(k, k_out);      // (no k meets nothing)
  if (places_repeat(q_out) || places_repeat(k_out)) return fail(MUON_E_ARG, "an output has two values in one place");
  if (places_meet(q_out, k_out, size)) return fail(MUON_E_ARG, "q_out and k_out overlap");
  if ((!q_same && places_meet(q_out, q, size)) || (!k_same && places_meet(k_out, k, size)))
    return fail(MUON_E_ARG, "an output overlaps its input and is not the same tensor");
  if (places_meet(q_out, k, size) || places_meet(k_out, q, size))
    return fail(MUON_E_ARG, "an output overlaps the other tensor's input");
  RotaryDev d{};
  d.tokens = a->batch * a->len;
  d.offset = a->offset; d.len = int32_t(a->len); d.heads = a->heads; d.kv_heads = a->kv_heads; d.dim = a->dim;
  d.pairs = a->pairs; d.axes = a->axes; d.interleaved = a->interleaved; d.inverse = a->inverse;
  d.f32 = a->dtype == MUON_F32; d.scale = a->scale;
  d.freqs = a->freqs; d.positions = a->positions; d.pos_batch = a->positions_batch;
  d.q = heads_dev(a->q); d.k = heads_dev(a->k); d.q_out = heads_dev(a->q_out); d.k_out = heads_dev(a->k_out);
  d.in_place = q_same && (a->kv_heads == 0 || k_same);
  // Pairs that move at once: whole chunks of a head (of halves, all of whose pairs
  // turn or none), and runs on their boundaries (0: not even a pair of neighbours
  // is).
  int vec = 0;
  for (int v : {8, 4, 2, 1}) {
    bool fits = vec == 0 && a->dim % (2 * v) == 0 && (a->interleaved || a->pairs % v == 0);
    for (const muon_heads* t : {&a->q, &a->q_out, &a->k, &a->k_out})
      fits = fits && ((a->kv_heads == 0 && (t == &a->k || t == &a->k_out)) || rotary_runs(*t, a->dtype, a->interleaved ? 2 * v : v));
    if (fits) vec = v;
  }
  return launched("muon_rotary", launch_rotary(static_cast<hipStream_t>(hip_stream), d, vec));
}

}  // extern "C"
