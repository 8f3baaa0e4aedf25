// Fused residual norm: the end of one transformer sub-block and the start of
// the next, forward and backward.
//
//   p = N_post(h) w_post;  r' = r + alpha gate_b p;
//   y = N_pre(r') w_pre (1 + scale_b) + shift_b          (b: the row's sample)
//
// Bound by memory: forward reads r and h and writes r' and y once, backward
// reads r', h, dr' and dy and writes dr and dh once.  One row is held in the
// registers of one wave (up to 512 columns) or of one workgroup, eight
// columns per thread, so that the two norms' statistics (mean first, then the
// centred squares, both fp32) cost no second pass over memory.
//
// Backward, with xhat and hhat the normalised rows and g = dy w_pre (1 + scale_b):
//
//   dr = dr' + rstd_r (g - [mean g] - xhat mean(g xhat))
//   dh = rstd_h (u - [mean u] - hhat mean(u hhat)),  u = alpha gate_b w_post dr
//
// (bracketed terms for LayerNorm only), and three column sums per sample,
//   S1 = sum dy xhat,  S2 = sum dr hhat,  S3 = sum dy,
// give all five vector gradients, because what multiplies them does not
// change along the rows of one sample:
//   dscale = w_pre S1, dshift = S3, dgate = alpha w_post S2,
//   dw_pre = sum_b (1 + scale_b) S1, dw_post = sum_b alpha gate_b S2.
// A workgroup keeps the three sums of its share of one sample's rows in
// registers and writes them once; a second kernel adds the shares in order
// (no atomics).
//
// Measured on one MI355X, where a large copy moves 5.1 TB/s: forward 16384 x
// 2048, fp32 stream and bf16 branch, modulated, 79 us (403 MB, 5.1 TB/s);
// backward 8192 x 5120 with every gradient 156 us for the rows (756 MB, 4.8
// TB/s) and 7.5 + 4.7 us for the sums; seven rows of 1001 columns 5.6 us.
#include <type_traits>

#include "block_device.h"

namespace muon {
namespace {

constexpr int kMaxWaves = 16;

// Sums of N values over the row's threads.  One wave per row: shuffles only.
// Otherwise one LDS exchange; `buf` alternates between two halves so that a
// row needs one barrier per sum.
template <int N, bool WAVE>
__device__ __forceinline__ void row_sum(float (&v)[N], float (*red)[2][kMaxWaves], int& phase, int nwaves) {
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = wave_sum(v[k]);
  if constexpr (!WAVE) {
    const int w = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int k = 0; k < N; ++k) red[phase][k][w] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
      float s = 0.f;
      for (int i = 0; i < nwaves; ++i) s += red[phase][k][i];
      v[k] = s;
    }
    phase ^= 1;
  }
}

// Columns of chunk c of this thread: VEC from col(c), none past the row.
// tid counts the threads of a row.
template <int VEC>
__device__ __forceinline__ int col_of(int c, int tid, int nthreads) { return (c * nthreads + tid) * VEC; }

// The start of a row: with the row's number in scalar registers, so is this,
// and a column takes one register as an offset where an address takes two.
template <typename T>
__device__ __forceinline__ T* row_of(const NormMat& m, int64_t row) { return static_cast<T*>(m.p) + row * m.ld; }

// Mean and 1 / deviation of a row held in v (zeros past its end).
template <int VEC, int NC, bool WAVE>
__device__ __forceinline__ void row_stats(const float (&v)[NC][VEC], int kind, int cols, float inv, float eps,
                                          int tid, int nt, float (*red)[2][kMaxWaves], int& phase, float& mean,
                                          float& rstd) {
  mean = 0.f;
  rstd = 1.f;
  if (kind == 0) return;
  if (kind == 2) {
    float s[1] = {0.f};
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int k = 0; k < VEC; ++k) s[0] += v[c][k];
    row_sum<1, WAVE>(s, red, phase, nt >> 6);
    mean = s[0] * inv;
  }
  float q[1] = {0.f};
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    if (col_of<VEC>(c, tid, nt) < cols) {
#pragma unroll
      for (int k = 0; k < VEC; ++k) { const float d = v[c][k] - mean; q[0] = fmaf(d, d, q[0]); }
    }
  }
  row_sum<1, WAVE>(q, red, phase, nt >> 6);
  rstd = 1.0f / sqrtf(fmaf(q[0], inv, eps));
}

// One row per wave (WAVE: four rows per workgroup) or per workgroup.  Every
// kernel's first workgroup is `from`, for grids that go out in pieces.
template <typename TR, typename TH, int VEC, int NC, bool WAVE>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void norm_fwd_kernel(NormDev a, int64_t from) {
  __shared__ float red[2][2][kMaxWaves];
  const int tid = WAVE ? threadIdx.x & 63 : threadIdx.x;
  const int nt = WAVE ? 64 : blockDim.x;
  const int64_t row = WAVE ? (from + blockIdx.x) * 4 + (threadIdx.x >> 6) : from + blockIdx.x;
  if (row >= a.rows) return;          // WAVE: whole waves, no barrier follows
  int phase = 0;
  const int64_t grp = row / a.group_rows;
  const float inv = 1.0f / float(a.cols);
  float r[NC][VEC], h[NC][VEC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int col = col_of<VEC>(c, tid, nt);
#pragma unroll
    for (int k = 0; k < VEC; ++k) { r[c][k] = 0.f; h[c][k] = 0.f; }
    if (col < a.cols) {
      load_vals<TR, VEC>(a.resid.p, row * a.resid.ld + col, r[c]);
      if (a.h.p) load_vals<TH, VEC>(a.h.p, row * a.h.ld + col, h[c]);
    }
  }
  float mh = 0.f, rh = 1.f, mr, rr;
  if (a.h.p) {
    row_stats<VEC, NC, WAVE>(h, a.post_kind, a.cols, inv, a.eps, tid, nt, red, phase, mh, rh);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int col = col_of<VEC>(c, tid, nt);
      if (col >= a.cols) continue;
      float w[VEC], g[VEC];
#pragma unroll
      for (int k = 0; k < VEC; ++k) { w[k] = 1.f; g[k] = 1.f; }
      if (a.post_weight.p) load_any<VEC>(a.post_weight.p, a.post_weight.dt, col, w);
      if (a.gate.p) load_any<VEC>(a.gate.p, a.gate.dt, grp * a.gate.ld + col, g);
#pragma unroll
      for (int k = 0; k < VEC; ++k) r[c][k] = fmaf(a.alpha * g[k], (h[c][k] - mh) * rh * w[k], r[c][k]);
      store_vals<TR, VEC>(a.resid_out.p, row * a.resid_out.ld + col, r[c]);
    }
  }
  row_stats<VEC, NC, WAVE>(r, a.pre_kind, a.cols, inv, a.eps, tid, nt, red, phase, mr, rr);
  if (a.y.p) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int col = col_of<VEC>(c, tid, nt);
      if (col >= a.cols) continue;
      float w[VEC], sc[VEC], sh[VEC];
#pragma unroll
      for (int k = 0; k < VEC; ++k) { w[k] = 1.f; sc[k] = 0.f; sh[k] = 0.f; }
      if (a.pre_weight.p) load_any<VEC>(a.pre_weight.p, a.pre_weight.dt, col, w);
      if (a.scale.p) load_any<VEC>(a.scale.p, a.scale.dt, grp * a.scale.ld + col, sc);
      if (a.shift.p) load_any<VEC>(a.shift.p, a.shift.dt, grp * a.shift.ld + col, sh);
#pragma unroll
      for (int k = 0; k < VEC; ++k) w[k] = fmaf((r[c][k] - mr) * rr * w[k], 1.f + sc[k], sh[k]);
      store_vals<TH, VEC>(a.y.p, row * a.y.ld + col, w);
    }
  }
  if (tid == 0 && a.stats) {
    *as_global(reinterpret_cast<f32x2_t*>(a.stats + row * 4)) = f32x2_t{mh, rh};
    *as_global(reinterpret_cast<f32x2_t*>(a.stats + row * 4 + 2)) = f32x2_t{mr, rr};
  }
}

// VEC values of a row as they were loaded, for rows read ahead.
template <typename T, int VEC>
struct Raw {
  using V = std::conditional_t<sizeof(T) == 4, f32x4_t, u32x4_t>;
  V a[sizeof(T) == 4 ? 2 : 1];
  __device__ __forceinline__ void load(const void* p, int64_t e) {
    const auto* q = as_global(reinterpret_cast<const V*>(static_cast<const T*>(p) + e));
    a[0] = q[0];
    if constexpr (sizeof(T) == 4) a[1] = q[1];
  }
  __device__ __forceinline__ void get(float (&v)[VEC]) const {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (sizeof(T) == 4) {
        v[k] = a[0][k];
        v[4 + k] = a[1][k];
      } else {
        v[2 * k] = bf16_to_f32(a[0][k] & 0xffffu);
        v[2 * k + 1] = __uint_as_float(a[0][k] & 0xffff0000u);
      }
    }
  }
  __device__ __forceinline__ void clear() {
    a[0] = V{};
    if constexpr (sizeof(T) == 4) a[1] = V{};
  }
};
template <typename T>
struct Raw<T, 1> {
  float a;
  __device__ __forceinline__ void load(const void* p, int64_t e) {
    float v[1];
    load_vals<T, 1>(p, e, v);
    a = v[0];
  }
  __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = a; }
  __device__ __forceinline__ void clear() { a = 0.f; }
};

// One share of one sample's rows per wave (WAVE: four shares per workgroup)
// or per workgroup; share = group * splits + split.  AHEAD: the next row is
// read while this one is worked on, in rows of up to 5120 columns, the widest
// timed with it (4096 x 5120 fp32 stream, bf16 branch: 92 us; 4096 x 5128 without
// it 106); up to 768 threads would have the registers.
template <typename TR, typename TH, int VEC, int NC, bool WAVE, bool AHEAD>
__global__ __launch_bounds__(WAVE ? 256 : AHEAD ? 640 : 1024) void norm_bwd_kernel(NormDev a, int64_t from,
                                                                                   int64_t shares) {
  __shared__ float red[2][2][kMaxWaves];
  const int tid = WAVE ? threadIdx.x & 63 : threadIdx.x;
  const int nt = WAVE ? 64 : blockDim.x;
  const int64_t share = WAVE ? (from + blockIdx.x) * 4 + (threadIdx.x >> 6) : from + blockIdx.x;
  if (share >= shares) return;
  int phase = 0;
  const int64_t grp = share / a.splits;
  const int64_t first = grp * a.group_rows + (share - grp * a.splits) * int64_t(a.split_rows);
  const int64_t end = min(first + a.split_rows, (grp + 1) * a.group_rows);
  const float inv = 1.0f / float(a.cols);
  const bool have_h = a.h.p != nullptr, have_y = a.d_y.p != nullptr, have_r = a.d_resid_out.p != nullptr;
  const float kpre = a.pre_kind == 2 ? inv : 0.f, kpost = a.post_kind == 2 ? inv : 0.f;
  const float npre = a.pre_kind ? inv : 0.f, npost = a.post_kind ? inv : 0.f;
  // what multiplies dy and dr in this share's columns, and its sums
  float wy[NC][VEC], wr[NC][VEC], s1[NC][VEC], s2[NC][VEC], s3[NC][VEC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int col = col_of<VEC>(c, tid, nt);
#pragma unroll
    for (int k = 0; k < VEC; ++k) { wy[c][k] = 1.f; wr[c][k] = a.alpha; s1[c][k] = s2[c][k] = s3[c][k] = 0.f; }
    if (col >= a.cols) continue;
    float t[VEC];
    if (a.pre_weight.p) load_any<VEC>(a.pre_weight.p, a.pre_weight.dt, col, wy[c]);
    if (a.scale.p) {
      load_any<VEC>(a.scale.p, a.scale.dt, grp * a.scale.ld + col, t);
#pragma unroll
      for (int k = 0; k < VEC; ++k) wy[c][k] *= 1.f + t[k];
    }
    if (a.post_weight.p) {
      load_any<VEC>(a.post_weight.p, a.post_weight.dt, col, t);
#pragma unroll
      for (int k = 0; k < VEC; ++k) wr[c][k] *= t[k];
    }
    if (a.gate.p) {
      load_any<VEC>(a.gate.p, a.gate.dt, grp * a.gate.ld + col, t);
#pragma unroll
      for (int k = 0; k < VEC; ++k) wr[c][k] *= t[k];
    }
  }
  Raw<TR, VEC> lx[NC], lr[NC];
  Raw<TH, VEC> ly[NC], lh[NC];
  f32x4_t lst;
  auto read = [&](int64_t row) {
    const TR *px = row_of<TR>(a.resid_out, row), *pr = row_of<TR>(a.d_resid_out, row);
    const TH *py = row_of<TH>(a.d_y, row), *ph = row_of<TH>(a.h, row);
    lst = *as_global(reinterpret_cast<const f32x4_t*>(a.stats + row * 4));
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const unsigned col = unsigned(col_of<VEC>(c, tid, nt));
      if (col >= unsigned(a.cols)) continue;
      if (have_y) {
        lx[c].load(px, col);
        ly[c].load(py, col);
      }
      if (have_r) lr[c].load(pr, col);
      if (have_h) lh[c].load(ph, col);
    }
  };
#pragma unroll
  for (int c = 0; c < NC; ++c) { lx[c].clear(); lr[c].clear(); ly[c].clear(); lh[c].clear(); }
  if (AHEAD && first < end) read(first);
  for (int64_t row = first; row < end; ++row) {
    if (!AHEAD) read(row);
    const f32x4_t st = lst;
    float x[NC][VEC], dy[NC][VEC], dr[NC][VEC], h[NC][VEC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      lx[c].get(x[c]);
      ly[c].get(dy[c]);
      lr[c].get(dr[c]);
      lh[c].get(h[c]);
    }
    if (AHEAD) read(min(row + 1, end - 1));
    if (have_y) {
      float t[2] = {0.f, 0.f};
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        if (col_of<VEC>(c, tid, nt) >= a.cols) continue;
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          x[c][k] = (x[c][k] - st[2]) * st[3];
          s3[c][k] += dy[c][k];
          s1[c][k] = fmaf(dy[c][k], x[c][k], s1[c][k]);
          dy[c][k] *= wy[c][k];
          t[0] += dy[c][k];
          t[1] = fmaf(dy[c][k], x[c][k], t[1]);
        }
      }
      if (a.pre_kind) row_sum<2, WAVE>(t, red, phase, nt >> 6);
      t[0] *= kpre;
      t[1] *= npre;
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int k = 0; k < VEC; ++k) dr[c][k] = fmaf(st[3], dy[c][k] - t[0] - x[c][k] * t[1], dr[c][k]);
    }
    float t[2] = {0.f, 0.f};
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const unsigned col = unsigned(col_of<VEC>(c, tid, nt));
      if (col >= unsigned(a.cols)) continue;
      store_vals<TR, VEC>(row_of<TR>(a.d_resid, row), col, dr[c]);
      if (have_h) {
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          h[c][k] = (h[c][k] - st[0]) * st[1];
          s2[c][k] = fmaf(dr[c][k], h[c][k], s2[c][k]);
          dr[c][k] *= wr[c][k];
          t[0] += dr[c][k];
          t[1] = fmaf(dr[c][k], h[c][k], t[1]);
        }
      }
    }
    if (!have_h) continue;
    if (a.post_kind) row_sum<2, WAVE>(t, red, phase, nt >> 6);
    t[0] *= kpost;
    t[1] *= npost;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const unsigned col = unsigned(col_of<VEC>(c, tid, nt));
      if (col >= unsigned(a.cols)) continue;
#pragma unroll
      for (int k = 0; k < VEC; ++k) dr[c][k] = st[1] * (dr[c][k] - t[0] - h[c][k] * t[1]);
      store_vals<TH, VEC>(row_of<TH>(a.d_h, row), col, dr[c]);
    }
  }
  if (!a.part) return;
  float* o = a.part + share * int64_t(kNormSums) * a.cols;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int col = col_of<VEC>(c, tid, nt);
    if (col >= a.cols) continue;
    store_vals<float, VEC>(o, col, s1[c]);
    store_vals<float, VEC>(o, int64_t(a.cols) + col, s2[c]);
    store_vals<float, VEC>(o, 2 * int64_t(a.cols) + col, s3[c]);
  }
}

// Sums over `n` rows, `stride` floats apart, of 64 columns per workgroup:
// 16 threads per column take every 16th row, then their sums are added in
// order.  The result is in the threads of the first wave.  UNROLL rows are read
// ahead of their additions.
template <int N, int UNROLL>
__device__ __forceinline__ void col_sums(const float* p, int64_t n, int64_t stride, int64_t next, int col, int cols,
                                         float (&v)[N], float (*red)[16][64]) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = 0.f;
  if (col < cols) {
#pragma unroll UNROLL
    for (int64_t i = w; i < n; i += 16)
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] += *as_global(p + i * stride + k * next + col);
  }
#pragma unroll
  for (int k = 0; k < N; ++k) red[k][w][lane] = v[k];
  __syncthreads();
  if (w == 0) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      v[k] = 0.f;
      for (int i = 0; i < 16; ++i) v[k] += red[k][i][lane];
    }
  }
}

// FEW: a sample has no more shares than that workgroup has waves, and a wave
// adds one sample's 64 columns by itself, in the same order.
template <bool FEW>
__global__ __launch_bounds__(FEW ? 256 : 1024) void norm_sums_kernel(NormDev a, int64_t from, int64_t groups) {
  const int tiles = (a.cols + 63) / 64;
  const int64_t item = FEW ? (from + blockIdx.x) * 4 + (threadIdx.x >> 6) : from + blockIdx.x;   // below 2^31
  if (FEW && item >= groups * tiles) return;
  const int64_t grp = unsigned(item) / unsigned(tiles);
  const int col = int(unsigned(item) % unsigned(tiles)) * 64 + (threadIdx.x & 63);
  const float* part = a.part + grp * a.splits * kNormSums * int64_t(a.cols);
  float s[kNormSums] = {0.f, 0.f, 0.f};
  if constexpr (FEW) {
    if (col >= a.cols) return;
    for (int i = 0; i < a.splits; ++i)
#pragma unroll
      for (int k = 0; k < kNormSums; ++k) s[k] += *as_global(part + (i * kNormSums + k) * int64_t(a.cols) + col);
  } else {
    __shared__ float red[kNormSums][16][64];
    col_sums<kNormSums, 1>(part, a.splits, kNormSums * int64_t(a.cols), a.cols, col, a.cols, s, red);
    if (threadIdx.x >= 64 || col >= a.cols) return;
  }
  const float wp = a.pre_weight.p ? load_any1(a.pre_weight.p, a.pre_weight.dt, col) : 1.f;
  const float wo = a.post_weight.p ? load_any1(a.post_weight.p, a.post_weight.dt, col) : 1.f;
  if (a.d_scale.p) store_any1(a.d_scale.p, a.d_scale.dt, grp * a.d_scale.ld + col, wp * s[0]);
  if (a.d_gate.p) store_any1(a.d_gate.p, a.d_gate.dt, grp * a.d_gate.ld + col, a.alpha * wo * s[1]);
  if (a.d_shift.p) store_any1(a.d_shift.p, a.d_shift.dt, grp * a.d_shift.ld + col, s[2]);
  const float sc = a.scale.p ? load_any1(a.scale.p, a.scale.dt, grp * a.scale.ld + col) : 0.f;
  const float g = a.gate.p ? load_any1(a.gate.p, a.gate.dt, grp * a.gate.ld + col) : 1.f;
  const float dp = (1.f + sc) * s[0], dq = a.alpha * g * s[1];
  if (groups == 1) {
    if (a.d_pre_weight.p) store_any1(a.d_pre_weight.p, a.d_pre_weight.dt, col, dp);
    if (a.d_post_weight.p) store_any1(a.d_post_weight.p, a.d_post_weight.dt, col, dq);
  } else if (a.gsum) {
    *as_global(a.gsum + grp * 2 * a.cols + col) = dp;
    *as_global(a.gsum + (grp * 2 + 1) * a.cols + col) = dq;
  }
}

__global__ __launch_bounds__(1024) void norm_weights_kernel(NormDev a, int64_t groups) {
  __shared__ float red[2][16][64];
  const int col = int(blockIdx.x) * 64 + (threadIdx.x & 63);
  float s[2];
  col_sums<2, 8>(a.gsum, groups, 2 * int64_t(a.cols), a.cols, col, a.cols, s, red);
  if (threadIdx.x >= 64 || col >= a.cols) return;
  if (a.d_pre_weight.p) store_any1(a.d_pre_weight.p, a.d_pre_weight.dt, col, s[0]);
  if (a.d_post_weight.p) store_any1(a.d_post_weight.p, a.d_post_weight.dt, col, s[1]);
}

// Threads per row and chunks per thread: eight columns per thread while a
// row fits 1024 threads, single columns (four, eight or sixteen) where a row is
// not whole aligned groups of eight.  The backward pass holds seven values per
// column: sixteen columns, in any form, spill some 250 registers and run at 2.1 -
// 2.5 TB/s in whole groups, 0.9 in single columns (4096 x 10001: 789 us; x 16384:
// 476), eight single ones none (4096 x 5001: 203 us, 963 with sixteen).
struct Shape { int threads; int nc; bool wave; };
Shape shape_of(int cols, bool vec) {
  const int per = (cols + (vec ? 8 : 1) - 1) / (vec ? 8 : 1);   // thread columns of a row
  const int nc = vec ? (per <= 1024 ? 1 : 2) : per <= 4096 ? 4 : per <= 8192 ? 8 : 16;
  const int threads = ((per + nc - 1) / nc + 63) / 64 * 64;
  return {threads, nc, threads == 64 && nc == (vec ? 1 : 4)};
}

#define FWD_KERNEL(TR, TH)                                                                                   \
  (vec ? (sh.wave ? norm_fwd_kernel<TR, TH, 8, 1, true> : sh.nc == 1 ? norm_fwd_kernel<TR, TH, 8, 1, false>     \
                                                                     : norm_fwd_kernel<TR, TH, 8, 2, false>)    \
       : (sh.wave ? norm_fwd_kernel<TR, TH, 1, 4, true> : sh.nc == 4 ? norm_fwd_kernel<TR, TH, 1, 4, false>     \
          : sh.nc == 8 ? norm_fwd_kernel<TR, TH, 1, 8, false> : norm_fwd_kernel<TR, TH, 1, 16, false>))
#define BWD_KERNEL(TR, TH)                                                                                   \
  (vec ? (sh.wave           ? norm_bwd_kernel<TR, TH, 8, 1, true, true>                                         \
          : sh.nc == 2        ? norm_bwd_kernel<TR, TH, 8, 2, false, false>                                     \
          : sh.threads <= 640 ? norm_bwd_kernel<TR, TH, 8, 1, false, true>                                      \
                              : norm_bwd_kernel<TR, TH, 8, 1, false, false>)                                    \
       : (sh.wave      ? norm_bwd_kernel<TR, TH, 1, 4, true, false>                                             \
          : sh.nc == 4 ? norm_bwd_kernel<TR, TH, 1, 4, false, false>                                            \
          : sh.nc == 8 ? norm_bwd_kernel<TR, TH, 1, 8, false, false>                                            \
                       : norm_bwd_kernel<TR, TH, 1, 16, false, false>))
#define BY_TYPES(K)                                                                                 \
  (a.resid_out.dt ? (hdt ? K(uint16_t, uint16_t) : K(uint16_t, float)) : (hdt ? K(float, uint16_t) : K(float, float)))

// Whether a wave or a workgroup adds a sample's shares: a workgroup's 16 waves
// read one share each where there are up to 16, so many samples wait for
// workgroups (30000 samples of one row of 512: 818 us, 178 a wave each; 300 of 13
// shares 11.9 and 7.6), while a wave reads them one after the other (16 samples
// of 16 shares, 1024 columns: 8.4 us for 4.0; 64 of 8 take 6.0 both ways).
bool sums_by_wave(int splits, int64_t items) { return splits <= 16 && items >= 128 * splits; }

// A launch has fewer than 2^32 threads: a larger grid goes out in pieces.
// launch(first workgroup, workgroups)
template <typename F>
hipError_t in_pieces(int64_t workgroups, int threads, F launch) {
  const int64_t most = 0xffffffffll / threads;
  for (int64_t from = 0; from < workgroups; from += most) {
    launch(from, dim3(unsigned(workgroups - from < most ? workgroups - from : most)));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

int norm_splits(int64_t groups, int64_t group_rows, int cols) {
  // About ten waves of shares on each of 256 CUs (one workgroup at 5120
  // columns, where 512 shares measured 3% slower: a share costs one write and
  // one read of its column sums), of at least eight rows.
  const int64_t waves = (cols + 511) / 512;
  const int64_t total = waves < 10 ? 2560 / waves : 256;
  const int64_t want = (total + groups - 1) / groups;
  const int64_t most = (group_rows + 7) / 8;
  const int64_t n = want < most ? want : most;
  return int(n < 1 ? 1 : n);
}

hipError_t launch_norm_fwd(hipStream_t s, const NormDev& a, bool vec) {
  const Shape sh = shape_of(a.cols, vec);
  const int hdt = a.h.p ? a.h.dt : a.y.dt;
  auto* k = BY_TYPES(FWD_KERNEL);
  const int threads = sh.wave ? 256 : sh.threads;
  return in_pieces(sh.wave ? (a.rows + 3) / 4 : a.rows, threads, [&](int64_t from, dim3 grid) {
    hipLaunchKernelGGL(k, grid, dim3(threads), 0, s, a, from);
  });
}

hipError_t launch_norm_bwd(hipStream_t s, const NormDev& a, bool vec, bool sums) {
  const Shape sh = shape_of(a.cols, vec);
  const int hdt = a.h.p ? a.h.dt : a.d_y.dt;
  const int64_t groups = a.rows / a.group_rows, shares = groups * a.splits;
  auto* k = BY_TYPES(BWD_KERNEL);
  const int threads = sh.wave ? 256 : sh.threads;
  hipError_t e = in_pieces(sh.wave ? (shares + 3) / 4 : shares, threads, [&](int64_t from, dim3 grid) {
    hipLaunchKernelGGL(k, grid, dim3(threads), 0, s, a, from, shares);
  });
  if (e != hipSuccess || !sums) return e;
  const unsigned tiles = unsigned((a.cols + 63) / 64);
  const bool few = sums_by_wave(a.splits, tiles * groups);
  auto* sum = few ? norm_sums_kernel<true> : norm_sums_kernel<false>;
  const int sum_threads = few ? 256 : 1024;
  e = in_pieces(few ? (tiles * groups + 3) / 4 : tiles * groups, sum_threads, [&](int64_t from, dim3 grid) {
    hipLaunchKernelGGL(sum, grid, dim3(sum_threads), 0, s, a, from, groups);
  });
  if (e != hipSuccess || groups == 1 || !(a.d_pre_weight.p || a.d_post_weight.p)) return e;
  hipLaunchKernelGGL(norm_weights_kernel, dim3(tiles), dim3(1024), 0, s, a, groups);
  return hipGetLastError();
}

}  // namespace muon
