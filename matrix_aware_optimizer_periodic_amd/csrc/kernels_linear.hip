// Linear layer with its epilogue on bf16 matrix cores, forward and backward.
//
//   z = x W^T + bias, y = residual + drop(act(z))
//   dz = drop(dy) act'(z), d_bias = column sums of dz, dx = dz W, dW = dz^T x
//
// Forward: one product; bias, activation, dropout and the residual's addition
// are its epilogue, on the fp32 sums.  Backward: one pass over dy and z forms dz
// and the column sums, then dx and dW are one launch of products, or two.  (The
// pass is left out where dz is dy itself, bf16 without activation and dropout, and
// there is no bias or rows are few.)  Small calls are one launch in fp32.
// Roundings to bf16: z as stored, dz as the products' operand, and the results.
// d_bias is summed from the unrounded dz.  dz's rounding puts d_x and dW off by
// 1.66e-3 of their norm (fp32 results too), as much as a bf16 result's own (2.35e-3
// together): the matrix cores take no wider operand at this rate, and a product of
// the remainder as well would double the backward pass's work.
//
// Bound by the matrix cores from some hundreds of rows on, by reading the weights
// (backward: and writing their gradient) below.  Measured on one MI355X (a large
// library product runs at 1520 - 1590 TFLOP/s, a copy at 4.9 - 5.5 TB/s), kernels
// alone: 4096 rows, 2048 -> 8192, bias, gelu and z 137 us (1006 TFLOP/s; all tiles
// of a round end together and then write 67 MB); 8192 -> 2048 with dropout and fp32
// residual 114 - 122 + 27 us (tiles in halves, joined: 134 MB at 5 TB/s); backward of
// 5120 -> 20480 dz 94 us (5.4 TB/s), products 1280 - 1380 (1240 - 1340 TFLOP/s).
#include "block_gemm.h"

namespace muon {
namespace {

constexpr double kEachUs = 0.14;       // plan_of

template <int BT, int ACT, bool DROP>
__global__ __launch_bounds__(256, BT == 256 ? 1 : 2) void linear_kernel(ProdArgs g, LinearExtra<DROP> ext) {
  product_tile<BT, ROWS_ROWS, EPI_LINEAR, ACT>(g, ext);
}
template <int BT, int ACT, bool DROP>
__global__ __launch_bounds__(256) void linear_join_kernel(ProdArgs g, LinearExtra<DROP> ext) {
  product_join<BT, EPI_LINEAR, ACT>(g, ext);
}
// ---- few rows -----------------------------------------------------------------
template <int MT, int NW>
__global__ __launch_bounds__(64 * NW, NW / 8) void linear_few_rows_kernel(Prod p, LinearExtra<true> ext, int act) {
  f32x4_t sum[1];
  int64_t m, n;
  if (!few_rows_sums<MT, false, NW>(p, sum, m, n)) return;
  asm volatile("" : "+v"(sum[0]));     // (nothing below moves up among the sum's reads, whose registers it would spill)
  float v[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = sum[0][k] + (ext.bias ? load_any1(ext.bias, ext.bias_bf16, n + k) : 0.f);
  if (p.c2) store4(p.c2, m * p.ldc2 + n, f32x4_t{v[0], v[1], v[2], v[3]});
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = act == 0 ? act_value<0>(v[k]) : act == 1 ? act_value<1>(v[k]) : v[k];
  if (ext.drop.on) drop<4>(ext.drop, rng_of(ext.drop), uint64_t(m) * unsigned(p.n) + n, v);
  const int64_t r = m * p.ldgu + n, c = m * p.ldc + n;
  if (p.gu) {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] += load_any1(p.gu, !p.f32, r + k);
  }
  if (p.f32) *as_global(reinterpret_cast<f32x4_t*>(static_cast<float*>(p.c) + c)) = f32x4_t{v[0], v[1], v[2], v[3]};
  else store4(p.c, c, f32x4_t{v[0], v[1], v[2], v[3]});
}

// Every workgroup reads all of x, so the time grows with rows x cols x out where
// tiles take the weights' time and 8 to 12 us.  In us, here against tiles, with
// weights from memory: 256 -> 2048 columns 4 against 8 for 64 rows; 2048 -> 2048 5
// against 12 for one row, 12.2 against 13.8 for 64; 2048 -> 12288 11 against 19,
// 16 against 19 for 16, 20 against 20 for 24; 8192 -> 2048 18 against 19 for 12;
// 5120 -> 5120 17 against 19 for 8, 24 against 19 for 12; 5120 -> 20480 43 against
// 44.5 for 4, 53 against 45 for 8; 5120 -> 30720 62 against 64 for 4, 76 against
// 64 for 8.
bool few_rows(int64_t t, int64_t d, int64_t n) {
  const double dn = double(d) * n;
  if (t <= 8) return t * dn <= 4.6e8;
  return t <= 64 && (t * dn <= 2.7e8 || (t * d <= 50000 && dn <= 3e7));
}

hipError_t run_few_rows(hipStream_t s, const Prod& p, const LinearExtra<true>& ext, int act) {
  const int cols = p.m <= 8 ? 8 : 16;
  const unsigned grid = unsigned((p.n + cols - 1) / cols);
  const bool wide = grid <= 256;      // a workgroup per CU at most: more waves to each
  auto* k = p.m <= 8    ? (wide ? linear_few_rows_kernel<0, 16> : linear_few_rows_kernel<0, 8>)
            : p.m <= 16 ? (wide ? linear_few_rows_kernel<1, 16> : linear_few_rows_kernel<1, 8>)
            : p.m <= 32 ? (wide ? linear_few_rows_kernel<2, 16> : linear_few_rows_kernel<2, 8>)
                        : (wide ? linear_few_rows_kernel<4, 16> : linear_few_rows_kernel<4, 8>);
  hipLaunchKernelGGL(k, dim3(grid), dim3(wide ? 1024 : 512), 0, s, p, ext, act);
  return hipGetLastError();
}

template <int ACT, bool DROP>
hipError_t run_linear(hipStream_t s, const ProdArgs& g, const LinearDev& f) {
  const Plan q = plan_of(g, false, kEachUs);
  const LinearExtra<DROP> ext{f.bias.p, f.bias.dt, f.drop};
  return q.bt == 256 ? launch_prod<256, EPI_LINEAR>(s, g, q, &linear_kernel<256, ACT, DROP>, &linear_join_kernel<256, ACT, DROP>, 0, ext)
                     : launch_prod<128, EPI_LINEAR>(s, g, q, &linear_kernel<128, ACT, DROP>, &linear_join_kernel<128, ACT, DROP>, 0, ext);
}

// ---- dz and d_bias --------------------------------------------------------------
// A thread has eight columns of every 256 / width-th row of its workgroup's
// share, `width` threads beside each other.  The shares' column sums are added in
// a fixed order: by the rows within a workgroup, then by the workgroups behind the
// gradients' products (or by a kernel of their own).  Bound by memory: the slope of
// an activation is some fifteen instructions (with divisions it was sixty, and
// 4096 x 20480 took 138 us).  Waves that hide each other's latency do better than
// rows read ahead: 4096 x 20480 with gelu 93 us (5.4 TB/s), 100 with four rows read
// ahead; 777 x 2728 with silu and dropout from fp32 7.8 and 10.2.
struct DzShape {
  int width_log;         // threads along the columns: 1 << width_log
  int blocks;            // workgroups along the columns
  int splits;            // shares of the rows
  int64_t rows;          // rows of a share
};
DzShape dz_shape(int64_t rows, int64_t out) {
  DzShape d{};
  const int64_t chunks = out / 8;
  while (d.width_log < 6 && (int64_t(1) << d.width_log) < chunks) ++d.width_log;
  d.blocks = int((chunks + (1 << d.width_log) - 1) >> d.width_log);
  const int64_t turn = 256 >> d.width_log;                       // rows at a time
  const int64_t turns = (rows + turn - 1) / turn;
  d.splits = int(std::max<int64_t>(1, std::min<int64_t>(turns, std::min<int64_t>(256, 1024 / d.blocks))));
  d.rows = (turns + d.splits - 1) / d.splits * turn;
  d.splits = int((rows + d.rows - 1) / d.rows);
  return d;
}

template <typename T, int ACT>
__global__ __launch_bounds__(256) void linear_dz_kernel(LinearDev a, DzShape d) {
  __shared__ float red[256][9];
  const int cc = threadIdx.x & ((1 << d.width_log) - 1), rr = threadIdx.x >> d.width_log, turn = 256 >> d.width_log;
  const int64_t n = (int64_t(blockIdx.x << d.width_log) + cc) * 8;
  const int64_t end = min(a.rows, (int64_t(blockIdx.y) + 1) * d.rows);
  const Rng rng = a.drop.on ? rng_of(a.drop) : Rng{};
  float sum[8] = {};
  if (n < a.out) {
    for (int64_t r = int64_t(blockIdx.y) * d.rows + rr; r < end; r += turn) {
      float v[8], z[8];
      load_vals<T, 8>(a.d_y.p, r * a.d_y.ld + n, v);
      if constexpr (ACT != 2) load_vals<uint16_t, 8>(a.z.p, r * a.z.ld + n, z);
      if (a.drop.on) drop<8>(a.drop, rng, uint64_t(r) * uint64_t(a.out) + n, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if constexpr (ACT != 2) v[k] *= act_slope<ACT>(z[k]);
        sum[k] += v[k];
      }
      if (a.dz) store_vals<uint16_t, 8>(a.dz, r * a.out + n, v);
    }
  }
  if (!a.d_bias.p) return;
#pragma unroll
  for (int k = 0; k < 8; ++k) red[threadIdx.x][k] = sum[k];
  __syncthreads();
  for (int i = threadIdx.x; i < (8 << d.width_log); i += 256) {
    const int64_t at = (int64_t(blockIdx.x) << d.width_log) * 8 + i;
    if (at >= a.out) return;
    float s = 0.f;
    for (int r = 0; r < turn; ++r) s += red[(r << d.width_log) + (i >> 3)][i & 7];
    if (d.splits > 1) a.sums[int64_t(blockIdx.y) * a.out + at] = s;
    else store_any1(a.d_bias.p, a.d_bias.dt, at, s);
  }
}

// Column sums of a few rows, 256 columns to a workgroup: of the shares' sums, or
// of dy itself where that is dz and has few rows.
struct BiasSums {
  const void* rows;
  int64_t ld;
  NormMat d_bias;
  int64_t out;
  int32_t count, bf16;
  int32_t item0;         // the first workgroup of a launch that does this
};
__device__ __forceinline__ void add_bias_sums(const BiasSums& b, int block) {
  const int64_t n = int64_t(block) * 256 + threadIdx.x;
  if (n >= b.out) return;
  float s = 0.f;
  if (b.bf16) {
#pragma unroll 8
    for (int i = 0; i < b.count; ++i) s += load_any1(b.rows, 1, i * b.ld + n);
  } else {
#pragma unroll 8
    for (int i = 0; i < b.count; ++i) s += load_any1(b.rows, 0, i * b.ld + n);
  }
  store_any1(b.d_bias.p, b.d_bias.dt, n, s);
}
// (a thread reads eight rows at a time; a launch less: 32 rows of 2048 -> 2048, both
// gradients and d_bias, 17.4 -> 14 us)
bool bias_from_rows(const LinearDev& f) { return f.d_bias.p && !f.dz && f.act == 2 && !f.drop.on && f.d_y.dt && f.rows <= 64; }
__global__ __launch_bounds__(256) void linear_bias_kernel(BiasSums b) { add_bias_sums(b, int(blockIdx.x)); }

template <int BT>
__global__ __launch_bounds__(256, BT == 256 ? 1 : 2) void linear_grads_kernel(ProdArgs g, BiasSums b) {
  if (int(blockIdx.x) >= b.item0) return add_bias_sums(b, int(blockIdx.x) - b.item0);
  product_tile<BT, MIXED_COLS, EPI_PLAIN, 0>(g, NoExtra{});
}
template <int BT>
__global__ __launch_bounds__(256) void linear_grads_join_kernel(ProdArgs g, BiasSums) {
  product_join<BT, EPI_PLAIN, 0>(g, NoExtra{});
}

// ---- small backward calls ---------------------------------------------------------
// Every gradient in one launch, in fp32 throughout: dz is formed where it is used and
// not rounded.  A workgroup has 32 x 32 results of dx or dW, each thread 2 x 2,
// and goes over 32 values of the sum at a time, the next ones read ahead; those of
// dW's first columns add up d_bias.  A turn of 32 takes about 1.4 us, the loads'
// latency, so sums are kept short.
//
// In us, both gradients and d_bias with gelu, here against two or three launches of
// the other forms, replayed and (called from Python): 5 rows 608 -> 104 columns 7.9
// against 7.8 (13.6 against 18.4), 41 rows 144 -> 40 5.8 against 7.6 (13.3 against
// 18.2), 64 rows 4096 -> 64 6.7 against 8.0 (13.6 against 18.4); 64 rows 256 -> 256
// 14.6 against 9.7 (14.7 against 18.3), 440 rows 64 -> 184 27 against 11.
struct SmallGrads {
  LinearDev f;
  int32_t col_blocks, dx_tiles, dw_cols;     // dw_cols: column blocks of dW (1 for d_bias alone)
};
bool small_grads(int64_t t, int64_t d, int64_t n) { return t <= 128 && n <= 128 && t * d * n <= 20000000; }

// Four values at element e, a multiple of four of rows that are 16-byte aligned.
__device__ __forceinline__ void load4(const void* p, int dt, int64_t e, float (&v)[4]) {
  if (dt) {
    const u32x2_t u = *as_global(reinterpret_cast<const u32x2_t*>(static_cast<const uint16_t*>(p) + e));
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = k & 1 ? __uint_as_float(u[k / 2] & 0xffff0000u) : bf16_to_f32(u[k / 2] & 0xffffu);
  } else {
    const f32x4_t u = *as_global(reinterpret_cast<const f32x4_t*>(static_cast<const float*>(p) + e));
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = u[k];
  }
}

// Four values of dz, row r, columns n .. n + 3, fp32.
__device__ __forceinline__ void dz4(const LinearDev& f, const Rng& rng, int64_t r, int64_t n, float (&v)[4]) {
  float z[4];
  load4(f.d_y.p, f.d_y.dt, r * f.d_y.ld + n, v);
  if (f.act != 2) load4(f.z.p, 1, r * f.z.ld + n, z);
  if (f.drop.on) drop<4>(f.drop, rng, uint64_t(r) * uint64_t(f.out) + uint64_t(n), v);
  if (f.act == 2) return;
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] *= f.act == 0 ? act_slope<0>(z[k]) : act_slope<1>(z[k]);
}

__global__ __launch_bounds__(256) void linear_small_grads_kernel(SmallGrads a) {
  __shared__ float sa[32][36], sb[32][36];             // [k][row of the result], [k][column]
  const LinearDev& f = a.f;
  const int id = int(blockIdx.x), tid = threadIdx.x;
  const bool is_w = id >= a.dx_tiles;
  const int blocks = is_w ? a.dw_cols : a.col_blocks, tile = is_w ? id - a.dx_tiles : id;
  const int64_t m0 = int64_t(tile / blocks) * 32, c0 = int64_t(tile % blocks) * 32;
  const int64_t rows = is_w ? f.out : f.rows, depth = is_w ? f.rows : f.out;
  const NormMat& o = is_w ? f.d_w : f.d_x;             // absent where dW's tiles are there for d_bias
  const Rng rng = f.drop.on ? rng_of(f.drop) : Rng{};
  const int i8 = tid >> 3, q4 = (tid & 7) * 4;         // this thread's four values of each operand
  float va[4], vb[4];
  auto fetch = [&](int64_t k0) {
    // dz: columns are k for dx, rows are k for dW
    const int64_t r = is_w ? k0 + i8 : m0 + i8, n = is_w ? m0 + q4 : k0 + q4;
#pragma unroll
    for (int k = 0; k < 4; ++k) va[k] = vb[k] = 0.f;
    if (r < f.rows && n < f.out) dz4(f, rng, r, n, va);
    const NormMat& b = is_w ? f.x : f.w;
    if (o.p && k0 + i8 < depth && c0 + q4 < f.cols) load4(b.p, 1, (k0 + i8) * b.ld + c0 + q4, vb);
  };
  const int ty = (tid >> 4) * 2, tx = (tid & 15) * 2;
  float acc[2][2] = {}, sum = 0.f;
  const bool bias = is_w && c0 == 0 && f.d_bias.p && tid < 32;
  fetch(0);
  for (int64_t k0 = 0; k0 < depth; k0 += 32) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (is_w) sa[i8][q4 + k] = va[k];
      else sa[q4 + k][i8] = va[k];
      sb[i8][q4 + k] = vb[k];
    }
    __syncthreads();
    if (k0 + 32 < depth) fetch(k0 + 32);
#pragma unroll 8
    for (int k = 0; k < 32; ++k) {
      const float a0 = sa[k][ty], a1 = sa[k][ty + 1], b0 = sb[k][tx], b1 = sb[k][tx + 1];
      acc[0][0] = fmaf(a0, b0, acc[0][0]);
      acc[0][1] = fmaf(a0, b1, acc[0][1]);
      acc[1][0] = fmaf(a1, b0, acc[1][0]);
      acc[1][1] = fmaf(a1, b1, acc[1][1]);
    }
    if (bias)
#pragma unroll 8
      for (int k = 0; k < 32; ++k) sum += sa[k][tid];
    __syncthreads();
  }
  if (bias && m0 + tid < f.out) store_any1(f.d_bias.p, f.d_bias.dt, m0 + tid, sum);
  if (!o.p || c0 + tx >= f.cols) return;
#pragma unroll
  for (int y = 0; y < 2; ++y)
    if (m0 + ty + y < rows)
#pragma unroll
      for (int x = 0; x < 2; ++x) store_any1(o.p, o.dt, (m0 + ty + y) * o.ld + c0 + tx + x, acc[y][x]);
}

hipError_t run_small_grads(hipStream_t s, const LinearDev& f) {
  SmallGrads a{f, int32_t((f.cols + 31) / 32), 0, 0};
  if (f.d_x.p) a.dx_tiles = int32_t((f.rows + 31) / 32) * a.col_blocks;
  a.dw_cols = f.d_w.p ? a.col_blocks : f.d_bias.p ? 1 : 0;
  const unsigned grid = unsigned(a.dx_tiles + int32_t((f.out + 31) / 32) * a.dw_cols);
  hipLaunchKernelGGL(linear_small_grads_kernel, dim3(grid), dim3(256), 0, s, a);
  return hipGetLastError();
}

// ---- the weight's gradient from few rows ----------------------------------------
// dW = dz^T x of up to 16 rows, bound by writing dW.  A wave keeps the x of 256
// columns as fragments and goes down the columns of dz, four at a time, with
// MFMAs of 16 blocks of 4 x 4: a block's rows are columns of x, so that a lane ends
// with eight consecutive values of a row of dW and 16 lanes write 256 bytes beside
// each other (512 in fp32).  MFMAs of one 16 x 16 block leave 64 bytes to four
// lanes: 8 rows of 5120 -> 30720 columns, both gradients, 187 us.  The stores are
// non-temporal: as others they leave the caches full of dW, and reading W for d_x
// next to it takes 98 us instead of 57 (in all 159, now 132: 4.8 TB/s; as tiles of
// one launch with d_x 158).  d_bias, where it is wanted here, comes from the same
// columns of dz.
constexpr int kOuterCols = 256;          // of a wave, four waves beside each other
constexpr int kOuterGroups = 1024;       // workgroups of a launch, about
constexpr int kOuterRows = 256;          // columns of dz that a workgroup holds
struct Outer {
  const void *dz, *x;
  int64_t ld_dz, ld_x, n, d;
  NormMat dw, d_bias;
  int32_t rows, span;                    // columns of dz to a workgroup, a multiple of four
};

// v_mfma_f32_4x4x4_16b_bf16: lane 4 b + i gives row (A) or column (B) i of block b,
// four k; result v of lane 4 b + j is row v, column j of block b.
__device__ __forceinline__ f32x4_t mfma4(u32x2_t a, u32x2_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(__builtin_bit_cast(s16x4_t, a), __builtin_bit_cast(s16x4_t, b), c, 0, 0, 0);
}

// Lane i of four holds row i of a 4 x 4 block of bf16; afterwards column i.
__device__ __forceinline__ u32x2_t turned4(u32x2_t a, int i) {
  unsigned v[4];
  auto from = [&](auto j) {
    constexpr int J = decltype(j)::value;
    const unsigned lo = unsigned(__builtin_amdgcn_mov_dpp(int(a[0]), J * 0x55, 0xf, 0xf, true));
    const unsigned hi = unsigned(__builtin_amdgcn_mov_dpp(int(a[1]), J * 0x55, 0xf, 0xf, true));
    v[J] = ((i & 2 ? hi : lo) >> (16 * (i & 1))) & 0xffffu;
  };
  from(std::integral_constant<int, 0>{});
  from(std::integral_constant<int, 1>{});
  from(std::integral_constant<int, 2>{});
  from(std::integral_constant<int, 3>{});
  return u32x2_t{v[0] | v[1] << 16, v[2] | v[3] << 16};
}

// KT: steps of four rows.
template <bool F32, int KT>
__global__ __launch_bounds__(256) void linear_outer_kernel(Outer o) {
  __shared__ __attribute__((aligned(16))) uint16_t z[kOuterRows * 4 * KT];        // [column of dz][row]
  const int lane = threadIdx.x & 63, b = lane >> 2, i = lane & 3;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = int64_t(blockIdx.x) * o.span, c0 = (int64_t(blockIdx.y) * 4 + wave) * kOuterCols;
  const int here = int(min(int64_t(o.span), o.n - n0));
  const auto* dz = as_global(static_cast<const uint16_t*>(o.dz));
  const auto* x = as_global(static_cast<const uint16_t*>(o.x));
  for (int t = wave; t < 4 * KT; t += 4)
    for (int n = lane; n < here; n += 64) z[n * 4 * KT + t] = t < o.rows ? dz[t * o.ld_dz + n0 + n] : uint16_t(0);
  constexpr int G = kOuterCols / 128;
  u32x2_t fx[G][2][KT];
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int k = 0; k < KT; ++k) {
        const int64_t c = c0 + 128 * g + 8 * b + 4 * h;
        u32x2_t v{0, 0};
        if (c < o.d && 4 * k + i < o.rows) v = *reinterpret_cast<const MUON_GLOBAL u32x2_t*>(x + (4 * k + i) * o.ld_x + c);
        fx[g][h][k] = turned4(v, i);
      }
  __syncthreads();
  if (blockIdx.y == 0 && o.d_bias.p && int(threadIdx.x) < here) {
    float s = 0.f;
#pragma unroll
    for (int t = 0; t < 4 * KT; ++t) s += bf16_to_f32(z[threadIdx.x * 4 * KT + t]);
    store_any1(o.d_bias.p, o.d_bias.dt, n0 + threadIdx.x, s);
  }
  if (c0 >= o.d) return;
  for (int n = i; n < here; n += 4) {        // (here is a multiple of four)
    u32x2_t fz[KT];
#pragma unroll
    for (int k = 0; k < KT; ++k) fz[k] = *(const MUON_LOCAL u32x2_t*)(const MUON_LOCAL uint16_t*)(z + n * 4 * KT + 4 * k);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      f32x4_t acc[2] = {(f32x4_t)(0.f), (f32x4_t)(0.f)};
#pragma unroll
      for (int k = 0; k < KT; ++k) {
        acc[0] = mfma4(fx[g][0][k], fz[k], acc[0]);
        acc[1] = mfma4(fx[g][1][k], fz[k], acc[1]);
      }
      const int64_t c = c0 + 128 * g + 8 * b;
      const float v[8] = {acc[0][0], acc[0][1], acc[0][2], acc[0][3], acc[1][0], acc[1][1], acc[1][2], acc[1][3]};
      using T = std::conditional_t<F32, float, uint16_t>;
      if (c < o.d) store_vals_past<T>(o.dw.p, (n0 + n) * o.dw.ld + c, v);
    }
  }
}

// In us, both gradients and d_bias, here against tiles: 8 rows 5120 -> 30720 131
// against 155, 20480 -> 5120 94 against 99, 5120 -> 5120 34 against 32, 2048 ->
// 12288 38 against 33; 16 rows 5120 -> 30720 136 against 155, 20480 -> 5120 98
// against 100; 24 rows 5120 -> 30720 157 against 155.
bool outer_rows(int64_t t, int64_t d, int64_t n) { return t <= 16 && d * n >= 100000000; }

hipError_t run_outer(hipStream_t s, const Outer& o0) {
  Outer o = o0;
  const int64_t groups = (o.d + 4 * kOuterCols - 1) / (4 * kOuterCols);
  o.span = int32_t(std::min<int64_t>(kOuterRows, std::max<int64_t>(16, (o.n * groups / kOuterGroups + 3) / 4 * 4)));
  const dim3 grid(unsigned((o.n + o.span - 1) / o.span), unsigned(groups));
  auto* k = o.rows <= 8 ? (o.dw.dt ? linear_outer_kernel<false, 2> : linear_outer_kernel<true, 2>)
                        : (o.dw.dt ? linear_outer_kernel<false, 4> : linear_outer_kernel<true, 4>);
  hipLaunchKernelGGL(k, grid, dim3(256), 0, s, o);
  return hipGetLastError();
}

// ---- the gradients' products --------------------------------------------------
// dx, dW or both, in one launch or two.  Only a launch's first product is divided
// where its sums are long for the tiles it has, so the one that needs it comes
// first, or each is launched alone (an allowance of 4 us), where that is a fifth
// less by the estimate: 16384 rows of 2048 -> 32 columns, whose dW has 16 tiles of
// 512 stages, 175 us with dW behind dx and 47 in two launches; 4096 rows of 2048 ->
// 8192, where the estimates are close, 235 with dx first and 255 turned.
struct GradPlan {
  ProdArgs g[2];
  Plan q[2];
  int launches;
};
GradPlan grad_plan(int64_t t, int64_t d, int64_t n, bool d_x, bool d_w) {
  const Prod dx = sizes(t, d, n);
  Prod dw = sizes(n, d, t);
  dw.acols = 1;
  auto one = [](const Prod& a, const Prod* b) {
    ProdArgs g = alone(a);
    if (b) g.p[g.count++] = *b;
    return g;
  };
  GradPlan best{};
  if (!d_x && !d_w) return best;
  best.launches = 1;
  best.g[0] = d_x && d_w ? one(dx, &dw) : one(d_x ? dx : dw, nullptr);
  best.q[0] = plan_of(best.g[0], false, kEachUs);
  if (!d_x || !d_w) return best;
  const ProdArgs turned = one(dw, &dx);
  const Plan q = plan_of(turned, false, kEachUs);
  if (q.us < 0.8 * best.q[0].us) { best.g[0] = turned; best.q[0] = q; }
  GradPlan apart{{one(dx, nullptr), one(dw, nullptr)}, {}, 2};
  for (int i = 0; i < 2; ++i) apart.q[i] = plan_of(apart.g[i], false, kEachUs);
  return apart.q[0].us + apart.q[1].us + 4 < 0.8 * best.q[0].us ? apart : best;
}
size_t grad_part_bytes(const GradPlan& p) {
  size_t most = 0;
  for (int i = 0; i < p.launches; ++i) most = std::max(most, part_bytes(p.g[i], p.q[i]));
  return most;
}

}  // namespace

size_t linear_fwd_part_bytes(int64_t t, int64_t d, int64_t n) {
  if (t == 0 || few_rows(t, d, n)) return 0;
  const ProdArgs g = alone(sizes(t, n, d));
  return part_bytes(g, plan_of(g, false, kEachUs));
}
size_t linear_bwd_part_bytes(int64_t t, int64_t d, int64_t n, bool d_x, bool d_w) {
  if (t == 0 || !(d_x || d_w)) return 0;
  return grad_part_bytes(grad_plan(t, d, n, d_x, d_w && !outer_rows(t, d, n)));
}
bool linear_small_grads(int64_t rows, int64_t cols, int64_t out) { return small_grads(rows, cols, out); }
int linear_sum_splits(int64_t rows, int64_t out) { return dz_shape(rows, out).splits; }

hipError_t launch_linear_fwd(hipStream_t s, const LinearDev& f) {
  ProdArgs g = alone(sizes(f.rows, f.out, f.cols));
  g.part = f.part;
  Prod& p = g.p[0];
  p.a = f.x.p; p.lda = f.x.ld;
  p.b = f.w.p; p.ldb = f.w.ld;
  p.c = f.y.p; p.ldc = f.y.ld; p.f32 = f.y.dt == 0;
  p.c2 = f.z.p; p.ldc2 = f.z.ld;
  p.gu = f.resid.p; p.ldgu = f.resid.ld;
  if (few_rows(f.rows, f.cols, f.out)) return run_few_rows(s, p, LinearExtra<true>{f.bias.p, f.bias.dt, f.drop}, f.act);
  if (f.drop.on) return f.act == 0 ? run_linear<0, true>(s, g, f) : f.act == 1 ? run_linear<1, true>(s, g, f) : run_linear<2, true>(s, g, f);
  return f.act == 0 ? run_linear<0, false>(s, g, f) : f.act == 1 ? run_linear<1, false>(s, g, f) : run_linear<2, false>(s, g, f);
}

template <typename T>
void launch_dz(hipStream_t s, const LinearDev& f, const DzShape& d) {
  auto* k = f.act == 0 ? linear_dz_kernel<T, 0> : f.act == 1 ? linear_dz_kernel<T, 1> : linear_dz_kernel<T, 2>;
  hipLaunchKernelGGL(k, dim3(unsigned(d.blocks), unsigned(d.splits)), dim3(256), 0, s, f, d);
}

hipError_t launch_linear_bwd(hipStream_t s, const LinearDev& f) {
  if (small_grads(f.rows, f.cols, f.out)) return run_small_grads(s, f);
  BiasSums b{};
  unsigned bias_blocks = 0;
  const bool outer = f.d_w.p && outer_rows(f.rows, f.cols, f.out), bias_there = outer && !f.dz && f.act == 2 && !f.drop.on && f.d_y.dt;
  if (!bias_there && bias_from_rows(f)) {
    b = BiasSums{f.d_y.p, f.d_y.ld, f.d_bias, f.out, int32_t(f.rows), 1, 0};
    bias_blocks = unsigned((f.out + 255) / 256);
  } else if (f.dz || (f.d_bias.p && !bias_there)) {
    const DzShape d = dz_shape(f.rows, f.out);
    if (f.d_y.dt) launch_dz<uint16_t>(s, f, d);
    else launch_dz<float>(s, f, d);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (f.d_bias.p && d.splits > 1) {
      b = BiasSums{f.sums, f.out, f.d_bias, f.out, d.splits, 0, 0};
      bias_blocks = unsigned((f.out + 255) / 256);
    }
  }
  if (outer) {
    const Outer o{f.dz ? f.dz : f.d_y.p, f.x.p, f.dz ? f.out : f.d_y.ld, f.x.ld, f.out, f.cols, f.d_w,
                  bias_there ? f.d_bias : NormMat{}, int32_t(f.rows), 0};
    const hipError_t e = run_outer(s, o);
    if (e != hipSuccess) return e;
  }
  if (!f.d_x.p && (!f.d_w.p || outer)) {
    if (bias_blocks) hipLaunchKernelGGL(linear_bias_kernel, dim3(bias_blocks), dim3(256), 0, s, b);
    return hipGetLastError();
  }
  GradPlan plan = grad_plan(f.rows, f.cols, f.out, f.d_x.p, f.d_w.p && !outer);
  const void* dz = f.dz ? f.dz : f.d_y.p;
  const int64_t ld = f.dz ? f.out : f.d_y.ld;
  hipError_t e = hipSuccess;
  for (int k = 0; k < plan.launches && e == hipSuccess; ++k) {
    ProdArgs& g = plan.g[k];
    const Plan& q = plan.q[k];
    g.part = f.part;                     // (a launch's join has read it before the next one begins)
    for (int i = 0; i < g.count; ++i) {
      Prod& p = g.p[i];
      p.a = dz; p.lda = ld;
      if (p.acols) {
        p.b = f.x.p; p.ldb = f.x.ld;
        p.c = f.d_w.p; p.ldc = f.d_w.ld; p.f32 = f.d_w.dt == 0;
      } else {
        p.b = f.w.p; p.ldb = f.w.ld;
        p.c = f.d_x.p; p.ldc = f.d_x.ld;
      }
    }
    b.item0 = items_of(g, q);
    e = q.bt == 256 ? launch_prod<256, EPI_PLAIN>(s, g, q, &linear_grads_kernel<256>, &linear_grads_join_kernel<256>, bias_blocks, b)
                    : launch_prod<128, EPI_PLAIN>(s, g, q, &linear_grads_kernel<128>, &linear_grads_join_kernel<128>, bias_blocks, b);
    bias_blocks = 0;
  }
  return e;
}

}  // namespace muon
