// Linear layer with its epilogue on bf16 matrix cores, forward and backward.
//
//   z = x W^T + bias, y = residual + drop(act(z))
//   dz = drop(dy) act'(z), d_bias = column sums of dz, dx = dz W, dW = dz^T x
//
// Forward: one product; bias, activation, dropout and the residual's addition
// are its epilogue, on the fp32 sums.  Backward: one pass over dy and z forms dz
// and the column sums, then dx and dW are one launch of products.  (The pass is
// left out where dz is dy itself: bf16, no activation, no dropout, no bias.)
// Roundings to bf16: z as stored, dz as the products' operand, and the results.
// d_bias is summed from the unrounded dz.
#include "block_gemm.h"

namespace muon {
namespace {

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

bool few_rows(int64_t t, int64_t d, int64_t n) {
  const double dn = double(d) * n, weights_us = 2 * dn / 5.1e6;
  if (t <= 8) return t * dn * (2.0 / 8) / 23e6 <= 12;
  return t <= 64 && t * dn * (2.0 / 16) / 7e6 <= 4 + weights_us / 8;
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
  const Plan q = plan_of(g, false);
  const LinearExtra<DROP> ext{f.bias.p, f.bias.dt, f.drop};
  return q.bt == 256 ? launch_prod<256, EPI_LINEAR>(s, g, q, &linear_kernel<256, ACT, DROP>, &linear_join_kernel<256, ACT, DROP>, 0, ext)
                     : launch_prod<128, EPI_LINEAR>(s, g, q, &linear_kernel<128, ACT, DROP>, &linear_join_kernel<128, ACT, DROP>, 0, ext);
}

// ---- dz and d_bias --------------------------------------------------------------
// A thread has eight columns of every 256 / width-th row of its workgroup's
// share, `width` threads beside each other, and reads kAhead rows before it works
// on them.  The shares' column sums are added in a fixed order: by the rows
// within a workgroup, then by the workgroups behind the gradients' products (or
// by a kernel of their own).  Bound by memory: the slope of an activation is some
// fifteen instructions (with divisions it was sixty, and as long as the memory).
constexpr int kAhead = 4;
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
  const int64_t turn = kAhead * (256 >> d.width_log);            // rows at a time
  const int64_t turns = (rows + turn - 1) / turn;
  d.splits = int(std::max<int64_t>(1, std::min<int64_t>(turns, std::min<int64_t>(512, 1024 / d.blocks))));
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
    for (int64_t r0 = int64_t(blockIdx.y) * d.rows + rr; r0 < end; r0 += kAhead * turn) {
      float v[kAhead][8], z[kAhead][8];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int64_t r = min(r0 + i * turn, end - 1);           // (past the end: the last one again)
        load_vals<T, 8>(a.d_y.p, r * a.d_y.ld + n, v[i]);
        if constexpr (ACT != 2) load_vals<uint16_t, 8>(a.z.p, r * a.z.ld + n, z[i]);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int64_t r = r0 + i * turn;
        if (r >= end) break;
        if (a.drop.on) drop<8>(a.drop, rng, uint64_t(r) * uint64_t(a.out) + n, v[i]);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if constexpr (ACT != 2) v[i][k] *= act_slope<ACT>(z[i][k]);
          sum[k] += v[i][k];
        }
        if (a.dz) store_vals<uint16_t, 8>(a.dz, r * a.out + n, v[i]);
      }
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

// The shares' sums of 256 columns: what a workgroup adds of them.
struct BiasSums {
  const float* sums;     // [splits][out]
  NormMat d_bias;
  int64_t out;
  int32_t splits;
  int32_t item0;         // the first workgroup of a launch that does this
};
__device__ __forceinline__ void add_bias_sums(const BiasSums& b, int block) {
  const int64_t n = int64_t(block) * 256 + threadIdx.x;
  if (n >= b.out) return;
  float s = 0.f;
#pragma unroll 8
  for (int i = 0; i < b.splits; ++i) s += as_global(b.sums)[i * b.out + n];
  store_any1(b.d_bias.p, b.d_bias.dt, n, s);
}
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

// ---- the gradients' products --------------------------------------------------
ProdArgs grad_sizes(int64_t t, int64_t d, int64_t n, bool d_x, bool d_w) {
  ProdArgs g{};
  if (d_x) g.p[g.count++] = sizes(t, d, n);
  if (d_w) {
    g.p[g.count] = sizes(n, d, t);
    g.p[g.count++].acols = 1;
  }
  return g;
}

}  // namespace

size_t linear_fwd_part_bytes(int64_t t, int64_t d, int64_t n) {
  if (t == 0 || few_rows(t, d, n)) return 0;
  const ProdArgs g = alone(sizes(t, n, d));
  return part_bytes(g, plan_of(g, false));
}
size_t linear_bwd_part_bytes(int64_t t, int64_t d, int64_t n, bool d_x, bool d_w) {
  if (t == 0 || !(d_x || d_w)) return 0;
  const ProdArgs g = grad_sizes(t, d, n, d_x, d_w);
  return part_bytes(g, plan_of(g, false));
}
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
  BiasSums b{};
  unsigned bias_blocks = 0;
  if (f.dz || f.d_bias.p) {
    const DzShape d = dz_shape(f.rows, f.out);
    if (f.d_y.dt) launch_dz<uint16_t>(s, f, d);
    else launch_dz<float>(s, f, d);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (f.d_bias.p && d.splits > 1) {
      b = BiasSums{f.sums, f.d_bias, f.out, d.splits, 0};
      bias_blocks = unsigned((f.out + 255) / 256);
    }
  }
  if (!f.d_x.p && !f.d_w.p) {
    if (bias_blocks) hipLaunchKernelGGL(linear_bias_kernel, dim3(bias_blocks), dim3(256), 0, s, b);
    return hipGetLastError();
  }
  ProdArgs g = grad_sizes(f.rows, f.cols, f.out, f.d_x.p, f.d_w.p);
  g.part = f.part;
  const void* dz = f.dz ? f.dz : f.d_y.p;
  const int64_t ld = f.dz ? f.out : f.d_y.ld;
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
  const Plan q = plan_of(g, false);
  b.item0 = items_of(g, q);
  return q.bt == 256 ? launch_prod<256, EPI_PLAIN>(s, g, q, &linear_grads_kernel<256>, &linear_grads_join_kernel<256>, bias_blocks, b)
                     : launch_prod<128, EPI_PLAIN>(s, g, q, &linear_grads_kernel<128>, &linear_grads_join_kernel<128>, bias_blocks, b);
}

}  // namespace muon
