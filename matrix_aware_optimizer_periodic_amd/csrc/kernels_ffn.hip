// Gated feed-forward block on bf16 matrix cores, forward and backward.
//
//   g = x Wg^T, u = x Wu^T, h = act(g) u, y = h Wd^T
//   dh = dy Wd, dg = dh u act'(g), du = dh act(g)
//   dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x, dWd = dy^T h
//
// Five products of one kernel template.  Every product is
// C[m][n] = sum_k A(m, k) B(n, k); an operand lies in memory either along k
// ("rows": x, h, dy, dg | du, and the weights of the forward pass) or along
// m / n ("cols": the weights in dh and dx, both operands of the weights'
// gradients).  Row operands are staged as rows of 64 k values and read as
// they are, column operands as 64 rows of the tile's width and read through the
// transposing LDS read, so that nothing is transposed in memory.
//
// Fusions: one product forms g and u side by side (the B tile takes 16 rows
// of Wg and 16 of Wu in turn, so a lane holds both for the same columns) and
// writes h; the dh product's epilogue reads g and u and writes dg, du and h;
// dx, one product over 2 f, and the three weights' gradients are one launch.
//
// Bound by the matrix cores from some hundreds of rows on, by reading the
// weights below.  Roundings to bf16: g and u as stored, h and dg, du as the
// next product's operands, and the results.
//
// Measured on one MI355X (a large library product runs at 1460 TFLOP/s), medians
// of twelve calls over several cards: 4096 rows, 2048 x 8192, gate and up 255 -
// 284 us (970 - 1080 TFLOP/s), down 118 - 124 + 14 us; 4096 rows, 5120 x 20480,
// dh 872 - 904 us (950 - 985; 160 us of it would take its epilogue's 0.84 GB
// alone), dx and the weights' gradients 3415 - 3450 us (1245 - 1258).
#include "block_gemm.h"

namespace muon {
namespace {

template <int BT, int LIE, int EPI, int ACT>
__global__ __launch_bounds__(256, BT == 256 ? 1 : 2) void ffn_gemm_kernel(ProdArgs g) {
  product_tile<BT, LIE, EPI, ACT>(g, NoExtra{});
}
template <int BT, int EPI, int ACT>
__global__ __launch_bounds__(256) void ffn_join_kernel(ProdArgs g) {
  product_join<BT, EPI, ACT>(g, NoExtra{});
}

template <int LIE, int EPI, int ACT = 0>
hipError_t run_prod(hipStream_t s, const ProdArgs& g) {
  const Plan q = plan_of(g, EPI == EPI_GATE);
  return q.bt == 256 ? launch_prod<256, EPI>(s, g, q, &ffn_gemm_kernel<256, LIE, EPI, ACT>, &ffn_join_kernel<256, EPI, ACT>, 0)
                     : launch_prod<128, EPI>(s, g, q, &ffn_gemm_kernel<128, LIE, EPI, ACT>, &ffn_join_kernel<128, EPI, ACT>, 0);
}

ProdArgs backward_sizes(int64_t t, int64_t d, int64_t h) {
  ProdArgs g{};
  g.p[0] = sizes(t, d, h, 2);
  g.p[1] = g.p[2] = sizes(h, d, t);
  g.p[3] = sizes(d, h, t);
  g.count = 4;
  return g;
}

// ---- few rows -----------------------------------------------------------------
template <int MT, bool GATE, int ACT, int NW>
__global__ __launch_bounds__(64 * NW, NW / 8) void ffn_few_rows_kernel(Prod p) {
  f32x4_t sum[GATE ? 2 : 1];
  int64_t m, n;
  if (!few_rows_sums<MT, GATE, NW>(p, sum, m, n)) return;
  if constexpr (GATE) {
    f32x4_t h;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float av, d;
      act_of<ACT>(sum[0][k], av, d);
      h[k] = av * sum[1][k];
    }
    if (p.c2) {
      store4(p.c2, m * p.ldc2 + n, sum[0]);
      store4(p.c2, m * p.ldc2 + p.n + n, sum[1]);
    }
    store4(p.c, m * p.ldc + n, h);
  } else {
    store4(p.c, m * p.ldc + n, sum[0]);
  }
}

// Every workgroup reads all of x: up to 8 rows at about 23 TB/s, as they are
// shared in L1, more at about 7 from L2; the tiled kernels take 25 us, and 8 us
// and an eighth of the weights' time, longer than reading them.  The whole call
// in us, here against tiles, with weights from memory: 2048 x 8192 27 against
// 41 for one row, 31 against 41 for 8, 40 against 42 for 16, 50 against 44 for
// 32; 5120 x 20480 121 against 150 for one, 148 against 150 for 8, 184 against
// 151 for 9; 8192 x 28672 254 against 261 for 4, 266 against 261 for 6.
bool few_rows(int64_t t, int64_t d, int64_t h) {
  const double dh = double(d) * h, weights_us = 6 * dh / 5.1e6;
  if (t <= 8) return t * dh * (4.0 / 8) / 23e6 <= 25;
  return t <= 64 && t * dh * (4.0 / 16) / 7e6 <= 8 + weights_us / 8;
}

template <bool GATE, int ACT>
hipError_t run_few_rows(hipStream_t s, const Prod& p) {
  const int cols = p.m <= 8 ? 8 : 16;
  const unsigned grid = unsigned((p.n + cols - 1) / cols);
  const bool wide = grid <= 256;      // a workgroup per CU at most: more waves to each
  auto* k = p.m <= 8    ? (wide ? ffn_few_rows_kernel<0, GATE, ACT, 16> : ffn_few_rows_kernel<0, GATE, ACT, 8>)
            : p.m <= 16 ? (wide ? ffn_few_rows_kernel<1, GATE, ACT, 16> : ffn_few_rows_kernel<1, GATE, ACT, 8>)
            : p.m <= 32 ? (wide ? ffn_few_rows_kernel<2, GATE, ACT, 16> : ffn_few_rows_kernel<2, GATE, ACT, 8>)
                        : (wide ? ffn_few_rows_kernel<4, GATE, ACT, 16> : ffn_few_rows_kernel<4, GATE, ACT, 8>);
  hipLaunchKernelGGL(k, dim3(grid), dim3(wide ? 1024 : 512), 0, s, p);
  return hipGetLastError();
}

}  // namespace

size_t ffn_fwd_part_bytes(int64_t t, int64_t d, int64_t h) {
  if (t == 0 || few_rows(t, d, h)) return 0;
  const ProdArgs up = alone(sizes(t, h, d)), down = alone(sizes(t, d, h));
  return std::max(part_bytes(up, plan_of(up, true)), part_bytes(down, plan_of(down, false)));
}
size_t ffn_bwd_part_bytes(int64_t t, int64_t d, int64_t h) {
  if (t == 0) return 0;
  const ProdArgs dh = alone(sizes(t, h, d)), rest = backward_sizes(t, d, h);
  return std::max(part_bytes(dh, plan_of(dh, false)), part_bytes(rest, plan_of(rest, false)));
}

hipError_t launch_ffn_fwd(hipStream_t s, const FfnDev& f) {
  const int64_t t = f.rows, d = f.cols, h = f.hidden;
  ProdArgs g = alone(sizes(t, h, d));
  g.part = f.part;
  Prod& p = g.p[0];
  p.a = f.x; p.lda = f.ld_x;
  p.b = f.w_gate; p.ldb = f.ld_wg; p.b2 = f.w_up; p.ldb2 = f.ld_wu;
  p.c = f.hid; p.ldc = h; p.c2 = f.gu; p.ldc2 = f.ld_gu;
  const bool few = few_rows(t, d, h);
  hipError_t e = few ? (f.act ? run_few_rows<true, 1>(s, p) : run_few_rows<true, 0>(s, p))
                 : f.act ? run_prod<ROWS_ROWS, EPI_GATE, 1>(s, g) : run_prod<ROWS_ROWS, EPI_GATE, 0>(s, g);
  if (e != hipSuccess) return e;
  p = sizes(t, d, h);
  p.a = f.hid; p.lda = h;
  p.b = f.w_down; p.ldb = f.ld_wd;
  p.c = f.y; p.ldc = f.ld_y;
  return few ? run_few_rows<false, 0>(s, p) : run_prod<ROWS_ROWS, EPI_PLAIN>(s, g);
}

hipError_t launch_ffn_bwd(hipStream_t s, const FfnDev& f) {
  const int64_t t = f.rows, d = f.cols, h = f.hidden;
  ProdArgs g = alone(sizes(t, h, d));
  g.part = f.part;
  Prod& p = g.p[0];
  p.a = f.d_y; p.lda = f.ld_dy;
  p.b = f.w_down; p.ldb = f.ld_wd;
  p.c = f.dgu; p.ldc = 2 * h; p.c2 = f.hid; p.ldc2 = h;
  p.gu = f.gu; p.ldgu = f.ld_gu;
  const hipError_t e = f.act ? run_prod<ROWS_COLS, EPI_DGATE, 1>(s, g) : run_prod<ROWS_COLS, EPI_DGATE, 0>(s, g);
  if (e != hipSuccess) return e;
  // dx, over the k range of dg and then that of du, and the weights' gradients
  g = backward_sizes(t, d, h);
  g.part = f.part;
  p.a = f.dgu; p.lda = 2 * h;
  p.b = f.w_gate; p.ldb = f.ld_wg; p.b2 = f.w_up; p.ldb2 = f.ld_wu;
  p.c = f.d_x; p.ldc = f.ld_dx;
  for (int i = 0; i < 3; ++i) {
    Prod& w = g.p[1 + i];
    w.acols = 1;
    w.f32 = !f.grad_bf16;
    if (i < 2) {
      w.a = static_cast<const uint16_t*>(f.dgu) + i * h; w.lda = 2 * h;
      w.b = f.x; w.ldb = f.ld_x;
      w.c = i ? f.d_wu : f.d_wg; w.ldc = i ? f.ld_dwu : f.ld_dwg;
    } else {
      w.a = f.d_y; w.lda = f.ld_dy;
      w.b = f.hid; w.ldb = h;
      w.c = f.d_wd; w.ldc = f.ld_dwd;
    }
  }
  return run_prod<MIXED_COLS, EPI_PLAIN>(s, g);
}

}  // namespace muon
