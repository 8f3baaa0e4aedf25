// Dropout from a counter-based generator: y = residual + keep x / (1 - p), the
// mask formed from the element's number (block_philox.h) and never stored.  The
// gradient is the same call on dy.
//
// Whole aligned groups of eight are bound by memory, and only just: ten rounds of
// two 64-bit products for four elements take about as long as four bytes of an
// element.  16384 x 2048 bf16 onto an fp32 residual 57 us (5.9 TB/s), 20000 x 1000
// bf16 17.5 (4.6).
//
// Rows off the groups (a width or stride that is no multiple of eight, rows apart)
// are not: a lane's four columns are loaded and stored one value at a time, and lie
// in two of the generator's blocks where they cross a group.  20000 x 1001 with rows
// 1004 apart in bf16 41 us (1.9 TB/s), onto an fp32 residual 56 (3.6); 300000 x 33
// with rows 40 apart in bf16 27 (1.5), in fp32 26 (3.0).  Rows beside each other
// count as one row, whatever their width: 300000 x 33 so 9.7 (4.1).
#include "block_philox.h"

namespace muon {
namespace {

// Eight columns per thread and turn, four one by one where rows are not whole
// aligned groups; an element's number goes by its row and column, not by where
// it lies.
template <typename TX, typename TY>
__device__ __forceinline__ void drop_some(const DropoutDev& a, const Rng& rng, int64_t row, int64_t col, int64_t end) {
  uint64_t group = ~uint64_t(0);
  u32x4_t w{0, 0, 0, 0};
  for (; col < end; ++col) {
    float v[1], r[1] = {0.f};
    load_vals<TX, 1>(a.x.p, row * a.x.ld + col, v);
    if (a.resid.p) load_vals<TY, 1>(a.resid.p, row * a.resid.ld + col, r);
    if (a.drop.on) {
      const uint64_t e = uint64_t(row) * uint64_t(a.cols) + uint64_t(col);
      if (e / 4 != group) {              // four columns are in two groups at most
        group = e / 4;
        w = philox(group, rng.offset, rng.seed);
      }
      const uint32_t mine = e % 4 == 0 ? w[0] : e % 4 == 1 ? w[1] : e % 4 == 2 ? w[2] : w[3];
      v[0] = mine <= a.drop.last ? 0.f : v[0] * a.drop.scale;
    }
    v[0] += r[0];
    store_vals<TY, 1>(a.y.p, row * a.y.ld + col, v);
  }
}

template <typename TX, typename TY, bool VEC>
__global__ __launch_bounds__(256) void dropout_kernel(DropoutDev a) {
  constexpr int N = VEC ? 8 : 4;
  const int64_t per = (a.cols + N - 1) / N;
  const Rng rng = rng_of(a.drop);
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < a.rows * per; i += int64_t(gridDim.x) * 256) {
    const int64_t row = i / per, col = (i - row * per) * N;
    if constexpr (VEC) {
      if (col + N <= a.cols) {
        float v[N], r[N] = {};
        load_vals<TX, N>(a.x.p, row * a.x.ld + col, v);
        if (a.resid.p) load_vals<TY, N>(a.resid.p, row * a.resid.ld + col, r);
        if (a.drop.on) drop<N>(a.drop, rng, uint64_t(row) * uint64_t(a.cols) + uint64_t(col), v);
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] += r[k];
        store_vals<TY, N>(a.y.p, row * a.y.ld + col, v);
        continue;
      }
    }
    drop_some<TX, TY>(a, rng, row, col, min(col + N, a.cols));
  }
}

}  // namespace

hipError_t launch_dropout(hipStream_t s, const DropoutDev& a, bool vec) {
  const int64_t n = vec ? 8 : 4, items = a.rows * ((a.cols + n - 1) / n);
  const unsigned grid = unsigned(items / 256 >= (1 << 20) ? 1 << 20 : (items + 255) / 256);
  using B = uint16_t;
  auto* k = a.x.dt ? (a.y.dt ? (vec ? dropout_kernel<B, B, true> : dropout_kernel<B, B, false>)
                             : (vec ? dropout_kernel<B, float, true> : dropout_kernel<B, float, false>))
                   : (a.y.dt ? (vec ? dropout_kernel<float, B, true> : dropout_kernel<float, B, false>)
                             : (vec ? dropout_kernel<float, float, true> : dropout_kernel<float, float, false>));
  hipLaunchKernelGGL(k, dim3(grid), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace muon
