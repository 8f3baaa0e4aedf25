// Rotary positions on queries and keys, forward and inverse.
//
//   t = sum_a pos[a] freqs[a][p],  (u, v) -> scale (u cos t - v sin t, v cos t + u sin t)
//
// A workgroup takes a few tokens: first each angle's cosine and sine once, for
// all heads of both tensors, then the heads.  Angles are formed in fp64 and
// brought to within half a turn there, so that far positions keep their digits
// (fp32 would leave 0.06 at a position of a million); the sine and cosine of
// what is left are fp32.
#include "block_device.h"

namespace muon {
namespace {

__device__ __forceinline__ uint32_t over(uint32_t n, const FastDiv& d) { return (__umulhi(n, d.mul) + n) >> d.shift; }

// N consecutive values, aligned to their size (to 16 bytes where that is more).
template <typename T, int N>
__device__ __forceinline__ void load_run(const void* p, int64_t e, float* v) {
  if constexpr (N == 16 || N == 8 || N == 1) {
    constexpr int M = N == 16 ? 8 : N;
#pragma unroll
    for (int i = 0; i < N; i += M) load_vals<T, M>(p, e + i, *reinterpret_cast<float(*)[M]>(v + i));
  } else {
    uint32_t w[N * sizeof(T) / 4];
    const auto* q = as_global(reinterpret_cast<const uint32_t*>(static_cast<const T*>(p) + e));
    if constexpr (sizeof w == 16) *reinterpret_cast<u32x4_t*>(w) = *(const MUON_GLOBAL u32x4_t*)q;
    else if constexpr (sizeof w == 8) *reinterpret_cast<u32x2_t*>(w) = *(const MUON_GLOBAL u32x2_t*)q;
    else w[0] = q[0];
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = sizeof(T) == 4 ? __uint_as_float(w[k]) : k & 1 ? __uint_as_float(w[k / 2] & 0xffff0000u) : bf16_to_f32(w[k / 2] & 0xffffu);
  }
}
template <typename T, int N>
__device__ __forceinline__ void store_run(void* p, int64_t e, const float* v) {
  if constexpr (N == 16 || N == 8 || N == 1) {
    constexpr int M = N == 16 ? 8 : N;
#pragma unroll
    for (int i = 0; i < N; i += M) store_vals<T, M>(p, e + i, *reinterpret_cast<const float(*)[M]>(v + i));
  } else {
    uint32_t w[N * sizeof(T) / 4];
#pragma unroll
    for (int k = 0; k < int(sizeof w / 4); ++k) w[k] = sizeof(T) == 4 ? __float_as_uint(v[k]) : pack_bf16x2(v[2 * k], v[2 * k + 1]);
    auto* q = as_global(reinterpret_cast<uint32_t*>(static_cast<T*>(p) + e));
    if constexpr (sizeof w == 16) *(MUON_GLOBAL u32x4_t*)q = *reinterpret_cast<u32x4_t*>(w);
    else if constexpr (sizeof w == 8) *(MUON_GLOBAL u32x2_t*)q = *reinterpret_cast<u32x2_t*>(w);
    else q[0] = w[0];
  }
}

constexpr int kAngles = 2048;          // cosines and sines of a workgroup

enum { HALVES = 0, NEIGHBOURS = 1, NEIGHBOURS_APART = 2 };   // the last: pairs off their boundary, value by value

// V: pairs of a thread's chunk.
template <typename T, int V, int LIE>
__global__ __launch_bounds__(256) void rotary_kernel(RotaryDev a, int group) {
  __shared__ f32x2_t cs[kAngles];
  const int heads = a.heads + a.kv_heads, turned = a.pairs / V;
  const uint32_t chunks = a.by_chunks.by;
  for (int64_t t0 = int64_t(blockIdx.x) * group; t0 < a.tokens; t0 += int64_t(gridDim.x) * group) {
    const int here = int(min(int64_t(group), a.tokens - t0));
    for (int i = threadIdx.x; i < here * a.pairs; i += 256) {
      const int tt = i / a.pairs, p = i - tt * a.pairs;
      const uint32_t token = uint32_t(t0 + tt), b = over(token, a.by_len), at = token - b * uint32_t(a.len);
      double t = 0.0;
      if (a.positions) {
        const int32_t* pos = a.positions + b * a.pos_batch + int64_t(at) * a.axes;
        for (int j = 0; j < a.axes; ++j) t += double(pos[j]) * a.freqs[j * a.pairs + p];
      } else {
        t = double(int64_t(at) + a.offset) * a.freqs[p];
      }
      t *= 0.15915494309189535;        // turns
      t -= rint(t);
      float s, c;
      sincospif(2.f * float(t), &s, &c);
      cs[i] = f32x2_t{c * a.scale, (a.inverse ? -s : s) * a.scale};
    }
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < uint32_t(here) * heads * chunks; i += 256) {
      const uint32_t rest = over(i, a.by_chunks), c = i - rest * chunks, tt = over(rest, a.by_heads);
      int h = int(rest - tt * heads);
      const uint32_t token = uint32_t(t0 + tt), b = over(token, a.by_len), at = token - b * uint32_t(a.len);
      const bool is_k = h >= a.heads;
      if (is_k) h -= a.heads;
      const HeadsDev& in = is_k ? a.k : a.q;
      const HeadsDev& out = is_k ? a.k_out : a.q_out;
      const int64_t from = b * in.sb + at * in.sl + h * in.sh, to = b * out.sb + at * out.sl + h * out.sh;
      const bool turn = int(c) < turned;
      // this chunk's 2 V values: one run, or one of each half
      const int first = turn && LIE == HALVES ? int(c) * V : int(c) * 2 * V;
      const int second = turn && LIE == HALVES ? first + a.pairs : first + V;
      float x[2 * V];
      if constexpr (LIE == NEIGHBOURS) {
        load_run<T, 2 * V>(in.p, from + first, x);
      } else {
        load_run<T, V>(in.p, from + first, x);
        load_run<T, V>(in.p, from + second, x + V);
      }
      if (turn) {
        const f32x2_t* w = cs + tt * a.pairs + c * V;
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const f32x2_t t = w[k];
          const int iu = LIE ? 2 * k : k, iv = LIE ? 2 * k + 1 : V + k;
          const float p = x[iu], q = x[iv];
          x[iu] = fmaf(p, t[0], -(q * t[1]));
          x[iv] = fmaf(q, t[0], p * t[1]);
        }
      }
      if constexpr (LIE == NEIGHBOURS) {
        store_run<T, 2 * V>(out.p, to + first, x);
      } else {
        store_run<T, V>(out.p, to + first, x);
        store_run<T, V>(out.p, to + second, x + V);
      }
    }
    __syncthreads();
  }
}

}  // namespace

hipError_t launch_rotary(hipStream_t s, const RotaryDev& a0, int vec) {
  RotaryDev a = a0;
  const int heads = a.heads + a.kv_heads, chunks = (a.in_place ? 2 * a.pairs : a.dim) / (vec ? 2 * vec : 2);
  a.by_len = fast_div(uint32_t(a.len));
  a.by_heads = fast_div(uint32_t(heads));
  a.by_chunks = fast_div(uint32_t(chunks));
  // tokens of a workgroup: enough chunks for its threads, angles that fit
  int group = 1;
  while (group * heads * chunks < 512 && 2 * group * a.pairs <= kAngles) group *= 2;
  const int64_t groups = (a.tokens + group - 1) / group;
  const unsigned grid = unsigned(groups < (1 << 20) ? groups : 1 << 20);
  auto pick = [&](auto type) {
    using T = decltype(type);
    if (a.interleaved)
      return vec == 8   ? rotary_kernel<T, 8, NEIGHBOURS>
             : vec == 4 ? rotary_kernel<T, 4, NEIGHBOURS>
             : vec == 2 ? rotary_kernel<T, 2, NEIGHBOURS>
             : vec == 1 ? rotary_kernel<T, 1, NEIGHBOURS>
                        : rotary_kernel<T, 1, NEIGHBOURS_APART>;
    return vec == 8   ? rotary_kernel<T, 8, HALVES>
           : vec == 4 ? rotary_kernel<T, 4, HALVES>
           : vec == 2 ? rotary_kernel<T, 2, HALVES>
                      : rotary_kernel<T, 1, HALVES>;
  };
  auto* k = a.f32 ? pick(float{}) : pick(uint16_t{});
  hipLaunchKernelGGL(k, dim3(grid), dim3(256), 0, s, a, group);
  return hipGetLastError();
}

}  // namespace muon
