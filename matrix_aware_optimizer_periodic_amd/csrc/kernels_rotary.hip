// Rotary positions on queries and keys, forward and inverse.
//
//   t = sum_a pos[a] freqs[a][p],  (u, v) -> scale (u cos t - v sin t, v cos t + u sin t)
//
// A workgroup takes a few tokens: first each angle's cosine and sine once, for
// all heads of both tensors, then the heads.  Angles are formed in fp64 and
// brought to within half a turn there, so that far positions keep their digits
// (fp32 would leave 0.06 at a position of a million); the sine and cosine of
// what is left are fp32.
//
// Bound by memory: 16 x 1024 tokens, 32 heads of 128 in bf16 44 us with operands
// partly in the caches (6.1 TB/s), 51 without (5.3, a copy's rate).
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

constexpr int kTokens = 64;            // tokens of a workgroup, at most

// The heads of one tensor: a thread keeps to one chunk of 2 V values of a head and
// goes down the rows (token, head), a few of which it reads before it writes the
// first (the compiler cannot: the output may be the input).  Of neighbours a chunk
// may be cut by the end of what turns: 16 bytes at a time instead of 8, and rows
// read ahead, take five samples of 1001 tokens, 32 heads of 72 with 36 turned,
// from 17 us to 12.
template <typename T, int V, int LIE>
__device__ __forceinline__ void turn_heads(const RotaryDev& a, const HeadsDev& in, const HeadsDev& out, uint32_t heads,
                                           const FastDiv& by_heads, const f32x2_t* cs, const int64_t (*base)[2], int here,
                                           uint32_t c0, uint32_t width, uint32_t row0, uint32_t step) {
  constexpr int AHEAD = V == 8 ? 2 : 4;
  const uint32_t chunks = a.by_chunks.by, rows = uint32_t(here) * heads;
  for (uint32_t c = c0; c < chunks; c += width) {
    // this chunk's 2 V values: one run, or one of each half
    const bool halves = LIE == HALVES && int(c) * V < a.pairs;
    const int first = halves ? int(c) * V : int(c) * 2 * V;
    const int second = halves ? first + a.pairs : first + V;
    const int left = min(a.pairs - int(c) * V, V);       // pairs of it that turn
    for (uint32_t r0 = row0; r0 < rows; r0 += step * AHEAD) {
      float x[AHEAD][2 * V];
      uint32_t tok[AHEAD];
      int64_t to[AHEAD];
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        const uint32_t r = min(r0 + j * step, rows - 1), tt = over(r, by_heads), h = r - tt * heads;
        const int64_t from = base[tt][0] + h * in.sh;
        tok[j] = tt;
        to[j] = base[tt][1] + h * out.sh;
        if constexpr (LIE == NEIGHBOURS) {
          load_run<T, 2 * V>(in.p, from + first, x[j]);
        } else {
          load_run<T, V>(in.p, from + first, x[j]);
          load_run<T, V>(in.p, from + second, x[j] + V);
        }
      }
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        if (r0 + j * step >= rows) break;
        if (left > 0) {
          const f32x2_t* w = cs + tok[j] * a.pairs + c * V;
#pragma unroll
          for (int k = 0; k < V; ++k) {
            if (LIE && k >= left) break;                 // (of halves, all turn or none)
            const f32x2_t t = w[k];
            const int iu = LIE ? 2 * k : k, iv = LIE ? 2 * k + 1 : V + k;
            const float p = x[j][iu], q = x[j][iv];
            x[j][iu] = fmaf(p, t[0], -(q * t[1]));
            x[j][iv] = fmaf(q, t[0], p * t[1]);
          }
        }
        if constexpr (LIE == NEIGHBOURS) {
          store_run<T, 2 * V>(out.p, to[j] + first, x[j]);
        } else {
          store_run<T, V>(out.p, to[j] + first, x[j]);
          store_run<T, V>(out.p, to[j] + second, x[j] + V);
        }
      }
    }
  }
}

// V: pairs of a thread's chunk.
template <typename T, int V, int LIE>
__global__ __launch_bounds__(256) void rotary_kernel(RotaryDev a, int group) {
  __shared__ f32x2_t cs[kAngles];
  __shared__ int64_t base_q[kTokens][2], base_k[kTokens][2];
  const uint32_t chunks = a.by_chunks.by, width = min(chunks, 256u), step = 256u / width;
  const uint32_t row0 = chunks < 256u ? over(threadIdx.x, a.by_chunks) : 0, c0 = threadIdx.x - row0 * chunks;
  for (int64_t t0 = int64_t(blockIdx.x) * group; t0 < a.tokens; t0 += int64_t(gridDim.x) * group) {
    const int here = int(min(int64_t(group), a.tokens - t0));
    if (int(threadIdx.x) < here) {
      const uint32_t token = uint32_t(t0) + threadIdx.x, b = over(token, a.by_len), l = token - b * uint32_t(a.len);
      base_q[threadIdx.x][0] = b * a.q.sb + l * a.q.sl;
      base_q[threadIdx.x][1] = b * a.q_out.sb + l * a.q_out.sl;
      base_k[threadIdx.x][0] = b * a.k.sb + l * a.k.sl;
      base_k[threadIdx.x][1] = b * a.k_out.sb + l * a.k_out.sl;
    }
    for (int i = threadIdx.x; i < here * a.pairs; i += 256) {
      const int tt = i / a.pairs, p = i - tt * a.pairs;
      const uint32_t token = uint32_t(t0 + tt), b = over(token, a.by_len), l = token - b * uint32_t(a.len);
      double t = 0.0;
      if (a.positions) {
        const int32_t* pos = a.positions + b * a.pos_batch + int64_t(l) * a.axes;
        for (int j = 0; j < a.axes; ++j) t += double(pos[j]) * a.freqs[j * a.pairs + p];
      } else {
        t = double(int64_t(l) + a.offset) * a.freqs[p];
      }
      t *= 0.15915494309189535;        // turns
      t -= rint(t);
      float s, c;
      sincospif(2.f * float(t), &s, &c);
      cs[i] = f32x2_t{c * a.scale, (a.inverse ? -s : s) * a.scale};
    }
    __syncthreads();
    if (row0 < step) {
      turn_heads<T, V, LIE>(a, a.q, a.q_out, uint32_t(a.heads), a.by_heads, cs, base_q, here, c0, width, row0, step);
      if (a.kv_heads > 0)
        turn_heads<T, V, LIE>(a, a.k, a.k_out, uint32_t(a.kv_heads), a.by_kv_heads, cs, base_k, here, c0, width, row0, step);
    }
    __syncthreads();
  }
}

}  // namespace

hipError_t launch_rotary(hipStream_t s, const RotaryDev& a0, int vec) {
  RotaryDev a = a0;
  const int heads = a.heads + a.kv_heads, per = vec ? 2 * vec : 2;
  const int chunks = ((a.in_place ? 2 * a.pairs : a.dim) + per - 1) / per;
  a.by_len = fast_div(uint32_t(a.len));
  a.by_heads = fast_div(uint32_t(a.heads));
  a.by_kv_heads = fast_div(uint32_t(a.kv_heads));
  a.by_chunks = fast_div(uint32_t(chunks));
  // tokens of a workgroup: enough chunks for its threads, angles that fit
  int group = 1;
  while (group * heads * chunks < 512 && 2 * group * a.pairs <= kAngles && group < kTokens && a.tokens > 2048 * group) group *= 2;
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
