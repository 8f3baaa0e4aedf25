// Counter-based random words for dropout: Philox4x32-10 (Salmon, Moraes, Dror
// and Shaw, "Parallel Random Numbers: As Easy as 1, 2, 3", SC11).  A block of
// four words depends on a 64-bit key and a 128-bit counter alone, so a mask is
// formed again where it is needed and never stored.
//
// Key: the seed.  Counter: the number of a group of four consecutive elements
// (row * cols + column, rows beside each other whatever their stride) and the
// caller's offset.  An element is dropped where its word is below
// round(p 2^32).
//
// All 32 bits decide: the probability is kept to 2^-33, where 16 bits of a word
// for each of two elements would keep it to 2^-17 in half the work.
#pragma once

#include "block_device.h"

namespace muon {

// One instruction (the table of x ^ y ^ z), where the compiler makes two.
__device__ __forceinline__ uint32_t xor3(uint32_t x, uint32_t y, uint32_t z) { return __builtin_amdgcn_bitop3_b32(x, y, z, 0x96); }

__device__ __forceinline__ u32x4_t philox(uint64_t index, uint64_t offset, uint64_t seed) {
  uint32_t c0 = uint32_t(index), c1 = uint32_t(index >> 32), c2 = uint32_t(offset), c3 = uint32_t(offset >> 32);
  uint32_t k0 = uint32_t(seed), k1 = uint32_t(seed >> 32);
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = uint64_t(0xD2511F53u) * c0, b = uint64_t(0xCD9E8D57u) * c2;
    c0 = xor3(uint32_t(b >> 32), c1, k0);
    c1 = uint32_t(b);
    c2 = xor3(uint32_t(a >> 32), c3, k1);
    c3 = uint32_t(a);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return u32x4_t{c0, c1, c2, c3};
}

// A call's seed and offset, from the caller's device memory where it gave some.
struct Rng { uint64_t seed, offset; };
__device__ __forceinline__ Rng rng_of(const DropDev& d) {
  if (!d.state) return Rng{d.seed, d.offset};
  const auto* s = as_global(d.state);
  return Rng{s[0], s[1]};
}

// Bit k: whether element e + k is dropped, for four elements from e (a multiple
// of four) on.
__device__ __forceinline__ uint32_t dropped4(const DropDev& d, const Rng& r, uint64_t e) {
  const u32x4_t w = philox(e / 4, r.offset, r.seed);
  return (w[0] <= d.last ? 1u : 0u) | (w[1] <= d.last ? 2u : 0u) | (w[2] <= d.last ? 4u : 0u) | (w[3] <= d.last ? 8u : 0u);
}
// Dropped elements as 0, whatever they held, the others scaled.
template <int N>
__device__ __forceinline__ void drop_by(const DropDev& d, uint32_t dropped, float (&v)[N]) {
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = dropped >> k & 1u ? 0.f : v[k] * d.scale;
}

// v[0 .. N - 1], elements e .. e + N - 1 (e a multiple of four): dropped ones 0,
// whatever they held, the others scaled.
template <int N>
__device__ __forceinline__ void drop(const DropDev& d, const Rng& r, uint64_t e, float (&v)[N]) {
  static_assert(N % 4 == 0, "whole groups");
#pragma unroll
  for (int g = 0; g < N / 4; ++g) {
    const u32x4_t w = philox(e / 4 + g, r.offset, r.seed);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[4 * g + k] = w[k] <= d.last ? 0.f : v[4 * g + k] * d.scale;
  }
}

}  // namespace muon
