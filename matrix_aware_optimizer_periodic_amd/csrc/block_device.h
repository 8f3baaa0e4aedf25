// Device helpers of the transformer-block kernels.
#pragma once

#include <hip/hip_runtime.h>

#include "block_internal.h"

namespace muon {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));

// Pointers out of argument structures carry no address space; as global
// pointers their accesses count against the vector-memory counter only.
#define MUON_GLOBAL __attribute__((address_space(1)))
#define MUON_LOCAL __attribute__((address_space(3)))
template <typename T>
__device__ __forceinline__ MUON_GLOBAL T* as_global(T* p) { return (MUON_GLOBAL T*)(p); }

__device__ __forceinline__ float bf16_to_f32(uint32_t bits16) { return __uint_as_float(bits16 << 16); }
// Round to nearest even, NaN stays NaN (v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{lo, hi}, bf16x2_t));
}

// VEC consecutive values at element e of p, as fp32.  VEC is 8 (16-byte
// aligned) or 1.  T: float or uint16_t (bf16 bits).
template <typename T, int VEC>
__device__ __forceinline__ void load_vals(const void* p, int64_t e, float (&v)[VEC]) {
  if constexpr (VEC == 8 && sizeof(T) == 4) {
    const auto* q = as_global(reinterpret_cast<const f32x4_t*>(static_cast<const float*>(p) + e));
    const f32x4_t a = q[0], b = q[1];
#pragma unroll
    for (int k = 0; k < 4; ++k) { v[k] = a[k]; v[4 + k] = b[k]; }
  } else if constexpr (VEC == 8) {
    const u32x4_t u = *as_global(reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(p) + e));
#pragma unroll
    for (int k = 0; k < 4; ++k) { v[2 * k] = bf16_to_f32(u[k] & 0xffffu); v[2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u); }
  } else if constexpr (sizeof(T) == 4) {
    v[0] = *as_global(static_cast<const float*>(p) + e);
  } else {
    v[0] = bf16_to_f32(*as_global(static_cast<const uint16_t*>(p) + e));
  }
}

template <typename T, int VEC>
__device__ __forceinline__ void store_vals(void* p, int64_t e, const float (&v)[VEC]) {
  if constexpr (VEC == 8 && sizeof(T) == 4) {
    auto* q = as_global(reinterpret_cast<f32x4_t*>(static_cast<float*>(p) + e));
    q[0] = f32x4_t{v[0], v[1], v[2], v[3]};
    q[1] = f32x4_t{v[4], v[5], v[6], v[7]};
  } else if constexpr (VEC == 8) {
    *as_global(reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(p) + e)) =
        u32x4_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
  } else if constexpr (sizeof(T) == 4) {
    *as_global(static_cast<float*>(p) + e) = v[0];
  } else {
    *as_global(static_cast<uint16_t*>(p) + e) = uint16_t(pack_bf16x2(v[0], 0.f));
  }
}

// The same with the type chosen at run time (vectors read once per row).
template <int VEC>
__device__ __forceinline__ void load_any(const void* p, int dt, int64_t e, float (&v)[VEC]) {
  if (dt) load_vals<uint16_t, VEC>(p, e, v);
  else load_vals<float, VEC>(p, e, v);
}
__device__ __forceinline__ float load_any1(const void* p, int dt, int64_t e) {
  float v[1];
  load_any<1>(p, dt, e, v);
  return v[0];
}
__device__ __forceinline__ void store_any1(void* p, int dt, int64_t e, float x) {
  const float v[1] = {x};
  if (dt) store_vals<uint16_t, 1>(p, e, v);
  else store_vals<float, 1>(p, e, v);
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

}  // namespace muon
