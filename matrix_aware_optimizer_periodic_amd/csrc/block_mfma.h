// Tile movement and matrix-core fragments shared by the attention and
// feed-forward kernels.
#pragma once

#include "block_device.h"

namespace muon {

// v_mfma_f32_32x32x16_bf16: lane l gives row (A) or column (B) l % 32, eight
// consecutive k from 8 (l / 32); result v of a lane is column l % 32, row
// 8 (v / 4) + 4 (l / 32) + v % 4.
__device__ __forceinline__ f32x16_t mfma32(u32x4_t a, u32x4_t b, f32x16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                 0, 0, 0);
}
// v_mfma_f32_16x16x32_bf16: row or column l % 16, k from 8 (l / 16); result v
// is column l % 16, row 4 (l / 16) + v.
__device__ __forceinline__ f32x4_t mfma16(u32x4_t a, u32x4_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                 0, 0, 0);
}

// Raw buffer resource that covers offsets below kBufBytes; an offset of
// kBufNone or more reads as zero.  Every caller keeps its valid offsets
// inside the tensor and sends what is not there to kBufNone.
constexpr unsigned kBufNone = 0x80000000u;
__device__ __forceinline__ u32x4_t buffer_at(const void* p) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  return u32x4_t{unsigned(a), unsigned(a >> 32) & 0xffffu, kBufNone, 0x00020000u};
}

// 16 (or 4) bytes per lane from a raw buffer straight into LDS: lane l lands
// at lds_addr + 16 l (4 l).  Inline asm without outputs, so that the compiler
// does not drain it before unrelated LDS reads; the kernels order it with
// wait_vm() and barriers.  The compiler does not see the load's operands either
// and puts no wait states between a vector instruction that writes one of its
// scalar registers (a spilled one's reload, say) and the load, which needs five:
// the write of m0 and 1 + NOP more.  A kernel that gives a smaller NOP has to
// have its scalar operands that far ahead; the scan of the compiled code among
// the tests holds it to that.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"   // m0 is reserved; naming it is what is meant
// soff is added to every lane's offset; kBufNone stays out of range with it.
template <int NOP = 3>
__device__ __forceinline__ void dma16(u32x4_t rsrc, unsigned lds_addr, unsigned voff, unsigned soff = 0) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop %4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :: "s"(lds_addr), "v"(voff), "s"(rsrc), "s"(__builtin_amdgcn_readfirstlane(int(soff))), "n"(NOP)
               : "m0", "memory");
}
__device__ __forceinline__ void dma4(u32x4_t rsrc, unsigned lds_addr, unsigned voff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dword %1, %2, 0 offen lds"
               :: "s"(lds_addr), "v"(voff), "s"(rsrc) : "m0", "memory");
}
#pragma clang diagnostic pop
template <int N>
__device__ __forceinline__ void wait_vm() { asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory"); }
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
// A bare barrier: __syncthreads() would also wait for the DMA in flight.
__device__ __forceinline__ void barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

__device__ __forceinline__ unsigned lds_offset(const void* p) {
  return unsigned(reinterpret_cast<uintptr_t>((const MUON_LOCAL void*)p));
}
__device__ __forceinline__ u32x4_t lds_read16(const unsigned char* base, unsigned off) {
  return *(const MUON_LOCAL u32x4_t*)((const MUON_LOCAL unsigned char*)base + off);
}
// ds_read_b64_tr_b16: in each group of 16 lanes, lane i receives element
// i % 4 of the 8 bytes that lanes 4 e + i / 4, e = 0 .. 3, address.  With lane
// s addressing row k0 + s / 4, columns c0 + 4 (s % 4) .., lane i gets column
// c0 + i of rows k0 .. k0 + 3.
__device__ __forceinline__ u32x2_t lds_read_tr(const unsigned char* base, unsigned off) {
  MUON_LOCAL s16x4_t* p = (MUON_LOCAL s16x4_t*)((MUON_LOCAL unsigned char*)base + off);
  return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16(p));
}

// Workgroups go round the eight XCDs in turn; give each XCD one contiguous
// run of work items, so that neighbours share its L2.
__device__ __forceinline__ unsigned xcd_item(unsigned id, unsigned n) {
  const unsigned x = id & 7u, slot = id >> 3, per = n >> 3, rem = n & 7u;
  return x * per + min(x, rem) + slot;
}

}  // namespace muon
