// Structures and device helpers shared by the transformer-block operators'
// host side (block_runtime.cpp) and kernels.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

namespace muon {

// ---- residual norm --------------------------------------------------------
// A matrix or a set of per-sample vectors: base, row stride in values, type.
struct NormMat {
  void* p;
  int64_t ld;
  int32_t dt;   // 0 = f32, 1 = bf16
  int32_t pad;
};

struct NormDev {
  int64_t rows, group_rows;
  int32_t cols, post_kind, pre_kind;
  float alpha, eps;
  NormMat resid, h, resid_out, y;
  NormMat gate, scale, shift, post_weight, pre_weight;
  float* stats;
  NormMat d_resid_out, d_y, d_resid, d_h;
  NormMat d_gate, d_scale, d_shift, d_post_weight, d_pre_weight;
  // backward: column sums.  part: [group][split][kNormSums][cols]; gsum:
  // [group][2][cols], a sample's share of the two weight gradients.
  float* part;
  float* gsum;
  int32_t splits;        // workgroup shares of one sample's rows
  int32_t split_rows;    // rows of a share (the last may have fewer)
};

constexpr int kNormSums = 3;
constexpr int kNormMaxCols = 16384;
hipError_t launch_norm_fwd(hipStream_t s, const NormDev& a, bool vec);
hipError_t launch_norm_bwd(hipStream_t s, const NormDev& a, bool vec, bool sums);
// Shares of a sample's rows that the backward pass sums apart.
int norm_splits(int64_t groups, int64_t group_rows, int cols);

// ---- attention ------------------------------------------------------------
struct HeadsDev {
  void* p;
  int64_t sb, sl, sh;    // strides in values
};

// Division of numbers below 2^31 by a fixed divisor: the high word of a
// product, an addition and a shift (the round-up method of Granlund and
// Montgomery, "Division by Invariant Integers using Multiplication").
struct FastDiv {
  uint32_t mul, shift, by;
};
inline FastDiv fast_div(uint32_t d) {
  if (d == 0) d = 1;       // nothing is divided where there is nothing
  uint32_t l = 0;
  while ((uint64_t(1) << l) < d) ++l;
  return FastDiv{uint32_t(((uint64_t(1) << 32) * ((uint64_t(1) << l) - d)) / d + 1), l, d};
}

struct AttnDev {
  int32_t batch, q_len, k_len, heads, kv_heads, dim, causal;
  int64_t offset;
  float scale;
  const int32_t* q_lens;
  const int32_t* k_lens;
  HeadsDev q, k, v, o, d_o, d_q, d_k, d_v;
  float* lse;
  float* delta;          // backward: rowsum(d_o * o), batch x heads x q_len
  float* part_o;         // split forward: [split][batch][heads][q_len][dim] unnormalised-to-own-sum fp32
  float* part_lse;       // split forward: [split][batch][heads][q_len]
  int32_t splits;        // key ranges worked on apart (1: no join)
  int32_t split_keys;    // keys per range, a multiple of the key tile
  int32_t parts;         // backward: workgroups that share a key block (1: no join)
  FastDiv row_blocks, key_blocks, by_kv_heads, by_group, by_splits, by_parts, by_bh;
  float* part_kv;        // [part][batch][kv_heads][k_len][2][dim] fp32 sums of dk / scale, dv
};

hipError_t launch_attn_fwd(hipStream_t s, const AttnDev& a);
hipError_t launch_attn_bwd(hipStream_t s, const AttnDev& a);
// Fills in splits, split_keys, parts and the divisors.
void attn_plan(AttnDev& a);

// ---- gated feed-forward -----------------------------------------------------
struct FfnDev {
  int64_t rows, cols, hidden;
  int32_t act, grad_bf16;
  const void *x, *w_gate, *w_up, *w_down;
  int64_t ld_x, ld_wg, ld_wu, ld_wd;
  void* y; int64_t ld_y;
  void* gu; int64_t ld_gu;
  void* hid;             // rows x hidden bf16: act(g) u
  const void* d_y; int64_t ld_dy;
  void* d_x; int64_t ld_dx;
  void *d_wg, *d_wu, *d_wd; int64_t ld_dwg, ld_dwu, ld_dwd;
  void* dgu;             // backward: rows x 2 hidden bf16 (dg then du)
  float* part;           // partial products of split sums
};

hipError_t launch_ffn_fwd(hipStream_t s, const FfnDev& a);
hipError_t launch_ffn_bwd(hipStream_t s, const FfnDev& a);
size_t ffn_fwd_part_bytes(int64_t rows, int64_t cols, int64_t hidden);
size_t ffn_bwd_part_bytes(int64_t rows, int64_t cols, int64_t hidden);

}  // namespace muon
