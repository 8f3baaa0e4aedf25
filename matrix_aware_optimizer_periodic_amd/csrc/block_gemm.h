// Products on bf16 matrix cores with fused epilogues: the tiles, their choice
// and the few-row form that the feed-forward and linear kernels are built from.
//
// Every product is C[m][n] = sum_k A(m, k) B(n, k); an operand lies in memory
// either along k ("rows": activations, and the weights of a forward pass) or
// along m / n ("cols": the weights in an input's gradient, both operands of a
// weight's gradient).  Row operands are staged as rows of 64 k values and read
// as they are, column operands as 64 rows of the tile's width and read through
// the transposing LDS read, so that nothing is transposed in memory.
//
// An epilogue takes what it needs beyond a Prod from an argument of its own
// (X: NoExtra, or the linear block's).
#pragma once

#include <algorithm>
#include <type_traits>

#include "block_mfma.h"
#include "block_philox.h"

namespace muon {
namespace {

constexpr int kStageK = 32;   // k values per stage: one MFMA deep

// ---- activation -------------------------------------------------------------
// SiLU g / (1 + e^-g); GELU in its tanh form, 0.5 g (1 + tanh z) = g / (1 + e^-2z)
// with z = sqrt(2/pi) (g + 0.044715 g^3).  Both are g e for a logistic e of
// some w(g), so the derivative is e + g e (1 - e) w'(g).
template <int ACT>
__device__ __forceinline__ void act_of(float g, float& a, float& da) {
  float w = g, dw = 1.f;
  if constexpr (ACT == 1) {
    const float c = 1.5957691216057308f;     // 2 sqrt(2 / pi)
    w = c * fmaf(0.044715f * g, g * g, g);
    dw = c * fmaf(3.f * 0.044715f * g, g, 1.f);
  }
  const float e = 1.0f / (1.0f + __expf(-w));
  a = g * e;
  // 1 - e as the logistic of -w keeps its digits where e is near 1
  da = fmaf(a * dw, 1.0f / (1.0f + __expf(w)), e);
}

// The same in one exponential and one reciprocal, as the linear kernels take it:
// t = e^-w, e = 1 / (1 + t), and 1 - e = t e, without a difference of numbers near
// 1.  The reciprocal is within 2^-23 of itself.  The exponential is 2 to a power
// that is rounded to fp32 after the product with log2 e (and, of GELU, after w's own
// roundings), so that t is off by some 2^-24 |w| and more far out.  On the side where
// t is small that does not show; on the other the value has t's error, and is small
// itself.  Over every bf16 value, relative: 2.5e-7 for |w| up to 2 and on the positive
// side, then SiLU 2^-21 at w = -8, 2^-20 at -20, 2^-18 at -80, GELU twice that; the
// absolute error is 6e-8 at most on the negative side, and a slope's 1.6e-7 anywhere.
// Where t overflows (w below -88.7), e is 0 and so is all that t stands in: of values
// below 1e-36.  w' is taken of a bounded g^2, so that far values give 0 times a
// number.  ACT 2: none.
template <int ACT>
__device__ __forceinline__ float act_value(float g) {
  if constexpr (ACT == 2) return g;
  const float w = ACT == 1 ? 1.5957691216057308f * fmaf(0.044715f * g, g * g, g) : g;
  return g * __builtin_amdgcn_rcpf(1.0f + __expf(-w));
}
template <int ACT>
__device__ __forceinline__ float act_slope(float g) {
  if constexpr (ACT == 2) return 1.f;
  float w = g, dw = 1.f;
  if constexpr (ACT == 1) {
    const float c = 1.5957691216057308f, g2 = fminf(g * g, 1e12f);     // 2 sqrt(2 / pi)
    w = c * fmaf(0.044715f * g, g * g, g);
    dw = c * fmaf(3.f * 0.044715f, g2, 1.f);
  }
  const float t = __expf(-w), e = __builtin_amdgcn_rcpf(1.0f + t);
  return fmaf(g * e * (fminf(t, 3.4e38f) * e), dw, e);
}

// ---- products ---------------------------------------------------------------
struct Prod {
  const void* a;
  const void* b;
  const void* b2;       // EPI_GATE: Wu; two segments: the second segment's B
  void* c;
  void* c2;             // EPI_GATE: g, u; EPI_DGATE: h; EPI_LINEAR: what act is taken of
  const void* gu;       // EPI_DGATE: g, u; EPI_LINEAR: the residual
  int64_t lda, ldb, ldb2, ldc, ldc2, ldgu;
  int32_t m, n, k;      // k of one segment
  int32_t segments;     // 1, or 2: the sum goes on over a second k range (A's
                        // columns k .. 2 k - 1, B in b2)
  int32_t acols;        // A lies along m (launches that mix both)
  int32_t f32;          // EPI_PLAIN, EPI_LINEAR: C is fp32, not bf16
  int32_t mt, nt;       // tiles
  // The first `full` tiles are one workgroup each; the others' sums are cut
  // into `splits` ranges of split_stages stages, a workgroup each, whose fp32
  // results go to the launch's part and are added by a second kernel.
  int32_t full, splits, split_stages;
  int32_t item0, part0, join0;   // its first workgroup, range and tile to join
};
constexpr int kProds = 4;
struct ProdArgs {
  Prod p[kProds];
  int32_t count;
  float* part;
};

struct NoExtra { static constexpr bool kDrop = false; };
// EPI_LINEAR: y = residual + drop(act(sum + bias)); a Prod's c is y (f32: its
// type), c2 what act is taken of, gu the residual, of y's type.  ACT 2 is none.
// The activation and whether anything is dropped are template arguments: chosen
// at run time, the epilogue of a 256-tile outgrows what the compiler unrolls, and
// its accumulators go through scratch memory (4096 x 2048 x 8192 with gelu 223 us
// instead of 147).
template <bool DROP>
struct LinearExtra {
  static constexpr bool kDrop = DROP;
  const void* bias;     // n values, or null
  int32_t bias_bf16;
  DropDev drop;
};
// A lane's eight values of it.
template <class X>
__device__ __forceinline__ void load_bias(const X& ext, const Prod& p, int64_t n, float (&bias)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) bias[k] = ext.bias && n < p.n ? load_any1(ext.bias, ext.bias_bf16, n + k) : 0.f;
}

// Stages of a tile's whole sum; a first segment's last unit is a whole one.
__host__ __device__ inline int stages_of(const Prod& p) {
  return (p.segments - 1) * ((p.k + 63) / 64) * 2 + (p.k + kStageK - 1) / kStageK;
}

enum { EPI_PLAIN = 0, EPI_GATE = 1, EPI_DGATE = 2, EPI_LINEAR = 3 };
enum { ROWS_ROWS = 0, ROWS_COLS = 1, MIXED_COLS = 2 };   // how A and B lie

// One operand's units: 64 k of BT rows (128 bytes each in LDS), or COLS, BT
// columns of 64 rows of k (2 BT bytes each).  Both are BT / 32 DMAs per wave, of
// 1 KB each, whose lanes' offsets differ by a step (COLS with BT = 256: from
// one of two starts in turn).
constexpr int kUnitK = 2 * kStageK;
template <int BT> constexpr int unit_bytes() { return BT * kUnitK * 2; }

struct Side {
  const char* base;
  int64_t kbytes;            // bytes per k
  int64_t kspan;             // bytes per k of what a buffer covers: 0, a row's k are beside each other
  unsigned limit;            // rows: bytes of the rows that are there
  unsigned v0, v1, step;
  int chunk;                 // rows: the lane's chunk of 8 k; COLS: 0

  // first: first row (column) of the tile; there: how many there are;
  // turns: every other block of 16 LDS rows is another matrix's (waves 0 and 1
  // bring one, 2 and 3 the other).
  template <int BT, bool COLS>
  __device__ __forceinline__ void init(const void* p, int64_t ld, int64_t first, int there, int wave, int lane,
                                       bool turns) {
    const int64_t ldbytes = ld * 2;
    if constexpr (!COLS) {
      base = static_cast<const char*>(p) + first * ldbytes;
      const int lds_row = 8 * wave + (lane >> 3);                   // + 32 per DMA
      const int row = turns ? 8 * (wave & 1) + (lane >> 3) : lds_row;
      chunk = (lane & 7) ^ ((lds_row >> 1) & 7);
      v0 = v1 = unsigned(row * ldbytes + chunk * 16);
      step = unsigned((turns ? 16 : 32) * ldbytes);
      limit = unsigned(min(there, turns ? BT / 2 : BT) * ldbytes);
      kbytes = 2;
      kspan = 0;
    } else {
      base = static_cast<const char*>(p) + first * 2;
      constexpr int CH = BT / 8, RPB = 64 / CH;                     // chunks per row, rows per DMA
      const int row = RPB * wave + lane / CH;                       // + 4 RPB per DMA
      const int sw = ((row & 3) << 2) ^ (RPB * 4 == 8 ? 0 : ((row >> 3) & 1) << 1);
      const int c0 = (lane % CH) ^ sw, c1 = c0 ^ 2;
      v0 = c0 * 8 < there ? unsigned(row * ldbytes + c0 * 16) : kBufNone;
      v1 = RPB * 4 == 8 ? (c1 * 8 < there ? unsigned(row * ldbytes + c1 * 16) : kBufNone) : v0;
      step = unsigned(4 * RPB * ldbytes);
      kbytes = kspan = ldbytes;
      limit = 0;
      chunk = 0;
    }
  }
};

// Fragment reads (16 rows or columns, 32 k: a half of a unit) of one operand.
template <int BT, bool COLS>
struct Frag {
  unsigned off[COLS ? BT / 32 : 1];
  __device__ __forceinline__ void init(int wpos, int lane) {
    const int r = lane & 15, q = lane >> 4;
    if constexpr (!COLS) {
      off[0] = unsigned((wpos * (BT / 2) + r) * 128 + ((q ^ ((r >> 1) & 7)) << 4));
    } else {
      const int row = 8 * q + (r >> 2);
      const int sw = ((row & 3) << 2) ^ (((row >> 3) & 1) << 1);
#pragma unroll
      for (int f = 0; f < BT / 32; ++f) {
        const int col = wpos * (BT / 2) + f * 16 + 4 * (lane & 3);
        off[f] = unsigned(row * (2 * BT) + (((col >> 3) ^ sw) << 4) + ((col & 7) << 1));
      }
    }
  }
  // The second half of a row's chunks has bit 2 of the chunk's number flipped.
  __device__ __forceinline__ void read(u32x4_t& o, const unsigned char* s, unsigned half, int f) const {
    if constexpr (!COLS) {
      o = lds_read16(s, (off[0] ^ (half * 64u)) + unsigned(f * 2048));
    } else {
      s += half * unsigned(kStageK * 2 * BT);
      const u32x2_t x = lds_read_tr(s, off[f]);
      const u32x2_t y = lds_read_tr(s, off[f] + unsigned(4 * 2 * BT));
      o = u32x4_t{x[0], x[1], y[0], y[1]};
    }
  }
};

// Place of a product's tile.  Bands of 8 tile rows, walked column by column,
// so that tiles near each other share operands in their XCD's L2.
struct Tile { int tm, tn; };
__device__ __forceinline__ Tile tile_of(const Prod& p, int item) {
  const int band = item / (8 * p.nt), inb = item - band * 8 * p.nt;
  const int bh = min(8, p.mt - band * 8);
  return Tile{band * 8 + inb % bh, inb / bh};
}

// Output columns of a tile.
template <int BT, int EPI>
constexpr int tile_cols() { return EPI == EPI_GATE ? BT / 2 : BT; }

// 16 XB rows of a wave's part of a tile, from its accumulators (a lane has
// four columns of one row per block) through a part of LDS of the wave's own:
// a lane then takes eight consecutive columns, so that rows are read and
// written 16 bytes at a time.  EPI_DGATE reads g and u for four such pieces
// at once, the first four before the accumulators go to LDS: read one by one,
// the dh product of 4096 x 20480 x 5120 took 967 us instead of 876.
template <int BT, int EPI, int ACT, int XB, class X>
__device__ __forceinline__ void emit_rows(const Prod& p, const X& ext, const float (&bias)[8], const f32x4_t (*acc)[BT / 32],
                                          float* er, int64_t mrow, int64_t ncol, int lane) {
  constexpr int F = BT / 32, W = BT / 2, LDR = W + 4;
  constexpr int WOUT = tile_cols<BT, EPI>() / 2;
  constexpr int CPR = WOUT / 8, NIT = 16 * XB * CPR / 64, GRP = NIT < 4 ? NIT : 4;
  static_assert(NIT * 64 == 16 * XB * CPR && NIT % GRP == 0, "whole pieces per lane");
  const int64_t m_at = mrow + lane / CPR, n = ncol + lane % CPR * 8;   // + 64 / CPR rows per piece
  const bool n_ok = n < p.n;
  Rng rng{};
  if constexpr (X::kDrop) rng = rng_of(ext.drop);
  u32x4_t raw[GRP][2];
  auto load_gu = [&](int it) {
    if constexpr (EPI == EPI_DGATE) {
#pragma unroll
      for (int j = 0; j < GRP; ++j) {
        const int64_t m = m_at + (it + j) * (64 / CPR);
        raw[j][0] = raw[j][1] = u32x4_t{0, 0, 0, 0};
        if (n_ok && m < p.m) {
          const uint16_t* gu = static_cast<const uint16_t*>(p.gu) + m * p.ldgu + n;
          raw[j][0] = *as_global(reinterpret_cast<const u32x4_t*>(gu));
          raw[j][1] = *as_global(reinterpret_cast<const u32x4_t*>(gu + p.n));
        }
      }
    }
    if constexpr (EPI == EPI_LINEAR) {
      if (!p.gu) return;
#pragma unroll
      for (int j = 0; j < GRP; ++j) {
        const int64_t m = m_at + (it + j) * (64 / CPR);
        raw[j][0] = raw[j][1] = u32x4_t{0, 0, 0, 0};
        if (n_ok && m < p.m) {
          const auto* r = as_global(reinterpret_cast<const u32x4_t*>(static_cast<const char*>(p.gu) +
                                                                     (m * p.ldgu + n) * (p.f32 ? 4 : 2)));
          raw[j][0] = r[0];
          if (p.f32) raw[j][1] = r[1];
        }
      }
    }
  };
  load_gu(0);
#pragma unroll
  for (int x = 0; x < XB; ++x)
#pragma unroll
    for (int y = 0; y < F; ++y) {
      const int col = EPI == EPI_GATE ? (y >> 1) * 16 + (y & 1) * WOUT : y * 16;
      *(MUON_LOCAL f32x4_t*)(MUON_LOCAL float*)(er + (16 * x + (lane & 15)) * LDR + col + 4 * (lane >> 4)) = acc[x][y];
    }
  __builtin_amdgcn_wave_barrier();
#pragma unroll 1
  for (int it = 0; it < NIT; it += GRP) {
    if (it > 0) load_gu(it);
    // all of a group's reads go out at once (pinned: they would be sunk into
    // the branches below, each to be waited for there)
    f32x4_t w[GRP][EPI == EPI_GATE ? 4 : 2];
#pragma unroll
    for (int j = 0; j < GRP; ++j) {
      const MUON_LOCAL f32x4_t* q =
          (const MUON_LOCAL f32x4_t*)(const MUON_LOCAL float*)(er + (lane / CPR + (it + j) * (64 / CPR)) * LDR + lane % CPR * 8);
      w[j][0] = q[0];
      w[j][1] = q[1];
      if constexpr (EPI == EPI_GATE) {
        w[j][2] = q[WOUT / 4];
        w[j][3] = q[WOUT / 4 + 1];
      }
    }
#pragma unroll
    for (int j = 0; j < GRP; ++j)
#pragma unroll
      for (int k = 0; k < (EPI == EPI_GATE ? 4 : 2); ++k) asm volatile("" : "+v"(w[j][k]));
    // The group's mask, two blocks of the generator at a time: formed in a loop,
    // as bits, for the code's size (see LinearExtra).
    uint32_t dropped = 0;
    if constexpr (X::kDrop) {
#pragma unroll 1
      for (int j = GRP - 1; j >= 0; --j) {
        const uint64_t e = uint64_t(m_at + (it + j) * (64 / CPR)) * unsigned(p.n) + uint64_t(n);
        dropped = dropped << 8 | dropped4(ext.drop, rng, e) | dropped4(ext.drop, rng, e + 4) << 4;
      }
    }
#pragma unroll
    for (int j = 0; j < GRP; ++j) {
      const int row = lane / CPR + (it + j) * (64 / CPR);
      const int64_t m = mrow + row;
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = w[j][k / 4][k % 4];
      if (!n_ok || m >= p.m) continue;
      if constexpr (EPI == EPI_GATE) {
        float u[8], h[8], d;
#pragma unroll
        for (int k = 0; k < 8; ++k) u[k] = w[j][2 + k / 4][k % 4];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          act_of<ACT>(v[k], h[k], d);
          h[k] *= u[k];
        }
        if (p.c2) {
          store_vals<uint16_t, 8>(p.c2, m * p.ldc2 + n, v);
          store_vals<uint16_t, 8>(p.c2, m * p.ldc2 + p.n + n, u);
        }
        store_vals<uint16_t, 8>(p.c, m * p.ldc + n, h);
      } else if constexpr (EPI == EPI_DGATE) {
        float h[8], dg[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const unsigned gb = raw[j][0][k / 2], ub = raw[j][1][k / 2];
          const float gv = k & 1 ? __uint_as_float(gb & 0xffff0000u) : bf16_to_f32(gb & 0xffffu);
          const float uv = k & 1 ? __uint_as_float(ub & 0xffff0000u) : bf16_to_f32(ub & 0xffffu);
          float av, da;
          act_of<ACT>(gv, av, da);
          h[k] = av * uv;
          dg[k] = v[k] * uv * da;
          v[k] *= av;
        }
        store_vals<uint16_t, 8>(p.c, m * p.ldc + n, dg);
        store_vals<uint16_t, 8>(p.c, m * p.ldc + p.n + n, v);
        store_vals<uint16_t, 8>(p.c2, m * p.ldc2 + n, h);
      } else if constexpr (EPI == EPI_LINEAR) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] += bias[k];
        if (p.c2) store_vals_past<uint16_t>(p.c2, m * p.ldc2 + n, v);
        if constexpr (ACT != 2) {
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = act_value<ACT>(v[k]);
        }
        if constexpr (X::kDrop) drop_by(ext.drop, dropped >> (8 * j), v);
        if (p.gu) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const unsigned half = raw[j][0][k / 2];
            v[k] += p.f32 ? __uint_as_float(raw[j][k / 4][k % 4])
                          : k & 1 ? __uint_as_float(half & 0xffff0000u) : bf16_to_f32(half & 0xffffu);
          }
        }
        if (p.f32) store_vals<float, 8>(p.c, m * p.ldc + n, v);
        else store_vals<uint16_t, 8>(p.c, m * p.ldc + n, v);
      } else if (p.f32) {
        store_vals<float, 8>(p.c, m * p.ldc + n, v);
      } else {
        store_vals<uint16_t, 8>(p.c, m * p.ldc + n, v);
      }
    }
  }
  __builtin_amdgcn_wave_barrier();
}

// Units in the LDS ring: all 160 KB with 256-tiles, 80 KB with 128-tiles, of
// which two workgroups run per CU.
constexpr int kUnits = 5;

// The sums of one BT x BT tile, four waves of (BT / 2) x (BT / 2) each, over
// `stages` stages of 32 k from stage `first`, an even one, on.
//
// Software pipeline: the fragments of one stage are in registers while its
// MFMAs run; each fragment is refilled with the next stage's once its last
// MFMA has been issued, and the DMA goes out between MFMAs.  A stage's 64 bytes
// of a row are half a line, and the caches take as long for that as for a
// whole one.  So 64 k (a unit, of two stages) of A come in one stage and of B in
// the next, through a ring of five units: A and B of the stages worked on and of
// the next two, and the one under way.  Stage s asks for unit s + 4; units
// s + 1 and s + 2 are wanted when an odd stage begins to read ahead.  (With A
// and B of 64 k in one stage and two such stages in LDS everything took twice
// as long: they then have one stage's time to arrive.)
//
// A unit is last read in the stage before its last one, so an odd stage waits
// for its own reads before the barrier, which then says that the two units of
// its pair are free: A's is refilled at once, B's in the next stage, which has
// no barrier.  The reads are behind the first PRE MFMAs by then (10, 13, 18 and
// 26 of 64: 4330, 4380, 4380 and 4390 us for the backward call of 4096 rows,
// 5120 x 20480; fewer than 10 change nothing).
//
// 4096 rows, 2048 x 8192, the whole forward call: 378 us where the rows of both
// operands came as half lines, 32 KB a stage all the same, in 407.  The backward
// call of 777 rows, 1000 x 2728, 70 us for 79.
template <int BT, bool ACOLS, bool BCOLS, int EPI>
__device__ __forceinline__ void sum_tile(f32x4_t (&acc)[BT / 32][BT / 32], const Prod& p, int64_t m0, int64_t n0, int first,
                                         int stages, unsigned char* smem, int lane, int wave) {
  constexpr bool GATE = EPI == EPI_GATE;
  constexpr int F = BT / 32;                       // fragments per wave and side
  constexpr int UNIT = unit_bytes<BT>(), DMA = UNIT / 1024 / 4;
  constexpr bool TWO = EPI == EPI_PLAIN && BCOLS && !ACOLS;
  const int per = (p.k + kUnitK - 1) / kUnitK, at = first / 2, seg = TWO && at >= per ? 1 : 0;
  const bool second = (GATE && wave >= 2) || seg;  // brings rows of Wu, not of Wg
  Side sa, sb;
  sa.init<BT, ACOLS>(p.a, p.lda, m0, int(min(int64_t(BT), p.m - m0)), wave, lane, false);
  sb.init<BT, BCOLS>(second ? p.b2 : p.b, second ? p.ldb2 : p.ldb, n0, int(min(int64_t(BT), p.n - n0)), wave, lane, GATE);
  Frag<BT, ACOLS> fa;
  Frag<BT, BCOLS> fb;
  fa.init(wave >> 1, lane);
  fb.init(wave & 1, lane);

  // The next unit to ask for: where the pair's A and B are, what is left of k,
  // pairs to go (past the end the last one is loaded again, so that every
  // stage waits for the same number of DMAs; nothing reads it), the unit's
  // place in the ring.  Kept up in registers: worked out from the arguments in
  // each stage, these are read again and waited for.
  const int k0 = (at - seg * per) * kUnitK;
  const uint64_t pa2 = uint64_t(sa.base) + uint64_t(p.k) * 2;
  const uint64_t pb2 = TWO ? uint64_t(p.b2) + uint64_t(n0) * 2 : 0;
  uint64_t pa = (seg ? pa2 : uint64_t(sa.base)) + uint64_t(k0 * sa.kbytes);
  uint64_t pb = uint64_t(sb.base) + uint64_t(k0 * sb.kbytes);
  const unsigned a_pair = unsigned(kUnitK * sa.kbytes);
  unsigned b_pair = unsigned(kUnitK * sb.kbytes);
  const int k_all = p.k;
  int left = p.k - k0, to_go = (stages + 1) / 2 - 1;
  unsigned ring = 0;
  const unsigned lds = lds_offset(smem) + unsigned(wave) * 1024u;
  u32x4_t rsrc;
  unsigned v0, v1, step, to;
  auto place = [&](bool is_b) {
    const uint64_t from = is_b ? pb : pa;
    const unsigned rows = unsigned(min(left, kUnitK));
    const unsigned covers = is_b ? (BCOLS ? rows * unsigned(sb.kspan) : sb.limit)
                                 : (ACOLS ? rows * unsigned(sa.kspan) : sa.limit);
    rsrc = u32x4_t{unsigned(__builtin_amdgcn_readfirstlane(int(from))),
                   unsigned(__builtin_amdgcn_readfirstlane(int(from >> 32))) & 0xffffu,
                   unsigned(__builtin_amdgcn_readfirstlane(int(covers))), 0x00020000u};
    to = lds + ring;
    ring = ring == (kUnits - 1) * UNIT ? 0 : ring + UNIT;
  };
  auto starts = [&](bool is_b) {
    v0 = is_b ? sb.v0 : sa.v0;
    v1 = is_b ? sb.v1 : sa.v1;
    step = is_b ? sb.step : sa.step;
    if ((is_b ? sb.chunk : sa.chunk) * 8 >= left) v0 = v1 = kBufNone;
    if (is_b && to_go > 0) {
      --to_go;
      pa += a_pair;
      pb += b_pair;
      left -= kUnitK;
      if (TWO && left <= 0) {
        pa = pa2;
        pb = pb2;
        left = k_all;
        // the second matrix's rows lie ldb2 apart
        sb.init<BT, BCOLS>(p.b2, p.ldb2, n0, int(min(int64_t(BT), p.n - n0)), wave, lane, false);
        b_pair = unsigned(kUnitK * sb.kbytes);
      }
    }
  };
  // Among the MFMAs the descriptor is formed two of them ahead of its first
  // load, which then waits for nothing more: five wait states in each load took
  // 4440 us for 4330 in the backward call of 4096 rows, 5120 x 20480.
  auto issue_one = [&](int i, auto ahead) {
    dma16<decltype(ahead)::value ? 0 : 3>(rsrc, to + unsigned(i) * 4096u, ((i & 1) ? v1 : v0) + unsigned(i) * step);
  };
  u32x4_t a[F], b[F];

#pragma unroll
  for (int u = 0; u < kUnits - 1; ++u) {
    place(u & 1);
    starts(u & 1);
#pragma unroll
    for (int i = 0; i < DMA; ++i) issue_one(i, std::false_type{});
  }
  wait_vm<2 * DMA>();
  barrier();
#pragma unroll
  for (int f = 0; f < F; ++f) fa.read(a[f], smem, 0, f);
#pragma unroll
  for (int f = 0; f < F; ++f) fb.read(b[f], smem + UNIT, 0, f);

  constexpr int NXY = F * F, HB = F / 2, PRE = F == 8 ? 10 : 6;
  for (int s = 0; s < stages; ++s) {
    auto mma = [&](int i) {
      const int x = (i % (F * HB)) / HB, y = (i / (F * HB)) * HB + i % HB;
      // operands swapped: a lane then holds four consecutive n of one m
      acc[x][y] = mfma16(b[y], a[x], acc[x][y]);
    };
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < PRE; ++i) mma(i);
    __builtin_amdgcn_sched_barrier(0);
    if (s & 1) {
      wait_vm<DMA>();
      wait_lds();
      barrier();
    }
    const unsigned pair = unsigned(s + 1) & ~1u, half = unsigned(s + 1) & 1u;
    const unsigned char* sA = smem + (pair % kUnits) * UNIT;
    const unsigned char* sB = smem + ((pair + 1) % kUnits) * UNIT;
    int nd = 0;
#pragma unroll
    for (int i = PRE; i < NXY; ++i) {
      mma(i);
      const int x = (i % (F * HB)) / HB, y = (i / (F * HB)) * HB + i % HB;
      if (i == PRE) place(s & 1);
      if (i == PRE + 1) starts(s & 1);
      if (i >= PRE + 2 && nd < DMA && i % 2 == 0) issue_one(nd++, std::true_type{});
      if (x == F - 1) fb.read(b[y], sB, half, y);
      if (y == F - 1) fa.read(a[x], sA, half, x);
      __builtin_amdgcn_sched_barrier(0);
    }
    static_assert(PRE <= F * HB - HB && DMA <= (NXY - PRE - 2) / 2, "no read before the barrier, a slot for every DMA");
  }
}

// One BT x BT tile per workgroup of four waves.
template <int BT, bool ACOLS, bool BCOLS, int EPI, int ACT, class X>
__device__ __forceinline__ void run_tile(const Prod& p, const X& ext, Tile tile, int range, float* part, unsigned char* smem, int lane,
                                         int wave) {
  constexpr int F = BT / 32, NSTEP = tile_cols<BT, EPI>();
  const int wm = wave >> 1, wn = wave & 1;
  const int64_t m0 = int64_t(tile.tm) * BT, n0 = int64_t(tile.tn) * NSTEP;
  const int all = stages_of(p);
  const int first = range < 0 ? 0 : range % p.splits * p.split_stages;
  const int stages = range < 0 ? all : max(0, min(all - first, p.split_stages));
  f32x4_t acc[F][F];
#pragma unroll
  for (int x = 0; x < F; ++x)
#pragma unroll
    for (int y = 0; y < F; ++y) acc[x][y] = (f32x4_t)(0.f);
  sum_tile<BT, ACOLS, BCOLS, EPI>(acc, p, m0, n0, first, stages, smem, lane, wave);
  // The reloads of the last stage may still be on their way into LDS.
  wait_vm<0>();
  barrier();

  if (range >= 0) {
    float* o = part + (int64_t(p.part0 + range) * 4 + wave) * (F * F * 256) + lane * 4;
    // blocks of 16 rows that the matrix has
#pragma unroll
    for (int x = 0; x < F; ++x)
      if (m0 + wm * (BT / 2) + x * 16 < p.m)
#pragma unroll
        for (int y = 0; y < F; ++y) *as_global(reinterpret_cast<f32x4_t*>(o + (x * F + y) * 256)) = acc[x][y];
    return;
  }
  float bias[8] = {};
  if constexpr (EPI == EPI_LINEAR) load_bias(ext, p, n0 + wn * (NSTEP / 2) + lane % (NSTEP / 16) * 8, bias);
  constexpr int XB = 2;
  static_assert(4 * 16 * XB * (BT / 2 + 4) * 4 <= kUnits * unit_bytes<BT>(), "epilogue rows fit");
  float* er = reinterpret_cast<float*>(smem) + wave * 16 * XB * (BT / 2 + 4);
#pragma unroll
  for (int x = 0; x < F; x += XB)
    emit_rows<BT, EPI, ACT, XB>(p, ext, bias, &acc[x], er, m0 + wm * (BT / 2) + x * 16, n0 + wn * (NSTEP / 2), lane);
}

// MIXED_COLS: products of both kinds of A in one launch.
template <int BT, int LIE, int EPI, int ACT, class X>
__device__ __forceinline__ void product_tile(const ProdArgs& g, const X& ext) {
  __shared__ __attribute__((aligned(1024))) unsigned char smem[kUnits * unit_bytes<BT>()];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int id = int(blockIdx.x), which = 0;
  while (which + 1 < g.count && id >= g.p[which + 1].item0) ++which;
  const Prod& p = g.p[which];
  id -= p.item0;
  // Whole tiles first, then the ranges of the split ones.
  int item, range = -1;
  if (id < p.full) {
    item = int(xcd_item(unsigned(id), unsigned(p.full)));
  } else {
    range = int(xcd_item(unsigned(id - p.full), unsigned((p.mt * p.nt - p.full) * p.splits)));
    item = p.full + range / p.splits;
  }
  const Tile tile = tile_of(p, item);
  if constexpr (LIE == MIXED_COLS) {
    if (p.acols) run_tile<BT, true, true, EPI, ACT>(p, ext, tile, range, g.part, smem, lane, wave);
    else run_tile<BT, false, true, EPI, ACT>(p, ext, tile, range, g.part, smem, lane, wave);
  } else {
    run_tile<BT, false, LIE == ROWS_COLS, EPI, ACT>(p, ext, tile, range, g.part, smem, lane, wave);
  }
}

// Adds the ranges of one split tile, 16 rows of each wave's part per
// workgroup, and finishes them as the product's own epilogue would.
template <int BT, int EPI, int ACT, class X>
__device__ __forceinline__ void product_join(const ProdArgs& g, const X& ext) {
  constexpr int F = BT / 32;
  __shared__ float rows[4 * 16 * (BT / 2 + 4)];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int tile = blockIdx.x / F, which = 0;
  const int x = blockIdx.x % F;
  while (which + 1 < g.count && tile >= g.p[which + 1].join0) ++which;
  const Prod& p = g.p[which];
  tile -= p.join0;
  const Tile t = tile_of(p, p.full + tile);
  if (int64_t(t.tm) * BT + (wave >> 1) * (BT / 2) + x * 16 >= p.m) return;   // a whole wave, no barrier follows
  f32x4_t acc[1][F];
#pragma unroll
  for (int y = 0; y < F; ++y) acc[0][y] = (f32x4_t)(0.f);
#pragma unroll 4
  for (int i = 0; i < p.splits; ++i) {
    const float* o = g.part + (int64_t(p.part0 + tile * p.splits + i) * 4 + wave) * (F * F * 256) + lane * 4;
#pragma unroll
    for (int y = 0; y < F; ++y) acc[0][y] += *as_global(reinterpret_cast<const f32x4_t*>(o + (x * F + y) * 256));
  }
  const int64_t ncol = int64_t(t.tn) * tile_cols<BT, EPI>() + (wave & 1) * (tile_cols<BT, EPI>() / 2);
  float bias[8] = {};
  if constexpr (EPI == EPI_LINEAR) load_bias(ext, p, ncol + lane % (tile_cols<BT, EPI>() / 16) * 8, bias);
  emit_rows<BT, EPI, ACT, 1>(p, ext, bias, acc, rows + wave * 16 * (BT / 2 + 4),
                             int64_t(t.tm) * BT + (wave >> 1) * (BT / 2) + x * 16, ncol, lane);
}


// How a list of products is run.  A workgroup of a 256-tile takes a CU, of
// 128-tiles two fit.  Where a product's tiles do not fill a round over the
// CUs, or take much longer than the launch's others, their sums over k are
// divided, if that is worth a second kernel.
//
// The choice goes by the time of each way, from what was measured on this
// card: a stage takes 0.78 us in 256-tiles and 0.58 us in two 128-tiles of a CU
// (which do half the work), a tile's start and epilogue 11 and 5 us, a launch
// of 256-tiles 8 us more until its first stages are in, and a join 4 us and its
// partial sums' writing and reading at 4.5 TB/s.  (The backward call of 777 x
// 1000 x 2728: 128-tiles with dx in three ranges 70 us, 256-tiles in four 76.
// Forward at 2048 x 8192: 256 rows 49 us in 128-tiles, 57 in 256-tiles; down
// product of 4096 rows 116 + 14 us in halves of 256-tiles, 6 more in 128-tiles.)
struct Plan {
  int bt;
  double us;
  struct { int tiles, full, splits, split_stages; } p[kProds];
};
Plan plan_with(const ProdArgs& g, int bt, bool gate, double each_us) {
  Plan q{};
  q.bt = bt;
  const int nstep = gate ? bt / 2 : bt, slots = bt == 256 ? 256 : 512;
  const double stage_us = bt == 256 ? 0.78 : 0.58, tile_us = bt == 256 ? 11 : 5;
  const double launch_us = bt == 256 ? 8 : 0;
  double others = 0, longest = 0, shortest = 1e30;    // of the products after the first
  for (int i = 0; i < g.count; ++i) {
    const int st = stages_of(g.p[i]), tiles = ((g.p[i].m + bt - 1) / bt) * ((g.p[i].n + nstep - 1) / nstep);
    q.p[i] = {tiles, tiles, 1, st};
    const double us = st * stage_us + tile_us;
    if (i > 0) {
      others += tiles * us;
      longest = us > longest ? us : longest;
      shortest = us < shortest ? us : shortest;
    }
  }
  // The first product, alone or ahead of the others, undivided or in n ranges.
  const int stages = stages_of(g.p[0]), tiles = q.p[0].tiles, rows = g.p[0].m;
  const int rem = g.count > 1 ? tiles : tiles % slots, whole = g.count > 1 ? 0 : tiles / slots;
  const double part_mb = double(bt) * (rows < bt ? (rows + 15) / 16 * 16 : bt) * 4e-6, tile = stages * stage_us + tile_us;
  // (at most 2^20 ranges: a launch's workgroups are counted without them)
  for (int n = 1; n == 1 || (rem > 0 && n <= stages / 4 && n <= (g.count > 1 ? std::min(32, (1 << 20) / rem) : slots / rem));
       ++n) {
    const int per = ((stages + n - 1) / n + 1) & ~1, got = (stages + per - 1) / per;   // whole units
    const double one = per * stage_us + tile_us, join = got > 1 ? 4 + 2 * rem * got * part_mb / 4.5 + each_us * got : 0;
    double us;
    if (g.count == 1) {
      us = whole * tile + (rem > 0 ? one : 0) + join + launch_us;
    } else {
      // workgroups of unequal length, the long ones first
      const double even = (others + rem * got * one) / slots, least = one < shortest ? one : shortest;
      us = std::max(std::max(one, longest), even + 0.5 * least) + join + launch_us;
    }
    if (n == 1 || us < q.us) {
      q.us = us;
      q.p[0] = {tiles, got > 1 ? tiles - rem : tiles, got, per};
    }
  }
  return q;
}
// each_us: a join's time for each range of a tile, which it reads one after the
// other (0.14 us: 365 ranges of one tile took 51; it tells where few tiles have long
// sums, which the feed-forward's do not).
Plan plan_of(const ProdArgs& g, bool gate, double each_us = 0) {
  const Plan big = plan_with(g, 256, gate, each_us), small = plan_with(g, 128, gate, each_us);
  return big.us <= small.us ? big : small;
}
size_t part_bytes(const ProdArgs& g, const Plan& q) {
  size_t ranges = 0;
  for (int i = 0; i < g.count; ++i) ranges += size_t(q.p[i].tiles - q.p[i].full) * q.p[i].splits;
  return ranges * q.bt * q.bt * 4;
}

// Workgroups of a launch's tiles and ranges.
int items_of(const ProdArgs& g, const Plan& q) {
  int items = 0;
  for (int i = 0; i < g.count; ++i) items += q.p[i].full + (q.p[i].tiles - q.p[i].full) * q.p[i].splits;
  return items;
}

// `more` workgroups behind the products' own do what the kernel has them do.
template <int BT, int EPI, class... X>
hipError_t launch_prod(hipStream_t s, ProdArgs g, const Plan& q, void (*gemm)(ProdArgs, X...), void (*join)(ProdArgs, X...),
                       unsigned more, X... ext) {
  constexpr int NSTEP = tile_cols<BT, EPI>();
  int items = 0, ranges = 0, joins = 0;
  for (int i = 0; i < g.count; ++i) {
    Prod& p = g.p[i];
    p.mt = (p.m + BT - 1) / BT;
    p.nt = (p.n + NSTEP - 1) / NSTEP;
    p.full = q.p[i].full;
    p.splits = q.p[i].splits;
    p.split_stages = q.p[i].split_stages;
    p.item0 = items;
    p.part0 = ranges;
    p.join0 = joins;
    const int split = q.p[i].tiles - p.full;
    items += p.full + split * p.splits;
    ranges += split * p.splits;
    joins += split;
  }
  hipLaunchKernelGGL(gemm, dim3(unsigned(items) + more), dim3(256), 0, s, g, ext...);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || joins == 0) return e;
  hipLaunchKernelGGL(join, dim3(unsigned(joins * (BT / 32))), dim3(256), 0, s, g, ext...);
  return hipGetLastError();
}

// Sizes of the launches, for their choice and the workspace.
Prod sizes(int64_t m, int64_t n, int64_t k, int segments = 1) {
  Prod p{};
  p.m = int32_t(m); p.n = int32_t(n); p.k = int32_t(k);
  p.segments = segments;
  return p;
}
ProdArgs alone(const Prod& p) {
  ProdArgs g{};
  g.p[0] = p;
  g.count = 1;
  return g;
}
__device__ __forceinline__ void store4(void* c, int64_t e, f32x4_t v) {
  *as_global(reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(c) + e)) =
      u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}

// ---- few rows -----------------------------------------------------------------
// Up to 16 MT rows of x against row operands, bound by reading the weights
// once: a few output columns (with GATE of both matrices) per workgroup, whose
// waves divide the sum over k among them; weights and x go from memory to
// registers as MFMA fragments, weight rows down and the x rows across.
//
// With up to 8 rows (MT = 0) a fragment has 8 weight rows at 64 consecutive k:
// rows 8 .. 15 are the same weights 32 k further on, and columns 8 .. 15 the
// same x there, so that the two diagonal quarters of the result are the two
// halves of the sum (the others are not used).  Twice the workgroups then
// read, and whole 128-byte lines: one row of 2048 x 8192 takes 16.6 and 7.8 us
// (4.0 and 4.3 TB/s, weights from memory) where 16 columns and 32 k take 17.3
// and 12.0, and 5120 x 20480 takes 71 and 40 (5.9 and 5.2) for 85 and 58.
//
// Returns whether the lane finishes a row: then sum holds columns n .. n + 3 of
// row m.
template <int MT, bool GATE, int NW>
__device__ __forceinline__ bool few_rows_sums(const Prod& p, f32x4_t (&sum)[GATE ? 2 : 1], int64_t& m, int64_t& n) {
  constexpr bool PAIR = MT == 0;
  constexpr int NB = GATE ? 2 : 1, T = PAIR ? 1 : MT, COLS = PAIR ? 8 : 16;
  constexpr int STEPS = 8 / T, STEPK = PAIR ? 64 : 32;      // k steps whose loads go out together
  __shared__ f32x4_t red[NW][NB][T][64];
  const int lane = threadIdx.x & 63, q = lane >> 4;
  const int r = PAIR ? lane & 7 : lane & 15, k0 = 8 * q + (PAIR ? 4 * (lane & 8) : 0);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = int64_t(xcd_item(blockIdx.x, gridDim.x)) * COLS;
  // Rows past the end repeat the last one: their results are not stored.
  const int64_t wrow = min(n0 + r, int64_t(p.n) - 1);
  const uint16_t* w[2] = {static_cast<const uint16_t*>(p.b) + wrow * p.ldb,
                          static_cast<const uint16_t*>(p.b2) + (GATE ? wrow * p.ldb2 : 0)};
  const uint16_t* x[T];
#pragma unroll
  for (int t = 0; t < T; ++t) x[t] = static_cast<const uint16_t*>(p.a) + min(16 * t + r, p.m - 1) * p.lda;
  f32x4_t acc[NB][T];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int t = 0; t < T; ++t) acc[i][t] = (f32x4_t)(0.f);
  // The waves take turns along k, STEPS steps each.
  const int steps = (p.k + STEPK - 1) / STEPK;
  for (int s0 = wave * STEPS; s0 < steps; s0 += NW * STEPS) {
    u32x4_t fw[STEPS][NB], fx[STEPS][T];
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int k = (s0 + s) * STEPK + k0;
      const bool ok = k < p.k;              // k is a multiple of 8: whole groups
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        fw[s][i] = u32x4_t{0, 0, 0, 0};
        if (ok) fw[s][i] = *as_global(reinterpret_cast<const u32x4_t*>(w[i] + k));
      }
#pragma unroll
      for (int t = 0; t < T; ++t) {
        fx[s][t] = u32x4_t{0, 0, 0, 0};
        if (ok) fx[s][t] = *as_global(reinterpret_cast<const u32x4_t*>(x[t] + k));
      }
    }
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int t = 0; t < T; ++t) acc[i][t] = mfma16(fw[s][i], fx[s][t], acc[i][t]);
  }
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int t = 0; t < T; ++t) red[wave][i][t][lane] = acc[i][t];
  __syncthreads();
  // Wave t finishes rows 16 t ..: a lane has columns n0 + 4 q .. + 3 of one.
  if (wave >= T || (PAIR && (q > 1 || (lane & 8)))) return false;
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    sum[i] = (f32x4_t)(0.f);
#pragma unroll
    for (int v = 0; v < NW; ++v) {
      sum[i] += red[v][i][wave][lane];
      if constexpr (PAIR) sum[i] += red[v][i][wave][lane + 40];    // column + 8, rows + 8
    }
  }
  m = 16 * wave + r;
  n = n0 + 4 * q;
  return m < p.m && n < p.n;                // p.n is a multiple of 8
}

}  // namespace
}  // namespace muon
