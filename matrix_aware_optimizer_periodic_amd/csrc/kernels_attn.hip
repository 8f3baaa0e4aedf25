// Softmax attention, forward and backward, on bf16 matrix cores.
//
//   s = scale q k^T (keys that a query sees), p = softmax(s), o = p v
//   delta_i = do_i . o_i,  ds = p (do v^T - delta)
//   dv = p^T do,  dq = scale ds k,  dk = scale ds^T q
//
// One pass over the keys with a running maximum and sum per query; nothing of
// size q_len x k_len is stored, and the backward pass recomputes p from q, k
// and the logarithm of the sum.  Bound by the matrix cores (4 D operations per
// visible pair forward, 14 D backward here: the scores and do v^T are formed
// in both backward kernels, so that neither needs atomics), for one query by
// reading the keys and values.
//
// Every product is arranged so that the scores stay in registers between the
// two products they sit between: the first product leaves a lane with one
// query (or key) and four consecutive keys (or queries) at a time, and as the
// second product's operand those are k indices, whose order is free as long
// as the other operand follows it.  That other operand is read from LDS
// through the transposing read, four consecutive k of one column at a time,
// in just that order.  So probabilities never go through LDS.
//
// LDS rows hold 64 or 128 values; 16-byte chunk c of row r is stored at chunk
// c ^ x(r).  The row reads (32 rows at one chunk) and the transposed reads
// (four rows at a 64-byte block) then both go to distinct banks.
//
// Rows of the forward and dq kernels are the (query, head) pairs that share a
// key head, the heads of one query next to each other: grouped heads and few
// queries share the key tiles of one workgroup.
//
// Measured on one MI355X (a large library product runs at 1460 TFLOP/s), medians
// of twelve calls, head size 128: forward 164 us at 16 x 1024, 16 heads (836
// TFLOP/s), 1018 us at 2 x 8192 (1080); dq 153 us and dk, dv 243 us at 4 x 1024,
// 40 heads (845 and 708 on the products they form; 138 and 203 us at best), 1213
// TFLOP/s for both at 16384; one query of 4 x 32 heads over 8191 keys of 8 25 us
// (134 MB, 5.3 TB/s) and 4.4 us for the join.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "block_mfma.h"

namespace muon {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kTile = 64;        // keys (dq, forward) or queries (dk, dv) per LDS tile
constexpr int kRowsWg = 128;     // rows of the forward and dq workgroups: four waves of 32

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
// The lane's number, formed where it is called (the compiler cannot keep it).
__device__ __forceinline__ int fresh_lane() {
  unsigned all = ~0u;
  asm volatile("" : "+s"(all));
  return int(__builtin_amdgcn_mbcnt_hi(all, __builtin_amdgcn_mbcnt_lo(all, 0u)));
}
// The value of the lane 32 away.
__device__ __forceinline__ float other_half(float x) {
  const unsigned u = __float_as_uint(x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);   // (low of both, high of both)
  return __uint_as_float(__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u)) < 32 ? r[1] : r[0]);
}

// Head geometry: DB blocks of 32 dims; LDS rows of PITCH 16-byte chunks.
template <int DB>
struct Geo {
  static constexpr int KS = 2 * DB;                 // 16-deep steps over the head's dims
  static constexpr int PITCH = DB <= 2 ? 8 : 16;
  static constexpr int ROWB = PITCH * 16;           // bytes of a row
  static constexpr int TILEB = kTile * ROWB;
  static __device__ __forceinline__ int swz(int row) {
    return PITCH == 16 ? ((row & 3) << 2) | ((row >> 2) & 3) : (((row >> 1) & 1) << 2) | ((row >> 2) & 3);
  }
};

// Moves one tile of kTile rows, `stride` values apart, into LDS.  What is past
// `there` rows or past dim values reads as zero.
template <int DB, int WAVES = 4>
struct TileMove {
  static constexpr int P = Geo<DB>::PITCH;
  static constexpr int STEP = WAVES * (64 / P);       // rows between a wave's DMAs
  static constexpr int N = kTile / STEP;
  static_assert(STEP % 16 == 0, "a lane's swizzle is the same in all of its rows");
  unsigned voff;
  int row0;
  unsigned step;                                      // bytes
  __device__ __forceinline__ TileMove(int64_t stride, int dim, int wave, int lane) {
    row0 = wave * (64 / P) + lane / P;
    const int chunk = (lane % P) ^ Geo<DB>::swz(row0);
    voff = chunk * 8 < dim ? unsigned(int64_t(row0) * stride * 2 + chunk * 16) : kBufNone;
    step = unsigned(STEP * stride * 2);
  }
  __device__ __forceinline__ void issue(const uint16_t* tile, int there, unsigned lds, int wave) const {
    const u32x4_t r = buffer_at(tile);
    if (there >= kTile) {
#pragma unroll
      for (int i = 0; i < N; ++i) dma16(r, lds + unsigned(wave + WAVES * i) * 1024u, voff, unsigned(i) * step);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        dma16(r, lds + unsigned(wave + WAVES * i) * 1024u, row0 + i * STEP < there ? voff : kBufNone,
              unsigned(i) * step);
    }
  }
};

// Fragments straight from global memory: one row per lane, 8 values from
// 16 ks + 8 half.  One branch for all loads where the head fills its blocks.
template <int DB>
__device__ __forceinline__ void load_rows(u32x4_t (&f)[2 * DB], const uint16_t* row, bool ok, int dim, int half) {
#pragma unroll
  for (int ks = 0; ks < 2 * DB; ++ks) f[ks] = u32x4_t{0, 0, 0, 0};
  if (!ok) return;
  const auto* g = as_global(reinterpret_cast<const u32x4_t*>(row + half * 8));
  if (dim == 32 * DB) {
#pragma unroll
    for (int ks = 0; ks < 2 * DB; ++ks) f[ks] = g[2 * ks];
  } else {
#pragma unroll
    for (int ks = 0; ks < 2 * DB; ++ks)
      if (ks * 16 + half * 8 < dim) f[ks] = g[2 * ks];
  }
}

__device__ __forceinline__ unsigned div_by(unsigned n, const FastDiv& d) { return (__umulhi(n, d.mul) + n) >> d.shift; }

// Makes the compiler wait for loaded fragments here.  Left to their first use
// in a loop it would wait there in every round, and so for the DMA in flight.
template <int N>
__device__ __forceinline__ void arrived(u32x4_t (&f)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+v"(f[i]));
}

// This lane's reads within a tile: row reads (32 rows of one chunk) and
// transposed reads (A operand: dims down, k across).  The chunk's number is
// xored into the low bits of an offset, so one offset serves all of them.
template <int DB>
struct TileRead {
  using G = Geo<DB>;
  unsigned row, tr;
  __device__ __forceinline__ explicit TileRead(int lane) {
    const int l = lane & 31, half = lane >> 5, s = lane & 15;
    row = unsigned(l * G::ROWB + ((half ^ G::swz(l)) << 4));
    const int r = 4 * half + (s >> 2), c = 2 * ((lane >> 4) & 1) + ((s & 3) >> 1);
    tr = unsigned(r * G::ROWB + ((c ^ G::swz(r)) << 4) + (s & 1) * 8);
  }
  // 16 dims from 16 ks of the rows of block `block` of 32
  __device__ __forceinline__ u32x4_t rows(const unsigned char* t, int ks, int block) const {
    return lds_read16(t + block * 32 * G::ROWB, row ^ unsigned(32 * ks));
  }
  // dims 32 db .. + 31, k step `step` of 16 rows: rows 4 half .. and 8 + 4 half ..
  __device__ __forceinline__ u32x4_t cols(const unsigned char* t, int db, int step) const {
    const unsigned char* at = t + step * 16 * G::ROWB;
    const u32x2_t a = lds_read_tr(at, tr ^ unsigned(64 * db));
    const u32x2_t b = lds_read_tr(at + 8 * G::ROWB, tr ^ unsigned(64 * db) ^ 32u);
    return u32x4_t{a[0], a[1], b[0], b[1]};
  }
};

// The same with every offset in a register of its own, for kernels that have
// room for them: no arithmetic per read (a quarter of the forward kernel's
// vector instructions were these xors).  `at` is a constant.
template <int DB>
struct TileOffsets {
  using G = Geo<DB>;
  unsigned row[2 * DB], tr[DB][2];
  __device__ __forceinline__ explicit TileOffsets(int lane, const unsigned char* smem) {
    const TileRead<DB> r(lane);
    const unsigned lds = lds_offset(smem);
#pragma unroll
    for (int ks = 0; ks < 2 * DB; ++ks) {
      row[ks] = lds + (r.row ^ unsigned(32 * ks));
      asm volatile("" : "+v"(row[ks]));
    }
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        tr[db][u] = lds + (r.tr ^ unsigned(64 * db) ^ unsigned(32 * u));
        asm volatile("" : "+v"(tr[db][u]));
      }
  }
  __device__ __forceinline__ u32x4_t rows(unsigned at, int ks, int block) const {
    return *(const MUON_LOCAL u32x4_t*)(uintptr_t)(row[ks] + at + unsigned(block * 32 * G::ROWB));
  }
  __device__ __forceinline__ u32x4_t cols(unsigned at, int db, int step) const {
    const unsigned o = at + unsigned(step * 16 * G::ROWB);
    const u32x2_t a = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                      (MUON_LOCAL s16x4_t*)(uintptr_t)(tr[db][0] + o)));
    const u32x2_t b = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                      (MUON_LOCAL s16x4_t*)(uintptr_t)(tr[db][1] + o + 8u * G::ROWB)));
    return u32x4_t{a[0], a[1], b[0], b[1]};
  }
};

// Eight results of a product as the next product's operand.
__device__ __forceinline__ u32x4_t pack8(const f32x16_t& s, int from) {
  return u32x4_t{pack_bf16x2(s[from], s[from + 1]), pack_bf16x2(s[from + 2], s[from + 3]),
                 pack_bf16x2(s[from + 4], s[from + 5]), pack_bf16x2(s[from + 6], s[from + 7])};
}

// Result block -> one row of global memory per lane: dims 32 db + 8 g + 4 half
// .. + 3 of every g.
template <int DB>
__device__ __forceinline__ void store_rows(const f32x16_t (&acc)[DB], float mul, uint16_t* row, int dim, int half) {
#pragma unroll
  for (int db = 0; db < DB; ++db)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int d = 32 * db + 8 * g + 4 * half;
      if (d < dim)
        *as_global(reinterpret_cast<u32x2_t*>(row + d)) =
            u32x2_t{pack_bf16x2(acc[db][4 * g] * mul, acc[db][4 * g + 1] * mul),
                    pack_bf16x2(acc[db][4 * g + 2] * mul, acc[db][4 * g + 3] * mul)};
    }
}

__device__ __forceinline__ int clamp_len(const int32_t* lens, int b, int most) {
  return __builtin_amdgcn_readfirstlane(lens ? min(max(lens[b], 0), most) : most);
}

// Which rows a workgroup of the forward or dq kernel has, and what they see.
struct Rows {
  int b, kvh, q_here, k_here;
  int row0;                  // first row of the workgroup
  int qi, head;              // this lane's query and head
  bool ok;                   // the lane's row is inside the tensor
  bool live;                 // ... and inside the sample's length
  int see;                   // keys that the lane's row sees: 0 .. see - 1
};

__device__ __forceinline__ int seen(const AttnDev& a, int qi, int k_here) {
  if (!a.causal) return k_here;
  const int64_t n = int64_t(qi) + a.offset + 1;
  return int(max(int64_t(0), min(int64_t(k_here), n)));
}

__device__ __forceinline__ Rows rows_of(const AttnDev& a, unsigned item, int wave, int lane) {
  Rows r;
  // Later rows see more keys under a causal border: they go first.
  const unsigned bh = div_by(item, a.row_blocks), blk = a.row_blocks.by - 1 - (item - bh * a.row_blocks.by);
  r.b = int(div_by(bh, a.by_kv_heads));
  r.kvh = int(bh) - r.b * a.kv_heads;
  r.q_here = clamp_len(a.q_lens, r.b, a.q_len);
  r.k_here = clamp_len(a.k_lens, r.b, a.k_len);
  r.row0 = int(blk) * kRowsWg;
  const int row = r.row0 + wave * 32 + (lane & 31);
  const int group = int(a.by_group.by);
  r.qi = int(div_by(unsigned(row), a.by_group));
  r.head = r.kvh * group + row - r.qi * group;
  r.ok = r.qi < a.q_len;
  r.live = r.qi < r.q_here;
  r.see = r.live ? seen(a, r.qi, r.k_here) : 0;
  return r;
}

__device__ __forceinline__ int wave_max(int v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = max(v, __shfl_xor(v, o, 64));
  return __builtin_amdgcn_readfirstlane(v);
}

// Keys that the last of the workgroup's rows sees (the most of any).
__device__ __forceinline__ int seen_most(const AttnDev& a, const Rows& r) {
  const int last = min(int(div_by(unsigned(r.row0 + kRowsWg - 1), a.by_group)), r.q_here - 1);
  return last < int(div_by(unsigned(r.row0), a.by_group)) ? 0 : seen(a, last, r.k_here);
}

// ---------------------------------------------------------------------------
// Forward.  Per tile of 64 keys: s^T = k q^T (a lane has one row, half of the
// keys), running maximum and sum, o^T += v^T p^T.  The maximum that the
// exponents are taken against follows the running one only when that has
// grown by more than 2^8 (the result does not depend on it), so that the
// accumulators are rarely rescaled.
//
// Software pipeline: the products of the next tile's scores run between this
// tile's exponentials, and the maxima of the next tile between the products
// with v, so that the matrix cores and the vector units work at once.  The
// order within a slot (one product, its fragment's successor, a piece of
// arithmetic) is fixed; left to itself the compiler waits for each read at
// once.  Two workgroups of four waves and 128 rows per CU: eight waves and 256
// rows, which bring in half as much, measured 5% slower (the waves meet at
// every tile), and what a longer way between asking for a tile and using it, or
// several row blocks per workgroup, could hide measured nothing.  Up to 64 dims
// three workgroups fit (168 registers, one of them spilled): calls of 98 us
// against 107 for 16 samples of 1024 queries and keys with 16 heads of 64, 591
// against 619 for 2 of 8192 (the kernel alone: 89 and 595).  The dq kernel gains
// 1% at most from that, with four spilled.
template <int DB, bool SPLIT>
__global__ __launch_bounds__(256, DB <= 2 ? 3 : 2) void attn_fwd_kernel(AttnDev a, unsigned items) {
  using G = Geo<DB>;
  constexpr int KS = G::KS, AHEAD = 3;
  __shared__ __attribute__((aligned(1024))) unsigned char smem[4 * G::TILEB];   // two of k, two of v
  const int lane = threadIdx.x & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const unsigned id = xcd_item(blockIdx.x, items);
  const unsigned item = SPLIT ? div_by(id, a.by_splits) : id, split = id - item * unsigned(a.splits);
  const Rows r = rows_of(a, item, wave, lane);
  const int first = SPLIT ? int(split) * a.split_keys : 0;
  const int most = seen_most(a, r), end = SPLIT ? min(most, first + a.split_keys) : most;
  const int tiles = end > first ? (end - first + kTile - 1) / kTile : 0;

  const uint16_t* kbase = static_cast<const uint16_t*>(a.k.p) + r.b * a.k.sb + r.kvh * a.k.sh + first * a.k.sl;
  const uint16_t* vbase = static_cast<const uint16_t*>(a.v.p) + r.b * a.v.sb + r.kvh * a.v.sh + first * a.v.sl;
  const TileMove<DB, 4> mk(a.k.sl, a.dim, wave, lane), mv(a.v.sl, a.dim, wave, lane);
  const unsigned lds = lds_offset(smem);
  auto fetch_k = [&](int t) {
    mk.issue(kbase + int64_t(t) * kTile * a.k.sl, most - first - t * kTile, lds + unsigned(t & 1) * G::TILEB, wave);
  };
  auto fetch_v = [&](int t) {
    mv.issue(vbase + int64_t(t) * kTile * a.v.sl, most - first - t * kTile, lds + unsigned(2 + (t & 1)) * G::TILEB, wave);
  };

  if (tiles > 0) fetch_k(0);
  u32x4_t q[2 * DB];
  const uint16_t* qrow = static_cast<const uint16_t*>(a.q.p) + r.b * a.q.sb + r.qi * a.q.sl + r.head * a.q.sh;
  load_rows<DB>(q, qrow, r.live, a.dim, half);
  const TileOffsets<DB> rd(lane, smem);
  f32x16_t o[DB];
#pragma unroll
  for (int db = 0; db < DB; ++db) o[db] = (f32x16_t)(0.f);
  const float c = a.scale * kLog2e;
  float top = -INFINITY, top_c = 0.f, sum = 0.f;
  const int wave_all = -wave_max(r.ok ? -r.see : -0x7fffffff);
  const bool work = wave_max(r.see) > 0;
  // Keys of a tile that a row does not see.
  auto mask = [&](f32x16_t (&s)[2], int key0) {
    if (key0 + kTile > wave_all) {
      const int n = r.see - key0 - 4 * half;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int v = 0; v < 16; ++v)
          if (32 * kb + 8 * (v >> 2) + (v & 3) >= n) s[kb][v] = -INFINITY;
    }
  };
  // Raises the maximum where a tile's is much larger.
  auto raise = [&](float m) {
    m = fmaxf(m, other_half(m));
    if (__any((m - top) * c > 8.f)) {        // also where top is -inf and m is not
      const float to = fmaxf(top, m);
      const float f = to == -INFINITY ? 1.f : exp2_fast((top - to) * c);
      top = to;
      top_c = to == -INFINITY ? 0.f : to * c;
      sum *= f;
#pragma unroll
      for (int db = 0; db < DB; ++db)
#pragma unroll
        for (int v = 0; v < 16; ++v) o[db][v] *= f;
    }
  };

  f32x16_t s0[2], s1[2];
  wait_vm<0>();
  arrived(q);
  barrier();
  if (tiles > 0) {
    fetch_v(0);
    if (tiles > 1) fetch_k(1);
    if (work) {
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) s0[kb] = mfma32(rd.rows(0, ks, kb), q[ks], ks ? s0[kb] : (f32x16_t)(0.f));
      mask(s0, first);
      float m = s0[0][0];
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int v = 0; v < 16; ++v) m = fmaxf(m, s0[kb][v]);
      raise(m);
    }
  }
  // Tile t, whose scores are in s; the next tile's go to sn (past the last
  // tile from what is in LDS, and unused).
  auto step = [&](int t, auto odd, f32x16_t (&s)[2], f32x16_t (&sn)[2]) {
    constexpr int ODD = decltype(odd)::value;
    // The next k and this v are in, and every wave has read k of tile t (in the
    // step before) and v of tile t - 1, whose buffers are refilled.
    wait_vm<0>();
    barrier();
    if (t + 2 < tiles) fetch_k(t + 2);
    if (t + 1 < tiles) fetch_v(t + 1);
    if (!work) return;
    constexpr unsigned kt = (ODD ^ 1) * G::TILEB, vt = (2 + ODD) * G::TILEB;
    constexpr int N1 = 2 * KS, N2 = 4 * DB;
    u32x4_t f[AHEAD], p[4];
    auto fragment = [&](int n) {
      return n < N1 ? rd.rows(kt, n / 2, n & 1) : rd.cols(vt, (n - N1) % DB, (n - N1) / DB);
    };
    auto slot_end = [&](int n) {
      if (n + AHEAD < N1 + N2) f[n % AHEAD] = fragment(n + AHEAD);
      __builtin_amdgcn_sched_barrier(0);
    };
#pragma unroll
    for (int n = 0; n < AHEAD; ++n) f[n] = fragment(n);
    __builtin_amdgcn_sched_barrier(0);
    // 8 pieces of four values
    auto probs = [&](int i) {
      const int kb = i / 4, g = i % 4;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        s[kb][4 * g + k] = exp2_fast(fmaf(s[kb][4 * g + k], c, -top_c));
        sum += s[kb][4 * g + k];
      }
      if (g & 1) {
        p[2 * kb + (g >> 1)] = pack8(s[kb], 8 * (g >> 1));
        // pins the work here: it would be sunk past the mask's branch
        asm volatile("" : "+v"(p[2 * kb + (g >> 1)]), "+v"(sum));
      }
    };
#pragma unroll
    for (int n = 0; n < N1; ++n) {
      sn[n & 1] = mfma32(f[n % AHEAD], q[n / 2], n > 1 ? sn[n & 1] : (f32x16_t)(0.f));
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i * N1 / 8 == n) probs(i);
      slot_end(n);
    }
    mask(sn, first + (t + 1) * kTile);
    __builtin_amdgcn_sched_barrier(0);
    float m = -INFINITY;
#pragma unroll
    for (int n = N1; n < N1 + N2; ++n) {
      const int j = (n - N1) / DB, db = (n - N1) % DB;
      o[db] = mfma32(f[n % AHEAD], p[j], o[db]);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i * N2 / 8 == n - N1) {
#pragma unroll
          for (int k = 0; k < 4; ++k) m = fmaxf(m, sn[i / 4][4 * (i % 4) + k]);
          asm volatile("" : "+v"(m));
        }
      slot_end(n);
    }
    if (t + 1 < tiles) raise(m);
  };
  for (int t = 0; t < tiles; t += 2) {
    step(t, std::integral_constant<int, 0>{}, s0, s1);
    if (t + 1 < tiles) step(t + 1, std::integral_constant<int, 1>{}, s1, s0);
  }
  sum += other_half(sum);
  const float inv = sum == 0.f ? 0.f : 1.0f / sum;
  const float lse = sum == 0.f ? -INFINITY : fmaf(top, a.scale, __builtin_amdgcn_logf(sum) * kLn2);
  if (!r.ok) return;
  if (sum == 0.f) {            // sees none of these keys, whatever they hold
#pragma unroll
    for (int db = 0; db < DB; ++db) o[db] = (f32x16_t)(0.f);
  }
  const int64_t line = (int64_t(r.b) * a.heads + r.head) * a.q_len + r.qi;
  if constexpr (SPLIT) {
    const int64_t at = int64_t(split) * a.batch * a.heads * a.q_len + line;
    float* po = a.part_o + at * a.dim;
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int d = 32 * db + 8 * g + 4 * half;
        if (d < a.dim)
          *as_global(reinterpret_cast<f32x4_t*>(po + d)) = f32x4_t{o[db][4 * g] * inv, o[db][4 * g + 1] * inv,
                                                                   o[db][4 * g + 2] * inv, o[db][4 * g + 3] * inv};
      }
    if (half == 0) *as_global(a.part_lse + at) = lse;
  } else {
    store_rows<DB>(o, inv, static_cast<uint16_t*>(a.o.p) + r.b * a.o.sb + r.qi * a.o.sl + r.head * a.o.sh, a.dim, half);
    if (half == 0) *as_global(a.lse + line) = lse;
  }
}

// Joins the key ranges of one row: weights exp(lse_i - lse) add up to 1.  A
// wave per row: its lanes take the ranges' weights at once, then groups of 16
// lanes, eight dims each, every fourth range.
__global__ __launch_bounds__(256) void attn_join_kernel(AttnDev a) {
  const int64_t lines = int64_t(a.batch) * a.heads * a.q_len;
  const int64_t line = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (line >= lines) return;
  const int lane = threadIdx.x & 63, d = (lane & 15) * 8;
  float top = -INFINITY;
  bool nan = false;
  for (int i = lane; i < a.splits; i += 64) {
    const float lse = *as_global(a.part_lse + i * lines + line);
    top = fmaxf(top, lse);
    nan |= lse != lse;
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
  // The maximum leaves NaN out; a row that has one in any range is NaN.
  if (__any(nan)) top = NAN;
  float sum = 0.f, o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (top != -INFINITY) {
#pragma unroll 4
    for (int i = lane >> 4; i < a.splits; i += 4) {
      const float w = exp2_fast((*as_global(a.part_lse + i * lines + line) - top) * kLog2e);
      sum += w;
      if (d < a.dim) {
        float t[8];
        load_vals<float, 8>(a.part_o, (i * lines + line) * a.dim + d, t);
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = fmaf(w, t[k], o[k]);
      }
    }
#pragma unroll
    for (int x = 16; x <= 32; x <<= 1) {
      sum += __shfl_xor(sum, x, 64);
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] += __shfl_xor(o[k], x, 64);
    }
  }
  const int qi = int(line % a.q_len);
  const int64_t bh = line / a.q_len;
  if (lane < 16 && d < a.dim) {
    const float inv = sum == 0.f ? 0.f : 1.0f / sum;
#pragma unroll
    for (int k = 0; k < 8; ++k) o[k] *= inv;
    store_vals<uint16_t, 8>(a.o.p, (bh / a.heads) * a.o.sb + qi * a.o.sl + (bh % a.heads) * a.o.sh + d, o);
  }
  if (lane == 0) *as_global(a.lse + line) = sum == 0.f ? -INFINITY : top + __builtin_amdgcn_logf(sum) * kLn2;
}

// ---------------------------------------------------------------------------
// dq, and per row delta = do . o and the exponent's offset for the dk, dv
// kernel.  Per tile of 64 keys: s^T = k q^T, dp^T = v do^T,
// ds^T = p^T (dp^T - delta), dq^T += k^T ds^T.  Both halves of the tile run
// side by side, so that no product waits for the one before it.
template <int DB>
__global__ __launch_bounds__(256, 2) void attn_dq_kernel(AttnDev a, unsigned items) {
  using G = Geo<DB>;
  constexpr int AHEAD = 3;
  __shared__ __attribute__((aligned(1024))) unsigned char smem[4 * G::TILEB];
  const int lane = threadIdx.x & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Rows r = rows_of(a, xcd_item(blockIdx.x, items), wave, lane);
  const int end = seen_most(a, r);
  const int tiles = (end + kTile - 1) / kTile;

  u32x4_t q[2 * DB], g[2 * DB];
  load_rows<DB>(q, static_cast<const uint16_t*>(a.q.p) + r.b * a.q.sb + r.qi * a.q.sl + r.head * a.q.sh, r.see > 0, a.dim,
                half);
  load_rows<DB>(g, static_cast<const uint16_t*>(a.d_o.p) + r.b * a.d_o.sb + r.qi * a.d_o.sl + r.head * a.d_o.sh, r.see > 0,
                a.dim, half);
  float delta = 0.f;
  {
    u32x4_t o[2 * DB];
    load_rows<DB>(o, static_cast<const uint16_t*>(a.o.p) + r.b * a.o.sb + r.qi * a.o.sl + r.head * a.o.sh, r.see > 0,
                  a.dim, half);
    // The diagonal of o do^T, summed in the same order as do v^T below: where
    // a row's o is one row of v (one key), dp - delta is then exactly 0.
    f32x16_t s = (f32x16_t)(0.f);
#pragma unroll
    for (int ks = 0; ks < G::KS; ++ks) s = mfma32(o[ks], g[ks], s);
#pragma unroll
    for (int v = 0; v < 16; ++v)
      if (8 * (v >> 2) + 4 * half + (v & 3) == (lane & 31)) delta = s[v];
    delta += other_half(delta);
  }
  // A row that sees nothing gets the offset +inf: its probabilities are 0.
  const int64_t line = (int64_t(r.b) * a.heads + r.head) * a.q_len + r.qi;
  float lse = INFINITY;
  if (r.see > 0) {
    lse = *as_global(a.lse + line);
    lse = lse == -INFINITY ? INFINITY : lse * kLog2e;
  }
  if (r.ok && half == 0) {
    *as_global(a.part_lse + line) = lse;
    *as_global(a.delta + line) = delta;
  }

  const uint16_t* kbase = static_cast<const uint16_t*>(a.k.p) + r.b * a.k.sb + r.kvh * a.k.sh;
  const uint16_t* vbase = static_cast<const uint16_t*>(a.v.p) + r.b * a.v.sb + r.kvh * a.v.sh;
  const TileMove<DB, 4> mk(a.k.sl, a.dim, wave, lane), mv(a.v.sl, a.dim, wave, lane);
  const TileRead<DB> rd(lane);
  const unsigned lds = lds_offset(smem);
  auto fetch = [&](int t) {
    const unsigned at = lds + unsigned(t & 1) * 2u * G::TILEB;
    mk.issue(kbase + int64_t(t) * kTile * a.k.sl, end - t * kTile, at, wave);
    mv.issue(vbase + int64_t(t) * kTile * a.v.sl, end - t * kTile, at + G::TILEB, wave);
  };
  f32x16_t acc[DB];
#pragma unroll
  for (int db = 0; db < DB; ++db) acc[db] = (f32x16_t)(0.f);
  const float c = a.scale * kLog2e;
  const int wave_see = wave_max(r.see), wave_all = -wave_max(r.ok ? -r.see : -0x7fffffff);

  if (tiles > 0) fetch(0);
  arrived(q);
  arrived(g);
  for (int t = 0; t < tiles; ++t) {
    wait_vm<0>();
    barrier();
    if (t + 1 < tiles) fetch(t + 1);
    if (t * kTile >= wave_see) continue;
    const unsigned char* kt = smem + (t & 1) * 2 * G::TILEB;
    const unsigned char* vt = kt + G::TILEB;
    // Slots as in the forward kernel: 2 KS row reads of k, 2 KS of v (the two
    // halves of the tile in turn), 4 DB transposed reads of k.
    constexpr int KS = G::KS, N = 4 * KS + 4 * DB;
    u32x4_t f[AHEAD], ds[4];
    f32x16_t s[2], dp[2];
    auto fragment = [&](int n) {
      if (n < 2 * KS) return rd.rows(kt, n / 2, n & 1);
      if (n < 4 * KS) return rd.rows(vt, (n - 2 * KS) / 2, n & 1);
      return rd.cols(kt, (n - 4 * KS) % DB, (n - 4 * KS) / DB);
    };
    auto slot_end = [&](int n) {
      if (n + AHEAD < N) f[n % AHEAD] = fragment(n + AHEAD);
      __builtin_amdgcn_sched_barrier(0);
    };
    auto grads = [&](int i) {
      const int kb = i / 4, g = i % 4;
#pragma unroll
      for (int k = 0; k < 4; ++k) s[kb][4 * g + k] *= dp[kb][4 * g + k] - delta;
      if (g & 1) ds[2 * kb + (g >> 1)] = pack8(s[kb], 8 * (g >> 1));
    };
#pragma unroll
    for (int n = 0; n < AHEAD; ++n) f[n] = fragment(n);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int n = 0; n < 2 * KS; ++n) {
      s[n & 1] = mfma32(f[n % AHEAD], q[n / 2], n > 1 ? s[n & 1] : (f32x16_t)(0.f));
      slot_end(n);
    }
    if ((t + 1) * kTile > wave_all) {
      const int n = r.see - t * kTile - 4 * half;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int v = 0; v < 16; ++v)
          if (32 * kb + 8 * (v >> 2) + (v & 3) >= n) s[kb][v] = -INFINITY;
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int n = 2 * KS; n < 4 * KS; ++n) {
      const int m = n - 2 * KS;
      dp[n & 1] = mfma32(f[n % AHEAD], g[m / 2], m > 1 ? dp[n & 1] : (f32x16_t)(0.f));
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (1 + i * (2 * KS - 1) / 8 == m) {
#pragma unroll
          for (int k = 0; k < 4; ++k) s[i / 4][4 * (i % 4) + k] = exp2_fast(fmaf(s[i / 4][4 * (i % 4) + k], c, -lse));
        }
      slot_end(n);
    }
    grads(0);
    grads(1);
#pragma unroll
    for (int n = 4 * KS; n < N; ++n) {
      const int m = n - 4 * KS;
      acc[m % DB] = mfma32(f[n % AHEAD], ds[m / DB], acc[m % DB]);
      // ahead of the products that take them
#pragma unroll
      for (int i = 2; i < 8; ++i)
        if ((i - 2) / 2 * DB + (i & 1 ? DB - 1 : 0) == m) grads(i);
      slot_end(n);
    }
  }
  if (r.see == 0) {            // no gradient, whatever the others' keys and values hold
#pragma unroll
    for (int db = 0; db < DB; ++db) acc[db] = (f32x16_t)(0.f);
  }
  if (r.ok)
    store_rows<DB>(acc, a.scale, static_cast<uint16_t*>(a.d_q.p) + r.b * a.d_q.sb + r.qi * a.d_q.sl + r.head * a.d_q.sh,
                   a.dim, half);
}

// ---------------------------------------------------------------------------
// dk and dv of 256 keys, 32 per wave: the wave's k rows stay in registers, the
// workgroup's v rows in LDS, as the first products' second operand.  Over the
// heads of the group and tiles of 64 queries, 32 at a time: s = q k^T,
// dp = do v^T (a lane has one key), then dv^T += do^T p, dk^T += q^T ds.
// The accumulators (2 x 32 keys x dim) and k take 160 of the 256 registers at
// 128 dims; with v there too 64 registers spilled (427 us where this took
// 206), and 64 keys per wave in 512 registers, one wave per SIMD, took 295: the
// compiler then puts every product's result into accumulation registers and
// moves the scores back and forth.  256 keys share a tile, since a CU takes in
// only some 25 bytes per cycle on the way into LDS.
//
// The (head, query tile) pairs of a key block may be divided over several
// workgroups (a.parts), whose fp32 sums a second kernel adds.
template <int DB, int AHEAD>
__global__ __launch_bounds__(512, 2) void attn_dkv_kernel(AttnDev a, unsigned items) {
  using G = Geo<DB>;
  constexpr int NW = 8, KEYS = 32 * NW;
  constexpr int BUF = 2 * G::TILEB + 2 * kTile * 4;     // q, do, offsets, deltas
  constexpr int VB = KEYS * G::ROWB;
  __shared__ __attribute__((aligned(1024))) unsigned char smem[VB + 2 * BUF];
  const int lane = threadIdx.x & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // Under a causal border the first keys are seen by the most queries: their
  // workgroups go first, those of all heads in turn.
  const unsigned parts = unsigned(a.parts);
  const unsigned id = a.causal ? blockIdx.x : xcd_item(blockIdx.x, items);
  const unsigned item = div_by(id, a.by_parts), part = id - item * parts;
  const unsigned up = div_by(item, a.causal ? a.by_bh : a.key_blocks);
  const unsigned rest = item - up * (a.causal ? a.by_bh.by : a.key_blocks.by);
  const unsigned bh = a.causal ? rest : up, blk = a.causal ? up : rest;
  const int b = int(div_by(bh, a.by_kv_heads)), kvh = int(bh) - b * a.kv_heads, group = int(a.by_group.by);
  const int q_here = clamp_len(a.q_lens, b, a.q_len);
  // keys that the last query sees (the most of any); the others are as if not there
  const int k_here = q_here > 0 ? seen(a, q_here - 1, clamp_len(a.k_lens, b, a.k_len)) : 0;
  const int key0 = int(blk) * KEYS;
  const int wkey = key0 + wave * 32, key = wkey + (lane & 31);
  // First query that sees a key.
  const int64_t border = a.causal ? -a.offset : int64_t(-0x7fffffff);
  auto first_query = [&](int k) { return int(max(int64_t(0), min(int64_t(q_here), int64_t(k) + border))); };
  // The tiles begin at the first query that sees any of the block's keys.
  const int begin = first_query(key0);
  const int per_head = key0 < k_here ? (q_here - begin + kTile - 1) / kTile : 0;
  const int all = per_head * group, share = (all + a.parts - 1) / a.parts;
  const int t0 = min(all, int(part) * share), tiles = min(all, t0 + share) - t0;
  const int wave_first = first_query(wkey), wave_all = first_query(wkey + 31);

  const uint16_t* kbase = static_cast<const uint16_t*>(a.k.p) + b * a.k.sb + kvh * a.k.sh;
  const uint16_t* vbase = static_cast<const uint16_t*>(a.v.p) + b * a.v.sb + kvh * a.v.sh;
  u32x4_t kf[2 * DB] = {};
  const TileRead<DB> rd(lane);
  const unsigned lds = lds_offset(smem);
  const uint16_t* qb0 = static_cast<const uint16_t*>(a.q.p) + b * a.q.sb + kvh * group * a.q.sh;
  const uint16_t* gb0 = static_cast<const uint16_t*>(a.d_o.p) + b * a.d_o.sb + kvh * group * a.d_o.sh;
  const int64_t line0 = (int64_t(b) * a.heads + kvh * group) * a.q_len;
  auto fetch = [&](int head, int q0, int t) {
    const unsigned at = lds + VB + unsigned(t & 1) * BUF;
    // Formed anew for each tile: kept, its registers would spill, and a
    // reload's wait would also wait for the DMA in flight.
    const int lane = fresh_lane();
    const TileMove<DB, NW> mq(a.q.sl, a.dim, wave, lane), mg(a.d_o.sl, a.dim, wave, lane);
    mq.issue(qb0 + head * a.q.sh + q0 * a.q.sl, q_here - q0, at, wave);
    mg.issue(gb0 + head * a.d_o.sh + q0 * a.d_o.sl, q_here - q0, at + G::TILEB, wave);
    const int64_t line = line0 + int64_t(head) * a.q_len + q0;
    const unsigned off = lane < q_here - q0 ? unsigned(lane) * 4u : kBufNone;
    if (wave == 0) dma4(buffer_at(a.part_lse + line), at + 2 * G::TILEB, off);
    if (wave == 1) dma4(buffer_at(a.delta + line), at + 2 * G::TILEB + kTile * 4, off);
  };
  f32x16_t dk[DB], dv[DB];
#pragma unroll
  for (int db = 0; db < DB; ++db) dk[db] = dv[db] = (f32x16_t)(0.f);
  const float c = a.scale * kLog2e;

  int head = 0, q0 = 0;                 // of the tile worked on
  if (tiles > 0) {
    head = t0 / per_head;
    q0 = begin + t0 % per_head * kTile;
    const TileMove<DB, NW> mv(a.v.sl, a.dim, wave, lane);
#pragma unroll
    for (int i = 0; i < KEYS / kTile; ++i)
      mv.issue(vbase + (key0 + i * kTile) * a.v.sl, k_here - key0 - i * kTile, lds + unsigned(i) * G::TILEB, wave);
    fetch(head, q0, 0);
    load_rows<DB>(kf, kbase + key * a.k.sl, key < k_here, a.dim, half);
  }
  arrived(kf);
  const unsigned char* vh = smem + wave * 32 * G::ROWB;
  for (int t = 0; t < tiles; ++t) {
    wait_vm<0>();
    barrier();
    int next_head = head, next_q0 = q0 + kTile;
    if (next_q0 >= q_here) { next_q0 = begin; ++next_head; }
    if (t + 1 < tiles) fetch(next_head, next_q0, t + 1);
    const unsigned char* qt = smem + VB + (t & 1) * BUF;
    const unsigned char* gt = qt + G::TILEB;
    const float* lt = reinterpret_cast<const float*>(gt + G::TILEB);
    if (q0 + kTile > wave_first && wkey < k_here) {
      // Fragment n of 32 queries: KS row reads of q, KS of do (and of v), 2 DB
      // transposed reads of do, 2 DB of q; AHEAD of them are on their way.
      // The order of a slot's products, reads and arithmetic is fixed: left to
      // itself the compiler waits for each read at once.
      constexpr int KS = G::KS, DB2 = 2 * DB, NF = 2 * KS + 2 * DB2;
      u32x4_t f[AHEAD], fv[AHEAD];
      auto fragment = [&](int qb, int n) {
        const unsigned char* qh = qt + qb * 32 * G::ROWB;
        const unsigned char* gh = gt + qb * 32 * G::ROWB;
        if (n < KS) return rd.rows(qh, n, 0);
        if (n < 2 * KS) return rd.rows(gh, n - KS, 0);
        if (n < 2 * KS + DB2) return rd.cols(gh, (n - 2 * KS) % DB, (n - 2 * KS) / DB);
        return rd.cols(qh, (n - 2 * KS - DB2) % DB, (n - 2 * KS - DB2) / DB);
      };
#pragma unroll
      for (int n = 0; n < AHEAD; ++n) f[n] = fragment(0, n);
#pragma unroll 1
      for (int qb = 0; qb < 2; ++qb) {
        const MUON_LOCAL float* lh = (const MUON_LOCAL float*)(lt + 32 * qb + 4 * half);
        f32x16_t s, dp;
        u32x4_t p[2];
        f32x4_t l[2];
        auto slot_end = [&](int n) {
          const int m = n + AHEAD;
          if (m < NF) f[n % AHEAD] = fragment(qb, m);
          else f[n % AHEAD] = fragment(1, m - NF);      // of the second half (read again there: unused)
          if (m >= KS && m < 2 * KS) fv[n % AHEAD] = rd.rows(vh, m - KS, 0);
          __builtin_amdgcn_sched_barrier(0);
        };
        // Quarter g of the rows: p = exp2(c s - offset), then ds = p (dp - delta)
        auto probs = [&](int g) {
#pragma unroll
          for (int k = 0; k < 4; ++k) s[4 * g + k] = exp2_fast(fmaf(s[4 * g + k], c, -l[g & 1][k]));
          if (g & 1) p[g >> 1] = pack8(s, 8 * (g >> 1));
          if (g + 2 < 4) l[g & 1] = *(const MUON_LOCAL f32x4_t*)(lh + 8 * (g + 2));
        };
        auto grads = [&](int g) {
#pragma unroll
          for (int k = 0; k < 4; ++k) s[4 * g + k] *= dp[4 * g + k] - l[g & 1][k];
          if (g & 1) p[g >> 1] = pack8(s, 8 * (g >> 1));
          if (g + 2 < 4) l[g & 1] = *(const MUON_LOCAL f32x4_t*)(lh + kTile + 8 * (g + 2));
        };
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int n = 0; n < KS; ++n) {
          s = mfma32(f[n % AHEAD], kf[n], n ? s : (f32x16_t)(0.f));
          if (n < 2) l[n] = *(const MUON_LOCAL f32x4_t*)(lh + 8 * n);
          slot_end(n);
        }
        const int qq = q0 + 32 * qb;
        if (qq < wave_all) {
          const int l = fresh_lane(), unseen = first_query(wkey + (l & 31)) - 4 * (l >> 5) - qq;
#pragma unroll
          for (int v = 0; v < 16; ++v)
            if (8 * (v >> 2) + (v & 3) < unseen) s[v] = -INFINITY;
        }
        __builtin_amdgcn_sched_barrier(0);
        // The pieces of arithmetic are spread over the slots of a phase, none
        // in its first (their inputs are the last results of the one before).
#pragma unroll
        for (int n = KS; n < 2 * KS; ++n) {
          dp = mfma32(f[n % AHEAD], fv[n % AHEAD], n > KS ? dp : (f32x16_t)(0.f));
#pragma unroll
          for (int g = 0; g < 4; ++g)
            if (1 + g * (KS - 1) / 4 == n - KS) probs(g);
          if (n == 2 * KS - 1) {
#pragma unroll
            for (int g = 0; g < 2; ++g) l[g] = *(const MUON_LOCAL f32x4_t*)(lh + kTile + 8 * g);
          }
          slot_end(n);
        }
#pragma unroll
        for (int n = 2 * KS; n < 2 * KS + DB2; ++n) {
          const int m = n - 2 * KS;
          dv[m % DB] = mfma32(f[n % AHEAD], p[m / DB], dv[m % DB]);
          // p's first half is overwritten once it has been used, the second
          // in the last slot
          if (m == DB) { grads(0); grads(1); }
          if (m == DB2 - 1) { grads(2); grads(3); }
          slot_end(n);
        }
#pragma unroll
        for (int n = 2 * KS + DB2; n < NF; ++n) {
          const int m = n - 2 * KS - DB2;
          dk[m % DB] = mfma32(f[n % AHEAD], p[m / DB], dk[m % DB]);
          slot_end(n);
        }
      }
    }
    head = next_head;
    q0 = next_q0;
  }
  if (key >= a.k_len) return;
  if (key >= k_here) {      // a key past the length, or that no query sees, has no gradient
#pragma unroll
    for (int db = 0; db < DB; ++db) dk[db] = dv[db] = (f32x16_t)(0.f);
  }
  if (parts > 1) {
    float* o = a.part_kv + (((int64_t(part) * a.batch + b) * a.kv_heads + kvh) * a.k_len + key) * 2 * a.dim;
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int d = 32 * db + 8 * g + 4 * half;
        if (d >= a.dim) continue;
        *as_global(reinterpret_cast<f32x4_t*>(o + d)) =
            f32x4_t{dk[db][4 * g], dk[db][4 * g + 1], dk[db][4 * g + 2], dk[db][4 * g + 3]};
        *as_global(reinterpret_cast<f32x4_t*>(o + a.dim + d)) =
            f32x4_t{dv[db][4 * g], dv[db][4 * g + 1], dv[db][4 * g + 2], dv[db][4 * g + 3]};
      }
    return;
  }
  store_rows<DB>(dk, a.scale, static_cast<uint16_t*>(a.d_k.p) + b * a.d_k.sb + key * a.d_k.sl + kvh * a.d_k.sh, a.dim,
                 half);
  store_rows<DB>(dv, 1.f, static_cast<uint16_t*>(a.d_v.p) + b * a.d_v.sb + key * a.d_v.sl + kvh * a.d_v.sh, a.dim,
                 half);
}

// Adds the parts of dk and dv, eight values per thread.
__global__ __launch_bounds__(256) void attn_dkv_join_kernel(AttnDev a, int64_t n, int64_t stride) {
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i >= n) return;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int p = 0; p < a.parts; ++p) {
    float t[8];
    load_vals<float, 8>(a.part_kv, p * stride + i * 8, t);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] += t[k];
  }
  const int cpr = a.dim / 8;
  const int c = int(i % (2 * cpr));
  const int64_t line = i / (2 * cpr);
  const int key = int(line % a.k_len);
  const int64_t bh = line / a.k_len, b = bh / a.kv_heads, h = bh % a.kv_heads;
  const bool is_v = c >= cpr;
  const HeadsDev& o = is_v ? a.d_v : a.d_k;
  if (!is_v) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] *= a.scale;
  }
  store_vals<uint16_t, 8>(o.p, b * o.sb + key * o.sl + h * o.sh + (is_v ? c - cpr : c) * 8, v);
}

unsigned row_blocks(const AttnDev& a) {
  const int64_t rows = int64_t(a.q_len) * (a.heads / a.kv_heads);
  return unsigned((rows + kRowsWg - 1) / kRowsWg);
}
unsigned key_blocks(const AttnDev& a) { return unsigned((a.k_len + 255) / 256); }

#define BY_DIM(K, ...)                                                                             \
  (a.dim <= 32 ? K<1 __VA_ARGS__> : a.dim <= 64 ? K<2 __VA_ARGS__> : a.dim <= 96 ? K<3 __VA_ARGS__> \
                                                                                 : K<4 __VA_ARGS__>)
#define COMMA ,

int attn_splits(const AttnDev& a, int* split_keys) {
  // At least two workgroups fit on each of 256 CUs.  With fewer than half of that,
  // the keys are divided, in ranges of at least four tiles.
  const int64_t items = int64_t(row_blocks(a)) * a.batch * a.kv_heads;
  const int tiles = (a.k_len + kTile - 1) / kTile;
  int64_t n = 1;
  if (items > 0 && items < 256) {
    n = 512 / items;
    if (n > tiles / 4) n = tiles / 4;
    if (n < 1) n = 1;
  }
  const int per = int((tiles + n - 1) / n);
  *split_keys = per * kTile;
  return tiles == 0 ? 1 : (tiles + per - 1) / per;
}

int attn_parts(const AttnDev& a) {
  // The time of the dk, dv kernel in tiles of one workgroup per CU: whole
  // rounds of workgroups, or under a causal border, where their work differs
  // and the long ones go first, the average and a little of the longest.  A
  // divided block's part costs about as much as six tiles more, to write its
  // sums and read them back.  (8192 keys and queries, 16 heads over 4: the
  // whole backward pass took 1152, 1023, 961, 1005 and 1000 us with 2, 3, 4, 5
  // and 8 parts.)
  const double items = double(key_blocks(a)) * a.batch * a.kv_heads;
  const double tiles = double((a.q_len + kTile - 1) / kTile) * (a.heads / a.kv_heads);
  int best = 1;
  double least = 0;
  for (int p = 1; p <= 16 && (p == 1 || tiles / p >= 4); ++p) {
    const double cost = p > 1 ? 6 : 0, one = tiles / p + cost;
    const double time = a.causal ? std::max(one, items * p * (0.55 * tiles / p + cost) / 256 + 0.1 * one)
                                 : std::ceil(items * p / 256) * one;
    if (p == 1 || time < 0.97 * least) {
      best = p;
      least = time;
    }
  }
  return best;
}

}  // namespace

void attn_plan(AttnDev& a) {
  int keys = 0;
  a.splits = attn_splits(a, &keys);
  a.split_keys = keys;
  a.parts = attn_parts(a);
  a.row_blocks = fast_div(row_blocks(a));
  a.key_blocks = fast_div(key_blocks(a));
  a.by_kv_heads = fast_div(unsigned(a.kv_heads));
  a.by_group = fast_div(unsigned(a.heads / a.kv_heads));
  a.by_splits = fast_div(unsigned(a.splits));
  a.by_parts = fast_div(unsigned(a.parts));
  a.by_bh = fast_div(unsigned(a.batch) * unsigned(a.kv_heads));
}

hipError_t launch_attn_fwd(hipStream_t s, const AttnDev& a) {
  const unsigned blocks = row_blocks(a);
  const unsigned items = blocks * unsigned(a.batch) * unsigned(a.kv_heads) * unsigned(a.splits);
  if (a.splits == 1) {
    auto* k = BY_DIM(attn_fwd_kernel, COMMA false);
    hipLaunchKernelGGL(k, dim3(items), dim3(256), 0, s, a, items);
    return hipGetLastError();
  }
  auto* k = BY_DIM(attn_fwd_kernel, COMMA true);
  hipLaunchKernelGGL(k, dim3(items), dim3(256), 0, s, a, items);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t lines = int64_t(a.batch) * a.heads * a.q_len;
  hipLaunchKernelGGL(attn_join_kernel, dim3(unsigned((lines + 3) / 4)), dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_attn_bwd(hipStream_t s, const AttnDev& a) {
  const unsigned bh = unsigned(a.batch) * unsigned(a.kv_heads);
  if (a.q_len > 0) {
    const unsigned blocks = row_blocks(a), items = blocks * bh;
    auto* k = BY_DIM(attn_dq_kernel, );
    hipLaunchKernelGGL(k, dim3(items), dim3(256), 0, s, a, items);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.k_len > 0) {
    const unsigned blocks = key_blocks(a), items = blocks * bh * unsigned(a.parts);
    auto* k = BY_DIM(attn_dkv_kernel, COMMA 2);
    hipLaunchKernelGGL(k, dim3(items), dim3(512), 0, s, a, items);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.parts == 1) return e;
    const int64_t stride = int64_t(a.batch) * a.kv_heads * a.k_len * 2 * a.dim, n = stride / 8;
    hipLaunchKernelGGL(attn_dkv_join_kernel, dim3(unsigned((n + 255) / 256)), dim3(256), 0, s, a, n, stride);
    return hipGetLastError();
  }
  return hipSuccess;
}

}  // namespace muon
