/*
 * muon_block.h - C ABI of the transformer-block operators for gfx950 that
 * produce the gradients muon_step consumes: the fused residual norm, softmax
 * attention, the gated feed-forward block, linear layers with their epilogue,
 * rotary positions and dropout, each forward and backward.
 *
 * All entries are stateless.  A call validates its arguments on the host,
 * enqueues kernels on the given stream and returns; nothing is allocated,
 * copied or synchronised, so every call may be captured into a HIP graph.
 *
 * Memory and ownership
 *   Tensor pointers are DEVICE pointers owned by the caller and must stay
 *   valid until the stream has passed the call.  Where a call takes a
 *   workspace, its size comes from the matching *_workspace function (a pure
 *   host function of the sizes, 0 possible); the workspace is 256-byte
 *   aligned, its contents mean nothing before or after the call, and calls
 *   that may overlap on the device need one each.  Outputs must not overlap
 *   inputs or each other unless said otherwise.
 *
 * Matrices are muon_tensor (muon.h) with ld >= cols (rows apart by ld
 * values); a tensor that an argument allows to be absent has ptr NULL.
 *
 * Errors
 *   As in muon.h: a status, never an exception or abort, and nothing is
 *   enqueued when a call returns anything but MUON_OK or MUON_E_HIP.
 *   muon_block_last_error() gives the text.  NaN and infinities propagate
 *   as in the formulas, except where a length says that a value is not there
 *   (and, near a causal border, as the attention section says).
 */
#ifndef MUON_BLOCK_H
#define MUON_BLOCK_H

#include "muon.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Text of the last error of a function of this header on this thread. */
const char* muon_block_last_error(void);

/* ---- Residual norm --------------------------------------------------------
 * Ends one sub-block and begins the next, in one pass over the rows:
 *
 *   p = N_post(h) * post_weight
 *   resid_out = resid + alpha * gate_b * p
 *   y = N_pre(resid_out) * pre_weight * (1 + scale_b) + shift_b
 *
 * b = row / group_rows is the row's sample.  N of a row x: RMS,
 * x / sqrt(mean(x^2) + eps); LAYER, (x - mean) / sqrt(var + eps); NONE, x.
 * y is formed from the unrounded fp32 resid_out.  Sums and statistics are
 * fp32.  Absent weights and gate count as 1, absent scale and shift as 0;
 * h absent (with gate and post_weight absent, post_kind NONE) leaves
 * resid_out = resid, which is then not written.  pre_kind NONE with y absent
 * only updates the residual stream. */
typedef enum muon_norm_kind { MUON_NORM_NONE = 0, MUON_NORM_RMS = 1, MUON_NORM_LAYER = 2 } muon_norm_kind;

typedef struct muon_norm_args {
  int64_t rows, cols;     /* 0 <= rows < 2^31; 1 <= cols <= 16384; rows /
                           * group_rows times cols / 64 (up) below 2^31       */
  int64_t group_rows;     /* rows of one sample; divides rows                 */
  int32_t post_kind;      /* muon_norm_kind of h                              */
  int32_t pre_kind;       /* muon_norm_kind of resid_out                      */
  float alpha, eps;       /* residual scale; eps >= 0                         */
  /* rows x cols, F32 or BF16; resid and resid_out share a type, so do h, y */
  muon_tensor resid, h, resid_out, y;
  /* rows / group_rows x cols, F32 or BF16 */
  muon_tensor gate, scale, shift;
  /* 1 x cols, F32 or BF16 */
  muon_tensor post_weight, pre_weight;
  /* rows x 4 fp32, contiguous, 16-byte aligned: mean and 1 / deviation of
   * h's row, then of resid_out's row (0 and 1 where there is no mean / norm) */
  float* stats;
  /* Backward only.  d_resid_out (may be absent: 0) and d_y come in; the
   * others go out and may be absent except d_resid (and d_h where h is
   * there).  Types: d_resid* as resid, d_y and d_h as h, the gradient of a
   * vector as that vector; d_gate, d_scale, d_shift rows / group_rows x cols. */
  muon_tensor d_resid_out, d_y, d_resid, d_h;
  muon_tensor d_gate, d_scale, d_shift, d_post_weight, d_pre_weight;
} muon_norm_args;

muon_status muon_norm_fwd(const muon_norm_args* args, void* hip_stream);
muon_status muon_norm_bwd_workspace(const muon_norm_args* args, size_t* bytes);
/* Reads resid_out, h and stats as the forward call left them (resid, y and
 * shift are not read).  Column sums are added in a fixed order: the same
 * inputs give the same bits. */
muon_status muon_norm_bwd(const muon_norm_args* args, void* workspace, size_t workspace_bytes, void* hip_stream);

/* ---- Attention ------------------------------------------------------------
 * s_ij = scale q_i . k_j over the keys j that query i sees, p = softmax_j(s),
 * o_i = sum_j p_ij v_j, lse_i = log sum_j exp(s_ij).  Query head h reads key
 * head h / (heads / kv_heads).  Key j is seen by query i of sample b when
 * i < q_lens[b], j < k_lens[b] (each q_len / k_len where absent) and, with
 * causal, j <= i + offset.  A query that sees no key has o = 0 and
 * lse = -inf, and no gradient; a key that no query sees has none either.
 * What lies past a length, a key that no query sees and a query that sees no
 * key are never used, so they may hold anything.  Between queries and keys
 * that others do see, the causal border is kept by probabilities of 0: a NaN
 * or infinity in a key or value (backward: also in a query or its d_o) may
 * pass it, to positions less than 128 away from the border.  Scores, softmax
 * and all sums are fp32; probabilities and their gradients are rounded to
 * bf16 as matrix-core operands. */
typedef struct muon_heads {
  void* ptr;              /* BF16 (batch, len, heads, dim), dim contiguous    */
  int64_t stride_batch, stride_len, stride_head;   /* in values, multiples of 8 */
} muon_heads;

typedef struct muon_attn_args {
  int64_t batch, q_len, k_len;    /* >= 0; below 2^24 batch x kv_heads, and
                                   * those x q_len x (heads / kv_heads) / 128
                                   * (up); backward below 2^23 x k_len / 256  */
  int32_t heads, kv_heads;        /* kv_heads divides heads                   */
  int32_t dim;                    /* multiple of 8, 8 .. 128                  */
  int32_t causal;                 /* 0 or 1                                   */
  int64_t offset;                 /* causal border: j <= i + offset           */
  float scale;                    /* finite, above 0                          */
  int32_t reserved;               /* must be 0                                */
  const int32_t* q_lens;          /* batch device integers, 0 .. q_len (values
                                   * outside are taken as the nearer end), or
                                   * NULL                                     */
  const int32_t* k_lens;          /* likewise for keys                        */
  muon_heads q, k, v, o;
  float* lse;                     /* batch x heads x q_len fp32, contiguous   */
  muon_heads d_o, d_q, d_k, d_v;  /* backward only                            */
} muon_attn_args;

muon_status muon_attn_fwd_workspace(const muon_attn_args* args, size_t* bytes);
muon_status muon_attn_fwd(const muon_attn_args* args, void* workspace, size_t workspace_bytes, void* hip_stream);
muon_status muon_attn_bwd_workspace(const muon_attn_args* args, size_t* bytes);
/* Recomputes the probabilities from q, k and lse; reads o and d_o; writes
 * d_q, d_k, d_v whole (zeros past the lengths).  No atomics: the same inputs
 * give the same bits. */
muon_status muon_attn_bwd(const muon_attn_args* args, void* workspace, size_t workspace_bytes, void* hip_stream);

/* ---- Gated feed-forward ---------------------------------------------------
 * g = x w_gate^T, u = x w_up^T, y = (act(g) * u) w_down^T, products with fp32
 * accumulation; act(g) * u is formed in fp32 and rounded to bf16 as the down
 * projection's operand.  gu (rows x 2 hidden: g then u) is what the backward
 * pass reads; absent, it is not written.  The backward pass forms, from the
 * stored g and u, dh = dy w_down, dg = dh u act'(g), du = dh act(g) (rounded
 * to bf16 as operands), dx = dg w_gate + du w_up, and the weights' gradients
 * dg^T x, du^T x, dy^T (act(g) u) in the weights' own layout, F32 or BF16:
 * what muon_step takes. */
typedef enum muon_act { MUON_ACT_SILU = 0, MUON_ACT_GELU_TANH = 1, MUON_ACT_NONE = 2 } muon_act;

typedef struct muon_ffn_args {
  int64_t rows, cols, hidden;     /* rows >= 0; cols, hidden multiples of 8,
                                   * up to 2^20; below 15 x 2^20 tiles of 128
                                   * rows and 64 hidden or 128 other columns  */
  int32_t act;                    /* muon_act, not NONE                       */
  int32_t reserved;               /* must be 0                                */
  muon_tensor x, y;               /* rows x cols, BF16                        */
  muon_tensor w_gate, w_up;       /* hidden x cols, BF16                      */
  muon_tensor w_down;             /* cols x hidden, BF16                      */
  muon_tensor gu;                 /* rows x 2 hidden, BF16                    */
  muon_tensor d_y, d_x;           /* rows x cols, BF16 (backward)             */
  muon_tensor d_w_gate, d_w_up, d_w_down;   /* F32 or BF16, one type          */
} muon_ffn_args;

muon_status muon_ffn_fwd_workspace(const muon_ffn_args* args, size_t* bytes);
muon_status muon_ffn_fwd(const muon_ffn_args* args, void* workspace, size_t workspace_bytes, void* hip_stream);
muon_status muon_ffn_bwd_workspace(const muon_ffn_args* args, size_t* bytes);
muon_status muon_ffn_bwd(const muon_ffn_args* args, void* workspace, size_t workspace_bytes, void* hip_stream);

/* ---- Dropout ----------------------------------------------------------------
 * y = residual + keep x / (1 - p).  The mask is a function of (seed, offset) and
 * of an element's number row * cols + column, whatever the strides, and is
 * never stored: the gradient of x is the same call on d_y without a residual.
 * Element i is dropped when word i % 4 of Philox4x32-10's block with key seed
 * and counter (i / 4, offset), each number's low word first, is below p 2^32
 * (rounded; the probability is off by 2^-33 at most).  A dropped element is 0
 * whatever it held.  p 0 copies; p 1 drops everything. */
typedef struct muon_rng {
  uint64_t seed, offset;
  const uint64_t* state;  /* two device integers that are read in their place
                           * when the call runs (a graph's replays then differ
                           * by what the caller writes there), or NULL        */
} muon_rng;

typedef struct muon_dropout_args {
  int64_t rows, cols;     /* >= 0; rows x cols below 2^56                     */
  double p;               /* 0 .. 1                                           */
  muon_rng rng;
  muon_tensor x;          /* rows x cols, F32 or BF16; row strides up to 2^40 */
  muon_tensor residual;   /* may be absent; else of y's type                  */
  muon_tensor y;          /* F32 or BF16                                      */
} muon_dropout_args;

muon_status muon_dropout(const muon_dropout_args* args, void* hip_stream);

/* ---- Linear -----------------------------------------------------------------
 * z = x weight^T + bias, y = residual + drop(act(z)), products with fp32
 * accumulation and the epilogue in fp32.  drop is muon_dropout's, of a rows x
 * out matrix.  z (BF16) is what the backward pass reads where act is not NONE;
 * absent, it is not written.  The backward pass forms dz = drop(d_y) act'(z),
 * rounded to bf16 as a matrix-core operand (kept in fp32 by small calls, which
 * take no workspace), and d_x = dz weight, d_weight =
 * dz^T x, d_bias = the column sums of dz before its rounding, added in a fixed
 * order: the same inputs give the same bits.  The gradient of the residual is
 * d_y itself. */
typedef struct muon_linear_args {
  int64_t rows, cols, out;        /* rows 0 .. 2^30; cols, out multiples of 8,
                                   * up to 2^20; below 15 x 2^20 tiles of 128 x
                                   * 128 results                              */
  int32_t act;                    /* muon_act                                 */
  int32_t reserved;               /* must be 0                                */
  double p;                       /* dropout: 0 (none) .. 1                   */
  muon_rng rng;                   /* read where p is not 0                    */
  muon_tensor x;                  /* rows x cols, BF16                        */
  muon_tensor weight;             /* out x cols, BF16                         */
  muon_tensor bias;               /* 1 x out, F32 or BF16; may be absent      */
  muon_tensor residual;           /* rows x out, of y's type; may be absent   */
  muon_tensor y;                  /* rows x out, F32 or BF16                  */
  muon_tensor z;                  /* rows x out, BF16; may be absent (forward,
                                   * and backward where act is NONE)          */
  /* Backward only: reads d_y and, as far as they are needed, x, weight and z;
   * writes those of the three gradients that are there. */
  muon_tensor d_y;                /* rows x out, F32 or BF16                  */
  muon_tensor d_x;                /* rows x cols, BF16                        */
  muon_tensor d_weight;           /* out x cols, F32 or BF16                  */
  muon_tensor d_bias;             /* 1 x out, F32 or BF16                     */
} muon_linear_args;

muon_status muon_linear_fwd_workspace(const muon_linear_args* args, size_t* bytes);
muon_status muon_linear_fwd(const muon_linear_args* args, void* workspace, size_t workspace_bytes, void* hip_stream);
muon_status muon_linear_bwd_workspace(const muon_linear_args* args, size_t* bytes);
muon_status muon_linear_bwd(const muon_linear_args* args, void* workspace, size_t workspace_bytes, void* hip_stream);

/* ---- Rotary positions ---------------------------------------------------------
 * Pair p of a head at token i of sample b turns by t = sum_a pos[a] freqs[a][p]:
 *   (u, v) -> scale (u cos t - v sin t, v cos t + u sin t)
 * with (u, v) values (2 p, 2 p + 1) where interleaved, else (p, p + pairs).
 * Values from 2 pairs on are copied.  inverse turns by -t (with the same scale):
 * the gradient.  Angles are formed in fp64, so that far positions keep their
 * digits.  q_out may be q itself (the same pointer and strides), and k_out k;
 * outputs that share a value's place with each other, within themselves or
 * otherwise with q or k are refused (slices of one buffer need not). */
typedef struct muon_rotary_args {
  int64_t batch, len;             /* >= 0; batch x len below 2^31             */
  int32_t heads, kv_heads;        /* of q and of k; kv_heads 0: there is no k.
                                   * Together up to 2^16                      */
  int32_t dim;                    /* even, 2 .. 1024                          */
  int32_t pairs;                  /* 1 .. dim / 2                             */
  int32_t axes;                   /* 1 .. 8; 1 where positions is NULL        */
  int32_t interleaved, inverse;   /* 0 or 1                                   */
  int32_t dtype;                  /* of all four tensors: F32 or BF16         */
  float scale;                    /* finite                                   */
  int32_t reserved;               /* must be 0                                */
  int64_t offset;                 /* position of token 0 without positions    */
  const double* freqs;            /* axes x pairs device values, radians per
                                   * position                                 */
  const int32_t* positions;       /* [sample][len][axes] device integers, or
                                   * NULL: a token's position is its number
                                   * in its sample, plus offset               */
  int64_t positions_batch;        /* integers between samples (0: shared)     */
  muon_heads q, k, q_out, k_out;  /* (batch, len, heads, dim), any strides of
                                   * 0 or more (outputs: no two values in one
                                   * place)                                   */
} muon_rotary_args;

muon_status muon_rotary(const muon_rotary_args* args, void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* MUON_BLOCK_H */
