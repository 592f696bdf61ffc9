/*
 * moe_block.h - the part of libmoe's C ABI around the expert layer in a
 * transformer block and beside its projections: the root-mean-square norm with
 * the residual's addition, dropout and an 8-bit output, dropout by itself, and
 * low-rank adapters of many requests beside a shared projection. The
 * conventions of moe.h hold for every entry point here (caller-owned device
 * memory, host validation before any launch, nothing allocated or
 * synchronized, MOE_* status codes); ranges "overlap" as moe_train.h says.
 *
 * One block around a layer whose GEMMs read MXFP8 activations:
 *   moe_rmsnorm (y for the router's projection, q and scales for the GEMM)
 *   -> moe_route -> moe_align -> moe_grouped_gemm -> ... -> moe_combine_routed
 *   -> the next block's moe_rmsnorm, which adds the layer's output (with
 *      dropout) to the residual stream before it normalises it.
 */
#ifndef MOE_BLOCK_H
#define MOE_BLOCK_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * Dropout. The generator is Philox 4x32 with 10 rounds (Salmon, Moraes, Dror,
 * Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011), a function of a
 * key and a counter, so a mask is computed where it is needed and never
 * stored. With rng (device) uint64 [2] = {seed, offset}, the eight elements
 * i, ..., i + 7 (i a multiple of 8) of a [rows][n] matrix, numbered
 * row * n + column whatever the row stride, take the 128 bits of key = seed
 * and counter = {i / 8, offset} (64 bits each, low words first), element
 * i + j the j-th 16 bits, low half-words first. An element is kept when its
 * 16 bits, as a number, are at least
 *   threshold = round(p * 65536)  (ties to even),
 * i.e. with probability 1 - threshold / 65536, and is then multiplied by
 * 65536 / (65536 - threshold). A dropped element is 0, also where it was NaN
 * or infinite; p = 1 drops every element.
 *
 * The same rng, p and matrix size give the same mask in every entry point and
 * call: the gradient is the call itself on the gradient. rng is read on the
 * device when the kernels run, so a replayed graph draws another mask when the
 * caller has changed it. Masks of different offsets are independent.
 * ---------------------------------------------------------------------- */

/* y[r][i] = bf16( keep(r, i) * x[r][i] / (1 - threshold / 65536) ).
 * x, y (device) bf16 [rows][n], row strides x_ld, y_ld (elements).
 * Requirements: rows >= 0; n a positive multiple of 8, below 2^31; rows * n < 2^60; strides
 * >= n and multiples of 8; x, y 16-byte aligned, rng 8-byte; 0 <= p <= 1; rng
 * may be NULL when threshold is 0. y may be x (the same pointer and stride) and
 * must not overlap it otherwise, nor rng. */
moe_status moe_dropout(const void* x, int64_t x_ld, int64_t rows, int64_t n, float p, const uint64_t* rng, void* y,
                       int64_t y_ld, moe_stream_t stream);

/* The 8-bit form of the norm's output. */
typedef enum {
  MOE_QUANT_NONE = 0,
  MOE_QUANT_MXFP8 = 1,    /* E4M3 codes, an E8M0 byte per 32 columns: what moe_grouped_gemm takes as MOE_E4M3 */
  MOE_QUANT_PER_TOKEN = 2 /* E4M3 codes, an fp32 scale per row: what moe_grouped_gemm_per_token takes */
} moe_quant;

/* ------------------------------------------------------------------------
 * The root-mean-square norm of a residual stream to which a layer's output is
 * added. For every row r, in fp32:
 *   v = residual[r] + drop(x[r])         (residual NULL: 0; p = 0: x[r])
 *   u = v / sqrt(mean_i v[i]^2 + eps) * weight
 *   sum[r] = v     (rounded to residual_dtype; NULL: not stored)
 *   y[r]   = bf16(u)                     (NULL: not stored)
 *   quant MXFP8: the rule of moe_quantize_mxfp8 on u, i.e. per 32 columns
 *     X = floor(log2 max|u|) - 8 clamped to [-127, 127] (-127 for zeros),
 *     scales = X + 127, q = E4M3 nearest to u / 2^X, ties to even, saturated at
 *     448; a block holding a NaN or infinity becomes scales 0xFF, q 0x7F
 *   quant PER_TOKEN: scales[r] = max(max|u| / 448, 2^-126), q = E4M3 nearest to
 *     the fp32 quotient u / scales[r], ties to even; a row holding a NaN or
 *     infinity becomes scales NaN, q 0x7F
 * The statistics and the 8-bit forms come from the unrounded v and u. A row
 * whose sum of squares passes fp32's range gives what that formula gives in
 * fp32. */
typedef struct {
  int64_t rows;
  int64_t n;
  const void* x;           /* (device) bf16 [rows][n] */
  int64_t x_ld;            /* row strides in elements (q_ld, scales_ld too) */
  float p;                 /* dropout of x, see above; 0: none */
  const uint64_t* rng;     /* (device) {seed, offset}; read when threshold > 0 */
  const void* residual;    /* (device) [rows][n] or NULL */
  int64_t residual_ld;
  int32_t residual_dtype;  /* of residual and sum: MOE_BF16 or MOE_FP32 */
  void* sum;               /* (device) [rows][n] or NULL */
  int64_t sum_ld;
  const void* weight;      /* (device) [n] */
  int32_t weight_dtype;    /* MOE_BF16 or MOE_FP32 */
  float eps;
  void* y;                 /* (device) bf16 [rows][n] or NULL */
  int64_t y_ld;
  int32_t quant;           /* moe_quant */
  void* q;                 /* (device) uint8 [rows][n] */
  int64_t q_ld;
  void* scales;            /* (device) uint8 [rows][n/32], or fp32 [rows] (per token; contiguous) */
  int64_t scales_ld;       /* MXFP8 only */
} moe_rmsnorm_args;

/* Requirements: 0 <= rows < 2^31 - 1; n a positive multiple of 8 (32 for MXFP8), at
 * most 16384; y or a quant; eps >= 0 and finite; 0 <= p <= 1. Strides cover a row
 * and are multiples of 8. x, residual, sum, weight, y 16-byte aligned; rng and q
 * 8-byte, per-token scales 4-byte. Strides and pointers of what is
 * not asked for are not read. Outputs must not overlap each other or an input,
 * but sum may be residual (the same pointer and stride), which updates the
 * residual stream in place. No workspace. */
moe_status moe_rmsnorm(const moe_rmsnorm_args* args, moe_stream_t stream);

/* Its gradient, from the sum that the forward pass stored (whose statistics it
 * computes again: the gradient is that of the norm at the stored values). For
 * every row, with g = dy[r] * weight, v = sum[r], s = 1 / sqrt(mean v^2 + eps):
 *   d = dsum[r] + s (g - v s^2 mean_i(g[i] v[i]))    (dsum NULL: 0)
 *   dresidual[r] = d       (sum_dtype; NULL: not stored)
 *   dx[r] = bf16(drop(d))  (NULL: not stored)
 *   dweight = sum_r dy[r] v s   (fp32 [n]; NULL: not computed. A workgroup's rows are
 *   added in 32 bits, their sums in 64, in one fixed order) */
typedef struct {
  int64_t rows;
  int64_t n;
  const void* dy;          /* (device) bf16 [rows][n] */
  int64_t dy_ld;
  const void* dsum;        /* (device) sum_dtype [rows][n] or NULL */
  int64_t dsum_ld;
  const void* sum;         /* (device) sum_dtype [rows][n] */
  int64_t sum_ld;
  int32_t sum_dtype;       /* MOE_BF16 or MOE_FP32: of sum, dsum, dresidual */
  const void* weight;      /* (device) [n] */
  int32_t weight_dtype;
  float eps;
  float p;                 /* dropout of x in the forward pass, with its rng */
  const uint64_t* rng;
  void* dresidual;         /* (device) sum_dtype [rows][n] or NULL */
  int64_t dresidual_ld;
  void* dx;                /* (device) bf16 [rows][n] or NULL */
  int64_t dx_ld;
  float* dweight;          /* (device) fp32 [n] or NULL; rows = 0 writes zeros */
  void* workspace;         /* (device, 16-byte aligned) read with dweight; not kept between calls,
                              and calls that may run at the same time need one each */
  int64_t workspace_bytes; /* >= moe_rmsnorm_backward_workspace_bytes(rows, n) */
} moe_rmsnorm_backward_args;

/* Requirements as above (n a multiple of 8); one of dresidual, dx and dweight at
 * least. Outputs and workspace must not overlap each other or an input, but
 * dresidual may be dsum (the same pointer and stride). */
moe_status moe_rmsnorm_backward(const moe_rmsnorm_backward_args* args, moe_stream_t stream);

/* Bytes of its workspace with dweight; -1 on bad sizes. */
int64_t moe_rmsnorm_backward_workspace_bytes(int64_t rows, int64_t n);

/* ------------------------------------------------------------------------
 * Low-rank adapters beside a shared projection. A "group" is one adapter (A, B):
 * that of a request, or of one expert, or of a request's expert; slots are
 * routed to groups by moe_align over group ids (slots of id -1 have none), and
 * the block list is kept for all projections of the batch. For every slot s in
 * a block of group g, with row = s / x_row_div:
 *   h[s] = A[g] x[row]                            (fp32; stored when h != NULL)
 *   C[s] = bf16( C[s] + scale[g] * B[g] h[s] )    (scale NULL: 1)
 * C is what the shared projection wrote (moe_grouped_gemm, for one). Rows of C
 * and h of slots in no block are left as they were, and nothing that is in them
 * or in rows of x that no block names reaches a result. Products of bf16
 * values are exact, sums fp32; the second product takes h as three bf16 terms
 * (all of fp32's bits), so an infinite value of B gives infinities or NaN. The
 * order of the sums depends on the sizes alone: repeated calls give equal bits.
 *
 * With groups = experts, moe_grouped_gemm's block list serves the adapters too
 * (block_m 8 and 64 are its block sizes). An adapter of each expert for several
 * requests is a group = adapter * experts + expert: 1024 groups at most, so 8 such
 * adapters of 128 experts and 4 of 256; more of them take several lists and calls. */
typedef struct {
  int64_t num_slots;
  int32_t num_groups;
  int32_t rank;
  int64_t k;               /* width of x */
  int64_t n;               /* width of C */
  const void* x;           /* (device) bf16 [(num_slots - 1) / x_row_div + 1][k] */
  int64_t x_ld;            /* strides in elements */
  int32_t x_row_div;
  const void* a;           /* (device) bf16 [num_groups][rank][k] */
  int64_t a_stride_g;
  int64_t a_ld;
  const void* b;           /* (device) bf16 [num_groups][n][rank] */
  int64_t b_stride_g;
  int64_t b_ld;
  const float* scale;      /* (device) fp32 [num_groups] or NULL */
  const int32_t* sorted_slot_ids; /* (device) moe_align's sorted_token_ids, [max_blocks * block_m] */
  const int32_t* group_ids;       /* (device) moe_align's expert_ids, [max_blocks] */
  int32_t block_m;
  int64_t max_blocks;
  void* c;                 /* (device) bf16 [num_slots][n], read and written */
  int64_t c_ld;
  float* h;                /* (device) fp32 [num_slots][rank], contiguous, or NULL */
  void* workspace;         /* (device, 16-byte aligned) not kept between calls; calls that may run
                              at the same time (other streams, graphs replayed side by side) need one each */
  int64_t workspace_bytes; /* >= moe_lora_workspace_bytes(...); where that is 0, workspace may be NULL */
} moe_lora_args;

/* Requirements: 0 <= num_slots <= 2^31 - 2^16; 1 <= num_groups <= 1024; rank a
 * multiple of 8 from 8 to 128; k and n positive multiples of 8, below 2^24;
 * x_row_div >= 1; strides cover their rows and matrices and are multiples of 8;
 * x, a, b, c, h and workspace 16-byte aligned; block_m 8, 16, 32 or 64,
 * max_blocks >= moe_align_max_blocks(num_slots, num_groups, block_m) and
 * max_blocks * block_m < 2^31. A block whose group id lies outside
 * [0, num_groups) and a slot id outside [0, num_slots) are skipped; no slot may
 * stand in the list twice, so num_slots is at most the number that the list was
 * aligned for, which its padding places hold, however many rows c, x and h have
 * behind those. c, h and workspace must not overlap each other or an input. */
moe_status moe_lora(const moe_lora_args* args, moe_stream_t stream);

/* The block size that suits num_slots slots over num_groups groups: 16, or 64
 * from 32 slots a group on. -1 on bad sizes. */
int32_t moe_lora_block_m(int64_t num_slots, int32_t num_groups);

/* Bytes of moe_lora's workspace; -1 on bad sizes. */
int64_t moe_lora_workspace_bytes(int64_t num_slots, int32_t num_groups, int32_t rank, int64_t k, int64_t n,
                                 int32_t block_m, int64_t max_blocks);

/* Its gradients, from dy = the gradient of C after the addition:
 *   dh[s]  = scale[g] * B[g]^T dy[s]
 *   dx[s] += A[g]^T dh[s]                         (bf16, one rounding; dx NULL: not computed)
 *   da[g]  = sum of dh[s] x[s / x_row_div]^T      (fp32 [num_groups][rank][k])
 *   db[g]  = scale[g] * sum of dy[s] h[s]^T       (fp32 [num_groups][n][rank])
 * dx has a row per slot (the shared projection's gradient, to which this adds);
 * where x_row_div > 1, moe_combine_routed adds the rows of a token. dy passes
 * through to the shared projection unchanged. da and db are written for every
 * group, zeros for one without slots; both NULL: not computed (h and x are then
 * not read, but x is checked all the same). The products take dh and h as three
 * bf16 terms (all of fp32's bits). Rows of dx of slots in no block are left as
 * they were. */
typedef struct {
  int64_t num_slots;
  int32_t num_groups;
  int32_t rank;
  int64_t k;
  int64_t n;
  const void* dy;          /* (device) bf16 [num_slots][n] */
  int64_t dy_ld;
  const void* x;           /* as in the forward pass, and so on */
  int64_t x_ld;
  int32_t x_row_div;
  const void* a;
  int64_t a_stride_g;
  int64_t a_ld;
  const void* b;
  int64_t b_stride_g;
  int64_t b_ld;
  const float* scale;
  const int32_t* sorted_slot_ids;
  const int32_t* group_ids;
  int32_t block_m;
  int64_t max_blocks;
  const float* h;          /* (device) fp32 [num_slots][rank] as the forward pass stored it */
  void* dx;                /* (device) bf16 [num_slots][k], read and written, or NULL */
  int64_t dx_ld;
  float* da;               /* (device) fp32, contiguous, or NULL */
  float* db;
  void* workspace;         /* as in the forward pass */
  int64_t workspace_bytes; /* >= moe_lora_backward_workspace_bytes(...) */
} moe_lora_backward_args;

/* Requirements as for moe_lora, and moe_align's order of the block list (groups
 * ascending, each group's blocks together, -1 behind the last); da and db both
 * or neither, and one of dx and the two at least; da and db 16-byte aligned.
 * dx, da, db and workspace must not overlap each other or an input. */
moe_status moe_lora_backward(const moe_lora_backward_args* args, moe_stream_t stream);

/* Bytes of its workspace; -1 on bad sizes. */
int64_t moe_lora_backward_workspace_bytes(int64_t num_slots, int32_t num_groups, int32_t rank, int64_t k, int64_t n,
                                          int32_t block_m, int64_t max_blocks);

#ifdef __cplusplus
}
#endif

#endif /* MOE_BLOCK_H */
