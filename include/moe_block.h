/*
 * moe_block.h - the part of libmoe's C ABI around the expert layer in a
 * transformer block: the root-mean-square norm with the residual's addition,
 * dropout and an 8-bit output, and dropout by itself. The
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
 * Requirements: rows >= 0; n a positive multiple of 8; rows * n < 2^60; strides
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
 *     u / scales[r]; a row holding a NaN or infinity becomes scales NaN, q 0x7F
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

/* Requirements: 0 <= rows < 2^31; n a positive multiple of 8 (32 for MXFP8), at
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
 *   dweight = sum_r dy[r] v s   (fp32 [n], one fixed order; NULL: not computed) */
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

#ifdef __cplusplus
}
#endif

#endif /* MOE_BLOCK_H */
