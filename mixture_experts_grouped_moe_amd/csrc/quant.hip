// MXFP8 conversion of bf16 activations: E4M3 codes plus one E8M0 scale per
// 32 consecutive K elements of a row, the operand form of the MXFP8 grouped
// GEMM of ROCm/aiter PR #5310 "Add MoE GEMM variants and weight-gradient
// kernel" (Summary; its second review's kernel excerpt decodes an a_scale and
// a b_scale byte per K block). The pages do not give the conversion; this is
// the one of the OCP Microscaling Formats v1.0 specification:
//   X = floor(log2(max |v|)) - 8 over the block (8: largest E4M3 exponent),
//       clamped to [-127, 127]; an all-zero block takes -127; byte X + 127;
//   code = E4M3 nearest to v / 2^X, ties to even, saturating at +-448,
//       sign bit set when v < 0.
// A block holding a NaN or an infinity has no finite shared exponent: it is
// written as a NaN block (scale byte 0xFF, every code 0x7F), so the
// non-finite input never turns into finite codes or leaks into the bytes of
// its neighbours.
//
// HBM-bound: one thread per (row, 32-element block) reads 64 bytes, writes
// 32 code bytes and one scale byte; a wave covers 4 KB of contiguous input.
// The codes come from gfx950's scaled conversion v_cvt_scalef32_pk_fp8_bf16
// (two elements per instruction), which divides by the power of two given
// as an E8M0 exponent and rounds to the nearest E4M3 value, ties to even,
// but turns results past 448 into NaN and keeps the sign of -0 (measured).
// So each element's magnitude is first clamped to 448 * 2^X (bf16 bits are
// ordered like magnitudes: one packed 16-bit min for two elements) and the
// sign of a zero is cleared; the conversion of v / 2^X is then exact up to
// its single rounding, which is the definition's.
#include "common.h"
#include "params.h"
#include "quant_util.h"

namespace moe {

constexpr int kQuantThreads = 256;

__global__ __launch_bounds__(kQuantThreads) void quant_mxfp8_kernel(
    const uint16_t* __restrict__ x, int64_t x_ld, int64_t rows, int32_t kb, uint8_t* __restrict__ q,
    int64_t q_ld, uint8_t* __restrict__ s, int64_t s_ld) {
  const int64_t total = rows * kb;
  for (int64_t i = (int64_t)blockIdx.x * kQuantThreads + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * kQuantThreads) {
    const int64_t row = i / kb;
    const int b = (int)(i % kb);
    const u32x4_t* src = reinterpret_cast<const u32x4_t*>(x + row * x_ld + (int64_t)b * 32);
    u32x4_t v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = src[j];
    u32x4_t out[2];
    const uint32_t byte = mx_quantize_block(v, out);
    u32x4_t* dst = reinterpret_cast<u32x4_t*>(q + row * q_ld + (int64_t)b * 32);
    dst[0] = out[0];
    dst[1] = out[1];
    s[row * s_ld + b] = (uint8_t)byte;
  }
}

hipError_t launch_quant_mxfp8(const uint16_t* x, int64_t x_ld, int64_t rows, int64_t k, uint8_t* q, int64_t q_ld,
                              uint8_t* s, int64_t s_ld, hipStream_t stream) {
  const int64_t total = rows * (k / 32);
  if (total == 0) return hipSuccess;
  const int64_t want = (total + kQuantThreads - 1) / kQuantThreads;
  const uint32_t grid = (uint32_t)(want < 65536 * 8 ? want : 65536 * 8);
  hipLaunchKernelGGL(quant_mxfp8_kernel, dim3(grid), dim3(kQuantThreads), 0, stream, x, x_ld, rows,
                     (int32_t)(k / 32), q, q_ld, s, s_ld);
  return hipGetLastError();
}

}  // namespace moe
