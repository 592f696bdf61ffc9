// Building blocks of the low-rank adapter kernels (lora.hip, lora_grad.hip).
#pragma once

#include "common.h"
#include "params.h"

namespace moe {

constexpr int kLoraThreads = 256;  // four waves
constexpr int kLoraCUs = 256;

typedef __bf16 lora_bf16x8 __attribute__((ext_vector_type(8)));

// 16 bytes as 8 bf16 of an MFMA operand.
__device__ __forceinline__ lora_bf16x8 lora_frag(u32x4_t v) { return __builtin_bit_cast(lora_bf16x8, v); }

// D[16 x 16] += A[16 x 32] B[32 x 16]: lane l gives row (of A) or column (of B)
// l % 16 at 8 consecutive k from 8 (l / 16), and holds column l % 16, rows
// 4 (l / 16) .. + 3 of D.
__device__ __forceinline__ f32x4_t lora_mfma(u32x4_t a, u32x4_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(lora_frag(a), lora_frag(b), c, 0, 0, 0);
}

// Two floats as bf16 in one dword, rounded to nearest even.
__device__ __forceinline__ uint32_t lora_pack(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}

// f = t[0] + t[1] + t[2] for two floats, the terms bf16 pairs, each the upper half
// of what the ones before it leave: 8 of a float's 24 bits at a time, so that all
// are there (to what bf16's smallest holds), and none passes bf16's range. An
// infinite f is the first term alone. (Two terms lose the products' last bits,
// which show where they cancel what they are added to.)
__device__ __forceinline__ void lora_split(float f0, float f1, uint32_t (&t)[3]) {
  uint32_t a = __float_as_uint(f0), b = __float_as_uint(f1);
  t[0] = __builtin_amdgcn_perm(b, a, 0x07060302u);
  f0 = fabsf(f0) == INFINITY ? 0.0f : f0 - __uint_as_float(a & 0xffff0000u);
  f1 = fabsf(f1) == INFINITY ? 0.0f : f1 - __uint_as_float(b & 0xffff0000u);
  a = __float_as_uint(f0);
  b = __float_as_uint(f1);
  t[1] = __builtin_amdgcn_perm(b, a, 0x07060302u);
  f0 -= __uint_as_float(a & 0xffff0000u);
  f1 -= __uint_as_float(b & 0xffff0000u);
  t[2] = __builtin_amdgcn_perm(__float_as_uint(f1), __float_as_uint(f0), 0x07060302u);
}

// floor(s / d) for s < 2^31 (lora_set_division).
__device__ __forceinline__ uint32_t lora_div(uint32_t s, uint32_t magic, int32_t shift) {
  return (uint32_t)(((uint64_t)s * magic) >> shift);
}

// The parts of four ranks of a place, added in order.
__device__ __forceinline__ f32x4_t lora_sum_parts(const float* at, int64_t step, int parts) {
  f32x4_t h = {0, 0, 0, 0};
  int k = 0;
  for (; k + 4 <= parts; k += 4, at += 4 * step) {
    f32x4_t v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const f32x4_t*>(at + j * step);
    h = (((h + v[0]) + v[1]) + v[2]) + v[3];
  }
  for (; k < parts; ++k, at += step) h += *reinterpret_cast<const f32x4_t*>(at);
  return h;
}

// Rank r in the kernels: padded to 8, 16, 32, 64 or 128.
template <class F>
inline hipError_t lora_rank(int r, F f) {
  if (r <= 8) return f(std::integral_constant<int, 1>{});
  if (r <= 16) return f(std::integral_constant<int, 2>{});
  if (r <= 32) return f(std::integral_constant<int, 4>{});
  if (r <= 64) return f(std::integral_constant<int, 8>{});
  return f(std::integral_constant<int, 16>{});
}

}  // namespace moe
