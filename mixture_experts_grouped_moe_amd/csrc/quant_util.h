// The MXFP8 conversion of a 32-element block of bf16 values, shared by the
// quantizer (quant.hip) and the activation with a checkpoint (act.hip).
#pragma once

#include <type_traits>

#include "common.h"

namespace moe {

typedef short q_v2s __attribute__((ext_vector_type(2)));
typedef __bf16 q_v2bf __attribute__((ext_vector_type(2)));
typedef unsigned short q_v2u16 __attribute__((ext_vector_type(2)));

// Two bf16 elements (bits of one dword) -> the dword with their magnitudes
// clamped to `lim2` (448 * 2^X in both halves) and the sign of a zero
// element cleared. Each half's magnitude plus 0x7FFF has bit 15 set exactly
// when the magnitude is non-zero, and never carries into the other half.
__device__ __forceinline__ uint32_t clamp_pair(uint32_t d, uint32_t lim2) {
  const uint32_t mag = d & 0x7FFF7FFFu;
  const uint32_t sgn = d & 0x80008000u & (mag + 0x7FFF7FFFu);
  const q_v2u16 m = __builtin_elementwise_min(__builtin_bit_cast(q_v2u16, mag), __builtin_bit_cast(q_v2u16, lim2));
  return __builtin_bit_cast(uint32_t, m) | sgn;
}

// The 32 bf16 elements of v (four 16-byte pieces) -> their E4M3 codes in out
// and the block's E8M0 scale byte as the result. A block holding a NaN or an
// infinity becomes a NaN block (byte 0xFF, every code 0x7F).
__device__ __forceinline__ uint32_t mx_quantize_block(const u32x4_t (&v)[4], u32x4_t (&out)[2]) {
  // block maximum of |v| on the bf16 bits (order of magnitudes = order of bits)
  uint32_t amax = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      amax = max(amax, v[j][w] & 0x7FFFu);
      amax = max(amax, (v[j][w] >> 16) & 0x7FFFu);
    }
  if (amax >= 0x7F80u) {  // exponent field all ones: a NaN or an infinity in the block
    const uint32_t nan4 = 0x7F7F7F7Fu;
    out[0] = u32x4_t{nan4, nan4, nan4, nan4};
    out[1] = out[0];
    return 0xFFu;
  }
  // floor(log2(max)) from the exponent field; a zero or subnormal maximum
  // (below 2^-126) gives X below -127, so the clamp decides
  const int e = (int)(amax >> 7);
  const int X = e == 0 ? -127 : min(max(e - 127 - 8, -127), 127);
  // the conversion's scale operand: E8M0 byte X + 127 in the exponent
  // field (byte 0 is 2^-127); X <= 119 for finite inputs, so 448 * 2^X
  // (bf16 exponent 135 + X, mantissa 0x60) is a finite bf16
  const float scale = __uint_as_float((uint32_t)(X + 127) << 23);
  const uint32_t lim = ((uint32_t)(135 + X) << 7) | 0x60u;
  const uint32_t lim2 = lim | (lim << 16);
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int w = 0; w < 4; w += 2) {
      // elements 8j + 2w .. 8j + 2w + 3 -> the four bytes of dword 2j + w/2
      const uint32_t lo = clamp_pair(v[j][w], lim2), hi = clamp_pair(v[j][w + 1], lim2);
      q_v2s r = {0, 0};
      r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(q_v2bf, lo), scale, false);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(q_v2bf, hi), scale, true);
      out[j / 2][2 * (j % 2) + w / 2] = __builtin_bit_cast(uint32_t, r);
    }
  return (uint32_t)(X + 127);
}

// The same for a block spread over four neighbouring lanes (a lane quad, all
// active), 8 elements each: v -> this lane's 8 codes in out; the result, the
// block's scale byte, is the same in the four.
__device__ __forceinline__ uint32_t mx_quantize_quarter(const u32x4_t v, u32x2_t& out) {
  auto mag = [](uint32_t d) { return __builtin_bit_cast(q_v2u16, d & 0x7FFF7FFFu); };
  q_v2u16 m = __builtin_elementwise_max(__builtin_elementwise_max(mag(v[0]), mag(v[1])),
                                        __builtin_elementwise_max(mag(v[2]), mag(v[3])));
  auto other = [&](auto ctrl) {
    const int x = __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, m), decltype(ctrl)::value, 0xF, 0xF, true);
    m = __builtin_elementwise_max(m, __builtin_bit_cast(q_v2u16, x));
  };
  other(std::integral_constant<int, 0xB1>{});  // lane ^ 1
  other(std::integral_constant<int, 0x4E>{});  // lane ^ 2
  const uint32_t amax = max((uint32_t)m[0], (uint32_t)m[1]);
  const int e = (int)(amax >> 7);
  const int X = e == 0 ? -127 : max(e - 127 - 8, -127);  // (255 - 135 < 127)
  const float scale = __uint_as_float((uint32_t)(X + 127) << 23);
  const uint32_t lim = ((uint32_t)(135 + X) << 7) | 0x60u;
  const uint32_t lim2 = lim | (lim << 16);
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const uint32_t lo = clamp_pair(v[2 * w], lim2), hi = clamp_pair(v[2 * w + 1], lim2);
    q_v2s r = {0, 0};
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(q_v2bf, lo), scale, false);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(q_v2bf, hi), scale, true);
    out[w] = __builtin_bit_cast(uint32_t, r);
  }
  const bool bad = amax >= 0x7F80u;  // a NaN or an infinity in the block
  out[0] = bad ? 0x7F7F7F7Fu : out[0];
  out[1] = bad ? 0x7F7F7F7Fu : out[1];
  return bad ? 0xFFu : (uint32_t)(X + 127);
}

}  // namespace moe
