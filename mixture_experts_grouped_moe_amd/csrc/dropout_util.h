// The dropout generator, shared by dropout.hip and norm.hip: Philox 4x32 with
// 10 rounds (Salmon, Moraes, Dror, Shaw, 2011), the mask of 8 elements at a
// time, and the host's reading of the probability.
#pragma once

#include <cmath>

#include "common.h"

namespace moe {

// 128 random bits of key `seed` at counter {index, offset}. A round is two
// 32 x 32 -> 64 bit products; the key's steps are scalar work. 10 rounds are
// about 20 wide multiplies per 8 elements, less time than the 32 bytes that
// they move.
__device__ __forceinline__ u32x4_t philox(uint64_t seed, uint64_t offset, uint64_t index) {
  uint32_t c0 = (uint32_t)index, c1 = (uint32_t)(index >> 32), c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return u32x4_t{c0, c1, c2, c3};
}

// What a kernel needs of a dropout: kept where the 16 bits reach `threshold`.
struct Dropout {
  const uint64_t* rng;  // {seed, offset}, on the device
  uint32_t threshold;   // 0 .. 65536
  float scale;          // 65536 / (65536 - threshold)
};

inline Dropout make_dropout(float p, const uint64_t* rng) {
  const uint32_t t = (uint32_t)std::nearbyint((double)p * 65536.0);
  return {rng, t, t < 65536 ? (float)(65536.0 / (65536 - t)) : 0.0f};
}

// f -> kept values times the scale, others 0 (a selection: NaN and infinities
// are dropped too).
__device__ __forceinline__ void drop8(const Dropout& d, uint64_t seed, uint64_t offset, uint64_t piece,
                                      float (&f)[8]) {
  const u32x4_t w = philox(seed, offset, piece);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = (w[j] & 0xffffu) >= d.threshold ? f[2 * j] * d.scale : 0.0f;
    f[2 * j + 1] = (w[j] >> 16) >= d.threshold ? f[2 * j + 1] * d.scale : 0.0f;
  }
}

// 8 bf16 as floats and back (nearest even).
__device__ __forceinline__ void unpack8(const u32x4_t v, float (&f)[8]) {
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    f[2 * w] = __uint_as_float(v[w] << 16);
    f[2 * w + 1] = __uint_as_float(v[w] & 0xffff0000u);
  }
}
__device__ __forceinline__ u32x4_t pack8(const float (&f)[8]) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  u32x4_t v;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const bf16x2 b = {(__bf16)f[2 * w], (__bf16)f[2 * w + 1]};
    v[w] = __builtin_bit_cast(uint32_t, b);
  }
  return v;
}

}  // namespace moe
