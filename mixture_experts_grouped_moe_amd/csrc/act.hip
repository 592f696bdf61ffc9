// moe_act_mxfp8 and moe_act_mxfp8_backward: the expert activation between the
// two grouped GEMMs of a training step, which keeps its input for the
// backward pass as MXFP8 (E4M3 codes, one E8M0 scale per 32), and its
// gradient from that checkpoint.
//
// HBM-bound: each input is read and each output written once. A thread takes
// 8 columns (SwiGLU: 8 of the gate and the 8 of up half a row further on), so
// that a wave's accesses are contiguous, 16 bytes of bf16 and 8 bytes of codes
// a lane, and small calls have four times the waves that one thread per
// 32-element block gave; the four lanes of a block share its maximum by two
// lane exchanges. SwiGLU over 32768 x 5760: 132 us (one thread per block 157), its
// gradient 165 us (230), 5.8 and 5.9 TB/s, where a large copy reaches 4.9 and a
// fill 6.8. Products and the sigmoid are fp32; h and dpre are rounded
// once to bf16. The checkpoint's bits are those of moe_quantize_mxfp8.
#include "common.h"
#include "params.h"
#include "quant_util.h"

namespace moe {

constexpr int kActThreads = 256;
constexpr int64_t kActMaxUnits = (int64_t)1 << 30;  // 8-column pieces per launch: indices and the row division fit 31 bits

typedef float act_f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 act_bf16x2 __attribute__((ext_vector_type(2)));

// 8 bf16 as floats and back (nearest even).
__device__ __forceinline__ void act_unpack(const u32x4_t v, float (&f)[8]) {
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    f[2 * w] = bf16_bits_to_f32(v[w] & 0xffffu);
    f[2 * w + 1] = __uint_as_float(v[w] & 0xffff0000u);
  }
}
__device__ __forceinline__ u32x4_t act_pack(const float (&f)[8]) {
  u32x4_t v;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const act_bf16x2 b = {(__bf16)f[2 * w], (__bf16)f[2 * w + 1]};
    v[w] = __builtin_bit_cast(uint32_t, b);
  }
  return v;
}
// 8 codes under one scale, exact in fp32.
__device__ __forceinline__ void act_decode(const u32x2_t q, uint32_t byte, float (&f)[8]) {
  const float s = e8m0_as_scale(byte);
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const act_f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q[w], s, false);
    const act_f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q[w], s, true);
    f[4 * w] = a[0];
    f[4 * w + 1] = a[1];
    f[4 * w + 2] = b[0];
    f[4 * w + 3] = b[1];
  }
}
// (the hardware's exponential and reciprocal, 1 ulp each: far below the bf16
// that h and dpre are rounded to)
__device__ __forceinline__ float act_sigmoid(float z) { return __builtin_amdgcn_rcpf(1.0f + __expf(-z)); }

// floor(i / d) for i < 2^31 by a multiply-high (see wgrad.hip's launch).
__device__ __forceinline__ uint32_t act_row(uint32_t i, uint32_t magic, int shift) {
  return (uint32_t)(((uint64_t)i * magic) >> shift);
}

template <bool SWIGLU>
__global__ __launch_bounds__(kActThreads) void act_kernel(ActParams p) {
  const uint32_t i = blockIdx.x * kActThreads + threadIdx.x;
  if (i >= p.units) return;  // (whole blocks of four lanes)
  const uint32_t r = act_row(i, p.magic, p.shift);
  const uint32_t col = (i - r * p.row_units) * 8;
  const int64_t row = p.row0 + r;
  const int half = p.n / 2;
  const uint16_t* pre = p.pre + row * p.pre_ld + col;
  uint8_t* q = p.q + row * p.q_ld + col;
  uint8_t* s = p.s + row * p.s_ld + col / 32;
  const u32x4_t gv = *reinterpret_cast<const u32x4_t*>(pre);
  float g[8], h[8];
  act_unpack(gv, g);
  if constexpr (SWIGLU) {
    const u32x4_t uv = *reinterpret_cast<const u32x4_t*>(pre + half);
    float u[8];
    act_unpack(uv, u);
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = g[j] * act_sigmoid(g[j]) * u[j];
    u32x2_t c;
    const uint32_t b = mx_quantize_quarter(uv, c);
    *reinterpret_cast<u32x2_t*>(q + half) = c;
    if (threadIdx.x % 4 == 0) s[half / 32] = (uint8_t)b;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = relu2_f32(g[j]);
  }
  *reinterpret_cast<u32x4_t*>(p.h + row * p.h_ld + col) = act_pack(h);
  u32x2_t c;
  const uint32_t b = mx_quantize_quarter(gv, c);
  *reinterpret_cast<u32x2_t*>(q) = c;
  if (threadIdx.x % 4 == 0) *s = (uint8_t)b;
}

template <bool SWIGLU>
__global__ __launch_bounds__(kActThreads) void act_backward_kernel(ActParams p) {
  const uint32_t i = blockIdx.x * kActThreads + threadIdx.x;
  if (i >= p.units) return;
  const uint32_t r = act_row(i, p.magic, p.shift);
  const uint32_t col = (i - r * p.row_units) * 8;
  const int64_t row = p.row0 + r;
  const int half = p.n / 2;
  const uint8_t* q = p.q + row * p.q_ld + col;
  const uint8_t* s = p.s + row * p.s_ld + col / 32;
  uint16_t* dpre = p.dpre + row * p.dpre_ld + col;
  float g[8], dh[8], h[8];
  const u32x2_t gq = *reinterpret_cast<const u32x2_t*>(q);
  const u32x4_t dv = *reinterpret_cast<const u32x4_t*>(p.dh + row * p.dh_ld + col);
  act_decode(gq, *s, g);
  act_unpack(dv, dh);
  if constexpr (SWIGLU) {
    float u[8];
    act_decode(*reinterpret_cast<const u32x2_t*>(q + half), s[half / 32], u);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float sg = act_sigmoid(g[j]);
      const float gs = g[j] * sg;
      h[j] = gs * u[j];
      const float dg = dh[j] * (u[j] * (sg * (1.0f + g[j] * (1.0f - sg))));
      u[j] = dh[j] * gs;
      g[j] = dg;
    }
    *reinterpret_cast<u32x4_t*>(dpre + half) = act_pack(u);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      h[j] = relu2_f32(g[j]);
      g[j] = g[j] > 0.0f ? 2.0f * (g[j] * dh[j]) : 0.0f;  // (2 g may overflow where the product does not)
    }
  }
  *reinterpret_cast<u32x4_t*>(dpre) = act_pack(g);
  if (p.h != nullptr) *reinterpret_cast<u32x4_t*>(p.h + row * p.h_ld + col) = act_pack(h);
}

// Launches `kernel` over all rows, as many rows at a time as kActMaxUnits
// pieces hold.
template <class F>
static hipError_t act_launch(ActParams p, bool swiglu, F kernel, hipStream_t stream) {
  p.row_units = (uint32_t)(p.n / (swiglu ? 16 : 8));
  // floor(i / d) = (i m) >> (31 + l) with l = ceil(log2 d), m = ceil(2^(31+l) / d)
  // for i < 2^31 (Granlund and Montgomery, 1994, Theorem 4.2)
  int l = 0;
  while (((uint32_t)1 << l) < p.row_units) ++l;
  p.magic = (uint32_t)((((uint64_t)1 << (31 + l)) + p.row_units - 1) / p.row_units);
  p.shift = 31 + l;
  const int64_t per = kActMaxUnits / p.row_units;  // at least 3: row_units < 2^28
  for (p.row0 = 0; p.row0 < p.rows; p.row0 += per) {
    const int64_t rows = p.rows - p.row0 < per ? p.rows - p.row0 : per;
    p.units = (uint32_t)(rows * p.row_units);
    hipLaunchKernelGGL(kernel, dim3((p.units + kActThreads - 1) / kActThreads), dim3(kActThreads), 0, stream, p);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

hipError_t launch_act(const ActParams& p, bool swiglu, hipStream_t stream) {
  return swiglu ? act_launch(p, true, act_kernel<true>, stream) : act_launch(p, false, act_kernel<false>, stream);
}

hipError_t launch_act_backward(const ActParams& p, bool swiglu, hipStream_t stream) {
  return swiglu ? act_launch(p, true, act_backward_kernel<true>, stream)
                : act_launch(p, false, act_backward_kernel<false>, stream);
}

}  // namespace moe
