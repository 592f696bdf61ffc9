// moe_act_mxfp8 and moe_act_mxfp8_backward: the expert activation between the
// two grouped GEMMs of a training step, which keeps its input for the
// backward pass as MXFP8 (E4M3 codes, one E8M0 scale per 32), and its
// gradient from that checkpoint.
//
// HBM-bound: one thread per 32-element block (SwiGLU: per gate block and the
// up block half a row further on) reads each input and writes each output
// once. Products and the sigmoid are fp32; h and dpre are rounded once to
// bf16. The checkpoint's bits are those of moe_quantize_mxfp8.
#include "common.h"
#include "params.h"
#include "quant_util.h"

namespace moe {

constexpr int kActThreads = 256;

struct ActBlock {
  u32x4_t v[4];  // 32 bf16
  __device__ __forceinline__ void load(const uint16_t* src) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = reinterpret_cast<const u32x4_t*>(src)[j];
  }
  __device__ __forceinline__ void store(uint16_t* dst) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) reinterpret_cast<u32x4_t*>(dst)[j] = v[j];
  }
  __device__ __forceinline__ float lo(int j, int w) const { return bf16_bits_to_f32(v[j][w] & 0xffffu); }
  __device__ __forceinline__ float hi(int j, int w) const { return bf16_bits_to_f32(v[j][w] >> 16); }
  __device__ __forceinline__ void set(int j, int w, float a, float b) {
    v[j][w] = f32_to_bf16_bits(a) | (f32_to_bf16_bits(b) << 16);
  }
  // the MXFP8 codes and scale byte of the block
  __device__ __forceinline__ void checkpoint(uint8_t* q, uint8_t* s) const {
    u32x4_t out[2];
    const uint32_t byte = mx_quantize_block(v, out);
    reinterpret_cast<u32x4_t*>(q)[0] = out[0];
    reinterpret_cast<u32x4_t*>(q)[1] = out[1];
    *s = (uint8_t)byte;
  }
  // the bf16 values that codes and a scale byte stand for
  __device__ __forceinline__ void decode(const uint8_t* q, const uint8_t* s) {
    const float scale = e8m0_as_scale(*s);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const u32x4_t c = reinterpret_cast<const u32x4_t*>(q)[j];
      const bf16x8_t a = dequant_e4m3x8(c[0], c[1], scale), b = dequant_e4m3x8(c[2], c[3], scale);
      __builtin_memcpy(&v[2 * j], &a, 16);
      __builtin_memcpy(&v[2 * j + 1], &b, 16);
    }
  }
};

template <bool SWIGLU>
__global__ __launch_bounds__(kActThreads) void act_kernel(ActParams p) {
  const int32_t nb = p.n / 32 / (SWIGLU ? 2 : 1);  // blocks (SwiGLU: pairs of blocks) per row
  const int64_t total = p.rows * nb;
  for (int64_t i = (int64_t)blockIdx.x * kActThreads + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * kActThreads) {
    const int64_t row = i / nb;
    const int b = (int)(i % nb);
    ActBlock g, u, h;
    g.load(p.pre + row * p.pre_ld + b * 32);
    if (SWIGLU) u.load(p.pre + row * p.pre_ld + p.n / 2 + b * 32);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int w = 0; w < 4; ++w)
        if (SWIGLU)
          h.set(j, w, silu_f32(g.lo(j, w)) * u.lo(j, w), silu_f32(g.hi(j, w)) * u.hi(j, w));
        else
          h.set(j, w, relu2_f32(g.lo(j, w)), relu2_f32(g.hi(j, w)));
    h.store(p.h + row * p.h_ld + b * 32);
    g.checkpoint(p.q + row * p.q_ld + b * 32, p.s + row * p.s_ld + b);
    if (SWIGLU) u.checkpoint(p.q + row * p.q_ld + p.n / 2 + b * 32, p.s + row * p.s_ld + nb + b);
  }
}

struct ActGrad {
  float h, dg, du;
};
__device__ __forceinline__ ActGrad swiglu_grad(float g, float u, float dh) {
  const float s = 1.0f / (1.0f + __expf(-g));
  const float gs = g * s;
  return {gs * u, dh * (u * (s * (1.0f + g * (1.0f - s)))), dh * gs};
}
__device__ __forceinline__ ActGrad relu2_grad(float v, float dh) {
  return {relu2_f32(v), v > 0.0f ? 2.0f * v * dh : 0.0f, 0.0f};
}

template <bool SWIGLU>
__global__ __launch_bounds__(kActThreads) void act_backward_kernel(ActParams p) {
  const int32_t nb = p.n / 32 / (SWIGLU ? 2 : 1);
  const int64_t total = p.rows * nb;
  for (int64_t i = (int64_t)blockIdx.x * kActThreads + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * kActThreads) {
    const int64_t row = i / nb;
    const int b = (int)(i % nb);
    ActBlock g, u, dh, h;
    g.decode(p.q + row * p.q_ld + b * 32, p.s + row * p.s_ld + b);
    if (SWIGLU) u.decode(p.q + row * p.q_ld + p.n / 2 + b * 32, p.s + row * p.s_ld + nb + b);
    dh.load(p.dh + row * p.dh_ld + b * 32);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float d0 = dh.lo(j, w), d1 = dh.hi(j, w);
        const ActGrad a = SWIGLU ? swiglu_grad(g.lo(j, w), u.lo(j, w), d0) : relu2_grad(g.lo(j, w), d0);
        const ActGrad c = SWIGLU ? swiglu_grad(g.hi(j, w), u.hi(j, w), d1) : relu2_grad(g.hi(j, w), d1);
        h.set(j, w, a.h, c.h);
        g.set(j, w, a.dg, c.dg);
        if (SWIGLU) u.set(j, w, a.du, c.du);
      }
    if (p.h != nullptr) h.store(p.h + row * p.h_ld + b * 32);
    g.store(p.dpre + row * p.dpre_ld + b * 32);
    if (SWIGLU) u.store(p.dpre + row * p.dpre_ld + p.n / 2 + b * 32);
  }
}

static uint32_t act_grid(const ActParams& p, bool swiglu) {
  const int64_t total = p.rows * (p.n / 32 / (swiglu ? 2 : 1));
  const int64_t want = (total + kActThreads - 1) / kActThreads;
  return (uint32_t)(want < 65536 * 8 ? want : 65536 * 8);
}

hipError_t launch_act(const ActParams& p, bool swiglu, hipStream_t stream) {
  const uint32_t grid = act_grid(p, swiglu);
  if (grid == 0) return hipSuccess;
  if (swiglu)
    hipLaunchKernelGGL(act_kernel<true>, dim3(grid), dim3(kActThreads), 0, stream, p);
  else
    hipLaunchKernelGGL(act_kernel<false>, dim3(grid), dim3(kActThreads), 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_act_backward(const ActParams& p, bool swiglu, hipStream_t stream) {
  const uint32_t grid = act_grid(p, swiglu);
  if (grid == 0) return hipSuccess;
  if (swiglu)
    hipLaunchKernelGGL(act_backward_kernel<true>, dim3(grid), dim3(kActThreads), 0, stream, p);
  else
    hipLaunchKernelGGL(act_backward_kernel<false>, dim3(grid), dim3(kActThreads), 0, stream, p);
  return hipGetLastError();
}

}  // namespace moe
