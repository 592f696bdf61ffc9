// moe_combine: y[t] = sum_j w[t, j] * C[t * top_k + j], fp32, j ascending,
// one bf16 rounding. The method's last step (top-k routing weights applied to
// the expert outputs); it runs after the padded rows were computed and writes
// only the rows it is asked for, which is the slice-back of TensorRT-LLM PR
// #15311 "Bound Triton MoE JIT specializations via token-dim bucketing and
// warmup", Description.
//
// HBM-bound: each thread owns 8 output columns of one token (one 16-byte load
// per expert slot, one 16-byte store).
#include "common.h"
#include "params.h"

namespace moe {

constexpr int kCombineThreads = 256;

constexpr int kCombineBatch = 8;  // slots whose loads are issued together
constexpr int64_t kCombineChunk = (int64_t)1 << 26;  // threads per launch at most (a grid holds fewer than 2^32)

// ROUTED: slots whose id lies outside [0, E) are skipped (their rows of C and
// their weights are not read). 8192 tokens of 8 slots, width 7168, an eighth of
// them padding: 183 us, 5.1 TB/s.
template <bool ROUTED>
__global__ __launch_bounds__(kCombineThreads) void combine_kernel(
    const uint16_t* __restrict__ c, int64_t c_ld, const float* __restrict__ w,
    const int32_t* __restrict__ ids, int32_t E, int64_t T, int32_t top_k, int32_t n8, uint16_t* __restrict__ y, int64_t y_ld) {
  const int64_t gid = (int64_t)blockIdx.x * kCombineThreads + threadIdx.x;
  const int64_t t = gid / n8;
  const int col = (int)(gid % n8) * 8;
  if (t >= T) return;
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
  // up to 8 slots' weights and rows are loaded before any is used (one
  // memory round trip instead of one per slot); the sum runs over j in order
  for (int j0 = 0; j0 < top_k; j0 += kCombineBatch) {
    float wj[kCombineBatch];
    u32x4_t v[kCombineBatch];
#pragma unroll
    for (int jj = 0; jj < kCombineBatch; ++jj) {
      const int64_t sl = t * top_k + j0 + jj;
      bool ok = j0 + jj < top_k;
      if (ROUTED) ok = ok && (uint32_t)ids[sl] < (uint32_t)E;
      wj[jj] = ok ? w[sl] : 0.0f;
      v[jj] = ok ? *reinterpret_cast<const u32x4_t*>(c + sl * c_ld + col) : u32x4_t{0, 0, 0, 0};
    }
#pragma unroll
    for (int jj = 0; jj < kCombineBatch; ++jj) {
      if (j0 + jj >= top_k) break;  // (a skipped slot adds 0 * 0)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        acc[2 * q] += wj[jj] * bf16_bits_to_f32(v[jj][q] & 0xffffu);
        acc[2 * q + 1] += wj[jj] * bf16_bits_to_f32(v[jj][q] >> 16);
      }
    }
  }
  u32x4_t o;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    o[q] = f32_to_bf16_bits(acc[2 * q]) | (f32_to_bf16_bits(acc[2 * q + 1]) << 16);
  *reinterpret_cast<u32x4_t*>(y + t * y_ld + col) = o;
}

// Backward: dC[s] = w[s] dy[t] and dw[s] = dy[t] . C[s]. HBM-bound: C is read
// and dC written once. One wave per slot: its lanes take 8 columns at a time,
// the dot product ends with one reduction inside the wave, and the neighbouring
// waves, whose slots are the same token's, find its dy in the cache. (One
// workgroup per token, which reads dy once, took as long for many tokens and
// longer for few: 9.8 us against 5.5 at 333 tokens of 4 slots, width 2880.)
// 8192 tokens of 8 slots, width 7168, an eighth of them padding: 351 us, 5.6 TB/s.
constexpr int kCombineBwdUnroll = 4;

__global__ __launch_bounds__(kCombineThreads) void combine_backward_kernel(
    const uint16_t* __restrict__ dy, int64_t dy_ld, const uint16_t* __restrict__ c, int64_t c_ld,
    const float* __restrict__ w, const int32_t* __restrict__ ids, int32_t E, int64_t s0, int64_t end, int32_t top_k, int32_t n8,
    uint16_t* __restrict__ dc, int64_t dc_ld, float* __restrict__ dw) {
  const int lane = threadIdx.x % 64;
  const int64_t sl = s0 + (int64_t)blockIdx.x * (kCombineThreads / 64) + threadIdx.x / 64;
  if (sl >= end) return;
  const u32x4_t* g = reinterpret_cast<const u32x4_t*>(dy + (int64_t)((uint32_t)sl / (uint32_t)top_k) * dy_ld);
  const u32x4_t* x = reinterpret_cast<const u32x4_t*>(c + sl * c_ld);
  u32x4_t* o = reinterpret_cast<u32x4_t*>(dc + sl * dc_ld);
  if (ids != nullptr && (uint32_t)ids[sl] >= (uint32_t)E) {
    for (int i = lane; i < n8; i += 64) o[i] = u32x4_t{0, 0, 0, 0};
    if (lane == 0) dw[sl] = 0.0f;
    return;
  }
  const float ws = w[sl];
  float dot = 0.0f;
  for (int i0 = lane; i0 < n8; i0 += 64 * kCombineBwdUnroll) {
    u32x4_t gv[kCombineBwdUnroll], xv[kCombineBwdUnroll];
#pragma unroll
    for (int u = 0; u < kCombineBwdUnroll; ++u) {
      const int i = i0 + 64 * u;
      gv[u] = i < n8 ? g[i] : u32x4_t{0, 0, 0, 0};
      xv[u] = i < n8 ? x[i] : u32x4_t{0, 0, 0, 0};
    }
#pragma unroll
    for (int u = 0; u < kCombineBwdUnroll; ++u) {
      u32x4_t r;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float lo = bf16_bits_to_f32(gv[u][q] & 0xffffu), hi = __uint_as_float(gv[u][q] & 0xffff0000u);
        dot += lo * bf16_bits_to_f32(xv[u][q] & 0xffffu);
        dot += hi * __uint_as_float(xv[u][q] & 0xffff0000u);
        const bf16x2_t b = {(__bf16)(ws * lo), (__bf16)(ws * hi)};
        r[q] = __builtin_bit_cast(uint32_t, b);
      }
      if (i0 + 64 * u < n8) o[i0 + 64 * u] = r;
    }
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) dot += __shfl_xor(dot, d, 64);
  if (lane == 0) dw[sl] = dot;
}

hipError_t launch_combine(const uint16_t* c, int64_t c_ld, const float* w, int64_t T,
                          int32_t top_k, int64_t N, uint16_t* y, int64_t y_ld,
                          hipStream_t stream) {
  if (T == 0) return hipSuccess;
  const int32_t n8 = (int32_t)(N / 8);
  const int64_t threads = T * n8;
  const int64_t blocks = (threads + kCombineThreads - 1) / kCombineThreads;
  hipLaunchKernelGGL(combine_kernel<false>, dim3((uint32_t)blocks), dim3(kCombineThreads), 0, stream,
                     c, c_ld, w, (const int32_t*)nullptr, 0, T, top_k, n8, y, y_ld);
  return hipGetLastError();
}

hipError_t launch_combine_routed(const uint16_t* c, int64_t c_ld, const float* w, const int32_t* ids, int64_t T,
                                 int32_t top_k, int32_t E, int64_t N, uint16_t* y, int64_t y_ld,
                                 hipStream_t stream) {
  const int32_t n8 = (int32_t)(N / 8);
  const int64_t per = kCombineChunk / n8 > 0 ? kCombineChunk / n8 : 1;  // tokens per launch
  for (int64_t t = 0; t < T; t += per) {
    const int64_t n = T - t < per ? T - t : per, s = t * top_k;
    const uint32_t blocks = (uint32_t)((n * n8 + kCombineThreads - 1) / kCombineThreads);
    hipLaunchKernelGGL(combine_kernel<true>, dim3(blocks), dim3(kCombineThreads), 0, stream, c + s * c_ld, c_ld, w + s,
                       ids + s, E, n, top_k, n8, y + t * y_ld, y_ld);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

hipError_t launch_combine_backward(const uint16_t* dy, int64_t dy_ld, const uint16_t* c, int64_t c_ld, const float* w,
                                   const int32_t* ids, int64_t T, int32_t top_k, int32_t E, int64_t N, uint16_t* dc,
                                   int64_t dc_ld, float* dw, hipStream_t stream) {
  const int64_t S = T * top_k, per = kCombineChunk / 64;  // slots (waves) per launch
  for (int64_t s0 = 0; s0 < S; s0 += per) {
    const int64_t end = S - s0 < per ? S : s0 + per;
    const uint32_t blocks = (uint32_t)((end - s0 + kCombineThreads / 64 - 1) / (kCombineThreads / 64));
    hipLaunchKernelGGL(combine_backward_kernel, dim3(blocks), dim3(kCombineThreads), 0, stream, dy, dy_ld, c, c_ld, w,
                       ids, E, s0, end, top_k, (int32_t)(N / 8), dc, dc_ld, dw);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

}  // namespace moe
