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

// ROUTED: slots whose id lies outside [0, E) are skipped (their rows of C and
// their weights are not read).
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

// Backward: dC[s] = w[s] dy[t] and dw[s] = dy[t] . C[s]. One workgroup per
// token; each thread takes 8 columns at a time of dy and of up to 8 slots'
// rows, so dy is read once per 8 slots.
__global__ __launch_bounds__(kCombineThreads) void combine_backward_kernel(
    const uint16_t* __restrict__ dy, int64_t dy_ld, const uint16_t* __restrict__ c, int64_t c_ld,
    const float* __restrict__ w, const int32_t* __restrict__ ids, int32_t E, int32_t top_k, int32_t n8,
    uint16_t* __restrict__ dc, int64_t dc_ld, float* __restrict__ dw) {
  __shared__ float s_dot[kCombineThreads / 64][kCombineBatch];
  const int64_t t = blockIdx.x;
  for (int j0 = 0; j0 < top_k; j0 += kCombineBatch) {
    float wj[kCombineBatch], dot[kCombineBatch];
    bool ok[kCombineBatch];
#pragma unroll
    for (int jj = 0; jj < kCombineBatch; ++jj) {
      const int64_t sl = t * top_k + j0 + jj;
      ok[jj] = j0 + jj < top_k && (ids == nullptr || (uint32_t)ids[sl] < (uint32_t)E);
      wj[jj] = ok[jj] ? w[sl] : 0.0f;
      dot[jj] = 0.0f;
    }
    for (int i = threadIdx.x; i < n8; i += kCombineThreads) {
      const u32x4_t g = *reinterpret_cast<const u32x4_t*>(dy + t * dy_ld + i * 8);
#pragma unroll
      for (int jj = 0; jj < kCombineBatch; ++jj) {
        if (j0 + jj >= top_k) break;
        const int64_t sl = t * top_k + j0 + jj;
        u32x4_t o = {0, 0, 0, 0};
        if (ok[jj]) {
          const u32x4_t v = *reinterpret_cast<const u32x4_t*>(c + sl * c_ld + i * 8);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float lo = bf16_bits_to_f32(g[q] & 0xffffu), hi = bf16_bits_to_f32(g[q] >> 16);
            dot[jj] += lo * bf16_bits_to_f32(v[q] & 0xffffu);
            dot[jj] += hi * bf16_bits_to_f32(v[q] >> 16);
            o[q] = f32_to_bf16_bits(wj[jj] * lo) | (f32_to_bf16_bits(wj[jj] * hi) << 16);
          }
        }
        *reinterpret_cast<u32x4_t*>(dc + sl * dc_ld + i * 8) = o;
      }
    }
#pragma unroll
    for (int jj = 0; jj < kCombineBatch; ++jj) {
#pragma unroll
      for (int d = 32; d >= 1; d >>= 1) dot[jj] += __shfl_xor(dot[jj], d, 64);
      if (threadIdx.x % 64 == 0) s_dot[threadIdx.x / 64][jj] = dot[jj];
    }
    __syncthreads();
    if (threadIdx.x < kCombineBatch && j0 + (int)threadIdx.x < top_k) {
      float v = 0.0f;
#pragma unroll
      for (int i = 0; i < kCombineThreads / 64; ++i) v += s_dot[i][threadIdx.x];
      dw[t * top_k + j0 + threadIdx.x] = v;
    }
    __syncthreads();
  }
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
  if (T == 0) return hipSuccess;
  const int32_t n8 = (int32_t)(N / 8);
  const int64_t blocks = (T * n8 + kCombineThreads - 1) / kCombineThreads;
  hipLaunchKernelGGL(combine_kernel<true>, dim3((uint32_t)blocks), dim3(kCombineThreads), 0, stream,
                     c, c_ld, w, ids, E, T, top_k, n8, y, y_ld);
  return hipGetLastError();
}

hipError_t launch_combine_backward(const uint16_t* dy, int64_t dy_ld, const uint16_t* c, int64_t c_ld, const float* w,
                                   const int32_t* ids, int64_t T, int32_t top_k, int32_t E, int64_t N, uint16_t* dc,
                                   int64_t dc_ld, float* dw, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  hipLaunchKernelGGL(combine_backward_kernel, dim3((uint32_t)T), dim3(kCombineThreads), 0, stream, dy, dy_ld, c,
                     c_ld, w, ids, E, top_k, (int32_t)(N / 8), dc, dc_ld, dw);
  return hipGetLastError();
}

}  // namespace moe
