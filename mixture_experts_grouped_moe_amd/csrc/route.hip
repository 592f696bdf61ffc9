// moe_route and moe_route_backward: the router's top-k experts and weights,
// its per-expert counts and probability sums, the balance and z losses, and
// their gradient.
//
// One wave per token row: lane l holds the VPL consecutive experts
// [VPL l, VPL l + VPL). The row's maximum, sum of exponentials and top-k are
// wave reductions over registers, so the logits are read once and nothing of
// size T x E is written by the forward pass. The probabilities are not kept:
// the backward pass recomputes them from the logits, which it would have to
// read in their place.
//
// Statistics: each wave adds its rows' probabilities into registers, a
// workgroup adds its waves' in order and writes one partial row per
// workgroup; a second launch adds those in order (in double) and forms the
// losses. No floating-point atomics, so repeated calls give equal bits.
#include <type_traits>

#include "common.h"
#include "params.h"

namespace moe {

constexpr int kRtWaves = 4;
constexpr int kRtThreads = kRtWaves * 64;
constexpr int kRtMaxGrid = 512;      // workgroups of the row kernels, the partial rows of the statistics
constexpr int kRtFinThreads = 1024;

__device__ __forceinline__ float rt_neg_inf() { return -__builtin_huge_valf(); }

__device__ __forceinline__ float rt_load(const float* p) { return *p; }
__device__ __forceinline__ float rt_load(const uint16_t* p) { return bf16_bits_to_f32(*p); }
__device__ __forceinline__ void rt_store(float* p, float v) { *p = v; }
__device__ __forceinline__ void rt_store(uint16_t* p, float v) { *p = (uint16_t)f32_to_bf16_bits(v); }

template <class F>
__device__ __forceinline__ float rt_reduce(float v, F f) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v = f(v, __shfl_xor(v, d, 64));
  return v;
}
__device__ __forceinline__ float rt_sum(float v) {
  return rt_reduce(v, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ float rt_max(float v) {
  return rt_reduce(v, [](float a, float b) { return fmaxf(a, b); });
}

// log of the unnormalised score: z itself, or log sigmoid(z) without
// cancellation on either side (NaN stays NaN)
__device__ __forceinline__ float rt_log_score(float z, bool sigmoid) {
  if (!sigmoid) return z;
  return (z > 0.0f ? 0.0f : z) - log1pf(expf(-fabsf(z)));
}

// A row's logits and log scores in registers with its maximum and sum.
template <int VPL>
struct RtRow {
  float z[VPL], a[VPL];
  float m, s;  // maximum of a, sum of exp(a - m)

  template <class T>
  __device__ __forceinline__ void load(const T* row, int E, int lane, bool sigmoid) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane * VPL + i;
      z[i] = e < E ? rt_load(row + e) : rt_neg_inf();
    }
    m = rt_neg_inf();
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      a[i] = rt_log_score(z[i], sigmoid);
      m = fmaxf(m, a[i]);
    }
    m = rt_max(m);
    const float m0 = m == rt_neg_inf() ? 0.0f : m;
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      a[i] -= m0;
      s += expf(a[i]);
    }
    s = rt_sum(s);
  }
};

template <class T, int VPL>
__global__ __launch_bounds__(kRtThreads) void route_kernel(RouteParams p) {
  __shared__ float s_p[kRtWaves][64 * VPL];
  __shared__ int32_t s_c[64 * VPL];
  __shared__ int32_t s_n[kRtWaves];
  __shared__ float s_z[kRtWaves];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const bool sigmoid = p.sigmoid != 0;
  for (int e = threadIdx.x; e < 64 * VPL; e += kRtThreads) s_c[e] = 0;
  __syncthreads();
  float psum[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) psum[i] = 0.0f;
  int n = 0;
  float z2 = 0.0f;
  for (int64_t t = (int64_t)blockIdx.x * kRtWaves + wave; t < p.T; t += (int64_t)gridDim.x * kRtWaves) {
    int sel = -1;        // lane j < k: the expert in place j and its log score
    float sel_z = 0.0f;
    float w = 0.0f;
    if (p.mask == nullptr || p.mask[t] != 0) {
      RtRow<VPL> r;
      r.load((const T*)p.logits + t * p.ld, p.E, lane, sigmoid);
      // the top-k by the logits themselves; -inf and NaN are never chosen
      float key[VPL];
      bool nan = false;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        nan |= r.z[i] != r.z[i];
        key[i] = r.z[i] == r.z[i] ? r.z[i] : rt_neg_inf();
      }
      for (int j = 0; j < p.k; ++j) {
        float best = key[0];
#pragma unroll
        for (int i = 1; i < VPL; ++i) best = fmaxf(best, key[i]);
        const float top = rt_max(best);
        if (top == rt_neg_inf()) break;
        const int owner = __builtin_ctzll(__ballot(best == top));
        int e = 0;
#pragma unroll
        for (int i = VPL - 1; i >= 0; --i)
          if (key[i] == top) e = i;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          if (lane == owner && i == e) key[i] = rt_neg_inf();
        const int id = owner * VPL + __builtin_amdgcn_readlane(e, owner);
        if (lane == j) {
          sel = id;
          sel_z = top;
        }
      }
      const bool any_nan = __ballot(nan) != 0;
      const bool live = __ballot(sel >= 0) != 0 || any_nan;
      const float inv = 1.0f / r.s;
      if (sel >= 0) {
        const float a = rt_log_score(sel_z, sigmoid);
        if (p.renorm)
          w = expf(a - rt_log_score(__shfl(sel_z, 0, 64), sigmoid));
        else
          w = sigmoid ? 1.0f / (1.0f + expf(-sel_z)) : expf(a - r.m) * inv;
      }
      if (p.renorm) {
        const float sum = rt_sum(w);
        if (sel >= 0) w = w / sum;
      }
      w *= p.scale;
      if (p.stats && live) {
        ++n;
#pragma unroll
        for (int i = 0; i < VPL; ++i) psum[i] += expf(r.a[i]) * inv;
        const float lse = r.m + logf(r.s);
        if (!sigmoid) z2 += lse * lse;
        if (sel >= 0) atomicAdd(&s_c[sel], 1);
      }
    }
    if (lane < p.k) {
      p.ids[t * p.k + lane] = sel;
      p.w[t * p.k + lane] = w;
    }
  }
  if (!p.stats) return;
#pragma unroll
  for (int i = 0; i < VPL; ++i) s_p[wave][lane * VPL + i] = psum[i];
  if (lane == 0) {
    s_n[wave] = n;
    s_z[wave] = z2;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += kRtThreads) {
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < kRtWaves; ++i) v += s_p[i][e];
    p.part_p[(int64_t)blockIdx.x * p.E + e] = v;
    p.part_c[(int64_t)blockIdx.x * p.E + e] = s_c[e];
  }
  if (threadIdx.x == 0) {
    int nn = 0;
    float zz = 0.0f;
#pragma unroll
    for (int i = 0; i < kRtWaves; ++i) {
      nn += s_n[i];
      zz += s_z[i];
    }
    p.part_n[blockIdx.x] = nn;
    p.part_z[blockIdx.x] = zz;
  }
}

// The partial rows of `grid` workgroups, added in order; the losses.
__global__ __launch_bounds__(kRtFinThreads) void route_finish_kernel(RouteParams p, int grid) {
  __shared__ double s_b[kRtFinThreads];
  double b = 0.0;
  for (int e = threadIdx.x; e < p.E; e += kRtFinThreads) {
    double v = 0.0;
    int64_t c = 0;
    for (int g = 0; g < grid; ++g) {
      v += (double)p.part_p[(int64_t)g * p.E + e];
      c += p.part_c[(int64_t)g * p.E + e];
    }
    p.prob_sum[e] = (float)v;
    p.counts[e] = (int32_t)c;
    b += (double)c * v;
  }
  s_b[threadIdx.x] = b;
  __syncthreads();
  if (threadIdx.x == 0) {
    double sum = 0.0, z = 0.0;
    int64_t n = 0;
    for (int i = 0; i < kRtFinThreads; ++i) sum += s_b[i];
    for (int g = 0; g < grid; ++g) {
      n += p.part_n[g];
      z += (double)p.part_z[g];
    }
    *p.num_routed = (int32_t)n;
    p.losses[0] = n > 0 ? (float)(sum * (double)p.E / ((double)p.k * (double)n * (double)n)) : 0.0f;
    p.losses[1] = n > 0 ? (float)(z / (double)n) : 0.0f;
  }
}

template <class T, int VPL>
__global__ __launch_bounds__(kRtThreads) void route_backward_kernel(RouteParams p) {
  __shared__ float s_u[kRtWaves][64 * VPL];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const bool sigmoid = p.sigmoid != 0;
  float* su = s_u[wave];
  float cost[VPL];
  float zcoef = 0.0f;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    cost[i] = 0.0f;
    su[lane * VPL + i] = 0.0f;
  }
  if (p.dlosses != nullptr) {
    const float n = (float)max(*p.num_routed, 1);
    const float f = p.dlosses[0] * (float)p.E / ((float)p.k * n * n);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane * VPL + i;
      if (e < p.E) cost[i] = f * (float)p.counts[e];
    }
    if (!sigmoid) zcoef = 2.0f * p.dlosses[1] / n;
  }
  for (int64_t t = (int64_t)blockIdx.x * kRtWaves + wave; t < p.T; t += (int64_t)gridDim.x * kRtWaves) {
    T* out = (T*)p.dlogits + t * p.dld;
    const int32_t* ids = p.ids + t * p.k;
    if (ids[0] < 0) {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (lane * VPL + i < p.E) rt_store(out + lane * VPL + i, 0.0f);
      continue;
    }
    const T* row = (const T*)p.logits + t * p.ld;
    RtRow<VPL> r;
    r.load(row, p.E, lane, sigmoid);
    const float inv = 1.0f / r.s;
    const int id = lane < p.k ? ids[lane] : -1;
    const bool chosen = id >= 0 && id < p.E;
    float v = 0.0f, g = 0.0f;
    if (chosen) {
      const float z = rt_load(row + id);
      const float a = rt_log_score(z, sigmoid);
      g = p.scale * p.dw[t * p.k + lane];
      if (p.renorm || !sigmoid)
        v = expf(a - r.m);
      else
        v = 1.0f / (1.0f + expf(-z));
    }
    float u, total = 0.0f;
    if (p.renorm) {
      // softmax over the chosen, relative to their own maximum
      float a = chosen ? rt_log_score(rt_load(row + id), sigmoid) : rt_neg_inf();
      const float top = rt_max(a);
      v = chosen ? expf(a - top) : 0.0f;
      v = v / rt_sum(v);
      const float gv = rt_sum(g * v);
      u = v * (g - gv);
    } else if (!sigmoid) {
      u = v * inv * g;
      total = rt_sum(u);
    } else {
      u = v * g;
    }
    if (chosen) su[id] = u;
    __builtin_amdgcn_wave_barrier();
    float q[VPL], dot = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      q[i] = expf(r.a[i]) * inv;
      dot += q[i] * cost[i];
    }
    dot = rt_sum(dot);
    float common = -dot - total;
    if (!sigmoid) common += zcoef * (r.m + logf(r.s));
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane * VPL + i;
      if (e < p.E) {
        float d = q[i] * (cost[i] + common) + su[e];
        if (sigmoid) d *= 1.0f / (1.0f + expf(r.z[i]));
        rt_store(out + e, d);
      }
    }
    __builtin_amdgcn_wave_barrier();
    if (chosen) su[id] = 0.0f;
    __builtin_amdgcn_wave_barrier();
  }
}

static uint32_t rt_grid(int64_t T) {
  const int64_t want = (T + kRtWaves - 1) / kRtWaves;
  return (uint32_t)(want < kRtMaxGrid ? want : kRtMaxGrid);
}

// Workspace: partial counts and probability sums [grid][E], tokens and z
// sums [grid] (4-byte elements).
int64_t route_workspace_bytes(int64_t T, int32_t E) {
  return (int64_t)rt_grid(T) * ((int64_t)E + 1) * 8;
}

template <class F>
static hipError_t rt_dispatch(int E, bool bf16, F&& f) {
  auto by_type = [&](auto vpl) {
    if (bf16) f(uint16_t{}, vpl); else f(float{}, vpl);
  };
  if (E <= 64) by_type(std::integral_constant<int, 1>{});
  else if (E <= 128) by_type(std::integral_constant<int, 2>{});
  else if (E <= 256) by_type(std::integral_constant<int, 4>{});
  else if (E <= 512) by_type(std::integral_constant<int, 8>{});
  else by_type(std::integral_constant<int, 16>{});
  return hipGetLastError();
}

hipError_t launch_route(RouteParams p, bool bf16, void* workspace, hipStream_t stream) {
  const uint32_t grid = rt_grid(p.T);
  if (p.stats) {
    p.part_p = static_cast<float*>(workspace);
    p.part_c = reinterpret_cast<int32_t*>(p.part_p + (int64_t)grid * p.E);
    p.part_z = reinterpret_cast<float*>(p.part_c + (int64_t)grid * p.E);
    p.part_n = reinterpret_cast<int32_t*>(p.part_z + grid);
  }
  hipError_t err = hipSuccess;
  if (grid > 0)
    err = rt_dispatch(p.E, bf16, [&](auto t, auto vpl) {
      hipLaunchKernelGGL((route_kernel<decltype(t), decltype(vpl)::value>), dim3(grid), dim3(kRtThreads), 0, stream, p);
    });
  if (err != hipSuccess || !p.stats) return err;
  hipLaunchKernelGGL(route_finish_kernel, dim3(1), dim3(kRtFinThreads), 0, stream, p, (int)grid);
  return hipGetLastError();
}

hipError_t launch_route_backward(const RouteParams& p, bool bf16, hipStream_t stream) {
  const uint32_t grid = rt_grid(p.T);
  if (grid == 0) return hipSuccess;
  return rt_dispatch(p.E, bf16, [&](auto t, auto vpl) {
    hipLaunchKernelGGL((route_backward_kernel<decltype(t), decltype(vpl)::value>), dim3(grid), dim3(kRtThreads), 0,
                       stream, p);
  });
}

}  // namespace moe
