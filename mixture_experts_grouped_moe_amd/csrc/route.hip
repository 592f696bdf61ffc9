// moe_route and moe_route_backward: the router's top-k experts and weights,
// its per-expert counts and probability sums, the balance and z losses, and
// their gradient.
//
// Forward (top_k <= 16). LPR lanes hold a row, VPL logits each, read once in
// whole cache lines (8 lanes of 16 for 128 experts: a wave takes 8 rows at
// once and its cross-lane steps serve all of them). The top-k is a merge, not k
// rounds of a maximum: every lane sorts its logits in groups of L >= top_k
// with a fixed network, merges the groups keeping L, and log2(LPR) exchanges
// merge the lanes' lists, after which every lane has the row's list. Keys
// carry the expert's index below the logit (route_util.h), so ties need no
// extra step and ordering a pair takes two instructions. Taking the maximum k
// times over one row per wave cost 335 us on 65536 x 256 fp32 logits with
// top 8 and statistics; this takes 30 us on logits that no cache holds (25 and
// the finishing launch; 27 where the 256 MB cache holds them), where the
// logits' bytes take 13 us at the rate of a large copy. Instructions, about
// 130 a row, take half of the kernel's cycles at one per SIMD and 4 cycles;
// the same logits in bf16, half the bytes, take 27 us. What the other half
// waits for is not taken apart. Loading a row ahead of its use changed nothing.
// Wider top_k (up to 64): k rounds of a wave's maximum, one row per wave. On
// 65536 x 512 fp32 the merging kernel takes 53 us at top 16, this one 241 at
// top 17, 423 at top 32 and 812 at top 64.
//
// Backward: the same layout. The probabilities are not kept by the forward
// pass but recomputed from the logits, which the gradient would otherwise
// replace by a read of the same size. The chosen experts' terms go through a
// row of LDS that is zero otherwise, so adding them costs one scattered add
// and one read however many there are. 65536 x 256 fp32, an eighth of the rows
// padding: 29 us (sigmoid 30.5) from logits and into gradients that no cache
// holds, 4.7 TB/s; 27.5 (30) where the 256 MB cache holds some. In bf16 25 us:
// bound by instructions.
//
// Statistics: each lane adds its rows' probabilities into registers, a
// workgroup adds its lanes' and writes one partial row, and a second launch
// adds those in order (in double) and forms the losses. No floating-point
// atomics, so repeated calls give equal bits. Scores and sums are fp32, the
// token counts integers.
#include <type_traits>

#include "common.h"
#include "params.h"
#include "route_util.h"

namespace moe {

constexpr int kRtWaves = 8;
constexpr int kRtThreads = kRtWaves * 64;
constexpr int kRtMaxGrid = 512;   // workgroups of the row kernels: partial rows of the statistics
constexpr int kRtListMax = 16;    // widest top_k of the merging kernel
constexpr int kRtFinThreads = 512;
constexpr int kRtFinExperts = 16; // experts per workgroup of the finishing kernel

// One partial row of a workgroup: its LDS sums s_p[waves][width], its counts,
// routed tokens and squared log sums.
template <int WIDTH>
__device__ __forceinline__ void rt_write_partial(const RouteParams& p, const float (&s_p)[kRtWaves][WIDTH],
                                                 const int32_t* s_c, const int32_t* s_n, const float* s_z) {
  for (int e = threadIdx.x; e < p.E; e += kRtThreads) {
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < kRtWaves; ++i) v += s_p[i][e];
    p.part_p[(int64_t)blockIdx.x * p.E + e] = v;
    p.part_c[(int64_t)blockIdx.x * p.E + e] = s_c[e];
  }
  if (threadIdx.x == 0) {
    int n = 0;
    float z = 0.0f;
#pragma unroll
    for (int i = 0; i < kRtWaves; ++i) {
      n += s_n[i];
      z += s_z[i];
    }
    p.part_n[blockIdx.x] = n;
    p.part_z[blockIdx.x] = z;
    if (blockIdx.x == 0) *p.ticket = 0;
  }
}

// Waves per SIMD that the registers leave room for: 32 logits a lane or lists
// of 16 double keys take more than 128 (4096 x 256 fp32 top 16: 6.4 us, with
// registers in scratch memory at four waves 8.7).
template <class T, int VPL, int L>
constexpr int kRtOccupancy = VPL > 16 || sizeof(typename RtVec<T>::key::type) * L > 64 ? 2 : 4;

template <class T, int LPR, int VPL, int L, bool SIGMOID>
__global__ __launch_bounds__(kRtThreads, (kRtOccupancy<T, VPL, L>)) void route_kernel(RouteParams p) {
  using V = RtVec<T>;
  using K = typename V::key;
  constexpr int RPW = 64 / LPR;        // rows of a wave
  constexpr int WIDTH = LPR * VPL;
  constexpr int G = VPL < L ? VPL : L; // logits sorted at a time
  __shared__ float s_p[kRtWaves][WIDTH];
  __shared__ int32_t s_c[WIDTH];
  __shared__ int32_t s_n[kRtWaves];
  __shared__ float s_z[kRtWaves];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int l = lane % LPR, group = lane / LPR;
  const T* logits = static_cast<const T*>(p.logits);
  if (p.stats) {
    for (int e = threadIdx.x; e < WIDTH; e += kRtThreads) s_c[e] = 0;
    __syncthreads();
  }
  float psum[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) psum[i] = 0.0f;
  int n = 0;
  float z2 = 0.0f;
  const int64_t step = (int64_t)gridDim.x * kRtWaves * RPW;
  for (int64_t t0 = ((int64_t)blockIdx.x * kRtWaves + wave) * RPW; t0 < p.T; t0 += step) {
    const int64_t t = t0 + group;
    const bool on = t < p.T && (p.mask == nullptr || p.mask[t] != 0);
    float z[VPL];
    rt_load_row<T, LPR, VPL>(logits + t * p.ld, p.E, l, on, z);
    typename K::type top[L];
#pragma unroll
    for (int g = 0; g < VPL / G; ++g) {
      typename K::type v[L];
#pragma unroll
      for (int i = 0; i < L; ++i) {
        const int at = g * G + i;
        v[i] = i < G ? K::make(z[i < G ? at : 0], ((at / V::N) * LPR + l) * V::N + at % V::N) : K::lowest();
      }
      rt_sort<K, L>(v);
      if (g == 0) {
#pragma unroll
        for (int i = 0; i < L; ++i) top[i] = v[i];
      } else {
        rt_merge<K, L>(top, v);
      }
    }
    rt_merge_lanes<K, L, LPR>(top);
    const float m = K::value(top[0]);
    const float base = rt_base<SIGMOID>(m);
    float s = 0.0f;
    bool live = false;
    if (p.stats || (!SIGMOID && !p.renorm)) {  // the sum over all experts
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        z[i] = rt_score<SIGMOID>(z[i], base);
        s += z[i];
      }
      s = rt_sum<LPR>(s);
      live = s != 0.0f;  // (NaN too)
    }
    const float inv = live ? 1.0f / s : 0.0f;
    if (p.stats) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) psum[i] += z[i] * inv;
      if (live && l == 0) {
        ++n;
        const float lse = base + rt_log(s);
        if (!SIGMOID) z2 += lse * lse;
      }
    }
    // the chosen experts: lane l takes places l, l + LPR, .. of the row's list
    constexpr int NJ = (L + LPR - 1) / LPR;
    const float wbase = SIGMOID && !p.renorm ? 0.0f : base;
    int id[NJ];
    float w[NJ], sum = 0.0f;
#pragma unroll
    for (int jj = 0; jj < NJ; ++jj) {
      typename K::type key = top[jj * LPR];
#pragma unroll
      for (int j = 1; j < LPR && jj * LPR + j < L; ++j)
        if (l == j) key = top[jj * LPR + j];
      const float zj = K::value(key);
      const bool ok = jj * LPR + l < p.k && (LPR <= L || l < L) && zj != rt_neg_inf();
      id[jj] = ok ? K::expert(key) : -1;
      w[jj] = ok ? rt_score<SIGMOID>(zj, wbase) : 0.0f;
      sum += w[jj];
    }
    float f = p.scale;
    if (p.renorm) {
      sum = rt_sum<LPR>(sum);
      f = sum != 0.0f ? f / sum : 0.0f;
    } else if (!SIGMOID) {
      f *= inv;
    }
#pragma unroll
    for (int jj = 0; jj < NJ; ++jj) {
      const int j = jj * LPR + l;
      if (t < p.T && j < p.k) {
        p.ids[t * p.k + j] = id[jj];
        p.w[t * p.k + j] = id[jj] >= 0 ? w[jj] * f : 0.0f;
        if (p.stats && id[jj] >= 0) atomicAdd(&s_c[id[jj]], 1);
      }
    }
  }
  if (!p.stats) return;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const float v = rt_sum_rows<LPR>(psum[i]);
    if (group == 0) s_p[wave][((i / V::N) * LPR + l) * V::N + i % V::N] = v;
  }
  const float zz = rt_sum_rows<LPR>(z2);
  const float nn = rt_sum_rows<LPR>((float)n);  // at most rows per wave: exact
  if (lane == 0) {
    s_n[wave] = (int)nn;
    s_z[wave] = zz;
  }
  __syncthreads();
  rt_write_partial(p, s_p, s_c, s_n, s_z);
}

// top_k > 16: one wave per row, VPL consecutive experts per lane, top_k
// rounds of the row's maximum.
template <class T, int VPL, bool SIGMOID>
__global__ __launch_bounds__(kRtThreads) void route_wide_kernel(RouteParams p) {
  using V = RtVec<T>;
  constexpr int WIDTH = 64 * VPL;
  __shared__ float s_p[kRtWaves][WIDTH];
  __shared__ int32_t s_c[WIDTH];
  __shared__ int32_t s_n[kRtWaves];
  __shared__ float s_z[kRtWaves];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  for (int e = threadIdx.x; e < WIDTH; e += kRtThreads) s_c[e] = 0;
  __syncthreads();
  float psum[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) psum[i] = 0.0f;
  int n = 0;
  float z2 = 0.0f;
  for (int64_t t = (int64_t)blockIdx.x * kRtWaves + wave; t < p.T; t += (int64_t)gridDim.x * kRtWaves) {
    int sel = -1;  // lane j < k: the expert in place j and its logit
    float sel_z = rt_neg_inf(), w = 0.0f;
    if (p.mask == nullptr || p.mask[t] != 0) {
      const T* row = static_cast<const T*>(p.logits) + t * p.ld;
      float z[VPL], key[VPL];
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int e = lane * VPL + i;
        z[i] = e < p.E ? V::one(row + e) : rt_neg_inf();
        key[i] = z[i] == z[i] ? z[i] : rt_neg_inf();
      }
      for (int j = 0; j < p.k; ++j) {
        float best = key[0];
#pragma unroll
        for (int i = 1; i < VPL; ++i) best = fmaxf(best, key[i]);
        const float top = rt_max<64>(best);
        if (top == rt_neg_inf()) break;
        const int owner = __builtin_ctzll(__ballot(best == top));
        int at = 0;
#pragma unroll
        for (int i = VPL - 1; i >= 0; --i)
          if (key[i] == top) at = i;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          if (lane == owner && i == at) key[i] = rt_neg_inf();
        const int id = owner * VPL + __builtin_amdgcn_readlane(at, owner);
        if (lane == j) {
          sel = id;
          sel_z = top;
        }
      }
      const float m = __shfl(sel_z, 0, 64);
      const float base = rt_base<SIGMOID>(m);
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        z[i] = rt_score<SIGMOID>(z[i], base);
        s += z[i];
      }
      s = rt_sum<64>(s);
      const bool live = s != 0.0f;
      const float inv = live ? 1.0f / s : 0.0f;
      w = sel >= 0 ? rt_score<SIGMOID>(sel_z, SIGMOID && !p.renorm ? 0.0f : base) : 0.0f;
      const float sum = rt_sum<64>(w);
      float f = p.scale;
      if (p.renorm)
        f = sum != 0.0f ? f / sum : 0.0f;
      else if (!SIGMOID)
        f *= inv;
      w = sel >= 0 ? w * f : 0.0f;
      if (p.stats && live) {
        ++n;
#pragma unroll
        for (int i = 0; i < VPL; ++i) psum[i] += z[i] * inv;
        const float lse = base + rt_log(s);
        if (!SIGMOID) z2 += lse * lse;
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
  rt_write_partial(p, s_p, s_c, s_n, s_z);
}

// The partial rows of `grid` workgroups, added in order (32 threads an
// expert take every 32nd row, then are added in order); the workgroup that
// finishes last forms the losses from the sums of all.
__global__ __launch_bounds__(kRtFinThreads) void route_finish_kernel(RouteParams p, int grid) {
  constexpr int ROWS = kRtFinThreads / kRtFinExperts;
  __shared__ double s_v[ROWS][kRtFinExperts];
  __shared__ int32_t s_k[ROWS][kRtFinExperts];
  __shared__ int s_last;
  const int col = threadIdx.x % kRtFinExperts, row = threadIdx.x / kRtFinExperts;
  const int e = blockIdx.x * kRtFinExperts + col;
  double v = 0.0;
  int32_t c = 0;
  if (e < p.E)
#pragma unroll 4
    for (int g = row; g < grid; g += ROWS) {
      v += (double)p.part_p[(int64_t)g * p.E + e];
      c += p.part_c[(int64_t)g * p.E + e];
    }
  s_v[row][col] = v;
  s_k[row][col] = c;
  __syncthreads();
  if (row == 0) {
    for (int r = 1; r < ROWS; ++r) {
      v += s_v[r][col];
      c += s_k[r][col];
    }
    if (e < p.E) {
      p.prob_sum[e] = (float)v;
      p.counts[e] = c;
    }
    s_v[0][col] = v * (double)c;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    double b = 0.0;
    for (int i = 0; i < kRtFinExperts; ++i) b += s_v[0][i];
    __hip_atomic_store(&p.part_b[blockIdx.x], b, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    s_last = __hip_atomic_fetch_add(p.ticket, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == (int)gridDim.x - 1;
  }
  __syncthreads();
  if (!s_last) return;
  double z = 0.0;
  int32_t n = 0;
  for (int g = threadIdx.x; g < grid; g += kRtFinThreads) {
    z += (double)p.part_z[g];
    n += p.part_n[g];
  }
  double* s_z = &s_v[0][0];
  int32_t* s_n = &s_k[0][0];
  s_z[threadIdx.x] = z;
  s_n[threadIdx.x] = n;
  __syncthreads();
  if (threadIdx.x < 64) {
    z = 0.0;
    n = 0;
    for (int i = threadIdx.x; i < kRtFinThreads; i += 64) {
      z += s_z[i];
      n += s_n[i];
    }
    double b = (int)threadIdx.x < (int)gridDim.x  // at most 64 workgroups: 1024 experts
                   ? __hip_atomic_load(&p.part_b[threadIdx.x], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)
                   : 0.0;
#pragma unroll
    for (int d = 32; d >= 1; d /= 2) {
      z += __shfl_xor(z, d, 64);
      b += __shfl_xor(b, d, 64);
      n += __shfl_xor(n, d, 64);
    }
    if (threadIdx.x == 0) {
      *p.num_routed = n;
      p.losses[0] = n > 0 ? (float)(b * (double)p.E / ((double)p.k * (double)n * (double)n)) : 0.0f;
      p.losses[1] = n > 0 ? (float)(z / (double)n) : 0.0f;
    }
  }
}

// NJ: places of a row per lane (top_k <= NJ * LPR).
template <class T, int LPR, int VPL, int NJ, bool SIGMOID>
__global__ __launch_bounds__(kRtThreads, NJ > 4 ? 2 : 4) void route_backward_kernel(RouteParams p) {
  using V = RtVec<T>;
  constexpr int RPW = 64 / LPR;
  constexpr int WIDTH = LPR * VPL + 32;  // (rows a bank group apart)
  __shared__ __attribute__((aligned(16))) float s_u[kRtWaves][RPW][WIDTH];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int l = lane % LPR, group = lane / LPR;
  float* su = s_u[wave][group];
  // A row's loads, before what does not need them and without a branch between
  // them: one that waits for another costs its latency. (So the logits also of
  // a row routed nowhere, and clamped places.)
  float z[VPL], dwj[NJ];
  int idj[NJ], first;
  const auto load = [&](int64_t t) {
    const int64_t s0 = min(t, p.T - 1) * p.k;
    first = p.ids[s0];
#pragma unroll
    for (int jj = 0; jj < NJ; ++jj) {
      const int64_t s = s0 + min(jj * LPR + l, p.k - 1);
      idj[jj] = p.ids[s];
      dwj[jj] = p.dw[s];
    }
    rt_load_row<T, LPR, VPL>(static_cast<const T*>(p.logits) + t * p.ld, p.E, l, t < p.T, z);
  };
  const int64_t step = (int64_t)gridDim.x * kRtWaves * RPW;
  int64_t t0 = ((int64_t)blockIdx.x * kRtWaves + wave) * RPW;
  int32_t count[VPL];
  if (p.dlosses != nullptr) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = ((i / V::N) * LPR + l) * V::N + i % V::N;
      count[i] = p.counts[min(e, p.E - 1)];
    }
  }
  load(t0 + group);
  float cost[VPL], zcoef = 0.0f;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = ((i / V::N) * LPR + l) * V::N + i % V::N;
    su[e] = 0.0f;
    cost[i] = 0.0f;
  }
  if (p.dlosses != nullptr) {
    const float n = (float)max(*p.num_routed, 1);
    const float f = p.dlosses[0] * (float)p.E / ((float)p.k * n * n);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = ((i / V::N) * LPR + l) * V::N + i % V::N;
      cost[i] = e < p.E ? f * (float)count[i] : 0.0f;
    }
    if (!SIGMOID) zcoef = 2.0f * p.dlosses[1] / n;
  }
  for (; t0 < p.T; t0 += step) {
    const int64_t t = t0 + group;
    const bool on = t < p.T && first >= 0;
    const T* row = static_cast<const T*>(p.logits) + t * p.ld;
    // the chosen experts in places l, l + LPR, ..
    int id[NJ];
    float g[NJ], zj[NJ];
    float top = rt_neg_inf();
#pragma unroll
    for (int jj = 0; jj < NJ; ++jj) {
      const bool ok = on && jj * LPR + l < p.k && (uint32_t)idj[jj] < (uint32_t)p.E;
      id[jj] = ok ? idj[jj] : -1;
      zj[jj] = ok ? V::one(row + id[jj]) : rt_neg_inf();
      g[jj] = ok ? p.scale * dwj[jj] : 0.0f;
      top = fmaxf(top, zj[jj]);
    }
    float m = rt_neg_inf();
#pragma unroll
    for (int i = 0; i < VPL; ++i) m = fmaxf(m, z[i]);
    m = rt_max<LPR>(m);
    const float base = rt_base<SIGMOID>(m);
    float x[VPL], s = 0.0f, dot = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      x[i] = rt_score<SIGMOID>(z[i], base);
      s += x[i];
      dot += x[i] * cost[i];
    }
    s = rt_sum<LPR>(s);
    const float inv = s != 0.0f ? 1.0f / s : 0.0f;
    dot = rt_sum<LPR>(dot) * inv;
    float common = -dot;
    if (!SIGMOID) common += zcoef * (base + rt_log(s));
    // u_j
    float v[NJ], sum = 0.0f, gv = 0.0f;
    const float vbase = p.renorm ? rt_base<SIGMOID>(rt_max<LPR>(top)) : SIGMOID ? 0.0f : base;
#pragma unroll
    for (int jj = 0; jj < NJ; ++jj) {
      v[jj] = id[jj] >= 0 ? rt_score<SIGMOID>(zj[jj], vbase) : 0.0f;
      sum += v[jj];
      gv += g[jj] * v[jj];
    }
    if (p.renorm) {
      sum = rt_sum<LPR>(sum);
      const float is = sum != 0.0f ? 1.0f / sum : 0.0f;
      gv = rt_sum<LPR>(gv) * is;
#pragma unroll
      for (int jj = 0; jj < NJ; ++jj) v[jj] = v[jj] * is * (g[jj] - gv);
    } else if (!SIGMOID) {
      common -= rt_sum<LPR>(gv) * inv;
#pragma unroll
      for (int jj = 0; jj < NJ; ++jj) v[jj] *= inv * g[jj];
    } else {
#pragma unroll
      for (int jj = 0; jj < NJ; ++jj) v[jj] *= g[jj];
    }
#pragma unroll
    for (int jj = 0; jj < NJ; ++jj)
      if (id[jj] >= 0) atomicAdd(&su[id[jj]], v[jj]);  // (added: a caller's ids may name an expert twice)
    __builtin_amdgcn_wave_barrier();
    T* out = static_cast<T*>(p.dlogits) + t * p.dld;
#pragma unroll
    for (int c = 0; c < VPL / V::N; ++c) {
      const int e = (c * LPR + l) * V::N;
      typename V::vec o;
      f32x4_t u[V::N / 4];
#pragma unroll
      for (int i = 0; i < V::N / 4; ++i) u[i] = *reinterpret_cast<const f32x4_t*>(su + e + 4 * i);
#pragma unroll
      for (int i = 0; i < V::N; ++i) {
        const int at = c * V::N + i;
        float d = x[at] * inv * (cost[at] + common) + u[i / 4][i % 4];
        if (SIGMOID) d *= __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z[at] * 1.44269504f));  // 1 - sigmoid(z)
        d = on ? d : 0.0f;
        if (e + V::N <= p.E)
          V::put(o, i, d);
        else if (t < p.T && e + i < p.E)
          V::put(out + e + i, d);
      }
      if (t < p.T && e + V::N <= p.E) *reinterpret_cast<typename V::vec*>(out + e) = o;
    }
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int jj = 0; jj < NJ; ++jj)
      if (id[jj] >= 0) su[id[jj]] = 0.0f;
    __builtin_amdgcn_wave_barrier();
    load(t + step);
  }
}

// Rows that one workgroup takes at a time (rt_layout, and with 32 and 8 logits a lane).
static int rt_rows(int E) { return kRtWaves * (E <= 128 ? 8 : E <= 256 ? 4 : E <= 512 ? 2 : 1); }
static int rt_rows_deep(int E) { return kRtWaves * (E <= 256 ? 8 : E <= 512 ? 4 : 2); }
static int rt_rows_spread(int E) { return kRtWaves * (E <= 128 ? 4 : E <= 256 ? 2 : 1); }

static uint32_t rt_grid(int64_t T, int rows, int most = kRtMaxGrid) {
  const int64_t want = (T + rows - 1) / rows;
  return (uint32_t)(want < most ? want : most);
}
// Workgroups that write a partial row of the statistics: without tokens one
// still does, so that the statistics of nothing are written.
static uint32_t rt_partials(uint32_t grid) { return grid > 0 ? grid : 1; }

// Forward pass above 128 experts: 32 logits a lane instead of 16 sorts more
// in a lane and merges less between lanes, a quarter fewer instructions, but
// has fewer waves. It pays from where 16 a lane fill their largest grid (both
// kernels, statistics included, on logits that no cache holds; fp32 top 8, 256
// experts: 65536 tokens 34 -> 31 us, 16384 17.6 -> 16.2, 4096 11.6 -> 13.9;
// 1024 experts: 65536 tokens 130 -> 96 us, 4096 20.4 -> 17.7, 512 12.2 -> 13.3).
static bool rt_deep(int64_t T, int E) { return E > 128 && T >= (int64_t)kRtMaxGrid * rt_rows(E); }

// Workspace for either forward kernel: the finishing kernel's 64 partial
// products (8 bytes each) and ticket, the partial probability sums and
// counts [rows][E], z sums and tokens [rows].
int64_t route_workspace_bytes(int64_t T, int32_t E) {
  return 64 * 8 + 8 + (int64_t)rt_partials(rt_grid(T, kRtWaves)) * ((int64_t)E + 1) * 8;
}

// Backward pass of 65 to 512 experts: with 8 logits a lane a wave has half the
// rows and half the instructions, which bound it while every wave takes its
// rows once. It pays up to one workgroup per CU of the usual 256 (with the
// losses: 4096 x 256 fp32 7.2 -> 5.7 us, bf16 9.3 -> 7.0; 8192 x 256 7.9 and
// 8.1; 65536 x 512 52 -> 56).
static bool rt_spread(int64_t T, int E) { return E > 64 && E <= 512 && T <= (int64_t)256 * rt_rows_spread(E); }

template <int N>
using rt_c = std::integral_constant<int, N>;

// f(type, LPR, VPL) for the row layout of E experts, VPL at most 16.
template <class F>
static void rt_layout(int E, bool bf16, F&& f) {
  auto by_type = [&](auto lpr, auto vpl) {
    if (bf16)
      f(uint16_t{}, lpr, vpl);
    else
      f(float{}, lpr, vpl);
  };
  if (E <= 64)
    by_type(rt_c<8>{}, rt_c<8>{});
  else if (E <= 128)
    by_type(rt_c<8>{}, rt_c<16>{});
  else if (E <= 256)
    by_type(rt_c<16>{}, rt_c<16>{});
  else if (E <= 512)
    by_type(rt_c<32>{}, rt_c<16>{});
  else
    by_type(rt_c<64>{}, rt_c<16>{});
}
// With 8 logits a lane (64 < E <= 512).
template <class F>
static void rt_layout_spread(int E, bool bf16, F&& f) {
  auto by_type = [&](auto lpr) {
    if (bf16)
      f(uint16_t{}, lpr, rt_c<8>{});
    else
      f(float{}, lpr, rt_c<8>{});
  };
  if (E <= 128)
    by_type(rt_c<16>{});
  else if (E <= 256)
    by_type(rt_c<32>{});
  else
    by_type(rt_c<64>{});
}
// With 32 logits a lane (E > 128).
template <class F>
static void rt_layout_deep(int E, bool bf16, F&& f) {
  auto by_type = [&](auto lpr) {
    if (bf16)
      f(uint16_t{}, lpr, rt_c<32>{});
    else
      f(float{}, lpr, rt_c<32>{});
  };
  if (E <= 256)
    by_type(rt_c<8>{});
  else if (E <= 512)
    by_type(rt_c<16>{});
  else
    by_type(rt_c<32>{});
}

hipError_t launch_route(RouteParams p, bool bf16, void* workspace, hipStream_t stream) {
  const bool wide = p.k > kRtListMax;
  const bool deep = !wide && rt_deep(p.T, p.E);
  uint32_t grid = wide   ? rt_grid(p.T, kRtWaves)
                  : deep ? rt_grid(p.T, rt_rows_deep(p.E), kRtMaxGrid / 2)  // (registers: half the waves)
                         : rt_grid(p.T, rt_rows(p.E));
  if (p.stats) {
    grid = rt_partials(grid);
    p.part_b = static_cast<double*>(workspace);
    p.ticket = reinterpret_cast<int32_t*>(p.part_b + 64);
    p.part_p = reinterpret_cast<float*>(p.ticket + 2);
    p.part_c = reinterpret_cast<int32_t*>(p.part_p + (int64_t)grid * p.E);
    p.part_z = reinterpret_cast<float*>(p.part_c + (int64_t)grid * p.E);
    p.part_n = reinterpret_cast<int32_t*>(p.part_z + grid);
  }
  if (grid == 0) return hipSuccess;
  auto launch = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(kRtThreads), 0, stream, p);
  };
  auto by_score = [&](auto with) {
    if (p.sigmoid)
      with(std::true_type{});
    else
      with(std::false_type{});
  };
  if (wide) {
    auto go = [&](auto t, auto vpl) {
      by_score([&](auto sig) { launch(route_wide_kernel<decltype(t), decltype(vpl)::value, decltype(sig)::value>); });
    };
    auto by_type = [&](auto vpl) {
      if (bf16)
        go(uint16_t{}, vpl);
      else
        go(float{}, vpl);
    };
    if (p.E <= 64)
      by_type(rt_c<1>{});
    else if (p.E <= 256)
      by_type(rt_c<4>{});
    else
      by_type(rt_c<16>{});
  } else {
    auto go = [&](auto t, auto lpr, auto vpl) {
      by_score([&](auto sig) {
        using T = decltype(t);
        constexpr int R = decltype(lpr)::value, N = decltype(vpl)::value;
        constexpr bool S = decltype(sig)::value;
        if (p.k <= 4)
          launch(route_kernel<T, R, N, 4, S>);
        else if (p.k <= 8)
          launch(route_kernel<T, R, N, 8, S>);
        else
          launch(route_kernel<T, R, N, 16, S>);
      });
    };
    if (deep)
      rt_layout_deep(p.E, bf16, go);
    else
      rt_layout(p.E, bf16, go);
  }
  hipError_t err = hipGetLastError();
  if (err != hipSuccess || !p.stats) return err;
  hipLaunchKernelGGL(route_finish_kernel, dim3((p.E + kRtFinExperts - 1) / kRtFinExperts), dim3(kRtFinThreads), 0,
                     stream, p, (int)grid);
  return hipGetLastError();
}

hipError_t launch_route_backward(const RouteParams& p, bool bf16, hipStream_t stream) {
  const bool spread = rt_spread(p.T, p.E);
  const uint32_t grid = rt_grid(p.T, spread ? rt_rows_spread(p.E) : rt_rows(p.E));
  if (grid == 0) return hipSuccess;
  auto go = [&](auto t, auto lpr, auto vpl) {
    using T = decltype(t);
    constexpr int R = decltype(lpr)::value, N = decltype(vpl)::value;
    auto launch = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(grid), dim3(kRtThreads), 0, stream, p); };
    auto by_score = [&](auto nj) {
      constexpr int J = decltype(nj)::value;
      if (p.sigmoid)
        launch(route_backward_kernel<T, R, N, J, true>);
      else
        launch(route_backward_kernel<T, R, N, J, false>);
    };
    if (p.k <= R)
      by_score(rt_c<1>{});
    else if (p.k <= 2 * R)
      by_score(rt_c<2>{});
    else
      by_score(rt_c<64 / R>{});
  };
  if (spread)
    rt_layout_spread(p.E, bf16, go);
  else
    rt_layout(p.E, bf16, go);
  return hipGetLastError();
}

}  // namespace moe
