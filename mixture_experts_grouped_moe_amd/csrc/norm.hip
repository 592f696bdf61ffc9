// moe_rmsnorm and moe_rmsnorm_backward: the root-mean-square norm of a
// residual stream, with the addition of a layer's output (and its dropout) in
// front and the 8-bit forms that the GEMMs read behind.
//
// HBM-bound: every matrix is read or written once. A row stays in the
// registers of its threads (LANES threads of a workgroup, V <= 2 pieces of 8
// columns each, neighbouring threads on neighbouring pieces), so the sum of
// squares, the row's largest magnitude and all outputs come from one pass over
// memory; workgroups take rows in turn with the next row's loads in flight.
// 4096 x 7168 with MXFP8: 49 us, 5.4 TB/s (a copy of as many bytes reaches 5.4);
// 6554 x 2880 of an fp32 stream with dropout: 38 us, 5.9 TB/s; 7 rows of 2688 with
// per-token codes: 4.0 to 4.7 us, latency; gradient of 16384 x 7168: 166 us, 5.65
// TB/s, and 5 for dweight's last sums; of 333 x 2880: 7.5 and 3.9 us. One row a
// workgroup without the loads ahead: 55 us the first, 204 the last but one.
#include <type_traits>

#include "dropout_util.h"
#include "params.h"

namespace moe {

constexpr int kNormCUs = 256;
// waves per SIMD that the forward kernel is compiled and launched for, and the
// backward kernel, whose every workgroup leaves a row of partial sums (16384 x
// 7168: 172 us at 2, 188 at 4; the forward pass 16384 x 2048: 49.4 us at 4, 51.3
// at 2, 49.9 at 8)
constexpr int kNormWaves = 4, kNormBwdWaves = 2;
constexpr int kNormFinCols = 64;

typedef short norm_v2s __attribute__((ext_vector_type(2)));

// ------------------------------------------------------- lane and row sums

template <int CTRL>
__device__ __forceinline__ uint32_t norm_dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}

// op over the LANES (16, 64: part of a wave; more: whole waves, through LDS)
// threads of a row, the result in each; `red` holds 2 floats per wave. op is
// symmetric and the order fixed.
template <int LANES, class T, class F>
__device__ __forceinline__ T norm_reduce(T v, T* red, F op) {
  constexpr int in_wave = LANES < 64 ? LANES : 64;
#pragma unroll
  for (int m = 1; m < in_wave; m *= 2) v = op(v, __shfl_xor(v, m));
  if constexpr (LANES > 64) {
    constexpr int waves = LANES / 64;
    const int wave = threadIdx.x / 64;
    const int first = wave / waves * waves;
    if (threadIdx.x % 64 == 0) red[wave] = v;
    __syncthreads();
    v = red[first];
#pragma unroll
    for (int i = 1; i < waves; ++i) v = op(v, red[first + i]);
  }
  return v;
}

// The same for two sums at once.
template <int LANES>
__device__ __forceinline__ void norm_reduce2(float& a, float& b, float* red) {
  constexpr int in_wave = LANES < 64 ? LANES : 64;
#pragma unroll
  for (int m = 1; m < in_wave; m *= 2) {
    a += __shfl_xor(a, m);
    b += __shfl_xor(b, m);
  }
  if constexpr (LANES > 64) {
    constexpr int waves = LANES / 64;
    const int wave = threadIdx.x / 64;
    const int first = wave / waves * waves;
    if (threadIdx.x % 64 == 0) {
      red[2 * wave] = a;
      red[2 * wave + 1] = b;
    }
    __syncthreads();
    a = red[2 * first];
    b = red[2 * first + 1];
#pragma unroll
    for (int i = 1; i < waves; ++i) {
      a += red[2 * (first + i)];
      b += red[2 * (first + i) + 1];
    }
  }
}

// 1 / sqrt(sum / n + eps) to half a step: one Newton step on the hardware's
// estimate (1 step off), with the residual 1 - m r^2 in two terms. What r is off
// shifts a whole row's 8-bit codes at their rounding borders (4096 x 7168
// MXFP8: 2.5 times the error of the plain fp32 formula without it).
__device__ __forceinline__ float norm_rstd(float sum, float n, float eps) {
  const float mean = sum / n + eps;
  const bool small = mean < 0x1p-96f;  // (the estimate takes no subnormals)
  const float m = small ? mean * 0x1p96f : mean;
  float r = __builtin_amdgcn_rsqf(m);
  const float t = m * r;
  const float e = __builtin_fmaf(-t, r, 1.0f) - __builtin_fmaf(m, r, -t) * r;
  if (m > 0.0f && m < INFINITY) r = __builtin_fmaf(0.5f * r, e, r);
  return small ? r * 0x1p48f : r;
}

// ------------------------------------------------------------------ pieces

// V pieces of a row as they lie in memory, bf16 or (WIDE) fp32; zeros past the row.
template <int LANES, int V, bool WIDE>
struct NormRaw {
  u32x4_t v[WIDE ? 2 * V : V];
  __device__ __forceinline__ void load(const void* base, int64_t row, int64_t ld, int lane, int pieces) {
    const u32x4_t* p = reinterpret_cast<const u32x4_t*>(static_cast<const uint8_t*>(base) + row * ld * (WIDE ? 4 : 2));
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int piece = lane + j * LANES;
      const bool in = piece < pieces;
      if constexpr (WIDE) {
        v[2 * j] = in ? p[2 * piece] : u32x4_t{0, 0, 0, 0};
        v[2 * j + 1] = in ? p[2 * piece + 1] : u32x4_t{0, 0, 0, 0};
      } else {
        v[j] = in ? p[piece] : u32x4_t{0, 0, 0, 0};
      }
    }
  }
  // Keeps the compiler from holding the floats of an earlier get() of piece j
  // in registers: a second get() converts again.
  __device__ __forceinline__ void again(int j) {
#pragma unroll
    for (int i = 0; i < (WIDE ? 2 : 1); ++i) asm volatile("" : "+v"(v[(WIDE ? 2 : 1) * j + i]));
  }
  __device__ __forceinline__ void get(int j, float (&f)[8]) const {
    if constexpr (WIDE) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[i] = __uint_as_float(v[2 * j][i]);
        f[4 + i] = __uint_as_float(v[2 * j + 1][i]);
      }
    } else {
      unpack8(v[j], f);
    }
  }
};

// Outputs of 8 and 16 contiguous bytes a lane go past the caches (200000 x 128
// bf16 16.7 against 21.0 us, 4096 x 7168 with MXFP8 50.0 against 52.3); an fp32
// piece's two halves, which the L2 joins to lines, do not (6554 x 2880 fp32
// 45.1 against 46.0).
template <int LANES, int V, bool WIDE>
__device__ __forceinline__ void norm_store(void* base, int64_t row, int64_t ld, int lane, int pieces,
                                           const float (&f)[V][8]) {
  u32x4_t* p = reinterpret_cast<u32x4_t*>(static_cast<uint8_t*>(base) + row * ld * (WIDE ? 4 : 2));
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int piece = lane + j * LANES;
    if (piece >= pieces) continue;
    if constexpr (WIDE) {
      u32x4_t a, b;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = __float_as_uint(f[j][i]);
        b[i] = __float_as_uint(f[j][4 + i]);
      }
      p[2 * piece] = a;
      p[2 * piece + 1] = b;
    } else {
      __builtin_nontemporal_store(pack8(f[j]), &p[piece]);
    }
  }
}

template <int LANES, int V>
__device__ __forceinline__ void norm_weight(const NormParams& p, int lane, float (&w)[V][8]) {
  if (p.w_wide) {
    NormRaw<LANES, V, true> r;
    r.load(p.w, 0, 0, lane, p.pieces);
#pragma unroll
    for (int j = 0; j < V; ++j) r.get(j, w[j]);
  } else {
    NormRaw<LANES, V, false> r;
    r.load(p.w, 0, 0, lane, p.pieces);
#pragma unroll
    for (int j = 0; j < V; ++j) r.get(j, w[j]);
  }
}

// f / s rounded to nearest, inv = 1 / s likewise: two corrections of f inv by the
// remainder, the first to less than a step, after which the second's remainder is
// exact and its result the rounded quotient (Markstein, 1990). f inv alone, up to
// a step and a half off, can lie on another side of a border between two codes.
// s >= 2^-60, so that no remainder loses bits. (Four more operations an element:
// 4096 x 7168 bf16 50.4 us, 50.3 without them; 200000 x 128 24.3, 22.2.)
__device__ __forceinline__ float norm_quotient(float f, float s, float inv) {
  float q = f * inv;
  q = __builtin_fmaf(__builtin_fmaf(-q, s, f), inv, q);
  return __builtin_fmaf(__builtin_fmaf(-q, s, f), inv, q);
}

// 8 values over `scale` (a power of two, or 1) -> 8 E4M3 codes, saturated at
// +-lim = 448 scale. Adding 0 takes the sign off a zero.
__device__ __forceinline__ u32x2_t norm_codes(const float (&f)[8], float lim, float scale) {
  u32x2_t out;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    float c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = fminf(fmaxf(f[4 * w + i] + 0.0f, -lim), lim);
    norm_v2s r = {0, 0};
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, c[0], c[1], scale, false);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, c[2], c[3], scale, true);
    out[w] = __builtin_bit_cast(uint32_t, r);
  }
  return out;
}

// The bits of the largest magnitude: they order as the magnitudes do, with
// infinity and NaN on top.
__device__ __forceinline__ uint32_t norm_top(const float (&f)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
  return m;
}

// ----------------------------------------------------------------- forward

// A workgroup takes rows in turn, the next row's pieces loaded before the
// present one's sums, and its columns' weights loaded once.
template <int THREADS, int LANES, int V, bool RES, bool WIDE, bool DROP>
__global__ __launch_bounds__(THREADS, kNormWaves) void norm_kernel(NormParams p, Dropout d) {
  constexpr int kRows = THREADS / LANES;
  __shared__ float red[2][THREADS / 64];
  __shared__ uint32_t red_top[2][THREADS / 64];
  const int lane = threadIdx.x % LANES;
  const int64_t stride = (int64_t)gridDim.x * kRows;
  int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / LANES;
  if (row >= p.rows) return;  // (a row of several waves is a whole workgroup's)
  const uint64_t seed = DROP ? d.rng[0] : 0, offset = DROP ? d.rng[1] : 0;
  NormRaw<LANES, V, false> x;
  NormRaw<LANES, V, WIDE> res;
  x.load(p.x, row, p.x_ld, lane, p.pieces);
  if constexpr (RES) res.load(p.res, row, p.res_ld, lane, p.pieces);
  float w[V][8];
  norm_weight<LANES, V>(p, lane, w);
  // (sums and maxima go through two buffers in turn: the next row's writes do
  // not pass a barrier that this row's reads have yet to reach)
  for (int turn = 0; row < p.rows; row += stride, turn ^= 1) {
    float v[V][8];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      x.get(j, v[j]);
      if constexpr (DROP) drop8(d, seed, offset, (uint64_t)row * p.pieces + lane + j * LANES, v[j]);
      if constexpr (RES) {
        float f[8];
        res.get(j, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] += f[i];
      }
    }
    if (row + stride < p.rows) {
      x.load(p.x, row + stride, p.x_ld, lane, p.pieces);
      if constexpr (RES) res.load(p.res, row + stride, p.res_ld, lane, p.pieces);
    }
    if (p.sum != nullptr) norm_store<LANES, V, WIDE>(p.sum, row, p.sum_ld, lane, p.pieces, v);
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[j][i] * v[j][i];
    s = norm_reduce<LANES>(s, red[turn], [](float a, float b) { return a + b; });
    const float r = norm_rstd(s, p.n, p.eps);
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = v[j][i] * r * w[j][i];
    if (p.y != nullptr) norm_store<LANES, V, false>(p.y, row, p.y_ld, lane, p.pieces, v);

    if (p.quant == 1) {  // MXFP8: four neighbouring lanes hold a block of 32
      uint8_t* scales = static_cast<uint8_t*>(p.scales) + row * p.scales_ld;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int piece = lane + j * LANES;
        uint32_t top = norm_top(v[j]);
        top = max(top, norm_dpp<0xB1>(top));  // lane ^ 1
        top = max(top, norm_dpp<0x4E>(top));  // lane ^ 2
        const bool bad = top >= 0x7F800000u;
        const int x2 = max((int)(top >> 23) - 127 - 8, -127);  // (a subnormal's field gives -135; 254 - 135 < 127)
        const float scale = __uint_as_float((uint32_t)(x2 + 127) << 23);  // (byte 0 stands for 2^-127)
        const float lim = __uint_as_float(((uint32_t)(x2 + 135) << 23) | 0x600000u);
        u32x2_t c = norm_codes(v[j], lim, scale);
        if (bad) c = u32x2_t{0x7F7F7F7Fu, 0x7F7F7F7Fu};
        if (piece < p.pieces) {
          __builtin_nontemporal_store(c, &reinterpret_cast<u32x2_t*>(p.q + row * p.q_ld)[piece]);
          if (lane % 4 == 0) scales[piece / 4] = bad ? (uint8_t)0xFF : (uint8_t)(x2 + 127);
        }
      }
    } else if (p.quant == 2) {
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < V; ++j) top = max(top, norm_top(v[j]));
      top = norm_reduce<LANES>(top, red_top[turn], [](uint32_t a, uint32_t b) { return max(a, b); });
      const bool bad = top >= 0x7F800000u;
      const float scale = fmaxf(__uint_as_float(top) / 448.0f, 0x1p-126f);
      const float up = scale < 0x1p-60f ? 0x1p64f : 1.0f, s = scale * up, inv = 1.0f / s;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int piece = lane + j * LANES;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] = norm_quotient(v[j][i] * up, s, inv);
        u32x2_t c = norm_codes(v[j], 448.0f, 1.0f);
        if (bad) c = u32x2_t{0x7F7F7F7Fu, 0x7F7F7F7Fu};
        if (piece < p.pieces) __builtin_nontemporal_store(c, &reinterpret_cast<u32x2_t*>(p.q + row * p.q_ld)[piece]);
      }
      if (lane == 0) static_cast<float*>(p.scales)[row] = bad ? __uint_as_float(0x7FC00000u) : scale;
    }
  }
}

// ---------------------------------------------------------------- backward

// Workgroups take rows in turn, loads a row ahead, and keep dweight's terms of
// their columns in registers; each leaves one row of partial sums.
template <int THREADS, int LANES, int V, bool WIDE, bool DROP>
__global__ __launch_bounds__(THREADS, kNormBwdWaves) void norm_backward_kernel(NormParams p, Dropout d) {
  constexpr int kRows = THREADS / LANES;
  __shared__ float red[2][2 * THREADS / 64];
  __shared__ f32x4_t weight[LANES * V * 2];
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
  const int64_t stride = (int64_t)gridDim.x * kRows;
  int64_t row = (int64_t)blockIdx.x * kRows + group;
  const bool more = p.res != nullptr;
  const uint64_t seed = DROP ? d.rng[0] : 0, offset = DROP ? d.rng[1] : 0;
  NormRaw<LANES, V, false> dy;
  NormRaw<LANES, V, WIDE> sum, dsum = {};
  if (row < p.rows) {
    sum.load(p.v, row, p.v_ld, lane, p.pieces);
    dy.load(p.x, row, p.x_ld, lane, p.pieces);
    if (more) dsum.load(p.res, row, p.res_ld, lane, p.pieces);
  }
  {
    float w[V][8];
    norm_weight<LANES, V>(p, lane, w);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      weight[j * LANES + lane] = f32x4_t{w[j][0], w[j][1], w[j][2], w[j][3]};
      weight[(V + j) * LANES + lane] = f32x4_t{w[j][4], w[j][5], w[j][6], w[j][7]};
    }
  }
  __syncthreads();
  float acc[V][8];
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[j][i] = 0.0f;
  for (int turn = 0; row < p.rows; row += stride, turn ^= 1) {
    NormRaw<LANES, V, WIDE> v_now = sum, a_now = dsum;
    NormRaw<LANES, V, false> g_now = dy;
    if (row + stride < p.rows) {
      sum.load(p.v, row + stride, p.v_ld, lane, p.pieces);
      dy.load(p.x, row + stride, p.x_ld, lane, p.pieces);
      if (more) dsum.load(p.res, row + stride, p.res_ld, lane, p.pieces);
    }
    float s = 0.0f, t = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float v[8], g[8];
      v_now.get(j, v);
      g_now.get(j, g);
      const f32x4_t w[2] = {weight[j * LANES + lane], weight[(V + j) * LANES + lane]};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s += v[i] * v[i];
        t += v[i] * (g[i] * w[i / 4][i % 4]);
      }
    }
    norm_reduce2<LANES>(s, t, red[turn]);
    const float r = norm_rstd(s, p.n, p.eps);
    const float c = r * (r * (t / p.n));  // (r r would pass fp32's range where rows are below 2^-64)
    float v[V][8];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float g[8], a[8];
      v_now.again(j);
      g_now.again(j);
      v_now.get(j, v[j]);
      g_now.get(j, g);
      a_now.get(j, a);
      const f32x4_t w[2] = {weight[j * LANES + lane], weight[(V + j) * LANES + lane]};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        acc[j][i] += g[i] * (v[j][i] * r);
        const float dv = r * (g[i] * w[i / 4][i % 4] - v[j][i] * c);
        v[j][i] = more ? a[i] + dv : dv;
      }
    }
    if (p.sum != nullptr) norm_store<LANES, V, WIDE>(p.sum, row, p.sum_ld, lane, p.pieces, v);
    if (p.y != nullptr) {
      if constexpr (DROP) {
#pragma unroll
        for (int j = 0; j < V; ++j)
          drop8(d, seed, offset, (uint64_t)row * p.pieces + lane + j * LANES, v[j]);
      }
      norm_store<LANES, V, false>(p.y, row, p.y_ld, lane, p.pieces, v);
    }
  }
  if (p.dw == nullptr) return;
  if constexpr (kRows > 1) {  // the row groups' terms, added in order, in 64 bits
    __shared__ f32x4_t terms[kRows][LANES * V * 2];
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        terms[group][(2 * j + h) * LANES + lane] =
            f32x4_t{acc[j][4 * h], acc[j][4 * h + 1], acc[j][4 * h + 2], acc[j][4 * h + 3]};
    __syncthreads();
    if (group != 0) return;
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        double a[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) a[e] = acc[j][4 * h + e];
        for (int i = 1; i < kRows; ++i) {
          const f32x4_t t = terms[i][(2 * j + h) * LANES + lane];
#pragma unroll
          for (int e = 0; e < 4; ++e) a[e] += t[e];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][4 * h + e] = (float)a[e];
      }
  }
  norm_store<LANES, V, true>(p.partial, blockIdx.x, (int64_t)p.pieces * 8, lane, p.pieces, acc);
}

// dweight[c] = the sum of the partial rows, in 64 bits: 64 strands of rows a
// workgroup, 8 loads of a strand in flight, the strands added in order.
__global__ __launch_bounds__(1024) void norm_dweight_kernel(const float* __restrict__ partial, int32_t parts, int32_t n,
                                                            float* __restrict__ dw) {
  constexpr int kStrands = 64, kAhead = 8;
  typedef double f64x4_t __attribute__((ext_vector_type(4)));
  __shared__ f64x4_t s[kStrands][kNormFinCols / 4];
  const int c = threadIdx.x % (kNormFinCols / 4), k = threadIdx.x / (kNormFinCols / 4);
  const int col = blockIdx.x * kNormFinCols + 4 * c;
  const f32x4_t* p = reinterpret_cast<const f32x4_t*>(partial + col);
  f64x4_t a = {0, 0, 0, 0};
  if (col < n) {
    for (int i = k; i < parts; i += kStrands * kAhead) {
      f32x4_t v[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int r = i + j * kStrands;
        v[j] = r < parts ? p[(int64_t)r * (n / 4)] : f32x4_t{0, 0, 0, 0};
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) a[e] += v[j][e];
    }
  }
  s[k][c] = a;
  __syncthreads();
  if (k < 8) {
    for (int i = 1; i < 8; ++i) a += s[k + 8 * i][c];
    s[k][c] = a;
  }
  __syncthreads();
  if (k == 0 && col < n) {
    for (int i = 1; i < 8; ++i) a += s[i][c];
#pragma unroll
    for (int i = 0; i < 4; ++i) dw[col + i] = (float)a[i];
  }
}

// ------------------------------------------------------------------ launch

// Calls f with the row layout for this many pieces: the fewest threads that
// hold the row in at most 2 pieces each.
template <class F>
static auto norm_layout(int pieces, F f) {
#define MOE_NORM(T, L, V) f(std::integral_constant<int, T>{}, std::integral_constant<int, L>{}, std::integral_constant<int, V>{})
  if (pieces <= 16) return MOE_NORM(256, 16, 1);
  if (pieces <= 64) return MOE_NORM(256, 64, 1);
  if (pieces <= 128) return MOE_NORM(256, 64, 2);
  if (pieces <= 256) return MOE_NORM(128, 128, 2);
  if (pieces <= 512) return MOE_NORM(256, 256, 2);
  if (pieces <= 1024) return MOE_NORM(512, 512, 2);
  return MOE_NORM(1024, 1024, 2);
#undef MOE_NORM
}

// Workgroups of `threads` threads that keep `waves` waves on every SIMD (at
// least one a CU), no more than the rows need.
static int64_t norm_blocks(int64_t rows, int threads, int lanes, int waves) {
  const int64_t want = (rows + threads / lanes - 1) / (threads / lanes);
  const int64_t most = (int64_t)kNormCUs * (4 * waves * 64 < threads ? 1 : 4 * waves * 64 / threads);
  return want < most ? want : most;
}

hipError_t launch_norm(const NormParams& p, const Dropout& d, hipStream_t stream) {
  if (p.rows == 0) return hipSuccess;
  return norm_layout(p.pieces, [&](auto threads, auto lanes, auto v) {
    constexpr int T = decltype(threads)::value, L = decltype(lanes)::value, V = decltype(v)::value;
    auto pick = [&](auto drop) {
      constexpr bool D = decltype(drop)::value;
      if (p.res == nullptr) return p.wide ? norm_kernel<T, L, V, false, true, D> : norm_kernel<T, L, V, false, false, D>;
      return p.wide ? norm_kernel<T, L, V, true, true, D> : norm_kernel<T, L, V, true, false, D>;
    };
    auto kernel = d.threshold ? pick(std::true_type{}) : pick(std::false_type{});
    hipLaunchKernelGGL(kernel, dim3((uint32_t)norm_blocks(p.rows, T, L, kNormWaves)), dim3(T), 0, stream, p, d);
    return hipGetLastError();
  });
}

int64_t norm_backward_workspace_bytes(int64_t rows, int64_t n) {
  return norm_layout((int)(n / 8), [&](auto threads, auto lanes, auto) {
    return norm_blocks(rows, threads, lanes, kNormBwdWaves) * n * 4;
  });
}

hipError_t launch_norm_backward(const NormParams& p, const Dropout& d, hipStream_t stream) {
  int64_t parts = 0;
  if (p.rows > 0) {
    const hipError_t err = norm_layout(p.pieces, [&](auto threads, auto lanes, auto v) {
      constexpr int T = decltype(threads)::value, L = decltype(lanes)::value, V = decltype(v)::value;
      auto kernel = d.threshold ? (p.wide ? norm_backward_kernel<T, L, V, true, true> : norm_backward_kernel<T, L, V, false, true>)
                                : (p.wide ? norm_backward_kernel<T, L, V, true, false> : norm_backward_kernel<T, L, V, false, false>);
      const int64_t blocks = norm_blocks(p.rows, T, L, kNormBwdWaves);
      parts = blocks;
      hipLaunchKernelGGL(kernel, dim3((uint32_t)blocks), dim3(T), 0, stream, p, d);
      return hipGetLastError();
    });
    if (err != hipSuccess) return err;
  }
  if (p.dw == nullptr) return hipSuccess;
  const int n = p.pieces * 8;
  hipLaunchKernelGGL(norm_dweight_kernel, dim3((n + kNormFinCols - 1) / kNormFinCols), dim3(1024), 0, stream, p.partial,
                     (int32_t)parts, n, p.dw);
  return hipGetLastError();
}

}  // namespace moe
