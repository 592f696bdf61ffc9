// moe_rmsnorm and moe_rmsnorm_backward: the root-mean-square norm of a
// residual stream, with the addition of a layer's output (and its dropout) in
// front and the 8-bit forms that the GEMMs read behind.
//
// HBM-bound: every matrix is read or written once. A row stays in the
// registers of its threads (LANES threads of a 256- or 512-thread workgroup, V
// pieces of 8 columns each, neighbouring threads on neighbouring pieces, so
// that every access is 16 contiguous bytes a lane), so the sum of squares, the
// row's largest magnitude and the outputs come from one pass over memory.
#include "dropout_util.h"
#include "params.h"

namespace moe {

constexpr int kNormMaxPieces = 2048;  // 16384 columns
constexpr int64_t kNormMaxBlocks = 1 << 22;  // workgroups per launch (a grid holds fewer than 2^32 threads)
constexpr int kNormBwdBlocks = 1024;  // most workgroups whose partial sums make dweight
constexpr int kNormFinCols = 32, kNormFinRows = 16;

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

// ------------------------------------------------------------------ pieces

// V pieces of row `row` as floats; zeros past the row.
template <int LANES, int V>
__device__ __forceinline__ void norm_load(const void* base, bool wide, int64_t row, int64_t ld, int lane, int pieces,
                                          float (&f)[V][8]) {
  if (wide) {
    const float* p = static_cast<const float*>(base) + row * ld;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int piece = lane + j * LANES;
      f32x4_t a = {0, 0, 0, 0}, b = {0, 0, 0, 0};
      if (piece < pieces) {
        a = reinterpret_cast<const f32x4_t*>(p)[2 * piece];
        b = reinterpret_cast<const f32x4_t*>(p)[2 * piece + 1];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[j][i] = a[i];
        f[j][4 + i] = b[i];
      }
    }
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(base) + row * ld;
    u32x4_t v[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int piece = lane + j * LANES;
      v[j] = u32x4_t{0, 0, 0, 0};
      if (piece < pieces) v[j] = reinterpret_cast<const u32x4_t*>(p)[piece];
    }
#pragma unroll
    for (int j = 0; j < V; ++j) unpack8(v[j], f[j]);
  }
}

template <int LANES, int V>
__device__ __forceinline__ void norm_store(void* base, bool wide, int64_t row, int64_t ld, int lane, int pieces,
                                           const float (&f)[V][8]) {
  if (wide) {
    float* p = static_cast<float*>(base) + row * ld;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int piece = lane + j * LANES;
      if (piece < pieces) {
        reinterpret_cast<f32x4_t*>(p)[2 * piece] = f32x4_t{f[j][0], f[j][1], f[j][2], f[j][3]};
        reinterpret_cast<f32x4_t*>(p)[2 * piece + 1] = f32x4_t{f[j][4], f[j][5], f[j][6], f[j][7]};
      }
    }
  } else {
    uint16_t* p = static_cast<uint16_t*>(base) + row * ld;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int piece = lane + j * LANES;
      if (piece < pieces) reinterpret_cast<u32x4_t*>(p)[piece] = pack8(f[j]);
    }
  }
}

// 8 values over `scale` (a power of two, or 1) -> 8 E4M3 codes, saturated at
// +-lim = 448 scale. Adding 0 takes the sign off a zero.
__device__ __forceinline__ u32x2_t norm_codes(const float (&f)[8], float mul, float lim, float scale) {
  u32x2_t out;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    float c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = fminf(fmaxf(f[4 * w + i] * mul + 0.0f, -lim), lim);
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

template <int THREADS, int LANES, int V, bool RES, bool DROP>
__global__ __launch_bounds__(THREADS) void norm_kernel(NormParams p, Dropout d) {
  constexpr int kRows = THREADS / LANES;
  __shared__ float red[THREADS / 64];
  __shared__ uint32_t red_top[THREADS / 64];
  const int lane = threadIdx.x % LANES;
  const int64_t row = p.row0 + (int64_t)blockIdx.x * kRows + threadIdx.x / LANES;
  if (LANES <= 64 && row >= p.rows) return;  // (beyond, a workgroup is one row and the grid has no more)

  float v[V][8], w[V][8];
  norm_load<LANES, V>(p.x, false, row, p.x_ld, lane, p.pieces, v);
  if constexpr (RES) norm_load<LANES, V>(p.res, p.wide, row, p.res_ld, lane, p.pieces, w);
  if constexpr (DROP) {
    const uint64_t seed = d.rng[0], offset = d.rng[1];
#pragma unroll
    for (int j = 0; j < V; ++j)
      drop8(d, seed, offset, (uint64_t)row * p.pieces + lane + j * LANES, v[j]);
  }
  if constexpr (RES) {
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] += w[j][i];
  }
  norm_load<LANES, V>(p.w, p.w_wide, 0, 0, lane, p.pieces, w);
  if (p.sum != nullptr) norm_store<LANES, V>(p.sum, p.wide, row, p.sum_ld, lane, p.pieces, v);
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) s += v[j][i] * v[j][i];
  s = norm_reduce<LANES>(s, red, [](float a, float b) { return a + b; });
  const float r = rsqrtf(s * p.inv_n + p.eps);
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) v[j][i] = v[j][i] * r * w[j][i];
  if (p.y != nullptr) norm_store<LANES, V>(p.y, false, row, p.y_ld, lane, p.pieces, v);

  if (p.quant == 1) {  // MXFP8: four neighbouring lanes hold a block of 32
    uint8_t* scales = static_cast<uint8_t*>(p.scales) + row * p.scales_ld;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int piece = lane + j * LANES;
      uint32_t top = norm_top(v[j]);
      top = max(top, norm_dpp<0xB1>(top));  // lane ^ 1
      top = max(top, norm_dpp<0x4E>(top));  // lane ^ 2
      const bool bad = top >= 0x7F800000u;
      const int x = max((int)(top >> 23) - 127 - 8, -127);  // (a subnormal's exponent field gives -135; 254 - 135 < 127)
      const float scale = __uint_as_float((uint32_t)(x + 127) << 23);  // (byte 0 stands for 2^-127)
      const float lim = __uint_as_float(((uint32_t)(x + 135) << 23) | 0x600000u);
      u32x2_t c = norm_codes(v[j], 1.0f, lim, scale);
      if (bad) c = u32x2_t{0x7F7F7F7Fu, 0x7F7F7F7Fu};
      if (piece < p.pieces) {
        reinterpret_cast<u32x2_t*>(p.q + row * p.q_ld)[piece] = c;
        if (lane % 4 == 0) scales[piece / 4] = bad ? (uint8_t)0xFF : (uint8_t)(x + 127);
      }
    }
  } else if (p.quant == 2) {
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) top = max(top, norm_top(v[j]));
    top = norm_reduce<LANES>(top, red_top, [](uint32_t a, uint32_t b) { return max(a, b); });
    const bool bad = top >= 0x7F800000u;
    const float scale = fmaxf(__uint_as_float(top) / 448.0f, 0x1p-126f);
    const float inv = 1.0f / scale;  // (at most 2^126)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int piece = lane + j * LANES;
      u32x2_t c = norm_codes(v[j], inv, 448.0f, 1.0f);
      if (bad) c = u32x2_t{0x7F7F7F7Fu, 0x7F7F7F7Fu};
      if (piece < p.pieces) reinterpret_cast<u32x2_t*>(p.q + row * p.q_ld)[piece] = c;
    }
    if (lane == 0) static_cast<float*>(p.scales)[row] = bad ? __uint_as_float(0x7FC00000u) : scale;
  }
}

// ---------------------------------------------------------------- backward

// Workgroups take rows in turn and keep dweight's terms of their columns in
// registers; each row group of a workgroup leaves one row of partial sums.
template <int THREADS, int LANES, int V, bool DROP>
__global__ __launch_bounds__(THREADS) void norm_backward_kernel(NormParams p, Dropout d) {
  constexpr int kRows = THREADS / LANES;
  __shared__ float red[2][2 * THREADS / 64];
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
  float w[V][8], acc[V][8];
  norm_load<LANES, V>(p.w, p.w_wide, 0, 0, lane, p.pieces, w);
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[j][i] = 0.0f;
  const uint64_t seed = DROP ? d.rng[0] : 0, offset = DROP ? d.rng[1] : 0;
  int turn = 0;
  for (int64_t row = (int64_t)blockIdx.x * kRows + group; row < p.rows; row += (int64_t)gridDim.x * kRows, turn ^= 1) {
    float v[V][8], g[V][8];
    norm_load<LANES, V>(p.v, p.wide, row, p.v_ld, lane, p.pieces, v);
    norm_load<LANES, V>(p.x, false, row, p.x_ld, lane, p.pieces, g);
    float s = 0.0f, t = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s += v[j][i] * v[j][i];
        t += v[j][i] * (g[j][i] * w[j][i]);
      }
    auto add = [](float a, float b) { return a + b; };
    // (two buffers in turn: the next row's writes do not pass a barrier that
    // this row's reads have yet to reach)
    s = norm_reduce<LANES>(s, red[turn], add);
    t = norm_reduce<LANES>(t, red[turn] + THREADS / 64, add);
    const float r = rsqrtf(s * p.inv_n + p.eps);
    const float c = r * r * (t * p.inv_n);
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        acc[j][i] += g[j][i] * (v[j][i] * r);
        v[j][i] = r * (g[j][i] * w[j][i] - v[j][i] * c);
      }
    if (p.res != nullptr) {
      norm_load<LANES, V>(p.res, p.wide, row, p.res_ld, lane, p.pieces, g);
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] += g[j][i];
    }
    if (p.sum != nullptr) norm_store<LANES, V>(p.sum, p.wide, row, p.sum_ld, lane, p.pieces, v);
    if (p.y != nullptr) {
      if constexpr (DROP) {
#pragma unroll
        for (int j = 0; j < V; ++j)
          drop8(d, seed, offset, (uint64_t)row * p.pieces + lane + j * LANES, v[j]);
      }
      norm_store<LANES, V>(p.y, false, row, p.y_ld, lane, p.pieces, v);
    }
  }
  if (p.dw != nullptr)
    norm_store<LANES, V>(p.partial, true, (int64_t)blockIdx.x * kRows + group, (int64_t)p.pieces * 8, lane, p.pieces,
                         acc);
}

// dweight[c] = the partial rows' sum, in order within each of 16 strands and
// then over the strands.
__global__ __launch_bounds__(kNormFinCols* kNormFinRows) void norm_dweight_kernel(const float* __restrict__ partial,
                                                                                  int32_t parts, int32_t n,
                                                                                  float* __restrict__ dw) {
  __shared__ float s[kNormFinRows][kNormFinCols];
  const int c = threadIdx.x % kNormFinCols, k = threadIdx.x / kNormFinCols;
  const int col = blockIdx.x * kNormFinCols + c;
  float a = 0.0f;
  if (col < n)
    for (int i = k; i < parts; i += kNormFinRows) a += partial[(int64_t)i * n + col];
  s[k][c] = a;
  __syncthreads();
  if (k == 0 && col < n) {
    for (int i = 1; i < kNormFinRows; ++i) a += s[i][c];
    dw[col] = a;
  }
}

// ------------------------------------------------------------------ launch

// Calls f with the row layout for this many pieces: the fewest threads that
// hold the row in at most 4 pieces each (8 beyond 8192 columns).
template <class F>
static hipError_t norm_layout(int pieces, F f) {
#define MOE_NORM(T, L, V) f(std::integral_constant<int, T>{}, std::integral_constant<int, L>{}, std::integral_constant<int, V>{})
  if (pieces <= 16) return MOE_NORM(256, 16, 1);
  if (pieces <= 64) return MOE_NORM(256, 64, 1);
  if (pieces <= 128) return MOE_NORM(256, 64, 2);
  if (pieces <= 256) return MOE_NORM(256, 64, 4);
  if (pieces <= 512) return MOE_NORM(256, 256, 2);
  if (pieces <= 1024) return MOE_NORM(256, 256, 4);
  return MOE_NORM(512, 512, 4);
#undef MOE_NORM
}

static int norm_rows_per_block(int pieces) { return pieces <= 16 ? 16 : pieces <= 256 ? 4 : 1; }

hipError_t launch_norm(const NormParams& p, const Dropout& d, hipStream_t stream) {
  if (p.rows == 0) return hipSuccess;
  return norm_layout(p.pieces, [&](auto threads, auto lanes, auto v) {
    constexpr int T = decltype(threads)::value, L = decltype(lanes)::value, V = decltype(v)::value;
    auto kernel = p.res != nullptr ? (d.threshold ? norm_kernel<T, L, V, true, true> : norm_kernel<T, L, V, true, false>)
                                   : (d.threshold ? norm_kernel<T, L, V, false, true> : norm_kernel<T, L, V, false, false>);
    for (NormParams q = p; q.row0 < p.rows; q.row0 += kNormMaxBlocks * (T / L)) {
      const int64_t blocks = (p.rows - q.row0 + T / L - 1) / (T / L);
      hipLaunchKernelGGL(kernel, dim3((uint32_t)(blocks < kNormMaxBlocks ? blocks : kNormMaxBlocks)), dim3(T), 0,
                         stream, q, d);
      const hipError_t err = hipGetLastError();
      if (err != hipSuccess) return err;
    }
    return hipSuccess;
  });
}

static int64_t norm_backward_blocks(int64_t rows, int pieces) {
  const int per = norm_rows_per_block(pieces);
  const int64_t want = (rows + per - 1) / per;
  return want < kNormBwdBlocks ? want : kNormBwdBlocks;
}

int64_t norm_backward_workspace_bytes(int64_t rows, int64_t n) {
  const int pieces = (int)(n / 8);
  return norm_backward_blocks(rows, pieces) * norm_rows_per_block(pieces) * n * 4;
}

hipError_t launch_norm_backward(const NormParams& p, const Dropout& d, hipStream_t stream) {
  const int64_t blocks = norm_backward_blocks(p.rows, p.pieces);
  if (blocks > 0) {
    const hipError_t err = norm_layout(p.pieces, [&](auto threads, auto lanes, auto v) {
      constexpr int T = decltype(threads)::value, L = decltype(lanes)::value, V = decltype(v)::value;
      auto kernel = d.threshold ? norm_backward_kernel<T, L, V, true> : norm_backward_kernel<T, L, V, false>;
      hipLaunchKernelGGL(kernel, dim3((uint32_t)blocks), dim3(T), 0, stream, p, d);
      return hipGetLastError();
    });
    if (err != hipSuccess) return err;
  }
  if (p.dw == nullptr) return hipSuccess;
  const int n = p.pieces * 8;
  hipLaunchKernelGGL(norm_dweight_kernel, dim3((n + kNormFinCols - 1) / kNormFinCols), dim3(kNormFinCols * kNormFinRows),
                     0, stream, p.partial, (int32_t)(blocks * norm_rows_per_block(p.pieces)), n, p.dw);
  return hipGetLastError();
}

}  // namespace moe
