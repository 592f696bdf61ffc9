// moe_lora: low-rank adapters beside a shared projection, C[s] += scale[g]
// B[g] (A[g] x[s / div]) over the slots s of every group g, routed by
// moe_align's block list.
//
// HBM-bound: x is read once, C read and written once, and a group's adapter is
// shared by its blocks through the caches; the products are 2 R flops a byte.
// Two launches, since every output column needs the whole of h = A x: `down`
// forms h, a block of slots and a part of K a workgroup; `up` adds B h, a block
// and a part of N a workgroup, the parts of h summed (in order) as it is read.
#include <type_traits>

#include "lora_util.h"

namespace moe {

// ------------------------------------------------------------------- down

// D rows are ranks, columns slots: a lane then holds 4 consecutive ranks of a
// slot, one 16-byte store. The waves take K in turn, 32 at a time, operands
// straight from memory in MFMA layout (a row's 64 bytes a load), and add their
// sums through LDS.
template <int RT, int MT>
__global__ __launch_bounds__(kLoraThreads) void lora_down_kernel(LoraParams p) {
  constexpr int U = MT + RT <= 3 ? 8 : MT + RT <= 6 ? 4 : 2;  // steps whose loads are issued together
  __shared__ f32x4_t red[4][RT * MT][64];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, q = lane / 16, m16 = lane % 16;
  const int b = p.block0 + blockIdx.x / p.splits, sp = blockIdx.x % p.splits;
  const int g = p.groups[b];
  if ((uint32_t)g >= (uint32_t)p.G) return;
  const int row0 = blockIdx.y * MT * 16;
  const uint16_t* xr[MT];
  bool live[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int row = row0 + 16 * m + m16;
    const uint32_t s = row < p.bm ? (uint32_t)p.sorted[(int64_t)b * p.bm + row] : 0xFFFFFFFFu;
    live[m] = s < (uint32_t)p.S;
    xr[m] = p.x + (int64_t)(live[m] ? lora_div(s, p.div_magic, p.div_shift) : 0) * p.x_ld + 8 * q;
  }
  const uint16_t* wr[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) wr[t] = p.w + (int64_t)g * p.w_g + (int64_t)(16 * t + m16) * p.w_ld + 8 * q;
  const int steps = (p.K + 31) / 32, per = (steps + p.splits - 1) / p.splits;
  const int end = min(steps, (sp + 1) * per);
  f32x4_t acc[RT][MT];
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[t][m] = f32x4_t{0, 0, 0, 0};
  for (int i = sp * per + wave; i < end; i += 4 * U) {
    u32x4_t xv[U][MT], wv[U][RT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = 32 * (i + 4 * u);
      const bool in = i + 4 * u < end && k + 8 * q < p.K;
#pragma unroll
      for (int m = 0; m < MT; ++m)
        xv[u][m] = in && live[m] ? *reinterpret_cast<const u32x4_t*>(xr[m] + k) : u32x4_t{0, 0, 0, 0};
#pragma unroll
      for (int t = 0; t < RT; ++t)
        wv[u][t] = in && 16 * t + m16 < p.R ? *reinterpret_cast<const u32x4_t*>(wr[t] + k) : u32x4_t{0, 0, 0, 0};
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[t][m] = lora_mfma(wv[u][t], xv[u][m], acc[t][m]);
  }
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int m = 0; m < MT; ++m) red[wave][t * MT + m][lane] = acc[t][m];
  __syncthreads();
  for (int i = wave; i < RT * MT; i += 4) {
    const int t = i / MT, m = i % MT, row = row0 + 16 * m + m16, r = 16 * t + 4 * q;
    const uint32_t s = row < p.bm ? (uint32_t)p.sorted[(int64_t)b * p.bm + row] : 0xFFFFFFFFu;
    if (s >= (uint32_t)p.S || r >= p.R) continue;
    const f32x4_t v = ((red[0][i][lane] + red[1][i][lane]) + red[2][i][lane]) + red[3][i][lane];
    *reinterpret_cast<f32x4_t*>(p.part + ((int64_t)sp * p.S + s) * p.R + r) = v;
  }
}

// --------------------------------------------------------------------- up

// 8 ranks from 8 * piece of h[s]: the sum of the parts.
__device__ __forceinline__ void lora_h8(const LoraParams& p, uint32_t s, int piece, float (&f)[8]) {
  const float* at = p.part + (int64_t)s * p.R + 8 * piece;
  f32x4_t a = {0, 0, 0, 0}, b = {0, 0, 0, 0};
  for (int i = 0; i < p.splits; ++i, at += (int64_t)p.S * p.R) {
    a += reinterpret_cast<const f32x4_t*>(at)[0];
    b += reinterpret_cast<const f32x4_t*>(at)[1];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[i] = a[i];
    f[4 + i] = b[i];
  }
}

// D rows are columns of C, D columns slots. Row i of tile j stands for column
// 32 (j / 2) + 8 (i / 4) + 4 (j % 2) + i % 4 of a 64-column piece, so that a lane
// holds twice 8 consecutive columns of one slot and C moves 16 bytes a lane, 64
// contiguous bytes a row. h enters as hi + lo: for ranks up to 16 both lie in
// one MFMA's k (RC = 2: hi hi lo lo, RC = 1: hi lo and two zeros, in pieces of 8),
// beyond, each piece of 32 ranks of B meets hi and lo in turn.
template <int RC, int MT>
__global__ __launch_bounds__(kLoraThreads) void lora_up_kernel(LoraParams p) {
  constexpr int F = RC < 4 ? 1 : RC / 4, P = RC < 4 ? 1 : 2;
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, q = lane / 16, m16 = lane % 16;
  const int b = p.block0 + blockIdx.x / p.n_splits, sp = blockIdx.x % p.n_splits;
  const int g = p.groups[b];
  if ((uint32_t)g >= (uint32_t)p.G) return;
  const int row0 = blockIdx.y * MT * 16;
  const float scale = p.scale != nullptr ? p.scale[g] : 1.0f;
  const int pieces = p.R / 8;
  u32x4_t hv[MT][F][P];
  uint16_t* cr[MT];
  bool live[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int row = row0 + 16 * m + m16;
    const uint32_t s = row < p.bm ? (uint32_t)p.sorted[(int64_t)b * p.bm + row] : 0xFFFFFFFFu;
    live[m] = s < (uint32_t)p.S;
    cr[m] = p.c + (int64_t)(live[m] ? s : 0) * p.c_ld + 8 * q;
#pragma unroll
    for (int f = 0; f < F; ++f) {
      const int piece = RC >= 4 ? 4 * f + q : RC == 2 ? q % 2 : 0;
      const bool in = live[m] && piece < pieces && (RC != 1 || q < 2);
      float h[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if (in) {
        lora_h8(p, s, piece, h);
        if (p.h != nullptr && p.h != p.part && sp == 0 && wave == 0 && (RC >= 4 || q < RC)) {
          f32x4_t* to = reinterpret_cast<f32x4_t*>(p.h + (int64_t)s * p.R + 8 * piece);
          to[0] = f32x4_t{h[0], h[1], h[2], h[3]};
          to[1] = f32x4_t{h[4], h[5], h[6], h[7]};
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t a, c;
        lora_split(h[2 * i] * scale, h[2 * i + 1] * scale, a, c);
        if constexpr (P == 2) {
          hv[m][f][0][i] = a;
          hv[m][f][1][i] = c;
        } else {
          hv[m][0][0][i] = q < RC ? a : c;
        }
      }
    }
  }
  const uint16_t* wr = p.w + (int64_t)g * p.w_g;
  const int chunks = (p.N + 63) / 64, per = (chunks + p.n_splits - 1) / p.n_splits;
  const int end = min(chunks, (sp + 1) * per);
  for (int i = sp * per + wave; i < end; i += 4) {
    const int n0 = 64 * i;
    u32x4_t cv[MT][2], wv[4][F];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        cv[m][e] = live[m] && n0 + 32 * e + 8 * q < p.N ? *reinterpret_cast<const u32x4_t*>(cr[m] + n0 + 32 * e)
                                                        : u32x4_t{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + 32 * (j / 2) + 8 * (m16 / 4) + 4 * (j % 2) + m16 % 4;
#pragma unroll
      for (int f = 0; f < F; ++f) {
        const int piece = RC >= 4 ? 4 * f + q : RC == 2 ? q % 2 : 0;
        const bool in = n < p.N && piece < pieces && (RC != 1 || q < 2);
        wv[j][f] = in ? *reinterpret_cast<const u32x4_t*>(wr + (int64_t)n * p.w_ld + 8 * piece) : u32x4_t{0, 0, 0, 0};
      }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        f32x4_t d[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          d[j] = f32x4_t{0, 0, 0, 0};
#pragma unroll
          for (int f = 0; f < F; ++f)
#pragma unroll
            for (int k = 0; k < P; ++k) d[j] = lora_mfma(wv[2 * e + j][f], hv[m][f][k], d[j]);
        }
        u32x4_t o;
#pragma unroll
        for (int w = 0; w < 4; ++w)
          o[w] = lora_pack(__uint_as_float(cv[m][e][w] << 16) + d[w / 2][2 * (w % 2)],
                           __uint_as_float(cv[m][e][w] & 0xffff0000u) + d[w / 2][2 * (w % 2) + 1]);
        if (live[m] && n0 + 32 * e + 8 * q < p.N) *reinterpret_cast<u32x4_t*>(cr[m] + n0 + 32 * e) = o;
      }
  }
}

// ------------------------------------------------------------------ launch

// Parts of K: enough workgroups for the chip, at least 256 columns each.
int lora_k_splits(int64_t max_blocks, int64_t k) {
  const int64_t want = (1024 + max_blocks - 1) / (max_blocks > 0 ? max_blocks : 1);
  const int64_t most = k / 256 > 1 ? k / 256 : 1;
  const int64_t n = want < most ? want : most;
  return (int)(n < 8 ? n : 8);
}

static int lora_n_splits(int64_t max_blocks, int64_t n) {
  const int64_t want = (1024 + max_blocks - 1) / (max_blocks > 0 ? max_blocks : 1);
  const int64_t most = (n + 255) / 256;
  return (int)(want < most ? want : most);
}

// Row tiles of 16 slots a workgroup takes, and workgroups a block.
template <int RC, class F>
static hipError_t lora_rows(int bm, F f) {
  if (bm <= 16) return f(std::integral_constant<int, 1>{}, 1);
  if (bm == 32 || RC == 16) return f(std::integral_constant<int, 2>{}, bm / 32);
  if constexpr (RC < 16) return f(std::integral_constant<int, 4>{}, 1);
  return hipErrorInvalidValue;
}

// Launches over all blocks, at most kLoraMaxGrid workgroups at a time (a grid
// holds fewer than 2^32 threads).
constexpr int64_t kLoraMaxGrid = 1 << 22;

template <class F>
static hipError_t lora_blocks(LoraParams p, int per_block, F launch) {
  const int64_t per = kLoraMaxGrid / per_block;
  for (int64_t b = 0; b < p.max_blocks; b += per) {
    p.block0 = (int32_t)b;
    launch(p, (uint32_t)((p.max_blocks - b < per ? p.max_blocks - b : per) * per_block));
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

hipError_t launch_lora_down(const LoraParams& p, hipStream_t stream) {
  return lora_rank(p.R, [&](auto rank) {
    constexpr int RC = decltype(rank)::value;
    return lora_rows<RC>(p.bm, [&](auto mt, int y) {
      return lora_blocks(p, p.splits, [&](const LoraParams& q, uint32_t grid) {
        hipLaunchKernelGGL((lora_down_kernel<(RC + 1) / 2, decltype(mt)::value>), dim3(grid, y), dim3(kLoraThreads), 0,
                           stream, q);
      });
    });
  });
}

hipError_t launch_lora_up(const LoraParams& p0, hipStream_t stream) {
  LoraParams p = p0;
  p.n_splits = lora_n_splits(p.max_blocks, p.N);
  return lora_rank(p.R, [&](auto rank) {
    constexpr int RC = decltype(rank)::value;
    return lora_rows<RC>(p.bm, [&](auto mt, int y) {
      return lora_blocks(p, p.n_splits, [&](const LoraParams& q, uint32_t grid) {
        hipLaunchKernelGGL((lora_up_kernel<RC, decltype(mt)::value>), dim3(grid, y), dim3(kLoraThreads), 0, stream, q);
      });
    });
  });
}

}  // namespace moe
