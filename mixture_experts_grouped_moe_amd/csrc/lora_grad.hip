// moe_lora_backward beside the two kernels of lora.hip, which form dh = B^T dy
// and dx += A^T dh from transposed adapters: the transposes, and the adapters'
// gradients dA[g] = sum dh^T x, dB[g] = sum dy^T h over a group's slots.
//
// HBM-bound: x and dy are read once; a group's slots are cut into segments so
// that few groups fill the chip, whose partial sums a last launch adds in order
// (no atomics: equal bits every time). A group of one segment writes its
// gradient directly.
#include <type_traits>

#include "lora_util.h"

namespace moe {

constexpr int kLgCols = 256;   // columns of x or dy a workgroup takes
constexpr int kLgSlots = 32;   // slots a step
constexpr int kLgMaxGroups = 1024;
constexpr int kLgSegInts = 5;  // group, first block, end, partial slot (-1: none), segments of the group (0: not its first)

// ---------------------------------------------------------------- prepare

// Workgroups 1, 2, ... transpose 32 x 32 tiles of B, then of A; workgroup 0
// writes the segments: table[0] their number, then kLgSegInts each. Segments
// hold seg_blocks blocks (a group's last one fewer), groups ascending.
__global__ __launch_bounds__(1024) void lora_prepare_kernel(LoraGradParams p) {
  const int tid = threadIdx.x;
  if (blockIdx.x > 0) {
    __shared__ uint16_t tile[32][33];
    const int tr = (p.R + 31) / 32, tn = (p.N + 31) / 32, tk = (p.K + 31) / 32;
    const int64_t of_b = (int64_t)p.G * tn * tr, all = of_b + (int64_t)p.G * tk * tr;
    const int x = tid % 32, y = tid / 32;
    for (int64_t at = blockIdx.x - 1; at < all; at += gridDim.x - 1) {
      const bool is_a = at >= of_b;
      const int64_t i = is_a ? at - of_b : at;
      const int rows = is_a ? p.R : p.N, cols = is_a ? p.K : p.R;  // of the matrix read
      const int tc = is_a ? tk : tr, per = tr * (is_a ? tk : tn);
      const int g = (int)(i / per), t = (int)(i % per), r0 = t / tc * 32, c0 = t % tc * 32;
      const uint16_t* from = is_a ? p.a + (int64_t)g * p.a_g : p.b + (int64_t)g * p.b_g;
      const int64_t ld = is_a ? p.a_ld : p.b_ld;
      uint16_t* to = (is_a ? p.at : p.bt) + (int64_t)g * rows * cols;
      if (r0 + y < rows && c0 + x < cols) tile[y][x] = from[(int64_t)(r0 + y) * ld + c0 + x];
      __syncthreads();
      if (c0 + y < cols && r0 + x < rows) to[(int64_t)(c0 + y) * rows + r0 + x] = tile[x][y];
      __syncthreads();
    }
    return;
  }
  __shared__ int first[kLgMaxGroups + 1], count[kLgMaxGroups], scan[2][kLgMaxGroups];
  if (tid < p.G) {
    first[tid] = 0;
    count[tid] = 0;
  }
  __syncthreads();
  for (int b = tid; b < p.max_blocks; b += 1024) {
    const int g = p.groups[b];
    if ((uint32_t)g >= (uint32_t)p.G) continue;
    if (b == 0 || p.groups[b - 1] != g) first[g] = b;
  }
  __syncthreads();
  for (int b = tid; b < p.max_blocks; b += 1024) {
    const int g = p.groups[b];
    if ((uint32_t)g >= (uint32_t)p.G) continue;
    if (b + 1 == p.max_blocks || p.groups[b + 1] != g) count[g] = b + 1 > first[g] ? b + 1 - first[g] : 0;
  }
  __syncthreads();
  // segments before each group, and partial slots before it
  const int n = tid < p.G ? count[tid] : 0;
  const int segs = tid < p.G ? (n + p.seg_blocks - 1) / p.seg_blocks : 0;
  const int mine = tid < p.G ? (segs > 1 ? segs : 1) : 0, parts = segs > 1 ? segs : 0;
  scan[0][tid] = mine;
  scan[1][tid] = parts;
  __syncthreads();
  for (int d = 1; d < 1024; d *= 2) {
    const int a = tid >= d ? scan[0][tid - d] : 0, b = tid >= d ? scan[1][tid - d] : 0;
    __syncthreads();
    scan[0][tid] += a;
    scan[1][tid] += b;
    __syncthreads();
  }
  if (tid == 1023) p.table[0] = scan[0][tid] < p.max_segs ? scan[0][tid] : p.max_segs;
  if (tid < p.G) {
    const int at = scan[0][tid] - mine, part = scan[1][tid] - parts;
    for (int i = 0; i < mine; ++i) {
      if (at + i >= p.max_segs || (parts && part + parts > p.max_parts)) break;  // (the sizes allow for every moe_align list)
      int32_t* e = p.table + 1 + (int64_t)(at + i) * kLgSegInts;
      e[0] = tid;
      e[1] = first[tid] + i * p.seg_blocks;
      e[2] = min(first[tid] + (i + 1) * p.seg_blocks, first[tid] + n);
      e[3] = parts ? part + i : -1;
      e[4] = parts && i == 0 ? segs : 0;
    }
  }
}

// ---------------------------------------------------------------- weights

// A slot's 512-byte row of the tile, 16-byte units exchanged so that a
// transposing read (4 slots x 2 units a 16-lane group, slots 8 apart between
// the groups) meets the banks evenly.
__device__ __forceinline__ int lora_swz(int m, int u) { return u ^ ((m % 4) * 4) ^ ((m / 8 % 2) * 2); }

typedef __attribute__((address_space(3))) uint8_t lora_lds_u8;
typedef __attribute__((__vector_size__(4 * sizeof(short)))) short lora_s16x4;

// One segment's terms of 256 columns: D[16 ranks x 16 columns] tiles over 32
// slots a step. The wide operand (x or dy rows) comes to LDS by row and is read
// transposed; the narrow one (dh or h, fp32) is split into two bf16 terms on
// the way and lies transposed. Each wave takes 64 columns of all ranks.
template <int RT>
__global__ __launch_bounds__(kLoraThreads) void lora_wgrad_kernel(LoraGradParams p) {
  constexpr int kNarrowLd = 40;  // slots of a rank, padded: 80 bytes
  __shared__ __attribute__((aligned(16))) uint8_t wide[kLgSlots * kLgCols * 2];
  __shared__ __attribute__((aligned(16))) uint16_t narrow[2][RT * 16][kNarrowLd];
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64, q = lane / 16, m16 = lane % 16;
  if ((int)blockIdx.y >= p.table[0]) return;
  const int32_t* e = p.table + 1 + (int64_t)blockIdx.y * kLgSegInts;
  const int g = e[0], slot = e[3];
  const int64_t pos0 = (int64_t)e[1] * p.bm, pos1 = (int64_t)e[2] * p.bm;
  const int chunks_k = (p.K + kLgCols - 1) / kLgCols;
  const bool of_a = (int)blockIdx.x < chunks_k;
  const int c0 = (of_a ? blockIdx.x : blockIdx.x - chunks_k) * kLgCols;
  const int width = of_a ? p.K : p.N;
  const uint16_t* big = of_a ? p.x : p.dy;
  const int64_t ld = of_a ? p.x_ld : p.dy_ld;
  const float* small = of_a ? p.dh : p.h;
  const int parts = of_a ? p.splits : 1;
  const float scale = p.scale != nullptr ? p.scale[g] : 1.0f;
  f32x4_t acc[RT][4];
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[t][j] = f32x4_t{0, 0, 0, 0};
  const int srow = tid / 8, piece = tid % 8;            // of the wide tile: 4 pieces of 8 columns, 8 apart
  const int nslot = tid % kLgSlots, nr = tid / kLgSlots;  // of the narrow one: ranks 4 nr, + 32, ...
  const lora_lds_u8* base = (const lora_lds_u8*)wide;
  for (int64_t pos = pos0; pos < pos1; pos += kLgSlots) {
    u32x4_t v[4];
    const uint32_t s = pos + srow < pos1 ? (uint32_t)p.sorted[pos + srow] : 0xFFFFFFFFu;
    const bool live = s < (uint32_t)p.S;
    const uint16_t* row = big + (int64_t)(live ? (of_a ? lora_div(s, p.div_magic, p.div_shift) : s) : 0) * ld + c0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = 8 * (piece + 8 * i);
      v[i] = live && c0 + c < width ? *reinterpret_cast<const u32x4_t*>(row + c) : u32x4_t{0, 0, 0, 0};
    }
    const uint32_t ns = pos + nslot < pos1 ? (uint32_t)p.sorted[pos + nslot] : 0xFFFFFFFFu;
    f32x4_t h[(RT + 1) / 2];
#pragma unroll
    for (int i = 0; i < (RT + 1) / 2; ++i) {
      const int r = 4 * nr + 32 * i;
      h[i] = f32x4_t{0, 0, 0, 0};
      if (ns < (uint32_t)p.S && r < p.R)
        for (int k = 0; k < parts; ++k)
          h[i] += *reinterpret_cast<const f32x4_t*>(small + ((int64_t)k * p.S + ns) * p.R + r);
    }
    __syncthreads();  // the last step's reads are done
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<u32x4_t*>(wide + srow * (kLgCols * 2) + 16 * lora_swz(srow, piece + 8 * i)) = v[i];
#pragma unroll
    for (int i = 0; i < (RT + 1) / 2; ++i) {
      const int r = 4 * nr + 32 * i;
      if (r >= RT * 16) continue;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t hi, lo;
        lora_split(h[i][2 * k] * scale, h[i][2 * k + 1] * scale, hi, lo);
        narrow[0][r + 2 * k][nslot] = (uint16_t)hi;
        narrow[0][r + 2 * k + 1][nslot] = (uint16_t)(hi >> 16);
        narrow[1][r + 2 * k][nslot] = (uint16_t)lo;
        narrow[1][r + 2 * k + 1][nslot] = (uint16_t)(lo >> 16);
      }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // column m16 of the tile at 8 slots from 8 q: two transposing reads of 4 slots
      const int col = 64 * wave + 16 * j + 4 * (m16 % 4);
      lora_s16x4 w[2];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int m = 8 * q + 4 * half + m16 / 4;
        w[half] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) lora_s16x4*)(base + m * (kLgCols * 2) + 16 * lora_swz(m, col / 8) +
                                                            2 * (col % 8)));
      }
      u32x4_t wv;
      __builtin_memcpy(&wv, w, 16);
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int k = 0; k < 2; ++k)
          acc[t][j] = lora_mfma(*reinterpret_cast<const u32x4_t*>(&narrow[k][16 * t + m16][8 * q]), wv, acc[t][j]);
    }
  }
  float* out = slot < 0 ? (of_a ? p.da : p.db) : (of_a ? p.da_part : p.db_part);
  out += (int64_t)(slot < 0 ? g : slot) * p.R * width;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int c = c0 + 64 * wave + 16 * j + m16;
    if (c >= width) continue;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int r = 16 * t + 4 * q;
      if (r >= p.R) continue;
      if (of_a) {
#pragma unroll
        for (int i = 0; i < 4; ++i) out[(int64_t)(r + i) * width + c] = acc[t][j][i];
      } else {
        *reinterpret_cast<f32x4_t*>(out + (int64_t)c * p.R + r) = acc[t][j];
      }
    }
  }
}

// The partial sums of groups of several segments, added in order.
__global__ __launch_bounds__(kLoraThreads) void lora_wgrad_join_kernel(LoraGradParams p) {
  if ((int)blockIdx.y >= p.table[0]) return;
  const int32_t* e = p.table + 1 + (int64_t)blockIdx.y * kLgSegInts;
  const int g = e[0], slot = e[3], segs = e[4];
  const int64_t na = (int64_t)p.R * p.K, nb = (int64_t)p.R * p.N;
  for (int64_t i = ((int64_t)blockIdx.x * kLoraThreads + threadIdx.x) * 4; segs > 0 && i < na + nb;
       i += (int64_t)gridDim.x * kLoraThreads * 4) {
    const bool of_a = i < na;
    const int64_t n = of_a ? na : nb, at = of_a ? i : i - na;
    const float* part = (of_a ? p.da_part : p.db_part) + slot * n + at;
    f32x4_t a = {0, 0, 0, 0};
    for (int k = 0; k < segs; ++k, part += n) a += *reinterpret_cast<const f32x4_t*>(part);
    *reinterpret_cast<f32x4_t*>((of_a ? p.da : p.db) + g * n + at) = a;
  }
}

// ------------------------------------------------------------------ launch

LoraGradSizes lora_grad_sizes(int64_t S, int32_t G, int32_t R, int64_t K, int64_t N, int64_t max_blocks) {
  LoraGradSizes z{};
  const int64_t chunks = (K + kLgCols - 1) / kLgCols + (N + kLgCols - 1) / kLgCols;
  // about 512 workgroups in all where few groups would leave the chip idle
  const int64_t want = (512 + chunks - 1) / chunks;
  z.seg_blocks = (int32_t)((max_blocks + want - 1) / want > 1 ? (max_blocks + want - 1) / want : 1);
  z.max_segs = (int32_t)(max_blocks / z.seg_blocks + G);
  // a group of several segments has more than (segments - 1) seg_blocks >= segments / 2 seg_blocks blocks
  z.max_parts = (int32_t)(2 * (max_blocks / z.seg_blocks));
  z.splits = lora_k_splits(max_blocks, N);
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t was = at;
    at += (bytes + 255) / 256 * 256;
    return was;
  };
  z.at = take((int64_t)G * R * K * 2);
  z.bt = take((int64_t)G * R * N * 2);
  z.dh = take((int64_t)z.splits * S * R * 4);
  z.table = take((1 + (int64_t)z.max_segs * kLgSegInts) * 4);
  z.da_part = take((int64_t)z.max_parts * R * K * 4);
  z.db_part = take((int64_t)z.max_parts * R * N * 4);
  z.bytes = at;
  return z;
}

hipError_t launch_lora_grad_prepare(const LoraGradParams& p, hipStream_t stream) {
  const int64_t tr = (p.R + 31) / 32;
  const int64_t tiles = (int64_t)p.G * tr * ((p.N + 31) / 32 + (p.K + 31) / 32);
  hipLaunchKernelGGL(lora_prepare_kernel, dim3((uint32_t)(tiles < 65536 ? tiles : 65536) + 1), dim3(1024), 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_lora_grad_weights(const LoraGradParams& p, hipStream_t stream) {
  const uint32_t chunks = (uint32_t)((p.K + kLgCols - 1) / kLgCols + (p.N + kLgCols - 1) / kLgCols);
  const hipError_t err = lora_rank(p.R, [&](auto rank) {
    constexpr int RT = (decltype(rank)::value + 1) / 2;
    hipLaunchKernelGGL(lora_wgrad_kernel<RT>, dim3(chunks, p.max_segs), dim3(kLoraThreads), 0, stream, p);
    return hipGetLastError();
  });
  if (err != hipSuccess || p.max_parts == 0) return err;
  const int64_t quads = (int64_t)p.R * (p.K + p.N) / 4;
  const int64_t want = (quads + kLoraThreads - 1) / kLoraThreads;
  hipLaunchKernelGGL(lora_wgrad_join_kernel, dim3((uint32_t)(want < 1024 ? want : 1024), p.max_segs),
                     dim3(kLoraThreads), 0, stream, p);
  return hipGetLastError();
}

}  // namespace moe
