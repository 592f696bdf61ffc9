// moe_lora: low-rank adapters beside a shared projection, C[s] += scale[g]
// B[g] (A[g] x[s / div]) over the slots s of every group g, routed by
// moe_align's block list. Its `up` also adds the input gradient of
// moe_lora_backward, dx[s] += A[g]^T dh[s].
//
// HBM-bound: x is read once, C read and written once, and a group's adapter is
// shared by its blocks through the caches; the products are 2 R flops a byte.
// Every output column needs the whole of h = A x, so `down` forms h, a block of
// slots and a part of K a workgroup, and `up` adds B h. h lies by place in the
// block list; `up` takes it scaled, as `down` writes it where K is not split and
// `join` leaves it over the first part where it is; with few slots a small `up`
// reads the parts, two launches in all, or one (`both`). The second product
// takes h as three bf16 terms, all of its bits (lora_split).
//
// Measured (kernel times): 8192 slots of 8 groups, K = 7168, N = 4096, rank 32:
// `down` 31 us (3.8 TB/s: a group's A is read again by each block, beside the
// rows), `join` 4.8, `up` 34 (3.7 TB/s). 32768 slots of 128 groups, four to a row
// of 2880, N = 5760, rank 16: `down` 36 (5.5 TB/s), `up` 156 (730 MB, 4.7 TB/s, what
// the rows alone read and written back reach). 28 slots of 16 groups, K = 2048,
// N = 1856, rank 16: 6.8, latency: ids, then rows and A, then the stores.
#include <type_traits>

#include "lora_util.h"

namespace moe {

// ------------------------------------------------------------------- down

// D rows are ranks, columns slots: a lane then holds 4 consecutive ranks of a
// slot, one 16-byte store. The waves take K in turn, whole cache lines of x at a
// time, operands straight from memory in MFMA layout, the next ones on their way
// during the products, and add their sums through LDS, into wave 0's. Loads are
// not masked: a place without a slot reads the block's first row, a rank past R
// the last one, and their rows and columns of D are not stored. `slot`: of each
// tile's place m16; part `sp` of `splits` of K.
template <int W, int RT, int MT>
__device__ __forceinline__ void lora_down(const LoraParams& p, int g, const uint32_t (&slot)[MT],
                                          const bool (&live)[MT], uint32_t spare, int sp, int splits,
                                          f32x4_t (&red)[W / 2][RT * MT][64], f32x4_t (&acc)[RT][MT]) {
  constexpr int U = RT + MT <= 2 ? 4 : RT >= 4 ? 1 : 2;  // steps of 32 columns of a turn
  constexpr int kTurn = 32 * U;
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, q = lane / 16, m16 = lane % 16;
  const uint16_t* xr[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
    xr[m] = p.x + (int64_t)lora_div(live[m] ? slot[m] : spare, p.div_magic, p.div_shift) * p.x_ld + 8 * q;
  const uint16_t* wr[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t)
    wr[t] = p.w + (int64_t)g * p.w_g + (int64_t)min(16 * t + m16, p.R - 1) * p.w_ld + 8 * q;
  #pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[t][m] = f32x4_t{0, 0, 0, 0};
  struct Turn {
    u32x4_t x[U][MT], w[U][RT];
  };
  auto load = [&](Turn& v, int turn) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = kTurn * turn + 32 * u;
#pragma unroll
      for (int m = 0; m < MT; ++m) v.x[u][m] = *reinterpret_cast<const u32x4_t*>(xr[m] + k);
#pragma unroll
      for (int t = 0; t < RT; ++t) v.w[u][t] = *reinterpret_cast<const u32x4_t*>(wr[t] + k);
    }
  };
  auto add = [&](const Turn& v) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[t][m] = lora_mfma(v.w[u][t], v.x[u][m], acc[t][m]);
  };
  const int turns = p.K / kTurn, per = (turns + splits - 1) / splits;
  const int end = min(turns, (sp + 1) * per);
  Turn v, next;
  int i = sp * per + wave;
  if (i < end) load(v, i);
  for (; i + W < end; i += 2 * W) {
    load(next, i + W);
    add(v);
    if (i + 2 * W < end) load(v, i + 2 * W);
    add(next);
  }
  if (i < end) add(v);
  if (kTurn * turns < p.K && sp == splits - 1 && wave == 0) {  // the columns behind the last whole turn
    Turn z = {};
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = kTurn * turns + 32 * u;
      if (k + 8 * q >= p.K) continue;
#pragma unroll
      for (int m = 0; m < MT; ++m) z.x[u][m] = *reinterpret_cast<const u32x4_t*>(xr[m] + k);
#pragma unroll
      for (int t = 0; t < RT; ++t) z.w[u][t] = *reinterpret_cast<const u32x4_t*>(wr[t] + k);
    }
    add(z);
  }
  // the waves' sums: the upper half's into the lower half's, and so on
#pragma unroll
  for (int half = W / 2; half > 0; half /= 2) {
    if (wave >= half && wave < 2 * half)
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int m = 0; m < MT; ++m) red[wave - half][t * MT + m][lane] = acc[t][m];
    __syncthreads();
    if (wave < half)
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[t][m] += red[wave][t * MT + m][lane];
    if (half > 1) __syncthreads();
  }
}

template <int RT, int MT>
__global__ __launch_bounds__(kLoraThreads) void lora_down_kernel(LoraParams p) {
  __shared__ f32x4_t red[2][RT * MT][64];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, q = lane / 16, m16 = lane % 16;
  const int b = p.block0 + blockIdx.x / p.splits, sp = blockIdx.x % p.splits;
  const int g = p.groups[b];
  const int row0 = blockIdx.y * MT * 16;
  const int32_t* ids = p.sorted + (int64_t)b * p.bm;
  const uint32_t first = (uint32_t)ids[0];
  uint32_t slot[MT];
  bool live[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) slot[m] = (uint32_t)ids[min(row0 + 16 * m + m16, p.bm - 1)];
  if ((uint32_t)g >= (uint32_t)p.G) return;
#pragma unroll
  for (int m = 0; m < MT; ++m) live[m] = row0 + 16 * m + m16 < p.bm && slot[m] < (uint32_t)p.S;
  f32x4_t acc[RT][MT];
  lora_down<4, RT, MT>(p, g, slot, live, first < (uint32_t)p.S ? first : 0, sp, p.splits, red, acc);
  if (wave > 0) return;
  const float scale = p.scaled && p.scale != nullptr ? p.scale[g] : 1.0f;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    if (!live[m]) continue;
    const int64_t pos = (int64_t)b * p.bm + row0 + 16 * m + m16;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int r = 16 * t + 4 * q;
      if (r >= p.R) continue;
      *reinterpret_cast<f32x4_t*>(p.part + ((int64_t)sp * p.max_blocks * p.bm + pos) * p.R + r) = acc[t][m] * scale;
      if (p.scaled && p.h != nullptr) *reinterpret_cast<f32x4_t*>(p.h + (int64_t)slot[m] * p.R + r) = acc[t][m];
    }
  }
}

// Several parts -> h where it is wanted, and scaled over the first part.
__global__ __launch_bounds__(kLoraThreads) void lora_join_kernel(LoraParams p) {
  const int64_t places = (int64_t)p.max_blocks * p.bm, n = places * (p.R / 4);
  for (int64_t i = (int64_t)blockIdx.x * kLoraThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kLoraThreads) {
    const int64_t pos = i / (p.R / 4);
    const int r = (int)(i % (p.R / 4)) * 4;
    const int g = p.groups[pos / p.bm];
    const uint32_t s = (uint32_t)p.sorted[pos];
    if ((uint32_t)g >= (uint32_t)p.G || s >= (uint32_t)p.S) continue;
    const float scale = p.scale != nullptr ? p.scale[g] : 1.0f;
    float* at = p.part + pos * p.R + r;
    const f32x4_t h = lora_sum_parts(at, places * p.R, p.splits);
    *reinterpret_cast<f32x4_t*>(at) = h * scale;
    if (p.h != nullptr) *reinterpret_cast<f32x4_t*>(p.h + (int64_t)s * p.R + r) = h;
  }
}

// ------------------------------------------------------ up, with few slots

// D rows are columns of C, D columns slots. Row i of tile j stands for column
// 32 (j / 2) + 8 (i / 4) + 4 (j % 2) + i % 4 of a 64-column piece, so that a lane
// holds twice 8 consecutive columns of one slot: one tile of 16 slots then
// spreads over four times the waves that `up` would use. h enters as there.
// Loads are not masked, as in `down`. (The first piece of C and B is on its way
// while h is made.)
template <int RC>
struct LoraFew {
  static constexpr int F = RC < 4 ? 1 : RC / 4, P = RC < 4 ? RC : 3;
  static constexpr int kRank = RC < 4 ? 16 : 8 * RC, kLd = kRank + 8;  // of a slot's row of h in LDS
  u32x4_t c[2], w[4][F];
  uint16_t* row;
  const uint16_t* matrix;
  int lane, q, m16;
  bool live;

  __device__ __forceinline__ LoraFew(const LoraParams& p, int g, uint32_t slot, bool live_, uint32_t spare)
      : live(live_) {
    lane = threadIdx.x % 64;
    q = lane / 16;
    m16 = lane % 16;
    row = p.c + (int64_t)(live ? slot : spare) * p.c_ld;
    matrix = p.w2 + (int64_t)g * p.w2_g;
  }
  __device__ __forceinline__ void load(const LoraParams& p, int i) {
    const int n0 = 64 * i, pieces = p.R / 8;
#pragma unroll
    for (int e = 0; e < 2; ++e) c[e] = *reinterpret_cast<const u32x4_t*>(row + min(n0 + 32 * e + 8 * q, p.N - 8));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = min(n0 + 32 * (j / 2) + 8 * (m16 / 4) + 4 * (j % 2) + m16 % 4, p.N - 1);
#pragma unroll
      for (int f = 0; f < F; ++f) {
        const int piece = RC >= 4 ? 4 * f + q : RC == 2 ? q % 2 : 0;
        const bool in = piece < pieces && (RC != 1 || q < 3);
        const u32x4_t v = *reinterpret_cast<const u32x4_t*>(matrix + (int64_t)n * p.w2_ld + (in ? 8 * piece : 0));
        w[j][f] = in ? v : u32x4_t{0, 0, 0, 0};
      }
    }
  }
  // Four ranks of a place to LDS.
  __device__ __forceinline__ static void put(uint16_t (&hs)[3][16][kLd], int place, int r, f32x4_t h) {
    uint32_t a[3], b[3];
    lora_split(h[0], h[1], a);
    lora_split(h[2], h[3], b);
#pragma unroll
    for (int k = 0; k < 3; ++k) *reinterpret_cast<u32x2_t*>(&hs[k][place][r]) = u32x2_t{a[k], b[k]};
  }
  // Adds the pieces i, i + step, ... below end, the first of which is loaded.
  __device__ __forceinline__ void add(const LoraParams& p, uint16_t (&hs)[3][16][kLd], int i, int step, int end) {
    u32x4_t h[F][P];
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
      for (int k = 0; k < P; ++k) {
        const int piece = RC >= 4 ? 4 * f + q : RC == 2 ? q % 2 : 0;
        const int term = RC >= 4 ? 2 - k : RC == 2 ? (k == 0 ? 2 : q / 2) : min(q, 2);
        h[f][k] = *reinterpret_cast<const u32x4_t*>(&hs[term][m16][8 * piece]);
        if ((RC == 1 && q == 3) || (RC == 2 && k == 0 && q >= 2)) h[f][k] = u32x4_t{0, 0, 0, 0};
      }
    for (; i < end; i += step) {
      const int n0 = 64 * i;
      f32x4_t d[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        d[j] = f32x4_t{0, 0, 0, 0};
#pragma unroll
        for (int f = 0; f < F; ++f)
#pragma unroll
          for (int k = 0; k < P; ++k) d[j] = lora_mfma(w[j][f], h[f][k], d[j]);
      }
      const u32x4_t now[2] = {c[0], c[1]};
      if (i + step < end) load(p, i + step);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        u32x4_t o;
#pragma unroll
        for (int v = 0; v < 4; ++v)
          o[v] = lora_pack(__uint_as_float(now[e][v] << 16) + d[2 * e + v / 2][2 * (v % 2)],
                           __uint_as_float(now[e][v] & 0xffff0000u) + d[2 * e + v / 2][2 * (v % 2) + 1]);
        const int n = n0 + 32 * e + 8 * q;
        if (live && n < p.N) *reinterpret_cast<u32x4_t*>(row + n) = o;
      }
    }
  }
};

// From the parts of h.
template <int RC>
__global__ __launch_bounds__(kLoraThreads) void lora_up_few_kernel(LoraParams p) {
  using Few = LoraFew<RC>;
  __shared__ __attribute__((aligned(16))) uint16_t hs[3][16][Few::kLd];
  const int wave = threadIdx.x / 64, m16 = threadIdx.x % 16;
  const int b = blockIdx.x / p.n_splits, sp = blockIdx.x % p.n_splits;
  const int g = p.groups[b];
  const int row0 = blockIdx.y * 16, rows = min(16, p.bm - row0);
  const int64_t pos0 = (int64_t)b * p.bm + row0;
  const int32_t* ids = p.sorted + pos0;
  const uint32_t slot = (uint32_t)ids[min(m16, rows - 1)], first = (uint32_t)p.sorted[(int64_t)b * p.bm];
  if ((uint32_t)g >= (uint32_t)p.G) return;
  Few few(p, g, slot, m16 < rows && slot < (uint32_t)p.S, first < (uint32_t)p.S ? first : 0);
  const int chunks = (p.N + 63) / 64, per = (chunks + p.n_splits - 1) / p.n_splits;
  const int end = min(chunks, (sp + 1) * per), i = sp * per + wave;
  if (i < end) few.load(p, i);
  const float scale = p.scale != nullptr ? p.scale[g] : 1.0f;
  for (int t = threadIdx.x; t < 16 * (Few::kRank / 4); t += kLoraThreads) {  // four ranks a thread
    const int row = t / (Few::kRank / 4), r = t % (Few::kRank / 4) * 4;
    const uint32_t s = row < rows ? (uint32_t)ids[row] : 0xFFFFFFFFu;
    f32x4_t h = {0, 0, 0, 0};
    if (s < (uint32_t)p.S && r < p.R) {
      h = lora_sum_parts(p.part + (pos0 + row) * p.R + r, (int64_t)p.max_blocks * p.bm * p.R, p.splits);
      if (p.h != nullptr && sp == 0) *reinterpret_cast<f32x4_t*>(p.h + (int64_t)s * p.R + r) = h;
    }
    Few::put(hs, row, r, h * scale);
  }
  __syncthreads();
  few.add(p, hs, i, 4, end);
}

// Both products in one launch: every workgroup of a tile forms its h, by 8 waves
// over K, and adds to its part of N.
template <int RC>
__global__ __launch_bounds__(512) void lora_both_kernel(LoraParams p) {
  using Few = LoraFew<RC>;
  constexpr int RT = (RC + 1) / 2;
  __shared__ f32x4_t red[4][RT][64];
  __shared__ __attribute__((aligned(16))) uint16_t hs[3][16][Few::kLd];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, q = lane / 16, m16 = lane % 16;
  const int b = blockIdx.x / p.n_splits, sp = blockIdx.x % p.n_splits;
  const int g = p.groups[b];
  const int row0 = blockIdx.y * 16, rows = min(16, p.bm - row0);
  const int32_t* ids = p.sorted + (int64_t)b * p.bm + row0;
  const uint32_t slot[1] = {(uint32_t)ids[min(m16, rows - 1)]}, first = (uint32_t)p.sorted[(int64_t)b * p.bm];
  if ((uint32_t)g >= (uint32_t)p.G) return;
  const bool live[1] = {m16 < rows && slot[0] < (uint32_t)p.S};
  const uint32_t spare = first < (uint32_t)p.S ? first : 0;
  Few few(p, g, slot[0], live[0], spare);
  const int chunks = (p.N + 63) / 64, per = (chunks + p.n_splits - 1) / p.n_splits;
  const int end = min(chunks, (sp + 1) * per), i = sp * per + wave;
  if (i < end) few.load(p, i);
  f32x4_t acc[RT][1];
  lora_down<8, RT, 1>(p, g, slot, live, spare, 0, 1, red, acc);
  if (wave == 0) {
    const float scale = p.scale != nullptr ? p.scale[g] : 1.0f;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int r = 16 * t + 4 * q;
      const bool in = live[0] && r < p.R;
      if (in && p.h != nullptr && sp == 0)
        *reinterpret_cast<f32x4_t*>(p.h + (int64_t)slot[0] * p.R + r) = acc[t][0];
      Few::put(hs, m16, r, in ? acc[t][0] * scale : f32x4_t{0, 0, 0, 0});
    }
  }
  __syncthreads();
  few.add(p, hs, i, 8, end);
}

// --------------------------------------------------------------------- up

// Waves per SIMD: three up to rank 16 (32768 slots of 128 groups, 5760 columns:
// 188 us for the whole call, 208 at two; with the parts' sums its registers do not
// suffice), two up to 64 (8192 slots of 8 groups, 4096 columns, rank 32: 69 us, 78
// at three).
constexpr int lora_up_waves(int RC, bool parts) { return RC == 1 || (RC == 2 && !parts) ? 3 : RC <= 8 ? 2 : 1; }

// A wave keeps 16 NT columns of a group's B in registers and takes the run's
// slots 16 at a time, ids two tiles ahead, C and h one ahead. D rows are slots,
// columns those of C: column m of tile j stands for column NT m + j, so that a
// lane holds NT consecutive columns of 4 slots and an access of C is 256
// contiguous bytes of 4 rows (28672 gathered rows of 5760, read and written back
// with no product: 4.7 TB/s so, 4.1 to 4.4 in 64-byte pieces of 16 rows). Every
// wave splits h: each piece of 32 ranks of B meets the three terms in turn, the
// smallest first; up to 16 ranks an MFMA's k of 32 holds several (RC = 2: the
// third term and zeros, then the first and the second; RC = 1: all three and
// zeros, in pieces of 8). PARTS: h comes from its parts, added and scaled by every
// wave. TURNED: the matrix is [R][N] (dx, whose
// matrix is A itself): a lane reads its 8 columns of each of 8 ranks and turns
// the 8 x 8 around in registers.
template <int RC, bool TURNED, bool PARTS>
__global__ __launch_bounds__(kLoraThreads, lora_up_waves(RC, PARTS)) void lora_up_kernel(LoraParams p) {
  constexpr int F = RC < 4 ? 1 : RC / 4, P = RC < 4 ? RC : 3;
  constexpr int NT = 8, kCols = 16 * NT;
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, q = lane / 16, m16 = lane % 16;
  const int run = blockIdx.x / p.n_splits, n0 = (blockIdx.x % p.n_splits * 4 + wave) * kCols;
  if (n0 >= p.N) return;
  const int shift = p.bm <= 16 ? 0 : p.bm / 32;  // log2 of a block's tiles (1, 2 or 4)
  const int t0 = run * p.run_tiles;                  // below 2^31 (as max_blocks * bm)
  const int tiles = min(p.run_tiles, (p.max_blocks << shift) - t0);
  const bool in = n0 + NT * m16 < p.N;
  const int pieces = p.R / 8;

  // Loads are not masked: a place without a slot reads the block's first row, a
  // column past N the last ones; what comes of them is not stored. (A tile of a
  // block without a group is passed over.)
  const int col = n0 + NT * m16 < p.N ? n0 + NT * m16 : p.N - NT;
  uint16_t* c0 = p.c + col;
  struct Ids {
    int slot[4], first, group;
  };
  struct Tile {
    u32x4_t c[4];
    f32x4_t h[F][2];  // 8 ranks of place m16
    int to[4];  // the rows' slots; -1: not stored
    int group;
  };
  auto load_ids = [&](Ids& v, int t) {
    const int b = (t0 + t) >> shift, row = 16 * ((t0 + t) & ((1 << shift) - 1)) + 4 * q;
    const int32_t* at = p.sorted + (int64_t)b * p.bm;
    v.group = p.groups[b];
    v.first = at[0];
    __builtin_memcpy(v.slot, at + (row < p.bm ? row : 0), 16);
  };
  auto load = [&](Tile& v, const Ids& ids, int t) {
    const int row = 16 * ((t0 + t) & ((1 << shift) - 1));
    v.group = __builtin_amdgcn_readfirstlane(ids.group);
    if ((uint32_t)v.group >= (uint32_t)p.G) return;
    const int first = (uint32_t)ids.first < (uint32_t)p.S ? ids.first : 0;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const bool live = row + 4 * q < p.bm && (uint32_t)ids.slot[r] < (uint32_t)p.S;
      v.to[r] = live && in ? ids.slot[r] : -1;
      v.c[r] = *reinterpret_cast<const u32x4_t*>(c0 + (int64_t)(live ? ids.slot[r] : first) * p.c_ld);
    }
    const int64_t pos = (int64_t)((t0 + t) >> shift) * p.bm + min(row + m16, p.bm - 1);
    const float scale = PARTS && p.scale != nullptr ? p.scale[v.group] : 1.0f;
#pragma unroll
    for (int f = 0; f < F; ++f) {
      const int piece = RC >= 4 ? 4 * f + q : RC == 2 ? q % 2 : 0;
      const bool here = piece < pieces;
      const float* at = p.part + pos * p.R + (here ? 8 * piece : 0);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        f32x4_t h;
        if constexpr (PARTS)
          h = lora_sum_parts(at + 4 * e, (int64_t)p.max_blocks * p.bm * p.R, p.splits) * scale;
        else
          h = *reinterpret_cast<const f32x4_t*>(at + 4 * e);
        v.h[f][e] = here ? h : f32x4_t{0, 0, 0, 0};
      }
    }
  };
  u32x4_t wv[NT][F];
  int have = -1;  // the group whose B is here
  auto matrix = [&](int group) {
    if (group != have && (uint32_t)group < (uint32_t)p.G) {
      have = group;
      const uint16_t* wr = p.w2 + (int64_t)have * p.w2_g;
#pragma unroll
      for (int f = 0; f < F; ++f) {
        const int piece = RC >= 4 ? 4 * f + q : RC == 2 ? q % 2 : 0;
        const bool here = piece < pieces && (RC != 1 || q < 3);
        u32x4_t w[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const int rank = here ? 8 * piece : 0;
          w[j] = *reinterpret_cast<const u32x4_t*>(TURNED ? wr + (int64_t)(rank + j) * p.w2_ld + col
                                                          : wr + (int64_t)(col + j) * p.w2_ld + rank);
        }
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t b = TURNED ? __builtin_amdgcn_perm(w[2 * e + 1][j / 2], w[2 * e][j / 2],
                                                              j % 2 ? 0x07060302u : 0x05040100u)
                                      : w[j][e];
            wv[j][f][e] = here ? b : 0u;
          }
      }
    }
  };
  auto add = [&](const Tile& v) {
    if ((uint32_t)v.group >= (uint32_t)p.G) return;
    f32x4_t d[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) d[j] = f32x4_t{0, 0, 0, 0};
#pragma unroll
    for (int f = 0; f < F; ++f) {
      u32x4_t t[3], h[P];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t w[3];
        lora_split(v.h[f][e / 2][2 * (e % 2)], v.h[f][e / 2][2 * (e % 2) + 1], w);
#pragma unroll
        for (int k = 0; k < 3; ++k) t[k][e] = w[k];
      }
      const u32x4_t none = {0, 0, 0, 0};
      if constexpr (RC >= 4) {
#pragma unroll
        for (int k = 0; k < 3; ++k) h[k] = t[2 - k];
      } else if constexpr (RC == 2) {
        h[0] = q < 2 ? t[2] : none;
        h[1] = q < 2 ? t[0] : t[1];
      } else {
        h[0] = q == 0 ? t[0] : q == 1 ? t[1] : q == 2 ? t[2] : none;
      }
#pragma unroll
      for (int k = 0; k < P; ++k)
#pragma unroll
        for (int j = 0; j < NT; ++j) d[j] = lora_mfma(h[k], wv[j][f], d[j]);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      u32x4_t o;
#pragma unroll
      for (int w = 0; w < 4; ++w)
        o[w] = lora_pack(__uint_as_float(v.c[r][w] << 16) + d[2 * w][r],
                         __uint_as_float(v.c[r][w] & 0xffff0000u) + d[2 * w + 1][r]);
      if (v.to[r] >= 0) *reinterpret_cast<u32x4_t*>(c0 + (int64_t)v.to[r] * p.c_ld) = o;
    }
  };
  Ids ids;
  Tile v, next;
  load_ids(ids, 0);
  load(v, ids, 0);
  matrix(v.group);
  if (tiles > 1) load_ids(ids, 1);
  for (int t = 0; t < tiles; t += 2) {
    matrix(v.group);
    if (t + 1 < tiles) {
      load(next, ids, t + 1);
      if (t + 2 < tiles) load_ids(ids, t + 2);
    }
    add(v);
    if (t + 1 >= tiles) break;
    matrix(next.group);
    if (t + 2 < tiles) {
      load(v, ids, t + 2);
      if (t + 3 < tiles) load_ids(ids, t + 3);
    }
    add(next);
  }
}

// ------------------------------------------------------------------ launch

// Whether the small `up` serves: up to 64 tiles of 16 slots. (28 slots of 16
// groups, 1856 columns, rank 16: 6.5 us for the whole call, 9.5 through `up`;
// 256 slots of 32 groups, 7168 columns: 13.2, and 14.9 us with `join` and `up`.)
static bool lora_few(int64_t max_blocks, int bm) { return max_blocks * (bm < 16 ? 1 : bm / 16) <= 64; }

// Parts of K: a workgroup for each CU, at least 256 columns and at most 32 parts.
// (8192 slots, 8 groups, K = 7168, rank 32: 69 us for the whole call at 2 parts,
// 76 at 3, 70 at 4, 79 at 1; 7 slots of 7 groups, rank 128: 15 us at 28 parts, 25
// at 8.)
int lora_k_splits(int64_t max_blocks, int64_t k) {
  const int64_t want = (kLoraCUs + max_blocks - 1) / (max_blocks > 0 ? max_blocks : 1);
  const int64_t most = k / 256 > 1 ? k / 256 : 1;
  const int64_t n = want < most ? want : most;
  return (int)(n < 32 ? n : 32);
}

// Whether both products go in one launch: with few slots and up to 64 KB of A,
// which every workgroup of a tile reads. (28 slots of 16 groups, K = 2048, rank
// 16: 6.4 us, 6.5 in two launches, and 8 us of the host's time in place of 12;
// one slot of 2048: 5.8 and 6.3; K = 2880, rank 16: 10.2 and 8.0 us, K = 7168,
// rank 8: 11.5 and 7.5. Past the border, at K R = 36864 to 46080 and ranks 8 to 32,
// one launch saves up to 1.0 us or costs up to 0.5 for one slot, saves up to 0.6 or
// costs up to 2.2 for 28 slots of 16 groups, and costs 0.2 to 5.4 for 200 of 8.)
static bool lora_both(int64_t max_blocks, int bm, int R, int64_t K) {
  return lora_few(max_blocks, bm) && R <= 32 && K * R <= 32768;
}

LoraSizes lora_sizes(int32_t R, int64_t K, int32_t bm, int64_t max_blocks) {
  LoraSizes z{};
  z.both = lora_both(max_blocks, bm, R, K);
  if (z.both) return z;
  z.few = lora_few(max_blocks, bm);
  z.splits = lora_k_splits(max_blocks, K);
  z.bytes = z.splits * max_blocks * bm * R * 4;
  return z;
}

hipError_t launch_lora_down(const LoraParams& p, hipStream_t stream) {
  return lora_rank(p.R, [&](auto rank) {
    constexpr int RT = (decltype(rank)::value + 1) / 2, MOST = RT == 8 ? 2 : 4;
    auto go = [&](auto mt) {
      constexpr int MT = decltype(mt)::value;
      const int y = p.bm <= 16 * MT ? 1 : p.bm / (16 * MT);
      // (a grid holds fewer than 2^32 threads)
      constexpr int64_t kMost = 1 << 21;
      const int64_t blocks = kMost / p.splits;
      LoraParams q = p;
      for (int64_t b = 0; b < p.max_blocks; b += blocks) {
        q.block0 = (int32_t)b;
        const int64_t n = p.max_blocks - b < blocks ? p.max_blocks - b : blocks;
        hipLaunchKernelGGL((lora_down_kernel<RT, MT>), dim3((uint32_t)(n * p.splits), y), dim3(kLoraThreads), 0, stream,
                           q);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
      }
      return hipSuccess;
    };
    if (p.bm <= 16) return go(std::integral_constant<int, 1>{});
    if (p.bm == 32) return go(std::integral_constant<int, 2>{});
    return go(std::integral_constant<int, MOST>{});
  });
}

hipError_t launch_lora_join(const LoraParams& p, hipStream_t stream) {
  const int64_t want = ((int64_t)p.max_blocks * p.bm * (p.R / 4) + kLoraThreads - 1) / kLoraThreads;
  if (want == 0) return hipSuccess;
  hipLaunchKernelGGL(lora_join_kernel, dim3((uint32_t)(want < 4096 ? want : 4096)), dim3(kLoraThreads), 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_lora_up(const LoraParams& p0, bool turned, hipStream_t stream) {
  LoraParams p = p0;
  p.n_splits = (p.N + 511) / 512;
  const int per = p.bm <= 16 ? 1 : p.bm / 16;
  const int64_t tiles = (int64_t)p.max_blocks * per, all = tiles * p.n_splits;  // of 16 slots; and 512 columns
  if (all == 0) return hipSuccess;
  // About 12 workgroups a CU: many more than run at once, so that they end together
  // (32768 slots of 128 groups, 5760 columns: 188 us for the whole call, 190 at 6
  // a CU), of whole blocks, whose slots are one group's (190 with 9 tiles in place
  // of 8). With fewer tiles 4 a workgroup, which reads its columns of B for them,
  // or what gives 512 workgroups (gradients of 1333 slots: 23.6 us, 27.0 at 4
  // tiles; 4096 slots of rank 64: 36 us at 4, 40 at 2).
  const int64_t share = all / (12 * kLoraCUs);
  const int64_t few = all / (2 * kLoraCUs) < 4 ? all / (2 * kLoraCUs) : 4;
  const int64_t run = share >= 8 ? share / per * per : share > 4 ? share : few > 1 ? few : 1;
  p.run_tiles = (int32_t)(run < tiles ? run : tiles);
  // (below 2^16 workgroups: 5 tiles for each of those 12 a CU where runs are short,
  // and a run that is not whole for each of at most 2^15 parts of the columns)
  const int64_t grid = (tiles + p.run_tiles - 1) / p.run_tiles * p.n_splits;
  return lora_rank(p.R, [&](auto rank) {
    constexpr int RC = decltype(rank)::value;
    auto kernel = !turned    ? lora_up_kernel<RC, false, false>
                  : p.scaled ? lora_up_kernel<RC, true, false>
                             : lora_up_kernel<RC, true, true>;
    hipLaunchKernelGGL(kernel, dim3((uint32_t)grid), dim3(kLoraThreads), 0, stream, p);
    return hipGetLastError();
  });
}

// The grid of the kernels for few slots: parts of N of at least `least` columns,
// below 1024 workgroups (lora_few: 64 tiles at most).
template <class F>
static hipError_t lora_few_grid(LoraParams p, int least, F launch) {
  const int y = p.bm <= 16 ? 1 : p.bm / 16;
  const int64_t tiles = (int64_t)p.max_blocks * y, most = (p.N + least - 1) / least;
  const int64_t want = (2 * kLoraCUs + tiles - 1) / (tiles > 0 ? tiles : 1);
  p.n_splits = (int32_t)(want < most ? want : most);
  launch(p, dim3(p.max_blocks * p.n_splits, y));
  return hipGetLastError();
}

hipError_t launch_lora_up_few(const LoraParams& p, hipStream_t stream) {
  return lora_rank(p.R, [&](auto rank) {
    return lora_few_grid(p, 256, [&](const LoraParams& q, dim3 grid) {
      hipLaunchKernelGGL(lora_up_few_kernel<decltype(rank)::value>, grid, dim3(kLoraThreads), 0, stream, q);
    });
  });
}

hipError_t launch_lora_both(const LoraParams& p, hipStream_t stream) {
  return lora_rank(p.R, [&](auto rank) {
    constexpr int RC = decltype(rank)::value < 4 ? decltype(rank)::value : 4;  // (ranks up to 32)
    return lora_few_grid(p, 512, [&](const LoraParams& q, dim3 grid) {
      hipLaunchKernelGGL(lora_both_kernel<RC>, grid, dim3(512), 0, stream, q);
    });
  });
}

}  // namespace moe
