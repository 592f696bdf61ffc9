// Building blocks of the weight-gradient kernels (wgrad.hip over bf16 rows,
// wgrad_mxfp8.hip over MXFP8 rows): the tile and its numbering, the LDS-DMA
// and scalar loads, the wait-and-barrier, the LDS swizzle and the transposing
// operand reads.
#pragma once

#include "common.h"
#include "params.h"

namespace moe {

constexpr int kWgBM = 64;                    // routing block
constexpr int kWgUM = 32;                    // slots per pipeline unit
constexpr int kWgTN = 256;                   // dW rows (N) per tile
constexpr int kWgTK = 256;                   // dW columns (K) per tile
constexpr int kWgGRowB = kWgTN * 2;          // 512 B: a slot's grad piece
constexpr int kWgXRowB = kWgTK * 2;          // 512 B: a slot's x piece
constexpr int kWgGUnitB = kWgUM * kWgGRowB;  // 16 KB
constexpr int kWgXUnitB = kWgUM * kWgXRowB;  // 16 KB
constexpr int kWgMaxExperts = 1024;
constexpr int kWgGroupN = 8;                 // N tiles per group of the tile order
constexpr uint32_t kWgOOB = 0x80000000u;     // buffer offset past x, grad and one expert's dW (each below 2 GB)
constexpr int kWgStoreNT = 2;                // cache-policy bits of the dW stores: non-temporal

typedef __attribute__((address_space(3))) uint8_t wg_lds_u8_t;
typedef __attribute__((__vector_size__(4 * sizeof(short)))) short wg_s16x4_t;

// Physical 16-byte unit of logical unit u in LDS row (slot) m. A
// transposing read covers 4 consecutive slots x 2 consecutive units per
// 16-lane group; XOR-ing the unit with 4 (m % 4) moves the four slots' pieces
// 64 bytes apart, onto distinct banks (rows are 256 or 512 bytes long).
__device__ __forceinline__ int wg_swz(int m, int u) { return u ^ ((m % 4) * 4); }

// 16 bytes per lane from `rsrc` at `voff` into LDS at lds_base + 16 * lane.
__device__ __forceinline__ void wg_dma16(__amdgpu_buffer_rsrc_t rsrc, uint32_t voff, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %1\n\tbuffer_load_dwordx4 %0, %2, 0 offen lds"
               :: "v"(voff), "s"(__builtin_amdgcn_readfirstlane(lds_base)), "s"(rsrc) : "m0");
}

typedef __attribute__((__vector_size__(4 * sizeof(int)))) int wg_i32x4_t;

template <class T>
using wg_const = __attribute__((address_space(4))) T;

// 4 consecutive slot ids through the scalar cache (a read). The load is the
// compiler's, which waits for it where the ids are used: one issued by inline
// asm may have its registers copied or reused before it lands.
__device__ __forceinline__ wg_i32x4_t wg_scalar_ids4(const wg_const<int32_t>* at) {
  return *(const wg_const<wg_i32x4_t>*)at;
}

// Wait until at most N of this wave's vector-memory operations are in
// flight and every LDS and scalar-memory operation is done, then barrier;
// `a` and `b` (ids loaded ahead) are loaded before it.
template <int N>
__device__ __forceinline__ void wg_wait_barrier(wg_i32x4_t& a, wg_i32x4_t& b) {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("s_waitcnt vmcnt(%2) lgkmcnt(0)\n\ts_barrier" : "+s"(a), "+s"(b) : "n"(N) : "memory");
}

// Operand of 8 consecutive slots [m0, m0 + 8) of tile column c0 + lane % 32,
// for the 32-wide MFMA fragment: lane l takes column c0 + l % 32 and slots
// m0 + 8 (l / 32) + i. Built from two transposing reads (slots +0..3, +4..7)
// of an LDS part whose rows are ROWB bytes.
template <int ROWB>
__device__ __forceinline__ bf16x8_t wg_operand(const wg_lds_u8_t* part, int c0, int m0, int lane) {
  const int g = lane / 16, s = lane % 16;
  const int col = c0 + 16 * (g % 2) + 4 * (s % 4);
  const int slot = m0 + 8 * (g / 2) + s / 4;
  bf16x8_t r;
  wg_s16x4_t v[2];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int m = slot + 4 * half;
    const int byte = m * ROWB + wg_swz(m, col / 8) * 16 + (col % 8) * 2;
    v[half] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) wg_s16x4_t*)(part + byte));
  }
  __builtin_memcpy(&r, v, 16);
  return r;
}

// Bytes of a buffer of rows: up to its last row's last element, since a view's
// last row may end with its allocation.
__device__ __forceinline__ int wg_span(int64_t rows, int64_t ld, int64_t width, int bytes) {
  return (int)(uint32_t)(rows > 0 ? ((rows - 1) * ld + width) * bytes : 0);
}

// A tile of dW and its expert's block range.
struct WgTile {
  int e, n0, k0, b0, b1;
};

// ---- expert block ranges in s_start [E + 1]: experts (lo, hi] start at
//      every block b where the expert id changes (lo = previous id, hi = this
//      id, or E for the first sentinel); experts past the last boundary start
//      at max_blocks
template <int THREADS>
__device__ __forceinline__ void wg_block_ranges(const WgradParams& p, int32_t* s_start) {
  const int tid = threadIdx.x;
  for (int e = tid; e <= p.E; e += THREADS) s_start[e] = p.max_blocks;
  __syncthreads();
  for (int b = tid; b < p.max_blocks; b += THREADS) {
    const int cur = p.expert_ids[b];
    const int prev = b > 0 ? p.expert_ids[b - 1] : -1;
    const int hi = (cur < 0 || cur > p.E) ? p.E : cur;
    const int lo = (b == 0 || prev < 0) ? -1 : prev;
    if ((b == 0 || prev != cur) && !(prev < 0 && cur < 0 && b > 0))
      for (int e = lo + 1; e <= hi; ++e) s_start[e] = b;
  }
  __syncthreads();
}

// Tile order: expert-major; within an expert, groups of group_n N tiles
// walked N-fastest then K, so any group_n x (64 / group_n) consecutive
// tiles share a few grad and x slices. XCD x (= hardware id % 8) owns the
// x-th eighth of the sequence, and its G/8 workgroups take consecutive
// tiles of it round by round (G = gridDim.x).
struct WgOrder {
  const WgradParams& p;
  const int32_t* s_start;
  int per_e, total, G, xcd, local, chunk, group_n;
  __device__ __forceinline__ WgOrder(const WgradParams& p_, const int32_t* s, int group = kWgGroupN)
      : p(p_), s_start(s), group_n(group) {
    per_e = p.tiles_n * p.tiles_k;
    total = p.E * per_e;  // below 2^31 (checked by the host API)
    G = gridDim.x;
    xcd = blockIdx.x % 8;
    local = blockIdx.x / 8;
    chunk = (total + 7) / 8;
  }
  // this workgroup's it-th tile, or total past its last
  __device__ __forceinline__ int index(int it) const {
    const int q = it * (G / 8) + local;
    const int T = xcd * chunk + q;
    return (q < chunk && T < total) ? T : total;
  }
  __device__ __forceinline__ WgTile at(int T) const {
    WgTile t;
    t.e = T / per_e;
    const int r = T % per_e;
    const int in_group = group_n * p.tiles_k;
    const int first_n = (r / in_group) * group_n;
    const int gsize = min(p.tiles_n - first_n, group_n);
    t.n0 = (first_n + (r % in_group) % gsize) * kWgTN;
    t.k0 = ((r % in_group) / gsize) * kWgTK;
    t.b0 = __builtin_amdgcn_readfirstlane(s_start[t.e]);
    t.b1 = __builtin_amdgcn_readfirstlane(s_start[t.e + 1]);
    return t;
  }
};

// Tile order for experts of unequal sizes: every XCD takes an eighth of each
// expert's tiles (numbered as in WgOrder), so all XCDs have the same work
// whatever the counts, where WgOrder gives each XCD whole experts. With
// tiles [lo(y), lo(y + 1)), lo(y) = per_e y / 8, the y-th eighth of an expert,
// XCD x takes eighth (x + e) % 8 of expert e, so that 8 consecutive experts
// give it per_e tiles also where 8 does not divide per_e. Its workgroups take
// consecutive tiles of its sequence round by round.
struct WgSplitOrder {
  WgOrder base;
  int per_e, step, xcd, local;
  int total;  // tiles of this XCD
  __device__ __forceinline__ WgSplitOrder(const WgradParams& p, const int32_t* s_start, int group)
      : base(p, s_start, group) {
    per_e = base.per_e;
    step = base.G / 8;
    xcd = base.xcd;
    local = base.local;
    total = p.E / 8 * per_e;
    for (int e = p.E / 8 * 8; e < p.E; ++e) total += lo((xcd + e) % 8 + 1) - lo((xcd + e) % 8);
  }
  __device__ __forceinline__ int lo(int y) const { return (int)((int64_t)per_e * y / 8); }
  // this workgroup's it-th tile of the XCD's sequence, or total past its last
  __device__ __forceinline__ int index(int it) const {
    const int64_t q = (int64_t)it * step + local;
    return q < total ? (int)q : total;
  }
  __device__ __forceinline__ WgTile at(int q) const {
    int e = q / per_e * 8, r = q % per_e;
    for (;; ++e) {
      const int y = (xcd + e) % 8, n = lo(y + 1) - lo(y);
      if (r < n) return base.at(e * per_e + lo(y) + r);
      r -= n;
    }
  }
};

// The division by top_k of the slots' token rows: with l = ceil(log2 d) and
// m = ceil(2^(31+l) / d), floor(s / d) = (s m) >> (31 + l) for every
// s < 2^31 (Granlund and Montgomery, "Division by invariant integers using
// multiplication", 1994, Theorem 4.2 with N = 31).
inline void wg_set_division(WgradParams& p) {
  int l = 0;
  while ((1 << l) < p.top_k) ++l;
  p.topk_magic = (uint32_t)((((uint64_t)1 << (31 + l)) + (uint64_t)p.top_k - 1) / (uint64_t)p.top_k);
  p.topk_shift = 31 + l;
}

}  // namespace moe
