// moe_lora_backward: the adapters' gradients dA[g] = sum dh^T x, dB[g] = scale
// sum dy^T h over a group's slots, and dh = scale B^T dy; dx += A^T dh is the
// `up` of lora.hip.
//
// HBM-bound: x and dy are read once (dh's parts come from the pass over dy that
// forms dB). A group's slots are cut into segments so that few groups fill the
// chip, whose partial sums a last launch adds in order (no atomics: equal bits
// every time); a group of one segment writes its gradient directly.
//
// Measured (kernel times): 32768 slots of 128 groups, K = 2880 (a row serves four),
// N = 5760, rank 16: the table 9 us, dy 104 (383 MB read and 69 written, 4.3 TB/s;
// gathered rows of this width are read at 4.5 to 4.9), h's join 6.8, dx 80 (4.8
// TB/s), x 32 (172 MB moved, 5.4 TB/s), the gradients' join 5.0. 1333 slots of 3 groups,
// 2688 x 1856, rank 8: four launches of 4 to 7 us each, all latency (dx and x,
// which both wait for dy alone, run one after the other).
#include <type_traits>

#include "lora_util.h"

namespace moe {

constexpr int kLgThreads = 512;
// columns of x or dy a workgroup takes: 64 a wave, 32 where all ranks' sums of 64 would not fit its registers
constexpr int lora_wide_cols(int R) { return R > 64 ? 256 : 512; }
constexpr int kLgSlots = 32;   // slots a step
constexpr int kLgMaxGroups = 1024;
constexpr int kLgSegInts = 4;   // group (-1: no segment), first place, end, partial slot (-1: none)
constexpr int kLgJoinInts = 3;  // group of several segments, its first partial slot, their number (0: no group)

// ------------------------------------------------------------------ table

// The segments where they hold several blocks, one workgroup: max_segs entries of kLgSegInts, then for the join
// an entry of kLgJoinInts for each group of several. Segments hold seg_blocks
// blocks (a group's last one fewer, and no places behind its last slot); a group
// without blocks has an empty one, which writes its zeros. Longest segments
// first, so that none is left for the end: by size in kBuckets steps (the order
// inside one, an atomic's, decides nothing but who runs when).
__global__ __launch_bounds__(1024) void lora_table_kernel(LoraGradParams p) {
  constexpr int kBuckets = 64;
  __shared__ int first[kLgMaxGroups], last[kLgMaxGroups], end[kLgMaxGroups], segs[kLgMaxGroups], parts[kLgMaxGroups];
  __shared__ int bucket[kBuckets + 1], joins;
  const int tid = threadIdx.x;
  first[tid] = 0;
  last[tid] = -1;
  end[tid] = 0;
  if (tid <= kBuckets) bucket[tid] = 0;
  if (tid == 0) joins = 0;
  for (int i = tid; i < p.max_segs; i += 1024) p.table[i * kLgSegInts] = -1;
  int32_t* join = p.table + p.max_segs * kLgSegInts;
  for (int i = tid; i < p.max_parts / 2; i += 1024) join[i * kLgJoinInts + 2] = 0;
  __syncthreads();
  for (int b = tid; b < p.max_blocks; b += 1024) {
    const int g = p.groups[b], before = b > 0 ? p.groups[b - 1] : -1;
    const int after = b + 1 < p.max_blocks ? p.groups[b + 1] : -1;
    if ((uint32_t)g >= (uint32_t)p.G) continue;
    if (before != g) first[g] = b;
    if (after != g) last[g] = b;
  }
  __syncthreads();
  // places up to the last slot of a group's last block, bm lanes a group (8 to 64,
  // a power of two); where one turn does not do, the loads of 8 together (128
  // groups: 9.0 us, 12.1 one by one)
  const int shift = __builtin_ctz(p.bm), at = tid & (p.bm - 1), lanes = p.max_blocks > 0 ? p.G * p.bm : 0;
  auto ends_of = [&](auto ahead) {
    constexpr int kAhead = decltype(ahead)::value;
    for (int i = tid; i < (lanes + 63) / 64 * 64; i += kAhead * 1024) {
      uint32_t slot[kAhead];
      bool here[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int g = (i + 1024 * j) >> shift, b = g < p.G ? last[g] : -1;
        here[j] = b >= 0;
        slot[j] = (uint32_t)p.sorted[here[j] ? (int64_t)b * p.bm + at : 0];
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const uint64_t live = __ballot(here[j] && slot[j] < (uint32_t)p.S);
        const uint64_t mine = live >> (tid % 64 - at) & (p.bm == 64 ? ~0ull : (1ull << p.bm) - 1);
        if (here[j] && at == 0) end[(i + 1024 * j) >> shift] = mine != 0 ? 64 - __builtin_clzll(mine) : 0;
      }
    }
  };
  if (lanes <= 1024)
    ends_of(std::integral_constant<int, 1>{});
  else
    ends_of(std::integral_constant<int, 8>{});
  const int n = tid < p.G && last[tid] >= first[tid] ? last[tid] + 1 - first[tid] : 0;
  const int many = (n + p.seg_blocks - 1) / p.seg_blocks, mine = tid < p.G ? (many > 1 ? many : 1) : 0;
  segs[tid] = mine;
  parts[tid] = many > 1 ? many : 0;
  __syncthreads();
  for (int d = 1; d < p.G; d *= 2) {  // running sums over the groups
    const int a = tid >= d ? segs[tid - d] : 0, b = tid >= d ? parts[tid - d] : 0;
    __syncthreads();
    segs[tid] += a;
    parts[tid] += b;
    __syncthreads();
  }
  const int total = min(segs[p.G - 1], p.max_segs);
  // a segment by its number: its group, and which of the group's it is
  auto find = [&](int i, int& g) {
    int lo = 0, hi = p.G - 1;
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (segs[mid] > i) hi = mid; else lo = mid + 1;
    }
    g = lo;
    return i - (lo > 0 ? segs[lo - 1] : 0);
  };
  auto size = [&](int g, int k) {
    const int blocks = last[g] >= first[g] ? last[g] + 1 - first[g] : 0;
    return min(p.seg_blocks, blocks - k * p.seg_blocks);
  };
  auto in = [&](int blocks) { return kBuckets - 1 - (int)((int64_t)blocks * (kBuckets - 1) / p.seg_blocks); };
  for (int i = tid; i < total; i += 1024) {
    int g;
    const int k = find(i, g);
    atomicAdd(&bucket[in(size(g, k)) + 1], 1);
  }
  __syncthreads();
  if (tid < 64) {  // running sums over the buckets
    int v = bucket[tid + 1];
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int a = __shfl_up(v, d);
      if (tid >= d) v += a;
    }
    bucket[tid + 1] = v;
  }
  __syncthreads();
  for (int i = tid; i < total; i += 1024) {
    int g;
    const int k = find(i, g), s = size(g, k), at = atomicAdd(&bucket[in(s)], 1);
    const int of = parts[g] - (g > 0 ? parts[g - 1] : 0), part = parts[g] - of;
    // (the sizes allow for every list of moe_align; of another one, whose groups
    // recur, what does not fit is left out)
    const bool fits = of == 0 || parts[g] <= p.max_parts, ends = (k + 1) * p.seg_blocks >= last[g] + 1 - first[g];
    const int b = first[g] + k * p.seg_blocks;
    int32_t* e = p.table + at * kLgSegInts;
    e[1] = fits && s > 0 ? b * p.bm : 0;
    e[2] = fits && s > 0 ? (ends ? (b + s - 1) * p.bm + end[g] : (b + s) * p.bm) : 0;
    e[3] = of && fits ? part + k : -1;
    e[0] = g;
    if (of && fits && k == 0) {
      const int j = atomicAdd(&joins, 1);
      if (j < p.max_parts / 2) {
        join[j * kLgJoinInts] = g;
        join[j * kLgJoinInts + 1] = part;
        join[j * kLgJoinInts + 2] = of;
      }
    }
  }
}

// Where every block is a segment (max_blocks <= 256: lora_grad_sizes), workgroups
// find theirs themselves: segment i is block i, its partial slot i too where the
// group has another block beside it, and those past max_blocks stand for groups
// without blocks. (1333 slots of 3 groups, 2688 x 1856, rank 8: 24.9 us for the
// whole call, 28.2 with the table; 700 slots of one, 4096 x 4096, rank 64: 44.0 and
// 46.4.) False: no segment.
__device__ __forceinline__ bool lora_segment(const LoraGradParams& p, int i, int& g, int& slot, int64_t& pos0,
                                             int64_t& pos1) {
  if (p.table != nullptr) {
    const int32_t* e = p.table + (int64_t)i * kLgSegInts;
    g = e[0];
    slot = e[3];
    pos0 = e[1];
    pos1 = e[2];
    return g >= 0;
  }
  slot = -1;
  pos0 = pos1 = 0;
  if (i >= p.max_blocks) {
    g = i - p.max_blocks;
    return g < p.G && !__syncthreads_or((int)threadIdx.x < p.max_blocks && p.groups[threadIdx.x] == g);
  }
  g = p.groups[i];
  const int before = i > 0 ? p.groups[i - 1] : -1, after = i + 1 < p.max_blocks ? p.groups[i + 1] : -1;
  const int lane = threadIdx.x % 64;
  pos0 = (int64_t)i * p.bm;
  const uint64_t live = __ballot(lane < p.bm && (uint32_t)p.sorted[pos0 + min(lane, p.bm - 1)] < (uint32_t)p.S);
  pos1 = pos0 + (live != 0 ? 64 - __builtin_clzll(live) : 0);
  if (before == g || after == g) slot = i;
  return (uint32_t)g < (uint32_t)p.G;
}

// ------------------------------------------------------------- x and dy

// A slot's row of the tile lies by 16-byte units, exchanged so that both reads
// meet the banks evenly: the transposing one (4 slots x 2 units a 16-lane group,
// slots 8 apart between the groups) and the one by rows (16 slots x 1 unit).
__device__ __forceinline__ int lora_swz(int m, int u) { return u ^ ((m % 4) * 4) ^ ((m / 8 % 2) * 2) ^ (m / 4 % 2); }

typedef __attribute__((address_space(3))) uint8_t lora_lds_u8;
typedef __attribute__((__vector_size__(4 * sizeof(short)))) short lora_s16x4;

// One segment's terms of 512 (ranks above 64: 256) columns of x (dA) or dy (dB), 32 slots a step.
// The wide operand (rows of x or dy) comes to LDS by row, the next step's on its
// way meanwhile; the narrow one (dh or h, fp32) is split into three bf16 terms,
// all its bits, and lies transposed. dA and dB: D[16 ranks x 16 columns], the
// sum over slots, the wide operand through transposing reads; a wave takes 16
// columns of every 128, at all ranks. dy also gives dh's part of these columns while it is
// here, D[16 ranks x 16 slots], the sum over columns, with B in registers: the
// 2 x RT tiles are dealt out to the 8 waves, in NP parts of the columns (32 of
// every 32 NP) where there are fewer than 8. (Addresses in LDS then differ by
// constants between a wave's tiles.)
template <int RT, bool OF_X>
__global__ __launch_bounds__(kLgThreads, RT == 1 ? 4 : 2) void lora_wide_kernel(LoraGradParams p) {
  constexpr int kLgCols = lora_wide_cols(16 * RT), NC = kLgCols / 128;  // 16-column tiles of a wave
  constexpr int NV = kLgCols / 128;                                     // wide loads a thread
  constexpr int kNarrowLd = 40;  // slots of a rank, padded: 80 bytes
  constexpr int NP = RT >= 4 ? 1 : 4 / RT, ST = RT == 8 ? 2 : 1;  // parts of the columns, slot tiles of a wave
  constexpr int KS = kLgCols / NP / 32;                           // steps of 32 columns of a part
  constexpr int NH = RT * 4 * kLgSlots > kLgThreads ? RT * 4 * kLgSlots / kLgThreads : 1;  // narrow loads a thread
  __shared__ __attribute__((aligned(16))) uint8_t wides[2][kLgSlots * kLgCols * 2];
  __shared__ __attribute__((aligned(16))) uint16_t narrows[2][3][RT * 16][kNarrowLd];
  __shared__ f32x4_t red[OF_X || NP == 1 ? 1 : NP][2 * RT][64];
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64, q = lane / 16, m16 = lane % 16;
  int g, slot;
  int64_t pos0, pos1;
  if (!lora_segment(p, blockIdx.y, g, slot, pos0, pos1)) return;
  const int c0 = blockIdx.x * kLgCols, width = OF_X ? p.K : p.N;
  const uint16_t* big = OF_X ? p.x : p.dy;
  const int64_t ld = OF_X ? p.x_ld : p.dy_ld;
  const float scale = p.scale != nullptr ? p.scale[g] : 1.0f;
  const float narrow_scale = OF_X && p.parts == 0 ? 1.0f : scale;  // (a joined dh is scaled)
  const bool weights = p.da != nullptr;
  f32x4_t acc[RT][NC];
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int j = 0; j < NC; ++j) acc[t][j] = f32x4_t{0, 0, 0, 0};

  const int srow = tid / 16, piece = tid % 16;            // of the wide tile: NV pieces of 8 columns, 16 apart
  const int nslot = tid % kLgSlots, nr = tid / kLgSlots;  // of the narrow one: ranks 4 nr, + 64
  const int rt = wave % RT, st = ST == 2 ? 0 : wave / RT % 2, np = NP == 1 ? 0 : wave / (2 * RT);
  u32x4_t bv[OF_X ? 1 : KS];
  // Loads are not masked: a place without a slot, or past the segment, reads the
  // segment's first row, a column past the width the last ones, and becomes zeros
  // on the way to LDS.
  struct {
    uint32_t wide, narrow;
  } ids;  // of the step after the one in `o`
  struct {
    u32x4_t v[NV];
    f32x4_t h[NH];
    uint32_t live;  // bit 0: the wide row's slot, bit 1: the narrow one's
  } o;  // a step's loads
  const uint32_t first = pos0 < pos1 ? (uint32_t)p.sorted[pos0] : 0;
  const uint32_t spare = first < (uint32_t)p.S ? first : 0;
  const int places = (int)(pos1 - pos0);
  const int32_t* ids_at = p.sorted + pos0;
  auto load_ids = [&](int at) {
    ids.wide = (uint32_t)ids_at[min(at + srow, places - 1)];
    ids.narrow = (uint32_t)ids_at[min(at + nslot, places - 1)];
  };
  const bool whole = c0 + kLgCols <= width;
  const uint16_t* big0 = big + (whole ? c0 + 8 * piece : 0);
  auto load = [&](int at) {
    const bool wide = at + srow < places && ids.wide < (uint32_t)p.S;
    const bool narrow = at + nslot < places && ids.narrow < (uint32_t)p.S;
    o.live = (wide ? 1 : 0) | (narrow ? 2 : 0);
    const uint32_t s = wide ? ids.wide : spare;
    const uint16_t* row = big0 + (int64_t)(OF_X ? lora_div(s, p.div_magic, p.div_shift) : s) * ld;
    if (whole) {
#pragma unroll
      for (int i = 0; i < NV; ++i) o.v[i] = *reinterpret_cast<const u32x4_t*>(row + 128 * i);
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        o.v[i] = *reinterpret_cast<const u32x4_t*>(row + min(c0 + 8 * (piece + 16 * i), width - 8));
    }
    if (!OF_X && !weights) return;
    const float* from = OF_X ? p.dh + (pos0 + min(at + nslot, places - 1)) * p.R
                             : p.h + (int64_t)(narrow ? ids.narrow : spare) * p.R;
#pragma unroll
    for (int i = 0; i < NH; ++i) {
      const float* at_r = from + min(4 * nr + 64 * i, p.R - 4);
      o.h[i] = OF_X && p.parts > 1 ? lora_sum_parts(at_r, (int64_t)p.max_blocks * p.bm * p.R, p.parts)
                                   : *reinterpret_cast<const f32x4_t*>(at_r);
    }
  };
  constexpr int kRowB = kLgCols * 2;
  auto put_dh = [&](int pos, int tile, f32x4_t d) {  // tile = 2 * rank tile + slot tile
    const int at = pos + 16 * (tile % 2) + m16;
    const int r = 16 * (tile / 2) + 4 * q;
    if (at < places && r < p.R)
      *reinterpret_cast<f32x4_t*>(p.dh + ((int64_t)blockIdx.x * p.max_blocks * p.bm + pos0 + at) * p.R + r) = d;
  };
  // A step's tile goes to one of two buffers while slower waves still read the
  // other, so a wave's next loads leave as soon as its last ones are here.
  auto step = [&](int pos, int turn) {
    uint8_t* wide = wides[turn];
    auto& narrow = narrows[turn];
    const lora_lds_u8* base = (const lora_lds_u8*)wide;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      *reinterpret_cast<u32x4_t*>(wide + srow * kRowB + 16 * lora_swz(srow, piece) + 256 * i) =
          (o.live & 1) && (whole || c0 + 8 * (piece + 16 * i) < width) ? o.v[i] : u32x4_t{0, 0, 0, 0};
    if (OF_X || weights) {
#pragma unroll
      for (int i = 0; i < NH; ++i) {
        const int r = 4 * nr + 64 * i;
        if (r >= RT * 16) continue;
        const f32x4_t h = (o.live & 2) && r < p.R ? o.h[i] * narrow_scale : f32x4_t{0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t term[3];
          lora_split(h[2 * k], h[2 * k + 1], term);
#pragma unroll
          for (int j = 0; j < 3; ++j) {
            narrow[j][r + 2 * k][nslot] = (uint16_t)term[j];
            narrow[j][r + 2 * k + 1][nslot] = (uint16_t)(term[j] >> 16);
          }
        }
      }
    }
    if (pos + kLgSlots < places) {
      load(pos + kLgSlots);
      load_ids(pos + 2 * kLgSlots);
    }
    __syncthreads();
    if constexpr (!OF_X) {
      f32x4_t d[ST];
#pragma unroll
      for (int t = 0; t < ST; ++t) d[t] = f32x4_t{0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int t = 0; t < ST; ++t) {
          const int m = 16 * (st + t) + m16, u = 4 * (s % (4 / NP) * NP + np) + q;
          const u32x4_t rows =
              *reinterpret_cast<const u32x4_t*>(wide + m * kRowB + 16 * lora_swz(m, u) + 256 * (s * NP / 4));
          d[t] = lora_mfma(bv[s], rows, d[t]);
        }
#pragma unroll
      for (int t = 0; t < ST; ++t) {
        const int tile = 2 * rt + st + t;
        if constexpr (NP > 1)
          red[np][tile][lane] = d[t];
        else
          put_dh(pos, tile, d[t]);
      }
    }
    if (OF_X || weights) {
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        // column m16 of the tile at 8 slots from 8 q: two transposing reads of 4 slots
        const int col = 16 * wave + 4 * (m16 % 4);
        lora_s16x4 w[2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int m = 8 * q + 4 * half + m16 / 4;
          w[half] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (__attribute__((address_space(3))) lora_s16x4*)(base + m * kRowB + 16 * lora_swz(m, col / 8) +
                                                              2 * (col % 8) + 256 * j));
        }
        u32x4_t wv;
        __builtin_memcpy(&wv, w, 16);
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
          for (int k = 2; k >= 0; --k)
            acc[t][j] = lora_mfma(*reinterpret_cast<const u32x4_t*>(&narrow[k][16 * t + m16][8 * q]), wv, acc[t][j]);
      }
    }
    if (!OF_X && NP > 1) {
      __syncthreads();
      for (int i = wave; i < 2 * RT; i += 8) {
        f32x4_t d = red[0][i][lane];
#pragma unroll
        for (int k = 1; k < NP; ++k) d += red[OF_X ? 0 : k][i][lane];
        put_dh(pos, i, d);
      }
    }
  };
  if (pos0 < pos1) {
    load_ids(0);
    load(0);
    load_ids(kLgSlots);
    // B of this wave's dh tiles, rank tile rt at its part of the columns: rows of
    // 16 ranks of the columns to LDS, where a rank tile after another is read
    // transposed
    if constexpr (!OF_X) {
      constexpr int kRowsB = kLgSlots * kLgCols * 2 / 32;  // columns of B that the tile's LDS holds at 16 ranks: all
      static_assert(kRowsB >= kLgCols, "B's rows fit");
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        if (t > 0) __syncthreads();
        for (int i = tid; i < kLgCols * 2; i += kLgThreads) {  // 16 bytes: 8 ranks of a column
          const int n = min(c0 + i / 2, width - 1), r = 16 * t + 8 * (i % 2);
          const u32x4_t v = *reinterpret_cast<const u32x4_t*>(p.b + (int64_t)g * p.b_g + (int64_t)n * p.b_ld +
                                                              min(r, p.R - 8));
          *reinterpret_cast<u32x4_t*>(wides[1] + 16 * i) = c0 + i / 2 < width && r < p.R ? v : u32x4_t{0, 0, 0, 0};
        }
        __syncthreads();
        if (t != rt) continue;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          lora_s16x4 w[2];
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int n = 128 * (k * NP / 4) + 32 * (k % (4 / NP) * NP + np) + 8 * q + 4 * half + m16 / 4;
            w[half] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) lora_s16x4*)((const lora_lds_u8*)wides[1] + n * 32 + 8 * (m16 % 4)));
          }
          __builtin_memcpy(&bv[k], w, 16);
        }
      }
    }
    for (int pos = 0; pos < places; pos += 2 * kLgSlots) {
      step(pos, 0);
      if (pos + kLgSlots < places) step(pos + kLgSlots, 1);
    }
  }
  if (!weights) return;
  float* out = slot < 0 ? (OF_X ? p.da : p.db) : (OF_X ? p.da_part : p.db_part);
  out += (int64_t)(slot < 0 ? g : slot) * p.R * width;
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const int c = c0 + 128 * j + 16 * wave + m16;
    if (c >= width) continue;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int r = 16 * t + 4 * q;
      if (r >= p.R) continue;
      if constexpr (OF_X) {
#pragma unroll
        for (int i = 0; i < 4; ++i) out[(int64_t)(r + i) * width + c] = acc[t][j][i];
      } else {
        *reinterpret_cast<f32x4_t*>(out + (int64_t)c * p.R + r) = acc[t][j];
      }
    }
  }
}

// The partial sums of groups of several segments, added in order.
__global__ __launch_bounds__(kLoraThreads) void lora_grad_join_kernel(LoraGradParams p) {
  int g, slot, segs;
  if (p.table != nullptr) {
    const int32_t* e = p.table + p.max_segs * kLgSegInts + (int64_t)blockIdx.y * kLgJoinInts;
    g = e[0], slot = e[1], segs = e[2];
  } else {  // a group's first block adds for its blocks (max_blocks <= kLoraThreads)
    __shared__ int stop;
    slot = blockIdx.y;
    if (slot + 1 >= p.max_blocks) return;
    g = p.groups[slot];
    if ((uint32_t)g >= (uint32_t)p.G || p.groups[slot + 1] != g || (slot > 0 && p.groups[slot - 1] == g)) return;
    const int i = threadIdx.x;
    if (i == 0) stop = p.max_blocks;
    __syncthreads();
    if (i > slot && i < p.max_blocks && p.groups[i] != g) atomicMin(&stop, i);
    __syncthreads();
    segs = stop - slot;
  }
  const int64_t na = (int64_t)p.R * p.K, nb = (int64_t)p.R * p.N;
  for (int64_t i = ((int64_t)blockIdx.x * kLoraThreads + threadIdx.x) * 4; segs > 0 && i < na + nb;
       i += (int64_t)gridDim.x * kLoraThreads * 4) {
    const bool of_a = i < na;
    const int64_t n = of_a ? na : nb, at = of_a ? i : i - na;
    const float* part = (of_a ? p.da_part : p.db_part) + slot * n + at;
    *reinterpret_cast<f32x4_t*>((of_a ? p.da : p.db) + g * n + at) = lora_sum_parts(part, n, segs);
  }
}

// ------------------------------------------------------------------ launch

LoraGradSizes lora_grad_sizes(int32_t G, int32_t R, int64_t K, int64_t N, int32_t bm, int64_t max_blocks) {
  LoraGradSizes z{};
  const int64_t cols = lora_wide_cols(R), of_k = (K + cols - 1) / cols, of_n = (N + cols - 1) / cols;
  z.n_parts = (int32_t)of_n;
  // segments for about 512 workgroups over both kernels, where few groups would leave the chip idle (one
  // group of 8192 slots, K = N = 4096: 89 us for the whole call, 120 at 2048 workgroups, whose partial sums cost more)
  const int64_t want = (2 * kLoraCUs + of_k + of_n - 1) / (of_k + of_n);
  const int64_t per = (max_blocks + want - 1) / want;
  z.seg_blocks = (int32_t)(per > 1 ? per : 1);
  z.max_segs = (int32_t)(max_blocks / z.seg_blocks + G);
  // (where a block is a segment, its number is its partial slot; else a group of s > 1 segments has more than
  // (s - 1) seg_blocks blocks, so s <= 2 blocks / seg_blocks)
  z.max_parts = (int32_t)(z.seg_blocks == 1 ? max_blocks : 2 * (max_blocks / z.seg_blocks));
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t was = at;
    at += (bytes + 255) / 256 * 256;
    return was;
  };
  // the join of dh's parts left to the readers, a launch less, where parts and ranks are few (1333 slots of 3 groups,
  // 2688 x 1856, rank 8, 4 parts: 23.7 us for the whole call, 24.9 with the join; rank 16 at 4 parts 17.6 and 19.2, 8
  // parts 20.9 and 20.8, 14 parts 28.5 and 25.3; rank 64 at 6 parts 31.4 and 30.4)
  z.direct = z.seg_blocks == 1 && z.n_parts * R <= 128;
  z.dh = take(z.n_parts * max_blocks * bm * R * 4);
  z.table = take(z.seg_blocks == 1 ? 0 : ((int64_t)z.max_segs * kLgSegInts + z.max_parts / 2 * kLgJoinInts) * 4);
  z.da_part = take((int64_t)z.max_parts * R * K * 4);
  z.db_part = take((int64_t)z.max_parts * R * N * 4);
  z.bytes = at;
  return z;
}

hipError_t launch_lora_grad_table(const LoraGradParams& p, hipStream_t stream) {
  hipLaunchKernelGGL(lora_table_kernel, dim3(1), dim3(1024), 0, stream, p);
  return hipGetLastError();
}

template <bool OF_X>
static hipError_t lora_wide(const LoraGradParams& p, hipStream_t stream) {
  const int cols = lora_wide_cols(p.R);
  return lora_rank(p.R, [&](auto rank) {
    constexpr int RT = (decltype(rank)::value + 1) / 2;
    hipLaunchKernelGGL((lora_wide_kernel<RT, OF_X>), dim3(((OF_X ? p.K : p.N) + cols - 1) / cols, p.max_segs),
                       dim3(kLgThreads), 0, stream, p);
    return hipGetLastError();
  });
}

hipError_t launch_lora_grad_dy(const LoraGradParams& p, hipStream_t stream) { return lora_wide<false>(p, stream); }
hipError_t launch_lora_grad_x(const LoraGradParams& p, hipStream_t stream) { return lora_wide<true>(p, stream); }

hipError_t launch_lora_grad_join(const LoraGradParams& p, hipStream_t stream) {
  if (p.max_parts == 0) return hipSuccess;
  const int64_t quads = (int64_t)p.R * (p.K + p.N) / 4;
  const int64_t want = (quads + kLoraThreads - 1) / kLoraThreads;
  const uint32_t groups = p.table != nullptr ? p.max_parts / 2 : p.max_parts;
  hipLaunchKernelGGL(lora_grad_join_kernel, dim3((uint32_t)(want < 1024 ? want : 1024), groups), dim3(kLoraThreads), 0, stream, p);
  return hipGetLastError();
}

}  // namespace moe
