// moe_wgrad: dW[e] = sum over the slots s routed to e of grad[s]^T x[s / top_k],
// fp32, straight from moe_align's sorted_token_ids / expert_ids.
//
// Follows ROCm/aiter PR #5310 "Add MoE GEMM variants and weight-gradient
// kernel": Summary (moe_wgrad replaces sort + pad + bmm and a host sync; its
// atomics needed dW reset between benchmark trials or results were corrupted)
// and Tests & Benchmarks (constant input, linearity, zero-padded tokens).
//
// Design for gfx950:
//  * dW is cut into (expert, 256 x 256) tiles. A persistent grid (one
//    workgroup of 8 waves per CU) walks them; each tile is accumulated over
//    its expert's routing blocks on v_mfma_f32_32x32x16_bf16 and written
//    once, so dW is overwritten (never accumulated into), empty experts get
//    zeros, nothing is atomic and repeated calls give identical bits.
//  * Slot rows of grad (256 columns) and x (256 columns), 512 bytes each, go
//    straight from global memory into LDS with buffer_load ... lds,
//    slot-major as they lie in memory, 32 slots per pipeline unit in four
//    32 KB stages. Units go in pairs (one 64-slot routing block): one
//    barrier per pair, after which the next pair's loads are issued (across
//    tile boundaries) and the pair is computed (one barrier per unit with
//    three stages measured 2% slower). Each wave computes 64 x 128 of the
//    tile: 16 MFMAs per unit. The
//    tile size is what the operand traffic asks for: loading both operands
//    costs (rows + columns) bytes per slot for rows x columns products, and
//    256 x 256 measured faster than 128 x 256 at two workgroups per CU
//    (5.7 against 6.5 ms on the E=256 gradient); larger tiles would need
//    more accumulator registers than two waves per SIMD allow.
//  * The contraction runs over slots, so an MFMA operand needs 8 consecutive
//    slots of one column: gfx950's transposing LDS read (ds_read_b64_tr_b16)
//    gathers them. Within each 16-lane group, lane j receives element j % 4
//    of the 8-byte reads of lanes j/4, j/4 + 4, j/4 + 8, j/4 + 12 (measured);
//    lane s of the group therefore points at slot (s / 4) and columns
//    4 (s % 4) .. + 3, and lane j ends up with column j of four consecutive
//    slots. Two such reads make one operand.
//  * A finished tile goes out through LDS: the MFMA output holds one column
//    per lane, so each wave passes 8 rows at a time through a scratch area
//    (the stage the next unit's loads will fill, free at that point; rows
//    4..7 of a pass XOR their columns with 32 so both halves of a write hit
//    distinct banks) and writes whole 512-byte row pieces with 16-byte
//    non-temporal stores.
//    Storing the MFMA output as it lies (one dword per lane, 128-byte row
//    stretches) issues four times the store instructions; four adjacent
//    columns per lane from swapped operands (32-byte stretches) measured
//    slower still.
//  * The 16-byte units of each LDS row are XOR-swizzled by slot.
//  * Tiles are numbered expert-major, then in groups of 8 N tiles walked
//    N-fastest, and each XCD takes consecutive tiles: the 64 workgroups an
//    XCD runs at once cover 8 x 8 tiles of one expert, whose grad and x
//    slices stay in its L2.
//  * Every expert's block range comes from one pass over expert_ids (sorted
//    by expert, sentinels last) into an LDS table at the start; slot ids are
//    read with scalar loads between the products of the pair before their use
//    (loads that the compiler tracks, placed where it waits for nothing else:
//    as fast as inline asm, whose registers it may copy before they are
//    loaded) and turned into row
//    offsets on the scalar unit (the token row s / top_k by a multiply-high),
//    so a load costs each lane only a select and an add. PAD slots and the
//    look-ahead past the last tile read zeros through the buffer bounds;
//    columns past N or K read whatever follows in memory and only reach dW
//    rows and columns that are never stored.
#include "common.h"
#include "params.h"
#include "wgrad_util.h"

namespace moe {

constexpr int kWgStageB = kWgGUnitB + kWgXUnitB;
constexpr int kWgStages = 4;                 // two pairs of units
constexpr int kWgWaves = 8;
constexpr int kWgThreads = kWgWaves * 64;
constexpr int kWgGLoads = kWgGUnitB / 1024 / kWgWaves;  // DMA instructions per wave per unit: 2 grad
constexpr int kWgXLoads = kWgXUnitB / 1024 / kWgWaves;  //   + 2 x (2 rows each)
constexpr int kWgStores = 8 * 4;             // 16-byte stores per lane per tile
constexpr int kWgWaitLds = 0xC07F;           // s_waitcnt lgkmcnt(0), no wait for vector memory
constexpr int kWgPerCU = 1;                  // resident workgroups per CU
static_assert(kWgGLoads == 2 && kWgXLoads == 2, "each wave loads the same 4 slot rows of both parts");

__global__ __launch_bounds__(kWgThreads, kWgPerCU) void wgrad_kernel(WgradParams p) {
  // four stages of [grad unit | x unit], slot-major
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kWgStages][kWgStageB];
  __shared__ int32_t s_start[kWgMaxExperts + 1];  // first block of expert e (s_start[E] = end)

  const int tid = threadIdx.x;
  const int lane = tid % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int l32 = lane % 32, h = lane / 32;

  wg_block_ranges<kWgThreads>(p, s_start);
  const WgOrder order(p, s_start);
  const int total = order.total;
  auto tile_index = [&](int it) { return order.index(it); };
  auto tile_at = [&](int T) { return order.at(T); };

  const __amdgpu_buffer_rsrc_t g_rsrc = __builtin_amdgcn_make_buffer_rsrc(
      (void*)p.grad, 0, wg_span(p.S, p.grad_ld, p.N, 2), 0x00020000);
  const __amdgpu_buffer_rsrc_t x_rsrc = __builtin_amdgcn_make_buffer_rsrc(
      (void*)p.x, 0, wg_span(p.S / p.top_k, p.x_ld, p.K, 2), 0x00020000);
  const uint32_t lds_base = (uint32_t)(uintptr_t)(wg_lds_u8_t*)&lds[0][0];
  const uint32_t g_row = (uint32_t)(p.grad_ld * 2), x_row = (uint32_t)(p.x_ld * 2);

  // ---- loader: walks the same tiles' units one pair ahead of the
  //      computation. Unit u of a tile is slots [32u, 32u + 32) of its block
  //      list; wave w loads slot rows 4w .. 4w + 3 of both parts (two
  //      instructions of 2 rows x 32 lanes each).
  //      Past the last tile it issues loads that read zeros, so every unit
  //      costs the same number of loads.
  // The 16-byte unit each lane fetches, as a byte offset within the row
  // piece (the LDS side is lane order, the global side the swizzled unit):
  // load i of either part has row % 4 = 2 (i % 2) + lane / 32.
  const uint32_t x_col0 = (uint32_t)wg_swz(lane / 32, lane % 32) * 16;
  const uint32_t x_col1 = (uint32_t)wg_swz(2 + lane / 32, lane % 32) * 16;
  // all-ones mask of the lanes that take the second row of a load (a
  // select by bit logic, one VALU operation)
  const uint32_t xm1 = lane >= 32 ? ~0u : 0u;
  auto pick = [](uint32_t mask, uint32_t a, uint32_t b) { return (a & mask) | (b & ~mask); };

  int ld_it = 0;
  WgTile ld = tile_at(tile_index(0));
  int ld_u = 0;
  bool ld_live = tile_index(0) < total;
  auto ld_skip_empty = [&]() {  // move to the next tile with a unit left (empty experts have none)
    while (ld_live && ld_u >= 2 * (ld.b1 - ld.b0)) {
      ++ld_it;
      ld_u = 0;
      const int T = tile_index(ld_it);
      ld_live = T < total;
      if (ld_live) ld = tile_at(T);
    }
  };
  // the ids of the pair of units the loader points at (a pair is one
  // 64-slot routing block, never split across tiles)
  auto ld_ids_pair = [&](wg_i32x4_t& a, wg_i32x4_t& b) {
    a = wg_i32x4_t{0, 0, 0, 0};
    b = a;
    if (ld_live) {
      const wg_const<int32_t>* at =
          (const wg_const<int32_t>*)p.sorted + (int64_t)ld.b0 * kWgBM + ld_u * kWgUM + wave * 4;
      a = wg_scalar_ids4(at);
      b = wg_scalar_ids4(at + kWgUM);
    }
  };
  ld_skip_empty();
  wg_i32x4_t ids, ids_b;
  ld_ids_pair(ids, ids_b);
  wg_wait_barrier<0>(ids, ids_b);

  auto issue_unit = [&](int stage, const wg_i32x4_t& uid) {
    // scalar row offsets of the wave's 8 slots within the tile's column
    // range (a PAD slot s = S lands at or past the end of both buffers)
    // (past the last tile the ids are 0 and the bases put every lane past
    // the buffers: s * row + kWgOOB stays below 2^32)
    const uint32_t g_base = ld_live ? (uint32_t)ld.n0 * 2 : kWgOOB;
    const uint32_t x_base = ld_live ? (uint32_t)ld.k0 * 2 : kWgOOB;
    uint32_t go[4], xo[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const uint32_t s = (uint32_t)uid[r];
      const uint64_t prod = ((uint64_t)__umulhi(s, p.topk_magic) << 32) | (s * p.topk_magic);
      const uint32_t xrow = (uint32_t)(prod >> p.topk_shift);
      go[r] = s * g_row + g_base;
      xo[r] = xrow * x_row + x_base;
    }
    const uint32_t dst = lds_base + (uint32_t)(stage * kWgStageB);
#pragma unroll
    for (int i = 0; i < kWgGLoads; ++i)
      wg_dma16(g_rsrc, pick(xm1, go[2 * i + 1], go[2 * i]) + (i % 2 ? x_col1 : x_col0),
               dst + (uint32_t)((wave * kWgGLoads + i) * 1024));
#pragma unroll
    for (int i = 0; i < kWgXLoads; ++i)
      wg_dma16(x_rsrc, pick(xm1, xo[2 * i + 1], xo[2 * i]) + (i % 2 ? x_col1 : x_col0),
               dst + (uint32_t)(kWgGUnitB + (wave * kWgXLoads + i) * 1024));
  };
  auto issue_pair = [&](int stage) {  // stages stage, stage + 1
    issue_unit(stage, ids);
    issue_unit(stage + 1, ids_b);
    if (ld_live) {
      ld_u += 2;
      ld_skip_empty();
    }
  };

  // waves 4 x 2: wave (wn, wk) computes dW rows n0 + wn*64 .. + 63 and
  // columns k0 + wk*128 .. + 127
  const int wn = wave / 2, wk = wave % 2;
  f32x16_t acc[2][4];  // [n sub-tile][k sub-tile]
  auto contract = [&](int stage, bool next_ids) {
    const wg_lds_u8_t* gt = (const wg_lds_u8_t*)&lds[stage][0];
    const wg_lds_u8_t* xt = gt + kWgGUnitB;
    // every operand of the unit first (their LDS latency overlaps), then the MFMAs
    constexpr int KS = kWgUM / 16;
    bf16x8_t af[KS][2], bfr[KS][4];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
      for (int i = 0; i < 2; ++i) af[ks][i] = wg_operand<kWgGRowB>(gt, wn * 64 + i * 32, ks * 16, lane);
#pragma unroll
      for (int j = 0; j < 4; ++j) bfr[ks][j] = wg_operand<kWgXRowB>(xt, wk * 128 + j * 32, ks * 16, lane);
    }
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      if (ks == KS - 1 && next_ids) {
        // the next pair's ids here: the last LDS results are awaited first, since
        // scalar loads return out of order and a wait for LDS with one in flight
        // waits for all, and the products that follow cover the load
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(kWgWaitLds);
        ld_ids_pair(ids, ids_b);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(af[ks][i], bfr[ks][j], acc[i][j], 0, 0, 0);
    }
  };

  // ---- computation, a pair of units (one routing block) per barrier:
  //      before a pair the wave waits until only the stores of a tile
  //      finished just before are in flight (the pair's loads were issued
  //      before them); the barrier makes every wave's DMA visible and
  //      guarantees all waves finished the previous pair, whose two stages
  //      the loads issued next overwrite.
  issue_pair(0);
  ld_ids_pair(ids, ids_b);
  int st = 0;  // first stage of the next pair computed
  bool stored = false;
  for (int it = 0; tile_index(it) < total; ++it) {
    const WgTile t = tile_at(tile_index(it));
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
    const int nu = 2 * (t.b1 - t.b0);
    for (int u = 0; u < nu; u += 2) {
      if (stored) {
        wg_wait_barrier<kWgStores>(ids, ids_b);
        stored = false;
      } else {
        wg_wait_barrier<0>(ids, ids_b);
      }
      issue_pair(st ^ 2);  // the pair computed last, now free
      contract(st, false);
      contract(st + 1, true);
      st ^= 2;
    }
    // store the tile through LDS: the first stage of the pair computed last
    // is free once every wave is past its last contraction (the next
    // pair's loads go to the other two). Each wave
    // passes 8 rows at a time through its own 4 KB of it and writes whole
    // 512-byte row pieces with 16-byte stores.
    __syncthreads();
    {
      // every lane issues its kWgStores stores, also at the N and K edges
      // (lanes past them write through an offset past the expert's dW, which
      // the buffer drops), so the waits above, which count them, stay exact
      const __amdgpu_buffer_rsrc_t dw_rsrc = __builtin_amdgcn_make_buffer_rsrc(
          (void*)(p.dw + (int64_t)t.e * p.N * p.K), 0, (int)(uint32_t)((int64_t)p.N * p.K * 4), 0x00020000);
      const int free_stage = st ^ 2;  // the last pair's first stage
      __attribute__((address_space(3))) float* scr =
          (__attribute__((address_space(3))) float*)&lds[free_stage][wave * 8 * 512];
#pragma unroll
      for (int pass = 0; pass < 8; ++pass) {
        const int i = pass / 4, q = pass % 4;
        // lane (l32, h) holds rows i*32 + 8q + 4h + (0..3) of columns j*32 + l32;
        // rows 4..7 of the scratch are stored with columns XOR 32 (distinct banks)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r) scr[(4 * h + r) * 128 + ((j * 32 + l32) ^ (32 * h))] = acc[i][j][4 * q + r];
#pragma unroll
        for (int rd = 0; rd < 4; ++rd) {
          const int lr = 2 * rd + h;  // local row 0..7 of the pass
          const f32x4_t v = *(const __attribute__((address_space(3))) f32x4_t*)&scr[lr * 128 + ((4 * l32) ^ (32 * (lr / 4)))];
          const int n = t.n0 + wn * 64 + i * 32 + 8 * q + lr;
          const int k = t.k0 + wk * 128 + 4 * l32;
          const uint32_t off = (n < p.N && k < p.K) ? (uint32_t)(((int64_t)n * p.K + k) * 4) : kWgOOB;
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(wg_i32x4_t, v), dw_rsrc, off, 0, kWgStoreNT);
        }
      }
    }
    stored = true;
  }
  // drain the look-ahead loads (past the last tile they read zeros)
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

int wgrad_block_m() { return kWgBM; }

hipError_t launch_wgrad(const WgradParams& p_in, hipStream_t stream) {
  WgradParams p = p_in;
  p.tiles_n = (p.N + kWgTN - 1) / kWgTN;
  p.tiles_k = (p.K + kWgTK - 1) / kWgTK;
  wg_set_division(p);
  const int64_t tiles = (int64_t)p.E * p.tiles_n * p.tiles_k;
  if (tiles == 0) return hipSuccess;
  int dev = 0, cus = 0;
  hipError_t err = hipGetDevice(&dev);
  if (err == hipSuccess) err = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
  if (err != hipSuccess) return err;
  // a persistent grid: kWgPerCU workgroups per CU, a multiple of 8 (one
  // stretch of tiles per XCD per round)
  int64_t grid = (int64_t)cus * kWgPerCU;
  grid = (grid + 7) / 8 * 8;
  hipLaunchKernelGGL(wgrad_kernel, dim3((uint32_t)grid), dim3(kWgThreads), 0, stream, p);
  return hipGetLastError();
}

}  // namespace moe
