// moe_wgrad_mxfp8: dW[e] = sum over the slots s routed to e of
// grad[s]^T xhat[s / top_k], fp32, with the activations kept as MXFP8 (E4M3
// codes, one E8M0 scale per 32 columns).
//
// The tiles, the ownership of dW and the transposing operand reads are those
// of wgrad.hip (256 x 256 tiles, one persistent workgroup of 8 waves per CU,
// every tile accumulated over its expert's routing blocks on
// v_mfma_f32_32x32x16_bf16 and written once). What differs:
//  * Every XCD takes an eighth of each expert's tiles (WgSplitOrder): whole
//    experts per XCD, as in wgrad.hip, left the fullest XCD 16% more blocks
//    than the average on routing whose experts have 430 to 1750 slots.
//  * x arrives as codes, half the bytes. An MFMA operand holds 8 slots of one
//    column, and every slot has a scale of its own, so decoding at the operand
//    would take a conversion per element in each of the four waves that share
//    a column. Instead the codes (and a scale byte per lane) go by LDS-DMA
//    into a ring of their own, and each wave decodes the rows that it loaded
//    itself, once per tile, to the bf16 rows that the operand reads expect
//    (32 columns under one scale: two elements per conversion, exact).
//  * The pipeline steps by units of 32 slots, two per loop iteration (a
//    routing block). Grads are loaded three units ahead and codes four
//    (decoded one ahead), so a load has three steps to land, and the stores of
//    a finished tile two to drain before a wait reaches them.
//  * The operands of 16 slots are read one half step before their MFMAs, the
//    second half's products running after the next barrier, and everything
//    else a wave issues (operand reads, addresses, DMA, decoding) is placed
//    between MFMAs in program order. A wave issues in order and both waves of
//    a SIMD leave a barrier together, so what stands before or after a run of
//    MFMAs adds to them: with the loader and the reads in front of the
//    products, and every XCD taking whole experts, the same pipeline ran at
//    2.6 ms on E = 64, N = 2048, K = 7168 over 65536 slots.
//
// Those sizes now take 2.02 to 2.16 ms from card to card, 0.9 PFLOP/s: the matrix pipe is busy 48% of
// the cycles, at a clock that the chip's power holds at 1.95 GHz (2.4 where
// the data are zeros). Changes that save cycles alone no longer save time:
// starting each XCD at an expert of its own took 1.4% fewer cycles and ran as
// long. A library's dense product of the same size, bf16 out, takes 1.90 ms.
#include "common.h"
#include "params.h"
#include "wgrad_util.h"

namespace moe {

constexpr int kMxWaves = 8;
constexpr int kMxThreads = kMxWaves * 64;
constexpr int kMxGRing = 4;   // units of grads in LDS
constexpr int kMxRRing = 4;   // units of codes
constexpr int kMxXRing = 2;   // units of decoded x
constexpr int kMxCodeB = kWgUM * kWgTK;     // 8 KB: a unit's codes
constexpr int kMxScaleB = kMxThreads * 4;   // 2 KB: one scale dword per lane
constexpr int kMxLoads = 4;   // DMA instructions per wave per unit: 2 grads, codes, scales
constexpr int kMxStores = 32; // 16-byte stores per lane per tile
// N tiles per group of the tile order: neighbouring tiles write long stretches
// of the same rows of dW and read the same codes (on the sizes above 2.02 ms,
// against 2.06 with 1, 2.03 with 3, 2.07 with 4 and 2.08 with 8).
constexpr int kMxGroupN = 2;
constexpr int kMxRowB = kWgTN * 2;
static_assert(kMxRowB == kWgTK * 2, "rows of both operands have one length");

// One byte per lane from `rsrc` at `voff` into LDS, zero-extended to the dword
// at lds_base + 4 * lane.
__device__ __forceinline__ void wg_dma_byte(__amdgpu_buffer_rsrc_t rsrc, uint32_t voff, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %1\n\tbuffer_load_ubyte %0, %2, 0 offen lds"
               :: "v"(voff), "s"(__builtin_amdgcn_readfirstlane(lds_base)), "s"(rsrc) : "m0");
}

template <class T>
using mx_lds = __attribute__((address_space(3))) T;

// Wait until at most N of this wave's vector-memory operations are in flight
// and its LDS operations are done, then barrier; without the barrier.
template <int N>
__device__ __forceinline__ void mx_wait_barrier() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" :: "n"(N) : "memory");
}
template <int N>
__device__ __forceinline__ void mx_wait() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" :: "n"(N) : "memory");
}

__global__ __launch_bounds__(kMxThreads, 1) void wgrad_mxfp8_kernel(WgradParams p) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds_g[kMxGRing][kWgGUnitB];
  __shared__ __attribute__((aligned(1024))) uint8_t lds_x[kMxXRing][kWgXUnitB];
  __shared__ __attribute__((aligned(1024))) uint8_t lds_c[kMxRRing][kMxCodeB];
  __shared__ __attribute__((aligned(1024))) uint8_t lds_s[kMxRRing][kMxScaleB];
  __shared__ int32_t s_start[kWgMaxExperts + 1];

  const int tid = threadIdx.x;
  const int lane = tid % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int l32 = lane % 32, h = lane / 32;

  wg_block_ranges<kMxThreads>(p, s_start);
  const WgSplitOrder order(p, s_start, kMxGroupN);

  // (PAD slots, s = S, lie past the buffers)
  const int64_t T = p.S / p.top_k;
  const __amdgpu_buffer_rsrc_t g_rsrc =
      __builtin_amdgcn_make_buffer_rsrc((void*)p.grad, 0, wg_span(p.S, p.grad_ld, p.N, 2), 0x00020000);
  const __amdgpu_buffer_rsrc_t x_rsrc =
      __builtin_amdgcn_make_buffer_rsrc((void*)p.x, 0, wg_span(T, p.x_ld, p.K, 1), 0x00020000);
  const __amdgpu_buffer_rsrc_t s_rsrc =
      __builtin_amdgcn_make_buffer_rsrc((void*)p.xs, 0, wg_span(T, p.xs_ld, p.K / 32, 1), 0x00020000);
  const uint32_t g_lds = (uint32_t)(uintptr_t)(wg_lds_u8_t*)&lds_g[0][0];
  const uint32_t x_lds = (uint32_t)(uintptr_t)(wg_lds_u8_t*)&lds_x[0][0];
  const uint32_t c_lds = (uint32_t)(uintptr_t)(wg_lds_u8_t*)&lds_c[0][0];
  const uint32_t s_lds = (uint32_t)(uintptr_t)(wg_lds_u8_t*)&lds_s[0][0];

  // ---- loader: walks the pairs of units (routing blocks) of the same tiles
  //      ahead of the computation; wave w loads slot rows 4w .. 4w + 3 of
  //      every unit. Past the last tile it issues loads that read zeros, so
  //      every step costs the same number of loads.
  const uint32_t g_col0 = (uint32_t)wg_swz(lane / 32, lane % 32) * 16;      // rows 0, 1 of the wave's four
  const uint32_t g_col1 = (uint32_t)wg_swz(2 + lane / 32, lane % 32) * 16;  // rows 2, 3
  const uint32_t c_col = (uint32_t)(lane % 16) * 16, s_col = (uint32_t)(lane % 8);
  const uint32_t g_row = (uint32_t)(p.grad_ld * 2), x_row = (uint32_t)p.x_ld, s_row = (uint32_t)p.xs_ld;
  // masks of the lanes whose row of the wave's four is at least 1, 2, 3
  uint32_t from[4] = {~0u, lane >= 16 ? ~0u : 0u, lane >= 32 ? ~0u : 0u, lane >= 48 ? ~0u : 0u};
  asm volatile("" : "+v"(from[1]), "+v"(from[2]), "+v"(from[3]));  // kept as masks: one AND each
  const int div_shift = p.topk_shift - 31;  // s / top_k = (2 s m) >> (32 + div_shift), top_k = 1 included

  int ld_it = 0, ld_u = 0, ld_n = 0;
  WgTile ld{};
  bool ld_live = true;
  wg_i32x4_t ids_e, ids_o;  // the wave's slots of the pair two ahead of the computation's
  uint32_t g_at0 = 0, g_at1 = 0, c_at = 0, s_at = 0;  // the lane's offsets in the tile's columns
  auto ld_tile = [&]() {  // the next tile with slots, from ld_it on
    for (;; ++ld_it) {
      const int at = order.index(ld_it);
      ld_live = at < order.total;
      if (!ld_live) break;
      ld = order.at(at);
      ld_n = 2 * (ld.b1 - ld.b0);
      if (ld_n > 0) break;
    }
    ++ld_it;
    ld_u = 0;
    g_at0 = g_col0 + (ld_live ? (uint32_t)ld.n0 * 2 : kWgOOB);
    g_at1 = g_col1 + (ld_live ? (uint32_t)ld.n0 * 2 : kWgOOB);
    c_at = c_col + (ld_live ? (uint32_t)ld.k0 : kWgOOB);
    s_at = s_col + (ld_live ? (uint32_t)ld.k0 / 32 : kWgOOB);
  };
  // the pair's ids, by scalar loads that the compiler tracks
  auto ld_ids = [&](wg_i32x4_t& e, wg_i32x4_t& o) {
    e = wg_i32x4_t{0, 0, 0, 0};
    o = e;
    if (ld_live) {
      const wg_const<int32_t>* at = (const wg_const<int32_t>*)p.sorted + (int64_t)ld.b0 * kWgBM + ld_u * kWgUM + wave * 4;
      e = wg_scalar_ids4(at);
      o = wg_scalar_ids4(at + kWgUM);
    }
  };
  auto ld_next = [&]() {
    ld_u += 2;
    if (ld_live && ld_u >= ld_n) ld_tile();
  };
  // Byte offsets of the lane's pieces of a unit: its two grad loads', its
  // codes' (16 lanes a row) and its scale's. The slots are scalars; a lane's
  // own is the first plus the differences up to its row, and the grads'
  // products are formed on the scalar unit. A PAD slot (s = S) lands at or
  // past the end of every buffer; past the last tile the ids are 0 and the
  // bases put every lane past them.
  struct Codes {
    uint32_t c, s, row;
  };
  auto codes_slot = [&](Codes& o, const wg_i32x4_t& id) {  // twice the lane's slot, in `row`
    const uint32_t i0 = (uint32_t)id[0], i1 = (uint32_t)id[1], i2 = (uint32_t)id[2], i3 = (uint32_t)id[3];
    o.row = (i0 + ((i1 - i0) & from[1]) + ((i2 - i1) & from[2]) + ((i3 - i2) & from[3])) << 1;
    asm volatile("" : "+v"(o.row));  // formed here, not where it is used (as the others below)
  };
  auto codes_row = [&](Codes& o) {
    o.row = __umulhi(o.row, p.topk_magic) >> div_shift;
    asm volatile("" : "+v"(o.row));
  };
  auto codes_offset = [&](Codes& o) {
    o.c = o.row * x_row + c_at;
    o.s = o.row * s_row + s_at;
    asm volatile("" : "+v"(o.c), "+v"(o.s));
  };
  auto grad_offset = [&](const wg_i32x4_t& id, int half) {
    const uint32_t a = (uint32_t)id[2 * half], b = (uint32_t)id[2 * half + 1];
    uint32_t off = (half ? g_at1 : g_at0) + a * g_row + (((b - a) * g_row) & from[2]);
    asm volatile("" : "+v"(off));
    return off;
  };
  const uint32_t g_dst = g_lds + (uint32_t)(wave * 2048), c_dst = c_lds + (uint32_t)(wave * 1024),
                 s_dst = s_lds + (uint32_t)(wave * 256);
  auto dma_grads = [&](int slot, int half, uint32_t off) {
    wg_dma16(g_rsrc, off, g_dst + (uint32_t)(slot * kWgGUnitB + half * 1024));
  };
  auto dma_codes = [&](int slot, const Codes& o) {
    wg_dma16(x_rsrc, o.c, c_dst + (uint32_t)(slot * kMxCodeB));
    wg_dma_byte(s_rsrc, o.s, s_dst + (uint32_t)(slot * kMxScaleB));
  };

  // ---- decoding: this wave's pieces of a unit's codes into its rows of x.
  //      Lane l takes 8 codes of either half of row l / 16, so that 16 lanes'
  //      pieces of a write are contiguous.
  u32x2_t raw_c[2];
  uint32_t raw_s[2];
  const uint32_t c_src = c_dst + (uint32_t)(lane / 16 * 256 + lane % 16 * 8),
                 s_src = s_dst + (uint32_t)(lane / 16 * 64 + lane % 16 / 4 * 4);
  // codes at c_rd[next] and scales at s_rd[next], `unit` slots on; [0] is the
  // ring slot of the current pair, [1] that of the next
  uint32_t c_rd[2] = {c_src, c_src + 2 * kMxCodeB}, s_rd[2] = {s_src, s_src + 2 * kMxScaleB};
  auto read_raw = [&](int next, int unit) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      raw_c[i] = *(const mx_lds<u32x2_t>*)(c_rd[next] + (uint32_t)(unit * kMxCodeB + i * 128));
      raw_s[i] = *(const mx_lds<uint32_t>*)(s_rd[next] + (uint32_t)(unit * kMxScaleB + i * 16));
    }
  };
  const int dm = wave * 4 + lane / 16;
  const uint32_t d_at = x_lds + (uint32_t)(dm * kMxRowB + wg_swz(dm, lane % 16) * 16);  // (+ 16 pieces keep the swizzle)
  auto decode = [&](int slot, int i) {
    *(mx_lds<bf16x8_t>*)(d_at + (uint32_t)(slot * kWgXUnitB + i * 256)) =
        dequant_e4m3x8(raw_c[i][0], raw_c[i][1], __uint_as_float(raw_s[i] << 23));
  };

  // ---- computation: wave (wn, wk) of 4 x 2 computes dW rows n0 + wn*64 ..
  //      + 63 and columns k0 + wk*128 .. + 127
  const int wn = wave / 2, wk = wave % 2;
  f32x16_t acc[2][4];
  struct Ops {
    bf16x8_t a[2], b[4];
  };
  // LDS addresses of the operand reads (see wg_operand in wgrad_util.h): lane
  // (group, s) points at slot 8 (group / 2) + s / 4 and columns
  // 16 (group % 2) + 4 (s % 4) of the operand's 32
  auto op_addr = [&](int c0) {
    const int g = lane / 16, s = lane % 16;
    const int col = c0 + 16 * (g % 2) + 4 * (s % 4), m = 8 * (g / 2) + s / 4;
    return (uint32_t)(m * kMxRowB + wg_swz(m, col / 8) * 16 + (col % 8) * 2);
  };
  uint32_t a_addr[2], b_addr[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) a_addr[i] = g_lds + op_addr(wn * 64 + i * 32);
#pragma unroll
  for (int j = 0; j < 4; ++j) b_addr[j] = x_lds + op_addr(wk * 128 + j * 32);
  // 8 consecutive slots, in two reads of 4 (adding 4 or 16 slots keeps the swizzle)
  auto read_op = [&](uint32_t at) {
    wg_s16x4_t v[2];
    v[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((mx_lds<wg_s16x4_t>*)at);
    v[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((mx_lds<wg_s16x4_t>*)(at + 4 * kMxRowB));
    bf16x8_t r;
    __builtin_memcpy(&r, v, 16);
    return r;
  };
  auto read_a = [&](Ops& o, int i, int unit, int ks) {  // unit 0 or 1 of the pair
    o.a[i] = read_op(a_addr[i] + (uint32_t)(unit * kWgGUnitB + ks * 16 * kMxRowB));
  };
  auto read_b = [&](Ops& o, int j, int unit, int ks) {
    o.b[j] = read_op(b_addr[j] + (uint32_t)(unit * kWgXUnitB + ks * 16 * kMxRowB));
  };
  auto mul = [&](const Ops& o, int i, int j) {
    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(o.a[i], o.b[j], acc[i][j], 0, 0, 0);
  };
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
  };
  // A finished tile goes out through the wave's own 2 KB of an x slot that
  // nothing reads: the MFMA output holds one column per lane, and 8 rows x 64
  // columns at a time become 16-byte pieces of 256-byte row stretches (rows
  // 4 .. 7 XOR their columns with 32: distinct banks for both halves of a
  // write). Every lane issues its kMxStores stores, also at the N and K edges
  // (through an offset past the expert's dW, which the buffer drops), so the
  // waits that count them stay exact.
  auto store_tile = [&](const WgTile& t, int x_slot) {
    const __amdgpu_buffer_rsrc_t dw_rsrc = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(p.dw + (int64_t)t.e * p.N * p.K), 0, (int)(uint32_t)((int64_t)p.N * p.K * 4), 0x00020000);
    mx_lds<float>* scr = (mx_lds<float>*)&lds_x[x_slot][wave * 2048];
    const int row0 = t.n0 + wn * 64, rows = p.N - row0;  // rows of this wave's part that exist
    const int k = t.k0 + wk * 128 + 4 * (lane % 16);
    const int row_b = p.K * 4;  // (one expert's dW spans less than 2 GB)
    const uint32_t base = (uint32_t)(((int64_t)(row0 + lane / 16) * p.K + k) * 4);  // (below 2^31 where it is used)
#pragma unroll
    for (int pass = 0; pass < 16; ++pass) {
      const int i = pass / 8, q = (pass / 2) % 4, jh = pass % 2;
#pragma unroll
      for (int jj = 0; jj < 2; ++jj)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          scr[(4 * h + r) * 64 + ((jj * 32 + l32) ^ (32 * h))] = acc[i][2 * jh + jj][4 * q + r];
#pragma unroll
      for (int rd = 0; rd < 2; ++rd) {
        const int lr = 4 * rd + lane / 16;  // local row 0 .. 7 of the pass
        const f32x4_t v =
            *(const mx_lds<f32x4_t>*)&scr[lr * 64 + ((4 * (lane % 16)) ^ (32 * rd))];
        const int r = i * 32 + 8 * q + 4 * rd;
        const uint32_t off = (r + lane / 16 < rows && k + jh * 64 < p.K) ? base : kWgOOB;
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(wg_i32x4_t, v), dw_rsrc, off,
                                               r * row_b + jh * 256, kWgStoreNT);
      }
    }
  };
  // an expert without slots: zeros
  auto store_zeros = [&](const WgTile& t) {
    const __amdgpu_buffer_rsrc_t dw_rsrc = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(p.dw + (int64_t)t.e * p.N * p.K), 0, (int)(uint32_t)((int64_t)p.N * p.K * 4), 0x00020000);
#pragma unroll 4
    for (int i = 0; i < 32; ++i) {
      const int n = t.n0 + wave * 32 + i, k = t.k0 + 4 * lane;
      const uint32_t off = (n < p.N && k < p.K) ? (uint32_t)(((int64_t)n * p.K + k) * 4) : kWgOOB;
      __builtin_amdgcn_raw_buffer_store_b128(wg_i32x4_t{0, 0, 0, 0}, dw_rsrc, off, 0, kWgStoreNT);
    }
  };

  // ---- prologue: codes of unit 0, then grads of units 0 .. 2 with codes of
  //      1 .. 3; unit 0 decoded
  Codes codes;
  uint32_t g0, g1;
  auto load_codes = [&](int slot, const wg_i32x4_t& id) {
    codes_slot(codes, id);
    codes_row(codes);
    codes_offset(codes);
    dma_codes(slot, codes);
  };
  auto load_grads = [&](int slot, const wg_i32x4_t& id) {
    dma_grads(slot, 0, grad_offset(id, 0));
    dma_grads(slot, 1, grad_offset(id, 1));
  };
  ld_tile();
  ld_ids(ids_e, ids_o);
  load_codes(0, ids_e);
  load_grads(0, ids_e);
  load_codes(1, ids_o);
  load_grads(1, ids_o);
  ld_next();
  ld_ids(ids_e, ids_o);
  load_codes(2, ids_e);
  load_grads(2, ids_e);
  load_codes(3, ids_o);
  g0 = grad_offset(ids_o, 0);
  g1 = grad_offset(ids_o, 1);
  ld_next();
  ld_ids(ids_e, ids_o);
  mx_wait<3 * kMxLoads>();
  read_raw(0, 0);
  decode(0, 0);
  decode(0, 1);

  // ---- step u, for the units of the workgroup's tiles in order. At its
  //      barrier: every wave's grads of u and codes of u + 1 have landed (the
  //      loads of the two steps before may be in flight, and the stores of a
  //      tile finished in those, which are younger), x of u is decoded, and
  //      nothing reads unit u - 1 any more. It multiplies the
  //      second half of u - 1 and the first of u, and starts the grads of
  //      u + 3 and the codes of u + 4.
  Ops even, odd;
  const bf16x8_t zero = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 2; ++i) odd.a[i] = zero;
#pragma unroll
  for (int j = 0; j < 4; ++j) odd.b[j] = zero;
  clear();
  WgTile t{}, done{};
  int it = 0, uu = 0, nu = 0;
  int since = 2;  // steps since a tile was stored
  int ring = 0;   // ring slot of the pair's first unit: 0 or 2
  // moves to the next tile with slots, writing zeros for those without;
  // false past the last
  auto next_tile = [&]() {
    for (;; ++it) {
      const int at = order.index(it);
      if (at >= order.total) return false;
      t = order.at(at);
      nu = 2 * (t.b1 - t.b0);
      if (nu > 0) break;
      store_zeros(t);
      since = 0;
    }
    ++it;
    uu = 0;
    return true;
  };
  auto fence = [] { __builtin_amdgcn_sched_barrier(0); };
  auto wait_step = [&]() {
    if (since < 2)
      mx_wait_barrier<2 * kMxLoads + kMxStores>();
    else
      mx_wait_barrier<2 * kMxLoads>();
    ++since;
  };
  // What a wave issues beside the products is spread over the gaps between
  // them, about ten operations each: with two waves on a SIMD, a gap lasts two
  // products.
  //
  // The products of unit u - 1's second half, with the first operand reads of
  // unit u (`unit` of its pair), the grad loads into g_slot (offsets g0, g1),
  // the raw codes of unit u + 1 and the offsets of the codes of slots `id`.
  auto first_half = [&](int unit, int g_slot, const wg_i32x4_t& id) {
    mul(odd, 0, 0);
    read_a(even, 0, unit, 0);
    read_b(even, 0, unit, 0);
    dma_grads(g_slot, 0, g0);
    fence();
    mul(odd, 0, 1);
    codes_slot(codes, id);
    fence();
    mul(odd, 0, 2);
    read_b(even, 1, unit, 0);
    read_b(even, 2, unit, 0);
    dma_grads(g_slot, 1, g1);
    fence();
    mul(odd, 0, 3);
    codes_row(codes);
    fence();
    mul(odd, 1, 0);
    read_b(even, 3, unit, 0);
    read_a(even, 1, unit, 0);
    read_raw(unit, 1 - unit);
    fence();
    mul(odd, 1, 1);
    codes_offset(codes);
    fence();
    mul(odd, 1, 2);
    fence();
    mul(odd, 1, 3);
    fence();
  };
  // The products of its first half, with the code loads (of slots `id`) into
  // c_slot and the offsets of their grads, the decoding of the next unit into
  // x_slot and the operand reads of the second half.
  auto second_half = [&](int unit, int c_slot, int x_slot, const wg_i32x4_t& id) {
    mul(even, 0, 0);
    dma_codes(c_slot, codes);
    fence();
    mul(even, 0, 1);
    decode(x_slot, 0);
    fence();
    mul(even, 0, 2);
    decode(x_slot, 1);
    fence();
    mul(even, 0, 3);
    read_a(odd, 0, unit, 1);
    read_b(odd, 0, unit, 1);
    g0 = grad_offset(id, 0);
    fence();
    mul(even, 1, 0);
    read_b(odd, 1, unit, 1);
    read_b(odd, 2, unit, 1);
    g1 = grad_offset(id, 1);
    fence();
    mul(even, 1, 1);
    // the next ids here: no LDS result is waited for before the barrier's own
    // wait (scalar loads return out of order, so a wait for LDS with one in
    // flight waits for all)
    if (unit == 1) {
      ld_next();
      ld_ids(ids_e, ids_o);
      fence();
    }
    read_b(odd, 3, unit, 1);
    read_a(odd, 1, unit, 1);
    fence();
    mul(even, 1, 2);
    mul(even, 1, 3);
    fence();
  };
  done.e = -1;
  for (bool go = next_tile(); go;) {
    wait_step();
    first_half(0, (ring ^ 2) + 1, ids_e);
    if (uu == 0) {
      if (done.e >= 0) {
        store_tile(done, 1);
        since = 0;
      }
      clear();
      fence();
    }
    second_half(0, ring, 1, ids_e);
    wait_step();
    first_half(1, ring, ids_o);
    second_half(1, ring + 1, 0, ids_o);
    ring ^= 2;
    const int to = ring ? 2 * kWgGUnitB : -2 * kWgGUnitB;
    static_assert(kWgGUnitB == 2 * kMxCodeB && kWgGUnitB == 8 * kMxScaleB, "one step for the three rings");
    a_addr[0] += to;
    a_addr[1] += to;
    c_rd[0] += to / 2, c_rd[1] -= to / 2;
    s_rd[0] += to / 8, s_rd[1] -= to / 8;
    uu += 2;
    if (uu == nu) {
      done = t;
      go = next_tile();
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) mul(odd, i, j);
  if (done.e >= 0) store_tile(done, 0);
  // drain the look-ahead loads
  mx_wait<0>();
}

hipError_t launch_wgrad_mxfp8(const WgradParams& p_in, hipStream_t stream) {
  WgradParams p = p_in;
  p.tiles_n = (p.N + kWgTN - 1) / kWgTN;
  p.tiles_k = (p.K + kWgTK - 1) / kWgTK;
  wg_set_division(p);
  if ((int64_t)p.E * p.tiles_n * p.tiles_k == 0) return hipSuccess;
  int dev = 0, cus = 0;
  hipError_t err = hipGetDevice(&dev);
  if (err == hipSuccess) err = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
  if (err != hipSuccess) return err;
  const uint32_t grid = (uint32_t)((cus + 7) / 8 * 8);  // one workgroup per CU, a multiple of 8 (the XCDs)
  hipLaunchKernelGGL(wgrad_mxfp8_kernel, dim3(grid), dim3(kMxThreads), 0, stream, p);
  return hipGetLastError();
}

}  // namespace moe
