// Host side of libmoe's block entry points (include/moe_block.h): argument
// validation before anything touches the GPU, and dispatch.
#include <hip/hip_runtime.h>

#include <climits>
#include <cmath>

#include "moe_block.h"

#include "dropout_util.h"
#include "host.h"
#include "lora_host.h"
#include "params.h"
#include "ranges.h"

namespace {

using moe::bad_ld;
using moe::check_device;
using moe::clash;
using moe::fail;
using moe::hip_status;
using moe::kAlignMaxExperts;
using moe::misaligned;
using moe::ok;
using moe::Range;
using moe::span;

constexpr int64_t kNormMaxWidth = 16384;
constexpr int32_t kLoraMaxRank = 128;
constexpr int64_t kLoraMaxWidth = (int64_t)1 << 24;

int64_t dtype_bytes(int32_t dtype) { return dtype == MOE_FP32 ? 4 : 2; }

// p and rng of a dropout: rng is needed where anything is dropped.
moe_status check_dropout(float p, const uint64_t* rng) {
  if (!(p >= 0.0f && p <= 1.0f)) return fail(MOE_ERR_INVALID_ARGUMENT, "p must be in [0, 1]");
  if (moe::make_dropout(p, rng).threshold > 0 && rng == nullptr)
    return fail(MOE_ERR_INVALID_ARGUMENT, "a dropout needs rng");
  if (misaligned(rng, 8)) return fail(MOE_ERR_INVALID_ARGUMENT, "rng must be 8-byte aligned");
  return MOE_OK;
}

// A bf16 or fp32 matrix of rows: its stride, and its alignment to 16 bytes.
moe_status check_rows(const char* name, const void* p, int64_t ld, int64_t rows, int64_t n, bool needed) {
  if (p == nullptr) {
    if (needed && rows > 0) return fail(MOE_ERR_INVALID_ARGUMENT, "%s is null", name);
    return MOE_OK;
  }
  if (bad_ld(ld, n, 8, rows))
    return fail(MOE_ERR_INVALID_ARGUMENT, "%s: row stride %lld must cover %lld and be a multiple of 8", name,
                (long long)ld, (long long)n);
  if (misaligned(p, 16)) return fail(MOE_ERR_INVALID_ARGUMENT, "%s must be 16-byte aligned", name);
  return MOE_OK;
}

// What the norm and its gradient check alike.
moe_status check_norm(int64_t rows, int64_t n, int64_t multiple, int32_t dtype, const void* weight,
                      int32_t weight_dtype, float eps, float p, const uint64_t* rng) {
  if (rows < 0 || rows >= INT32_MAX) return fail(MOE_ERR_INVALID_ARGUMENT, "rows must be in [0, 2^31 - 1)");
  if (n < multiple || n % multiple != 0)
    return fail(MOE_ERR_INVALID_ARGUMENT, "n must be a positive multiple of %lld", (long long)multiple);
  if (n > kNormMaxWidth) return fail(MOE_ERR_UNSUPPORTED, "n %lld > %lld", (long long)n, (long long)kNormMaxWidth);
  if ((dtype != MOE_BF16 && dtype != MOE_FP32) || (weight_dtype != MOE_BF16 && weight_dtype != MOE_FP32))
    return fail(MOE_ERR_UNSUPPORTED, "the residual stream and weight must be MOE_BF16 or MOE_FP32");
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(MOE_ERR_INVALID_ARGUMENT, "eps must be finite and >= 0");
  if (weight == nullptr) return fail(MOE_ERR_INVALID_ARGUMENT, "weight is null");
  if (misaligned(weight, 16)) return fail(MOE_ERR_INVALID_ARGUMENT, "weight must be 16-byte aligned");
  return check_dropout(p, rng);
}

// What the adapters' two entry points share: their arguments but the matrices
// by slot.
struct LoraCommon {
  int64_t S, K, N;
  int32_t G, R;
  const void* x;
  int64_t x_ld;
  int32_t x_row_div;
  const void* a;
  int64_t a_stride_g, a_ld;
  const void* b;
  int64_t b_stride_g, b_ld;
  const float* scale;
  const int32_t* sorted;
  const int32_t* groups;
  int32_t block_m;
  int64_t max_blocks;
};

template <class T>
LoraCommon lora_common(const T& a) {
  return {a.num_slots, a.k,          a.n,    a.num_groups, a.rank,           a.x,
          a.x_ld,      a.x_row_div,  a.a,    a.a_stride_g, a.a_ld,           a.b,
          a.b_stride_g, a.b_ld,      a.scale, a.sorted_slot_ids, a.group_ids, a.block_m,
          a.max_blocks};
}

moe_status check_lora_sizes(int64_t S, int32_t G, int32_t R, int64_t K, int64_t N, int32_t bm, int64_t max_blocks) {
  if (S < 0 || S > INT32_MAX - 65536)
    return fail(MOE_ERR_INVALID_ARGUMENT, "num_slots must be in [0, 2^31 - 2^16]");
  if (G < 1) return fail(MOE_ERR_INVALID_ARGUMENT, "num_groups < 1");
  if (G > kAlignMaxExperts) return fail(MOE_ERR_UNSUPPORTED, "num_groups %d > %d", G, kAlignMaxExperts);
  if (R < 8 || R % 8 != 0) return fail(MOE_ERR_INVALID_ARGUMENT, "rank must be a positive multiple of 8");
  if (R > kLoraMaxRank) return fail(MOE_ERR_UNSUPPORTED, "rank %d > %d", R, kLoraMaxRank);
  if (K < 8 || K % 8 != 0 || N < 8 || N % 8 != 0 || K >= kLoraMaxWidth || N >= kLoraMaxWidth)
    return fail(MOE_ERR_INVALID_ARGUMENT, "k and n must be positive multiples of 8, below 2^24");
  if (bm != 8 && bm != 16 && bm != 32 && bm != 64)
    return fail(MOE_ERR_INVALID_ARGUMENT, "block_m must be 8, 16, 32 or 64");
  const int64_t need = moe_align_max_blocks(S, G, bm);
  if (max_blocks < need)
    return fail(MOE_ERR_INVALID_ARGUMENT, "max_blocks %lld < required %lld", (long long)max_blocks, (long long)need);
  if (max_blocks * bm >= INT32_MAX) return fail(MOE_ERR_INVALID_ARGUMENT, "max_blocks too large");
  return MOE_OK;
}

moe_status check_lora(const LoraCommon& a) {
  moe_status st = check_lora_sizes(a.S, a.G, a.R, a.K, a.N, a.block_m, a.max_blocks);
  if (st != MOE_OK) return st;
  if (a.x_row_div < 1) return fail(MOE_ERR_INVALID_ARGUMENT, "x_row_div < 1");
  const int64_t rows = a.S > 0 ? (a.S - 1) / a.x_row_div + 1 : 0;
  st = check_rows("x", a.x, a.x_ld, rows, a.K, true);
  if (st == MOE_OK) st = check_rows("a", a.a, a.a_ld, a.R, a.K, true);
  if (st == MOE_OK) st = check_rows("b", a.b, a.b_ld, a.N, a.R, true);
  if (st != MOE_OK) return st;
  if (bad_ld(a.a_stride_g, a.R * a.a_ld, 8, a.G) || bad_ld(a.b_stride_g, a.N * a.b_ld, 8, a.G))
    return fail(MOE_ERR_INVALID_ARGUMENT, "a_stride_g and b_stride_g must cover a matrix and be multiples of 8");
  if (a.max_blocks > 0 && (a.sorted == nullptr || a.groups == nullptr))
    return fail(MOE_ERR_INVALID_ARGUMENT, "the block list is null");
  if (misaligned(a.scale, 4) || misaligned(a.sorted, 4) || misaligned(a.groups, 4))
    return fail(MOE_ERR_INVALID_ARGUMENT, "scale and the block list must be 4-byte aligned");
  return MOE_OK;
}

// One of `outs` overlaps another or an input of both entry points.
bool lora_clash(const LoraCommon& a, std::initializer_list<Range> outs) {
  const int64_t rows = a.S > 0 ? (a.S - 1) / a.x_row_div + 1 : 0;
  return clash(outs, {span(a.x, rows, a.x_ld, a.K, 2), {a.a, ((a.G - 1) * a.a_stride_g + (a.R - 1) * a.a_ld + a.K) * 2},
                      {a.b, ((a.G - 1) * a.b_stride_g + (a.N - 1) * a.b_ld + a.R) * 2}, {a.scale, a.G * 4},
                      {a.sorted, a.max_blocks * a.block_m * 4}, {a.groups, a.max_blocks * 4}});
}

moe::LoraParams lora_params(const LoraCommon& a) {
  moe::LoraParams p{};
  p.S = (int32_t)a.S;
  p.G = a.G;
  p.R = a.R;
  p.K = (int32_t)a.K;
  p.N = (int32_t)a.N;
  p.bm = a.block_m;
  p.max_blocks = (int32_t)a.max_blocks;
  p.sorted = a.sorted;
  p.groups = a.groups;
  p.scale = a.scale;
  return p;
}

}  // namespace

extern "C" {

moe_status moe_dropout(const void* x, int64_t x_ld, int64_t rows, int64_t n, float p, const uint64_t* rng, void* y,
                       int64_t y_ld, moe_stream_t stream) {
  if (rows < 0) return fail(MOE_ERR_INVALID_ARGUMENT, "rows < 0");
  if (n < 8 || n % 8 != 0 || n >= INT32_MAX)
    return fail(MOE_ERR_INVALID_ARGUMENT, "n must be a positive multiple of 8, below 2^31");
  if (rows >= moe::kMaxElements / n) return fail(MOE_ERR_INVALID_ARGUMENT, "rows * n must be below 2^60");
  moe_status st = check_dropout(p, rng);
  if (st == MOE_OK) st = check_rows("x", x, x_ld, rows, n, true);
  if (st == MOE_OK) st = check_rows("y", y, y_ld, rows, n, true);
  if (st != MOE_OK) return st;
  const Range in = x == y && x_ld == y_ld ? Range{nullptr, 0} : span(x, rows, x_ld, n, 2);
  if (clash({span(y, rows, y_ld, n, 2)}, {in, {rng, 16}}))
    return fail(MOE_ERR_INVALID_ARGUMENT, "y overlaps rng, or x without being x");
  st = check_device();
  if (st != MOE_OK) return st;
  return hip_status(moe::launch_dropout(static_cast<const uint16_t*>(x), x_ld, rows, n, p, rng,
                                        static_cast<uint16_t*>(y), y_ld, (hipStream_t)stream),
                    "moe_dropout launch");
}

moe_status moe_rmsnorm(const moe_rmsnorm_args* args, moe_stream_t stream) {
  if (args == nullptr) return fail(MOE_ERR_INVALID_ARGUMENT, "args is null");
  const moe_rmsnorm_args& a = *args;
  const int64_t rows = a.rows, n = a.n;
  if (a.quant != MOE_QUANT_NONE && a.quant != MOE_QUANT_MXFP8 && a.quant != MOE_QUANT_PER_TOKEN)
    return fail(MOE_ERR_INVALID_ARGUMENT, "unknown quant %d", a.quant);
  const bool mx = a.quant == MOE_QUANT_MXFP8, codes = a.quant != MOE_QUANT_NONE;
  moe_status st =
      check_norm(rows, n, mx ? 32 : 8, a.residual_dtype, a.weight, a.weight_dtype, a.eps, a.p, a.rng);
  if (st == MOE_OK) st = check_rows("x", a.x, a.x_ld, rows, n, true);
  if (st == MOE_OK) st = check_rows("residual", a.residual, a.residual_ld, rows, n, false);
  if (st == MOE_OK) st = check_rows("sum", a.sum, a.sum_ld, rows, n, false);
  if (st == MOE_OK) st = check_rows("y", a.y, a.y_ld, rows, n, !codes);
  if (st != MOE_OK) return st;
  if (codes) {
    if (rows > 0 && (a.q == nullptr || a.scales == nullptr))
      return fail(MOE_ERR_INVALID_ARGUMENT, "a quant needs q and scales");
    if (bad_ld(a.q_ld, n, 8, rows))
      return fail(MOE_ERR_INVALID_ARGUMENT, "q_ld must be >= n and a multiple of 8");
    if (mx && bad_ld(a.scales_ld, n / 32, 1, rows))
      return fail(MOE_ERR_INVALID_ARGUMENT, "scales_ld must be >= n / 32");
    if (misaligned(a.q, 8) || (!mx && misaligned(a.scales, 4)))
      return fail(MOE_ERR_INVALID_ARGUMENT, "q must be 8-byte aligned, per-token scales 4-byte");
  }
  const int64_t es = dtype_bytes(a.residual_dtype), on = codes ? 1 : 0;
  const bool in_place = a.sum != nullptr && a.sum == a.residual && a.sum_ld == a.residual_ld;
  const Range res = span(a.residual, rows, a.residual_ld, n, es), sum = span(a.sum, rows, a.sum_ld, n, es);
  const Range y = span(a.y, rows, a.y_ld, n, 2), q = span(a.q, on * rows, a.q_ld, n, 1);
  const Range scales = mx ? span(a.scales, rows, a.scales_ld, n / 32, 1) : Range{a.scales, on * rows * 4};
  const Range x = span(a.x, rows, a.x_ld, n, 2);
  const Range w = {a.weight, n * dtype_bytes(a.weight_dtype)}, rng = {a.rng, 16};
  if (clash({sum, y, q, scales}, {x, w, rng}) || clash({y, q, scales}, {res}) || (!in_place && clash({sum}, {res})))
    return fail(MOE_ERR_INVALID_ARGUMENT, "the outputs overlap each other or an input");
  st = check_device();
  if (st != MOE_OK) return st;
  moe::NormParams p{};
  p.rows = rows;
  p.pieces = (int32_t)(n / 8);
  p.eps = a.eps;
  p.n = (float)n;
  p.x = static_cast<const uint16_t*>(a.x);
  p.x_ld = a.x_ld;
  p.res = a.residual;
  p.res_ld = a.residual_ld;
  p.sum = a.sum;
  p.sum_ld = a.sum_ld;
  p.wide = a.residual_dtype == MOE_FP32;
  p.w = a.weight;
  p.w_wide = a.weight_dtype == MOE_FP32;
  p.y = static_cast<uint16_t*>(a.y);
  p.y_ld = a.y_ld;
  p.quant = a.quant;
  p.q = static_cast<uint8_t*>(a.q);
  p.q_ld = a.q_ld;
  p.scales = a.scales;
  p.scales_ld = a.scales_ld;
  return hip_status(moe::launch_norm(p, moe::make_dropout(a.p, a.rng), (hipStream_t)stream), "moe_rmsnorm launch");
}

int64_t moe_rmsnorm_backward_workspace_bytes(int64_t rows, int64_t n) {
  if (rows < 0 || rows >= INT32_MAX || n < 8 || n % 8 != 0 || n > kNormMaxWidth) return -1;
  return moe::norm_backward_workspace_bytes(rows, n);
}

moe_status moe_rmsnorm_backward(const moe_rmsnorm_backward_args* args, moe_stream_t stream) {
  if (args == nullptr) return fail(MOE_ERR_INVALID_ARGUMENT, "args is null");
  const moe_rmsnorm_backward_args& a = *args;
  const int64_t rows = a.rows, n = a.n;
  moe_status st = check_norm(rows, n, 8, a.sum_dtype, a.weight, a.weight_dtype, a.eps, a.p, a.rng);
  if (st == MOE_OK) st = check_rows("dy", a.dy, a.dy_ld, rows, n, true);
  if (st == MOE_OK) st = check_rows("sum", a.sum, a.sum_ld, rows, n, true);
  if (st == MOE_OK) st = check_rows("dsum", a.dsum, a.dsum_ld, rows, n, false);
  if (st == MOE_OK) st = check_rows("dresidual", a.dresidual, a.dresidual_ld, rows, n, false);
  if (st == MOE_OK) st = check_rows("dx", a.dx, a.dx_ld, rows, n, false);
  if (st != MOE_OK) return st;
  if (a.dresidual == nullptr && a.dx == nullptr && a.dweight == nullptr && rows > 0)
    return fail(MOE_ERR_INVALID_ARGUMENT, "one of dresidual, dx and dweight is needed");
  const int64_t need = a.dweight != nullptr ? moe_rmsnorm_backward_workspace_bytes(rows, n) : 0;
  if (a.workspace_bytes < need || (need > 0 && a.workspace == nullptr))
    return fail(MOE_ERR_INVALID_ARGUMENT, "workspace of %lld bytes, %lld needed", (long long)a.workspace_bytes,
                (long long)need);
  if (misaligned(a.dweight, 4) || (need > 0 && misaligned(a.workspace, 16)))
    return fail(MOE_ERR_INVALID_ARGUMENT, "dweight must be 4-byte aligned, workspace 16-byte");
  const int64_t es = dtype_bytes(a.sum_dtype);
  const bool in_place = a.dresidual != nullptr && a.dresidual == a.dsum && a.dresidual_ld == a.dsum_ld;
  const Range dres = span(a.dresidual, rows, a.dresidual_ld, n, es), dsum = span(a.dsum, rows, a.dsum_ld, n, es);
  const Range dx = span(a.dx, rows, a.dx_ld, n, 2), dw = {a.dweight, n * 4}, ws = {a.workspace, need};
  const Range dy = span(a.dy, rows, a.dy_ld, n, 2), sum = span(a.sum, rows, a.sum_ld, n, es);
  const Range w = {a.weight, n * dtype_bytes(a.weight_dtype)}, rng = {a.rng, 16};
  if (clash({dres, dx, dw, ws}, {dy, sum, w, rng}) || clash({dx, dw, ws}, {dsum}) || (!in_place && clash({dres}, {dsum})))
    return fail(MOE_ERR_INVALID_ARGUMENT, "the outputs overlap each other, the workspace or an input");
  st = check_device();
  if (st != MOE_OK) return st;
  moe::NormParams p{};
  p.rows = rows;
  p.pieces = (int32_t)(n / 8);
  p.eps = a.eps;
  p.n = (float)n;
  p.x = static_cast<const uint16_t*>(a.dy);
  p.x_ld = a.dy_ld;
  p.res = a.dsum;
  p.res_ld = a.dsum_ld;
  p.v = a.sum;
  p.v_ld = a.sum_ld;
  p.sum = a.dresidual;
  p.sum_ld = a.dresidual_ld;
  p.wide = a.sum_dtype == MOE_FP32;
  p.w = a.weight;
  p.w_wide = a.weight_dtype == MOE_FP32;
  p.y = static_cast<uint16_t*>(a.dx);
  p.y_ld = a.dx_ld;
  p.dw = a.dweight;
  p.partial = static_cast<float*>(a.workspace);
  return hip_status(moe::launch_norm_backward(p, moe::make_dropout(a.p, a.rng), (hipStream_t)stream),
                    "moe_rmsnorm_backward launch");
}

int32_t moe_lora_block_m(int64_t num_slots, int32_t num_groups) {
  if (num_slots < 0 || num_groups < 1) return -1;
  return num_slots >= 32 * (int64_t)num_groups ? 64 : 16;
}

int64_t moe_lora_workspace_bytes(int64_t num_slots, int32_t num_groups, int32_t rank, int64_t k, int64_t n,
                                 int32_t block_m, int64_t max_blocks) {
  if (check_lora_sizes(num_slots, num_groups, rank, k, n, block_m, max_blocks) != MOE_OK) return -1;
  return moe::lora_sizes(rank, k, block_m, max_blocks).bytes;
}

moe_status moe_lora(const moe_lora_args* args, moe_stream_t stream) {
  if (args == nullptr) return fail(MOE_ERR_INVALID_ARGUMENT, "args is null");
  const LoraCommon a = lora_common(*args);
  moe_status st = check_lora(a);
  if (st == MOE_OK) st = check_rows("c", args->c, args->c_ld, a.S, a.N, true);
  if (st != MOE_OK) return st;
  if (misaligned(args->h, 16) || misaligned(args->workspace, 16))
    return fail(MOE_ERR_INVALID_ARGUMENT, "h and workspace must be 16-byte aligned");
  const int64_t need = moe_lora_workspace_bytes(a.S, a.G, a.R, a.K, a.N, a.block_m, a.max_blocks);
  if (args->workspace_bytes < need || (need > 0 && args->workspace == nullptr))
    return fail(MOE_ERR_INVALID_ARGUMENT, "workspace of %lld bytes, %lld needed", (long long)args->workspace_bytes,
                (long long)need);
  if (lora_clash(a, {span(args->c, a.S, args->c_ld, a.N, 2), {args->h, a.S * a.R * 4}, {args->workspace, need}}))
    return fail(MOE_ERR_INVALID_ARGUMENT, "c, h or workspace overlaps another or an input");
  st = check_device();
  if (st != MOE_OK) return st;
  if (a.S == 0) return ok();
  moe::LoraParams p = lora_params(a);
  p.x = static_cast<const uint16_t*>(a.x);
  p.x_ld = a.x_ld;
  moe::lora_set_division(a.x_row_div, p.div_magic, p.div_shift);
  p.w = static_cast<const uint16_t*>(a.a);
  p.w_g = a.a_stride_g;
  p.w_ld = a.a_ld;
  const moe::LoraSizes z = moe::lora_sizes(a.R, a.K, a.block_m, a.max_blocks);
  p.splits = z.splits;
  p.h = args->h;
  p.w2 = static_cast<const uint16_t*>(a.b);
  p.w2_g = a.b_stride_g;
  p.w2_ld = a.b_ld;
  p.c = static_cast<uint16_t*>(args->c);
  p.c_ld = args->c_ld;
  if (z.both) return hip_status(moe::launch_lora_both(p, (hipStream_t)stream), "moe_lora launch");
  p.part = static_cast<float*>(args->workspace);
  p.scaled = !z.few && z.splits == 1;
  st = hip_status(moe::launch_lora_down(p, (hipStream_t)stream), "moe_lora launch");
  if (st != MOE_OK) return st;
  if (!z.few && z.splits > 1) {
    st = hip_status(moe::launch_lora_join(p, (hipStream_t)stream), "moe_lora launch");
    if (st != MOE_OK) return st;
    p.scaled = true;
  }
  return hip_status(z.few ? moe::launch_lora_up_few(p, (hipStream_t)stream)
                          : moe::launch_lora_up(p, false, (hipStream_t)stream),
                    "moe_lora launch");
}

int64_t moe_lora_backward_workspace_bytes(int64_t num_slots, int32_t num_groups, int32_t rank, int64_t k, int64_t n,
                                          int32_t block_m, int64_t max_blocks) {
  if (check_lora_sizes(num_slots, num_groups, rank, k, n, block_m, max_blocks) != MOE_OK) return -1;
  return moe::lora_grad_sizes(num_groups, rank, k, n, block_m, max_blocks).bytes;
}

moe_status moe_lora_backward(const moe_lora_backward_args* args, moe_stream_t stream) {
  if (args == nullptr) return fail(MOE_ERR_INVALID_ARGUMENT, "args is null");
  const LoraCommon a = lora_common(*args);
  const bool weights = args->da != nullptr;
  if (weights != (args->db != nullptr)) return fail(MOE_ERR_INVALID_ARGUMENT, "da and db: both or neither");
  moe_status st = check_lora(a);
  if (st == MOE_OK) st = check_rows("dy", args->dy, args->dy_ld, a.S, a.N, true);
  if (st == MOE_OK) st = check_rows("dx", args->dx, args->dx_ld, a.S, a.K, false);
  if (st != MOE_OK) return st;
  if (!weights && args->dx == nullptr && a.S > 0)
    return fail(MOE_ERR_INVALID_ARGUMENT, "one of dx and the weights' gradients is needed");
  if (weights && a.S > 0 && args->h == nullptr) return fail(MOE_ERR_INVALID_ARGUMENT, "h is null");
  if (misaligned(args->h, 16) || misaligned(args->da, 16) || misaligned(args->db, 16) ||
      misaligned(args->workspace, 16))
    return fail(MOE_ERR_INVALID_ARGUMENT, "h, da, db and workspace must be 16-byte aligned");
  const moe::LoraGradSizes z = moe::lora_grad_sizes(a.G, a.R, a.K, a.N, a.block_m, a.max_blocks);
  if (args->workspace_bytes < z.bytes || (z.bytes > 0 && args->workspace == nullptr))
    return fail(MOE_ERR_INVALID_ARGUMENT, "workspace of %lld bytes, %lld needed", (long long)args->workspace_bytes,
                (long long)z.bytes);
  const Range dy = span(args->dy, a.S, args->dy_ld, a.N, 2), h = {args->h, a.S * a.R * 4};
  const Range dx = span(args->dx, a.S, args->dx_ld, a.K, 2), ws = {args->workspace, z.bytes};
  const Range da = {args->da, a.G * a.R * a.K * 4}, db = {args->db, a.G * a.R * a.N * 4};
  if (lora_clash(a, {dx, da, db, ws}) || clash({dx, da, db, ws}, {dy, h}))
    return fail(MOE_ERR_INVALID_ARGUMENT, "dx, da, db or workspace overlaps another or an input");
  st = check_device();
  if (st != MOE_OK) return st;
  if (a.S == 0 && !weights) return ok();
  char* base = static_cast<char*>(args->workspace);
  moe::LoraGradParams q{};
  q.S = (int32_t)a.S;
  q.G = a.G;
  q.R = a.R;
  q.K = (int32_t)a.K;
  q.N = (int32_t)a.N;
  q.bm = a.block_m;
  q.max_blocks = (int32_t)a.max_blocks;
  q.sorted = a.sorted;
  q.groups = a.groups;
  q.scale = a.scale;
  q.x = static_cast<const uint16_t*>(a.x);
  q.x_ld = a.x_ld;
  moe::lora_set_division(a.x_row_div, q.div_magic, q.div_shift);
  q.dy = static_cast<const uint16_t*>(args->dy);
  q.dy_ld = args->dy_ld;
  q.h = args->h;
  q.da = args->da;
  q.db = args->db;
  q.b = static_cast<const uint16_t*>(a.b);
  q.b_g = a.b_stride_g;
  q.b_ld = a.b_ld;
  q.dh = reinterpret_cast<float*>(base + z.dh);
  if (z.seg_blocks > 1) q.table = reinterpret_cast<int32_t*>(base + z.table);
  if (z.direct) q.parts = z.n_parts;
  q.seg_blocks = z.seg_blocks;
  q.max_segs = z.max_segs;
  q.max_parts = z.max_parts;
  q.da_part = reinterpret_cast<float*>(base + z.da_part);
  q.db_part = reinterpret_cast<float*>(base + z.db_part);
  if (a.S == 0) q.max_blocks = 0;  // (a list then names no slot)
  moe::LoraParams p = lora_params(a);
  p.max_blocks = q.max_blocks;
  p.part = q.dh;
  p.splits = z.n_parts;
  p.scaled = !z.direct;
  const hipStream_t on = (hipStream_t)stream;
  hipError_t err = z.seg_blocks > 1 ? moe::launch_lora_grad_table(q, on) : hipSuccess;
  if (err == hipSuccess) err = moe::launch_lora_grad_dy(q, on);
  if (err == hipSuccess && !z.direct) err = moe::launch_lora_join(p, on);
  if (err == hipSuccess && args->dx != nullptr) {
    p.N = (int32_t)a.K;
    p.w2 = static_cast<const uint16_t*>(a.a);
    p.w2_g = a.a_stride_g;
    p.w2_ld = a.a_ld;
    p.c = static_cast<uint16_t*>(args->dx);
    p.c_ld = args->dx_ld;
    err = moe::launch_lora_up(p, true, on);
  }
  if (err == hipSuccess && weights) err = moe::launch_lora_grad_x(q, on);
  if (err == hipSuccess && weights) err = moe::launch_lora_grad_join(q, on);
  return hip_status(err, "moe_lora_backward launch");
}

}  // extern "C"
