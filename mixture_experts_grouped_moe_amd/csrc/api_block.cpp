// Host side of libmoe's block entry points (include/moe_block.h): argument
// validation before anything touches the GPU, and dispatch.
#include <hip/hip_runtime.h>

#include <climits>
#include <cmath>

#include "moe_block.h"

#include "dropout_util.h"
#include "host.h"
#include "params.h"
#include "ranges.h"

namespace {

using moe::bad_ld;
using moe::check_device;
using moe::clash;
using moe::fail;
using moe::hip_status;
using moe::misaligned;
using moe::ok;
using moe::Range;
using moe::span;

constexpr int64_t kNormMaxWidth = 16384;

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
  if (rows < 0 || rows >= INT32_MAX) return fail(MOE_ERR_INVALID_ARGUMENT, "rows must be in [0, 2^31)");
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

}  // extern "C"
