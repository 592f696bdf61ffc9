// Host side of libmoe's training entry points (include/moe_train.h):
// argument validation before anything touches the GPU, and dispatch.
#include <hip/hip_runtime.h>

#include <climits>
#include <cmath>
#include <initializer_list>
#include <utility>

#include "moe_train.h"

#include "host.h"
#include "params.h"

namespace {

using moe::check_device;
using moe::fail;
using moe::hip_status;
using moe::kAlignMaxExperts;
using moe::ok;

constexpr int32_t kRouteMaxTopK = 64;
constexpr int64_t kBufMax = (int64_t)0x80000000;
constexpr int64_t kMaxElements = (int64_t)1 << 60;  // rows * stride at most: byte offsets fit 64 bits

// `rows` rows of `width` bytes, `ld` bytes apart, from p.
struct Range {
  const void* p;
  int64_t width;
  int64_t rows = 1, ld = 0;
};

// `rows` rows of `width` elements, `ld` elements apart.
Range span(const void* p, int64_t rows, int64_t ld, int64_t width, int64_t bytes) {
  if (rows <= 1 || ld == width) return {p, rows * width * bytes};
  return {p, width * bytes, rows, ld * bytes};
}

// a and b share a byte. Exact for blocks and for rows of equal strides; rows
// of unequal strides count as sharing one where their first-to-last bytes do.
// (Null and empty ranges share none.)
bool share(Range a, Range b) {
  uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  if (x == 0 || y == 0 || a.width <= 0 || b.width <= 0) return false;
  if (y < x) {
    std::swap(a, b);
    std::swap(x, y);
  }
  const uint64_t off = y - x;  // b starts at this byte of a's
  if (off >= (uint64_t)((a.rows - 1) * a.ld + a.width)) return false;
  if (a.rows == 1 || (b.rows > 1 && b.ld != a.ld)) return true;
  // b's first row starts in a row of a or in the gap behind one; a further row
  // of a follows that gap, so b has to end before it. b's other rows, at the
  // same stride, repeat this.
  const uint64_t at = off % (uint64_t)a.ld;
  return at < (uint64_t)a.width || at + (uint64_t)b.width > (uint64_t)a.ld;
}

// One of `outs` shares a byte with another of them or with one of `ins`.
bool clash(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
  for (const Range* a = outs.begin(); a != outs.end(); ++a) {
    for (const Range* b = a + 1; b != outs.end(); ++b)
      if (share(*a, *b)) return true;
    for (const Range& b : ins)
      if (share(*a, b)) return true;
  }
  return false;
}

// A row stride that does not cover `width`, is no multiple of `multiple`, or
// takes `rows` rows past kMaxElements.
bool bad_ld(int64_t ld, int64_t width, int64_t multiple, int64_t rows) {
  return ld < width || ld % multiple != 0 || ld > kMaxElements / (rows > 1 ? rows : 1);
}

bool misaligned(const void* p, uintptr_t to) { return (uintptr_t)p % to != 0; }

// What moe_route and moe_route_backward check alike.
moe_status check_route(const void* logits, int32_t dtype, int64_t ld, int64_t T, int32_t E, int32_t k, int32_t score,
                       float scale, const int32_t* ids) {
  if (T < 0) return fail(MOE_ERR_INVALID_ARGUMENT, "num_tokens < 0");
  if (k < 1 || E < k) return fail(MOE_ERR_INVALID_ARGUMENT, "need 1 <= top_k (%d) <= num_experts (%d)", k, E);
  if (E > kAlignMaxExperts) return fail(MOE_ERR_UNSUPPORTED, "num_experts %d > %d", E, kAlignMaxExperts);
  if (k > kRouteMaxTopK) return fail(MOE_ERR_UNSUPPORTED, "top_k %d > %d", k, kRouteMaxTopK);
  if (T > (INT32_MAX - 65536) / k)
    return fail(MOE_ERR_INVALID_ARGUMENT, "num_tokens * top_k must be <= 2^31 - 2^16");
  if (dtype != MOE_FP32 && dtype != MOE_BF16)
    return fail(MOE_ERR_UNSUPPORTED, "logits must be MOE_FP32 or MOE_BF16");
  if (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID)
    return fail(MOE_ERR_INVALID_ARGUMENT, "unknown score %d", score);
  if (!std::isfinite(scale)) return fail(MOE_ERR_INVALID_ARGUMENT, "scale is not finite");
  if (bad_ld(ld, E, 1, T)) return fail(MOE_ERR_INVALID_ARGUMENT, "logits_ld must be >= num_experts");
  if (T > 0 && (logits == nullptr || ids == nullptr)) return fail(MOE_ERR_INVALID_ARGUMENT, "null pointer argument");
  if (misaligned(logits, dtype == MOE_FP32 ? 4 : 2) || misaligned(ids, 4))
    return fail(MOE_ERR_INVALID_ARGUMENT, "logits and topk_ids must be aligned to their elements");
  return MOE_OK;
}

// The sizes, strides and alignment that both combine entry points share.
moe_status check_combine(int64_t T, int32_t k, int64_t n) {
  if (T < 0 || k < 1) return fail(MOE_ERR_INVALID_ARGUMENT, "num_tokens < 0 or top_k < 1");
  if (n < 8 || n % 8 != 0 || n >= INT32_MAX)
    return fail(MOE_ERR_INVALID_ARGUMENT, "n must be a positive multiple of 8");
  if (T > (INT32_MAX - 65536) / k)
    return fail(MOE_ERR_INVALID_ARGUMENT, "num_tokens * top_k must be <= 2^31 - 2^16");
  return MOE_OK;
}

// What both activation entry points check alike; `out` is the width of h.
moe_status check_act(int32_t act, int64_t rows, int64_t n, const void* q, int64_t q_ld, const uint8_t* scales,
                     int64_t scales_ld, int64_t* out) {
  if (act != MOE_EPILOGUE_SWIGLU && act != MOE_EPILOGUE_RELU2)
    return fail(MOE_ERR_INVALID_ARGUMENT, "act must be MOE_EPILOGUE_SWIGLU or MOE_EPILOGUE_RELU2");
  const bool swiglu = act == MOE_EPILOGUE_SWIGLU;
  if (rows < 0 || rows >= INT32_MAX) return fail(MOE_ERR_INVALID_ARGUMENT, "rows must be in [0, 2^31)");
  const int64_t unit = swiglu ? 64 : 32;
  if (n < unit || n % unit != 0 || n >= INT32_MAX)
    return fail(MOE_ERR_INVALID_ARGUMENT, "n must be a positive multiple of %lld", (long long)unit);
  if (bad_ld(q_ld, n, 16, rows))
    return fail(MOE_ERR_INVALID_ARGUMENT, "q_ld must be >= n and a multiple of 16");
  if (bad_ld(scales_ld, n / 32, 1, rows)) return fail(MOE_ERR_INVALID_ARGUMENT, "scales_ld must be >= n / 32");
  if (rows > 0 && (q == nullptr || scales == nullptr)) return fail(MOE_ERR_INVALID_ARGUMENT, "null pointer argument");
  *out = swiglu ? n / 2 : n;
  return MOE_OK;
}

}  // namespace

extern "C" {

int64_t moe_route_workspace_bytes(int64_t num_tokens, int32_t num_experts) {
  if (num_tokens < 0 || num_experts < 1 || num_experts > kAlignMaxExperts) return -1;
  return moe::route_workspace_bytes(num_tokens, num_experts);
}

moe_status moe_route(const void* logits, int32_t logits_dtype, int64_t logits_ld, const uint8_t* token_mask,
                     int64_t num_tokens, int32_t num_experts, int32_t top_k, int32_t score, int32_t renormalize,
                     float scale, int32_t* topk_ids, float* topk_w, int32_t stats, int32_t* counts,
                     int32_t* num_routed, float* prob_sum, float* losses, void* workspace, int64_t workspace_bytes,
                     moe_stream_t stream) {
  moe_status st =
      check_route(logits, logits_dtype, logits_ld, num_tokens, num_experts, top_k, score, scale, topk_ids);
  if (st != MOE_OK) return st;
  if (num_tokens > 0 && topk_w == nullptr) return fail(MOE_ERR_INVALID_ARGUMENT, "null pointer argument");
  if (misaligned(topk_w, 4)) return fail(MOE_ERR_INVALID_ARGUMENT, "topk_w must be 4-byte aligned");
  if (stats) {
    if (counts == nullptr || num_routed == nullptr || prob_sum == nullptr || losses == nullptr)
      return fail(MOE_ERR_INVALID_ARGUMENT, "the statistics need counts, num_routed, prob_sum and losses");
    if (misaligned(counts, 4) || misaligned(num_routed, 4) || misaligned(prob_sum, 4) || misaligned(losses, 4))
      return fail(MOE_ERR_INVALID_ARGUMENT, "the statistics must be 4-byte aligned");
    const int64_t need = moe_route_workspace_bytes(num_tokens, num_experts);
    if (workspace_bytes < need || (need > 0 && workspace == nullptr))
      return fail(MOE_ERR_INVALID_ARGUMENT, "workspace of %lld bytes, %lld needed", (long long)workspace_bytes,
                  (long long)need);
    if (misaligned(workspace, 8)) return fail(MOE_ERR_INVALID_ARGUMENT, "workspace must be 8-byte aligned");
  }
  const int64_t T = num_tokens, E = num_experts, slots = T * top_k, on = stats ? 1 : 0;
  if (clash({{topk_ids, slots * 4}, {topk_w, slots * 4}, {counts, on * E * 4}, {num_routed, on * 4},
             {prob_sum, on * E * 4}, {losses, on * 8}, {workspace, on * moe_route_workspace_bytes(T, num_experts)}},
            {span(logits, T, logits_ld, E, logits_dtype == MOE_FP32 ? 4 : 2), {token_mask, T}}))
    return fail(MOE_ERR_INVALID_ARGUMENT, "the outputs overlap each other, the workspace or an input");
  st = check_device();
  if (st != MOE_OK) return st;
  moe::RouteParams p{};
  p.logits = logits;
  p.ld = logits_ld;
  p.mask = token_mask;
  p.T = num_tokens;
  p.E = num_experts;
  p.k = top_k;
  p.sigmoid = score == MOE_SCORE_SIGMOID;
  p.renorm = renormalize != 0;
  p.stats = stats != 0;
  p.scale = scale;
  p.ids = topk_ids;
  p.w = topk_w;
  p.counts = counts;
  p.num_routed = num_routed;
  p.prob_sum = prob_sum;
  p.losses = losses;
  return hip_status(moe::launch_route(p, logits_dtype == MOE_BF16, workspace, (hipStream_t)stream),
                    "moe_route launch");
}

moe_status moe_route_backward(const void* logits, int32_t logits_dtype, int64_t logits_ld, int64_t num_tokens,
                              int32_t num_experts, int32_t top_k, int32_t score, int32_t renormalize, float scale,
                              const int32_t* topk_ids, const float* dtopk_w, const int32_t* counts,
                              const int32_t* num_routed, const float* dlosses, void* dlogits, int64_t dlogits_ld,
                              moe_stream_t stream) {
  moe_status st =
      check_route(logits, logits_dtype, logits_ld, num_tokens, num_experts, top_k, score, scale, topk_ids);
  if (st != MOE_OK) return st;
  if (bad_ld(dlogits_ld, num_experts, 1, num_tokens))
    return fail(MOE_ERR_INVALID_ARGUMENT, "dlogits_ld must be >= num_experts");
  if (num_tokens > 0 && (dtopk_w == nullptr || dlogits == nullptr))
    return fail(MOE_ERR_INVALID_ARGUMENT, "null pointer argument");
  if (dlosses != nullptr && (counts == nullptr || num_routed == nullptr))
    return fail(MOE_ERR_INVALID_ARGUMENT, "dlosses need counts and num_routed");
  const int64_t es = logits_dtype == MOE_FP32 ? 4 : 2;
  if (misaligned(dtopk_w, 4) || misaligned(counts, 4) || misaligned(num_routed, 4) || misaligned(dlosses, 4) ||
      misaligned(dlogits, (uintptr_t)es))
    return fail(MOE_ERR_INVALID_ARGUMENT, "pointers must be aligned to their elements");
  const int64_t T = num_tokens, E = num_experts, slots = T * top_k, on = dlosses != nullptr ? 1 : 0;
  if (clash({span(dlogits, T, dlogits_ld, E, es)},
            {span(logits, T, logits_ld, E, es), {topk_ids, slots * 4}, {dtopk_w, slots * 4}, {counts, on * E * 4},
             {num_routed, on * 4}, {dlosses, 8}}))
    return fail(MOE_ERR_INVALID_ARGUMENT, "dlogits overlaps an input");
  st = check_device();
  if (st != MOE_OK) return st;
  moe::RouteParams p{};
  p.logits = logits;
  p.ld = logits_ld;
  p.T = num_tokens;
  p.E = num_experts;
  p.k = top_k;
  p.sigmoid = score == MOE_SCORE_SIGMOID;
  p.renorm = renormalize != 0;
  p.scale = scale;
  p.ids = const_cast<int32_t*>(topk_ids);
  p.counts = const_cast<int32_t*>(counts);
  p.num_routed = const_cast<int32_t*>(num_routed);
  p.dw = dtopk_w;
  p.dlosses = dlosses;
  p.dlogits = dlogits;
  p.dld = dlogits_ld;
  return hip_status(moe::launch_route_backward(p, logits_dtype == MOE_BF16, (hipStream_t)stream),
                    "moe_route_backward launch");
}

moe_status moe_combine_routed(const void* c, int64_t c_ld, const float* topk_w, const int32_t* topk_ids,
                              int64_t num_tokens, int32_t top_k, int32_t num_experts, int64_t n, void* y, int64_t y_ld,
                              moe_stream_t stream) {
  moe_status st = check_combine(num_tokens, top_k, n);
  if (st != MOE_OK) return st;
  if (num_experts < 1) return fail(MOE_ERR_INVALID_ARGUMENT, "num_experts < 1");
  const int64_t S = num_tokens * top_k;
  if (bad_ld(c_ld, n, 8, S) || bad_ld(y_ld, n, 8, num_tokens))
    return fail(MOE_ERR_INVALID_ARGUMENT, "c_ld and y_ld must be >= n and multiples of 8");
  if (num_tokens > 0 && (c == nullptr || topk_w == nullptr || topk_ids == nullptr || y == nullptr))
    return fail(MOE_ERR_INVALID_ARGUMENT, "null pointer argument");
  if (misaligned(c, 16) || misaligned(y, 16) || misaligned(topk_w, 4) || misaligned(topk_ids, 4))
    return fail(MOE_ERR_INVALID_ARGUMENT, "c and y must be 16-byte aligned, topk_w and topk_ids 4-byte");
  if (clash({span(y, num_tokens, y_ld, n, 2)}, {span(c, S, c_ld, n, 2), {topk_w, S * 4}, {topk_ids, S * 4}}))
    return fail(MOE_ERR_INVALID_ARGUMENT, "y overlaps an input");
  st = check_device();
  if (st != MOE_OK) return st;
  return hip_status(moe::launch_combine_routed(static_cast<const uint16_t*>(c), c_ld, topk_w, topk_ids, num_tokens,
                                               top_k, num_experts, n, static_cast<uint16_t*>(y), y_ld,
                                               (hipStream_t)stream),
                    "moe_combine_routed launch");
}

moe_status moe_combine_backward(const void* dy, int64_t dy_ld, const void* c, int64_t c_ld, const float* topk_w,
                                const int32_t* topk_ids, int64_t num_tokens, int32_t top_k, int32_t num_experts,
                                int64_t n, void* dc, int64_t dc_ld, float* dtopk_w, moe_stream_t stream) {
  moe_status st = check_combine(num_tokens, top_k, n);
  if (st != MOE_OK) return st;
  if (topk_ids != nullptr && num_experts < 1) return fail(MOE_ERR_INVALID_ARGUMENT, "num_experts < 1");
  const int64_t S = num_tokens * top_k;
  if (bad_ld(dy_ld, n, 8, num_tokens) || bad_ld(c_ld, n, 8, S) || bad_ld(dc_ld, n, 8, S))
    return fail(MOE_ERR_INVALID_ARGUMENT, "dy_ld, c_ld and dc_ld must be >= n and multiples of 8");
  if (num_tokens > 0 && (dy == nullptr || c == nullptr || topk_w == nullptr || dc == nullptr || dtopk_w == nullptr))
    return fail(MOE_ERR_INVALID_ARGUMENT, "null pointer argument");
  if (misaligned(dy, 16) || misaligned(c, 16) || misaligned(dc, 16) || misaligned(topk_w, 4) ||
      misaligned(topk_ids, 4) || misaligned(dtopk_w, 4))
    return fail(MOE_ERR_INVALID_ARGUMENT, "dy, c and dc must be 16-byte aligned, the others 4-byte");
  if (clash({span(dc, S, dc_ld, n, 2), {dtopk_w, S * 4}},
            {span(c, S, c_ld, n, 2), span(dy, num_tokens, dy_ld, n, 2), {topk_w, S * 4}, {topk_ids, S * 4}}))
    return fail(MOE_ERR_INVALID_ARGUMENT, "dc and dtopk_w must not overlap each other or an input");
  st = check_device();
  if (st != MOE_OK) return st;
  return hip_status(
      moe::launch_combine_backward(static_cast<const uint16_t*>(dy), dy_ld, static_cast<const uint16_t*>(c), c_ld,
                                   topk_w, topk_ids, num_tokens, top_k, num_experts, n, static_cast<uint16_t*>(dc),
                                   dc_ld, dtopk_w, (hipStream_t)stream),
      "moe_combine_backward launch");
}

moe_status moe_act_mxfp8(int32_t act, const void* pre, int64_t pre_ld, int64_t rows, int64_t n, void* h, int64_t h_ld,
                         void* q, int64_t q_ld, uint8_t* scales, int64_t scales_ld, moe_stream_t stream) {
  int64_t out = 0;
  moe_status st = check_act(act, rows, n, q, q_ld, scales, scales_ld, &out);
  if (st != MOE_OK) return st;
  if (bad_ld(pre_ld, n, 8, rows) || bad_ld(h_ld, out, 8, rows))
    return fail(MOE_ERR_INVALID_ARGUMENT, "pre_ld and h_ld must cover a row and be multiples of 8");
  if (rows > 0 && (pre == nullptr || h == nullptr)) return fail(MOE_ERR_INVALID_ARGUMENT, "null pointer argument");
  if (misaligned(pre, 16) || misaligned(h, 16) || misaligned(q, 16))
    return fail(MOE_ERR_INVALID_ARGUMENT, "pre, h and q must be 16-byte aligned");
  if (clash({span(h, rows, h_ld, out, 2), span(q, rows, q_ld, n, 1), span(scales, rows, scales_ld, n / 32, 1)},
            {span(pre, rows, pre_ld, n, 2)}))
    return fail(MOE_ERR_INVALID_ARGUMENT, "pre, h, q and scales must not overlap");
  st = check_device();
  if (st != MOE_OK) return st;
  moe::ActParams p{};
  p.pre = static_cast<const uint16_t*>(pre);
  p.pre_ld = pre_ld;
  p.rows = rows;
  p.n = (int32_t)n;
  p.h = static_cast<uint16_t*>(h);
  p.h_ld = h_ld;
  p.q = static_cast<uint8_t*>(q);
  p.q_ld = q_ld;
  p.s = scales;
  p.s_ld = scales_ld;
  return hip_status(moe::launch_act(p, act == MOE_EPILOGUE_SWIGLU, (hipStream_t)stream), "moe_act_mxfp8 launch");
}

moe_status moe_act_mxfp8_backward(int32_t act, const void* q, int64_t q_ld, const uint8_t* scales, int64_t scales_ld,
                                  const void* dh, int64_t dh_ld, int64_t rows, int64_t n, void* dpre, int64_t dpre_ld,
                                  void* h, int64_t h_ld, moe_stream_t stream) {
  int64_t out = 0;
  moe_status st = check_act(act, rows, n, q, q_ld, scales, scales_ld, &out);
  if (st != MOE_OK) return st;
  if (bad_ld(dh_ld, out, 8, rows) || bad_ld(dpre_ld, n, 8, rows) || (h != nullptr && bad_ld(h_ld, out, 8, rows)))
    return fail(MOE_ERR_INVALID_ARGUMENT, "dh_ld, dpre_ld and h_ld must cover a row and be multiples of 8");
  if (rows > 0 && (dh == nullptr || dpre == nullptr)) return fail(MOE_ERR_INVALID_ARGUMENT, "null pointer argument");
  if (misaligned(dh, 16) || misaligned(dpre, 16) || misaligned(h, 16) || misaligned(q, 16))
    return fail(MOE_ERR_INVALID_ARGUMENT, "q, dh, dpre and h must be 16-byte aligned");
  if (clash({span(dpre, rows, dpre_ld, n, 2), span(h, rows, h_ld, out, 2)},
            {span(q, rows, q_ld, n, 1), span(scales, rows, scales_ld, n / 32, 1), span(dh, rows, dh_ld, out, 2)}))
    return fail(MOE_ERR_INVALID_ARGUMENT, "dpre and h must not overlap each other or the inputs");
  st = check_device();
  if (st != MOE_OK) return st;
  moe::ActParams p{};
  p.q = const_cast<uint8_t*>(static_cast<const uint8_t*>(q));
  p.q_ld = q_ld;
  p.s = const_cast<uint8_t*>(scales);
  p.s_ld = scales_ld;
  p.rows = rows;
  p.n = (int32_t)n;
  p.dh = static_cast<const uint16_t*>(dh);
  p.dh_ld = dh_ld;
  p.dpre = static_cast<uint16_t*>(dpre);
  p.dpre_ld = dpre_ld;
  p.h = static_cast<uint16_t*>(h);
  p.h_ld = h_ld;
  return hip_status(moe::launch_act_backward(p, act == MOE_EPILOGUE_SWIGLU, (hipStream_t)stream),
                    "moe_act_mxfp8_backward launch");
}

moe_status moe_wgrad_mxfp8(const void* xq, int64_t xq_ld, const uint8_t* xs, int64_t xs_ld, const void* grad,
                           int64_t grad_ld, const int32_t* sorted_token_ids, const int32_t* expert_ids,
                           const int32_t* num_tokens_post_pad, int64_t num_tokens, int32_t top_k, int32_t num_experts,
                           int64_t n, int64_t k, int32_t block_m, int64_t max_blocks, float* dw, moe_stream_t stream) {
  if (num_tokens < 0) return fail(MOE_ERR_INVALID_ARGUMENT, "num_tokens < 0");
  if (top_k < 1 || num_experts < top_k)
    return fail(MOE_ERR_INVALID_ARGUMENT, "need 1 <= top_k (%d) <= num_experts (%d)", top_k, num_experts);
  if (num_experts > kAlignMaxExperts)
    return fail(MOE_ERR_UNSUPPORTED, "num_experts %d > %d", num_experts, kAlignMaxExperts);
  if (n < 32 || n % 32 != 0 || k < 32 || k % 32 != 0 || n >= INT32_MAX || k >= INT32_MAX)
    return fail(MOE_ERR_INVALID_ARGUMENT, "n and k must be positive multiples of 32");
  if (xq_ld < k || xq_ld % 16 != 0 || xq_ld >= kBufMax || grad_ld < n || grad_ld % 8 != 0 ||
      grad_ld >= kBufMax)
    return fail(MOE_ERR_INVALID_ARGUMENT, "xq_ld / grad_ld must cover a row and be multiples of 16 / 8");
  if (xs_ld < k / 32 || xs_ld >= kBufMax) return fail(MOE_ERR_INVALID_ARGUMENT, "xs_ld must be >= k / 32");
  if (block_m != moe::wgrad_block_m())
    return fail(MOE_ERR_INVALID_ARGUMENT, "block_m %d, expected %d", block_m, moe::wgrad_block_m());
  if (num_tokens >= INT32_MAX / top_k) return fail(MOE_ERR_INVALID_ARGUMENT, "num_tokens * top_k must be < 2^31");
  const int64_t S = num_tokens * top_k;
  const int64_t need = moe_align_max_blocks(S, num_experts, block_m);
  if (max_blocks < need)
    return fail(MOE_ERR_INVALID_ARGUMENT, "max_blocks %lld < required %lld", (long long)max_blocks,
                (long long)need);
  // sorted_token_ids is read through 32-bit byte offsets too
  if (max_blocks >= kBufMax / 4 / block_m) return fail(MOE_ERR_INVALID_ARGUMENT, "max_blocks too large");
  if (dw == nullptr || (S > 0 && (xq == nullptr || xs == nullptr || grad == nullptr)) ||
      (max_blocks > 0 && (sorted_token_ids == nullptr || expert_ids == nullptr)))
    return fail(MOE_ERR_INVALID_ARGUMENT, "null pointer argument");
  if (misaligned(xq, 16) || misaligned(grad, 16) || misaligned(dw, 16) || misaligned(sorted_token_ids, 4) ||
      misaligned(expert_ids, 4))
    return fail(MOE_ERR_INVALID_ARGUMENT, "xq, grad and dw must be 16-byte aligned, the routing 4-byte");
  const int64_t tiles = (int64_t)num_experts * ((n + 255) / 256) * ((k + 255) / 256);
  if (tiles >= (int64_t)INT32_MAX) return fail(MOE_ERR_UNSUPPORTED, "too many dW tiles");
  // xq, xs and grad are read through 32-bit buffer offsets
  if (num_tokens * xq_ld >= kBufMax || num_tokens * xs_ld >= kBufMax || S * grad_ld * 2 >= kBufMax ||
      n * k * 4 >= kBufMax)
    return fail(MOE_ERR_UNSUPPORTED, "xq, xs, grad or one expert's dW spans 2 GB or more");
  if (clash({{dw, num_experts * n * k * 4}},
            {span(xq, num_tokens, xq_ld, k, 1), span(xs, num_tokens, xs_ld, k / 32, 1), span(grad, S, grad_ld, n, 2),
             {sorted_token_ids, max_blocks * block_m * 4}, {expert_ids, max_blocks * 4}}))
    return fail(MOE_ERR_INVALID_ARGUMENT, "dw overlaps an input");
  (void)num_tokens_post_pad;
  moe_status st = check_device();
  if (st != MOE_OK) return st;
  moe::WgradParams p{};
  p.x = static_cast<const uint16_t*>(xq);
  p.x_ld = xq_ld;
  p.xs = xs;
  p.xs_ld = xs_ld;
  p.grad = static_cast<const uint16_t*>(grad);
  p.grad_ld = grad_ld;
  p.sorted = sorted_token_ids;
  p.expert_ids = expert_ids;
  p.S = (int32_t)S;
  p.top_k = top_k;
  p.E = num_experts;
  p.N = (int32_t)n;
  p.K = (int32_t)k;
  p.max_blocks = (int32_t)max_blocks;
  p.dw = dw;
  return hip_status(moe::launch_wgrad_mxfp8(p, (hipStream_t)stream), "moe_wgrad_mxfp8 launch");
}

}  // extern "C"
