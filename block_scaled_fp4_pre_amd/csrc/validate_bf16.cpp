// Host-side argument checks of the bfloat16 operators (validate.h): plain C++,
// no HIP.
#include "validate.h"

#include <initializer_list>

namespace moe {
namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
size_t dtype_size(int32_t dtype) { return dtype == 1 ? 4 : 2; }
bool dtype_ok(int32_t dtype) { return dtype == 0 || dtype == 1; }
uint64_t up256(uint64_t v) { return (v + 255) & ~uint64_t(255); }

// What the linear and the grouped linear have in common; `rows` of out, `x_rows` of x.
int check_product(int64_t rows, int64_t x_rows, int32_t K, int32_t N, const void* x, int64_t ldx, const void* w,
                  int32_t fn, int32_t gated, int32_t bias_dtype, const void* bias, const void* row_scale,
                  int32_t add_dtype, const void* addend, int64_t lda, int32_t out_dtype, const void* out, int64_t ldo,
                  bool* noop) {
  if (!dtype_ok(bias_dtype) || !dtype_ok(add_dtype) || !dtype_ok(out_dtype)) return MOE_EUNSUPPORTED;
  if (fn < MOE_FN_NONE || fn > MOE_FN_GELU_TANH || (gated != 0 && gated != 1)) return MOE_EUNSUPPORTED;
  if (rows < 0 || x_rows < 0 || K <= 0 || N <= 0) return MOE_EINVAL;
  if (K % 8 != 0 || K > kBf16MaxK || N > kBf16MaxN || rows > kBf16MaxRows || x_rows > kBf16MaxRows ||
      rows * N > kBf16MaxOut)
    return MOE_EUNSUPPORTED;
  if (rows == 0) {
    *noop = true;
    return MOE_OK;
  }
  if (x == nullptr || w == nullptr || out == nullptr || x_rows == 0) return MOE_EINVAL;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(out, dtype_size(out_dtype)) || !aligned(row_scale, 4) ||
      !aligned(bias, dtype_size(bias_dtype)) || !aligned(addend, dtype_size(add_dtype)))
    return MOE_EINVAL;
  if (ldx < K || ldo < N || (addend != nullptr && lda < N)) return MOE_EINVAL;
  if (ldx % 8 != 0 || ldx > kBf16MaxStride || ldo > kBf16MaxStride || (addend != nullptr && lda > kBf16MaxStride))
    return MOE_EUNSUPPORTED;
  // Workgroups read the inputs while others write out; an addend's value is read by
  // the lane that writes in its place, which needs the two to be laid out alike.
  if (out == x || out == w || out == bias || out == row_scale ||
      (out == addend && (add_dtype != out_dtype || lda != ldo)))
    return MOE_EINVAL;
  return MOE_OK;
}

}  // namespace

int check_linear_bf16_args(int64_t num_tokens, int32_t K, int32_t N, const void* x, int64_t ldx, const void* w,
                           int32_t fn, int32_t gated, int32_t bias_dtype, const void* bias, const void* row_scale,
                           int32_t add_dtype, const void* addend, int64_t lda, int32_t out_dtype, const void* out,
                           int64_t ldo, bool* noop) {
  *noop = false;
  return check_product(num_tokens, num_tokens, K, N, x, ldx, w, fn, gated, bias_dtype, bias, row_scale, add_dtype,
                       addend, lda, out_dtype, out, ldo, noop);
}

int check_grouped_bf16_args(int32_t E, int64_t num_rows, int32_t K, int32_t N, const void* offsets, const void* x,
                            int64_t x_rows, int64_t ldx, const void* rows, int32_t row_divisor, const void* w,
                            int32_t fn, int32_t gated, int32_t bias_dtype, const void* bias, const void* row_scale,
                            int32_t add_dtype, const void* addend, int64_t lda, int32_t out_dtype, const void* out,
                            int64_t ldo, bool* noop) {
  *noop = false;
  if (E <= 0 || row_divisor <= 0) return MOE_EINVAL;
  if (E > kMaxExperts || (int64_t)E * N > kBf16MaxGroupCols) return MOE_EUNSUPPORTED;
  const int st = check_product(num_rows, x_rows, K, N, x, ldx, w, fn, gated, bias_dtype, bias, row_scale, add_dtype,
                               addend, lda, out_dtype, out, ldo, noop);
  if (st != MOE_OK || *noop) return st;
  if (offsets == nullptr || !aligned(offsets, 4) || !aligned(rows, 4)) return MOE_EINVAL;
  if (rows == nullptr && x_rows < num_rows) return MOE_EINVAL;
  if (out == offsets || out == rows) return MOE_EINVAL;
  // (the gathered rows' places in x are 32-bit byte offsets)
  if (rows != nullptr && x_rows * ldx >= (int64_t)1 << 31) return MOE_EUNSUPPORTED;
  return MOE_OK;
}

int check_experts_bf16_cfg(const moe_w4a4_experts_bf16_cfg* c) {
  if (c == nullptr) return MOE_EINVAL;
  if (c->hidden <= 0 || c->inter <= 0 || c->num_experts <= 0 || c->topk <= 0 || c->max_tokens < 0) return MOE_EINVAL;
  if (c->hidden % 8 != 0 || c->inter % 8 != 0 || c->hidden > kBf16MaxK || c->inter > kBf16MaxK ||
      c->num_experts > kMaxExperts || c->topk > kMaxTopk || (int64_t)c->max_tokens * c->topk > kBf16MaxRows ||
      (int64_t)c->max_tokens * c->hidden >= (int64_t)1 << 31 ||
      (int64_t)c->num_experts * c->inter > kBf16MaxGroupCols || (int64_t)c->num_experts * c->hidden > kBf16MaxGroupCols ||
      (int64_t)c->max_tokens * c->topk * c->hidden > kBf16MaxOut || (int64_t)c->max_tokens * c->topk * c->inter > kBf16MaxOut)
    return MOE_EUNSUPPORTED;
  if (c->function < MOE_FN_NONE || c->function > MOE_FN_GELU_TANH) return MOE_EUNSUPPORTED;
  return MOE_OK;
}

ExpertsBf16Layout experts_bf16_layout(const moe_w4a4_experts_bf16_cfg* c) {
  ExpertsBf16Layout L{};
  const uint64_t R = (uint64_t)c->max_tokens * c->topk, E = c->num_experts;
  uint64_t at = 0;
  auto take = [&](uint64_t bytes) {
    const uint64_t here = at;
    at += up256(bytes);
    return here;
  };
  L.counts = take(E * 4);
  L.offsets = take((E + 1) * 4);
  L.sorted_rows = take(R * 4);
  L.pos = take(R * 4);
  L.hist = take((R + kRouteRowsPerBlock - 1) / kRouteRowsPerBlock * E * 4);
  L.h = take(R * c->inter * 2);
  L.y = take(R * c->hidden * 2);
  L.total = at;
  return L;
}

int check_experts_bf16_args(const moe_w4a4_experts_bf16_cfg* cfg, const void* w1, const void* w2, int32_t num_tokens,
                            const void* x, const void* topk_ids, const void* topk_weights, const void* out,
                            const void* workspace, size_t workspace_bytes, bool* noop) {
  *noop = false;
  const int st = check_experts_bf16_cfg(cfg);
  if (st != MOE_OK) return st;
  if (num_tokens < 0) return MOE_EINVAL;
  if (num_tokens > cfg->max_tokens) return MOE_ECAPACITY;
  if (num_tokens == 0) {
    *noop = true;
    return MOE_OK;
  }
  if (!w1 || !w2 || !x || !topk_ids || !topk_weights || !out || !workspace) return MOE_EINVAL;
  if (!aligned(w1, 16) || !aligned(w2, 16) || !aligned(x, 16) || !aligned(topk_ids, 4) || !aligned(topk_weights, 4) ||
      !aligned(out, 16) || !aligned(workspace, 256))
    return MOE_EINVAL;
  // (out may be x: every token's row was gathered before the combine writes it)
  for (const void* in : {w1, w2, topk_ids, topk_weights})
    if (out == in || workspace == in) return MOE_EINVAL;
  if (workspace == x || workspace == out) return MOE_EINVAL;
  if (workspace_bytes < experts_bf16_layout(cfg).total) return MOE_EWORKSPACE;
  return MOE_OK;
}

int check_post_norm_args(int32_t mma_type, int32_t res_dtype, int32_t w_dtype, int32_t gate_dtype, int32_t gate_kind,
                         int64_t rows, int32_t cols, const void* x, const void* residual, const void* post_weight,
                         const void* gate, float scale, const void* next_weight, float eps, float g,
                         const void* residual_out, const void* y, const void* codes, const void* scales, bool* noop) {
  *noop = false;
  if (!dtype_ok(res_dtype) || !dtype_ok(w_dtype) || !dtype_ok(gate_dtype)) return MOE_EUNSUPPORTED;
  if (gate_kind < MOE_GATE_NONE || gate_kind > MOE_GATE_FULL) return MOE_EUNSUPPORTED;
  if (rows < 0 || cols <= 0 || !(eps > 0.0f && eps <= 3.402823466e38f)) return MOE_EINVAL;
  if (!(scale >= -3.402823466e38f && scale <= 3.402823466e38f)) return MOE_EINVAL;
  if (cols % 32 != 0 || cols > kNormMaxCols || rows >= (int64_t)1 << 31) return MOE_EUNSUPPORTED;
  if (rows == 0) {
    *noop = true;
    return MOE_OK;
  }
  if (x == nullptr || residual == nullptr || residual_out == nullptr) return MOE_EINVAL;
  if ((gate == nullptr) != (gate_kind == MOE_GATE_NONE) || (codes == nullptr) != (scales == nullptr)) return MOE_EINVAL;
  // the norm before the next block goes with what it makes
  if ((next_weight == nullptr) != (y == nullptr && codes == nullptr)) return MOE_EINVAL;
  for (const void* p : {x, residual, post_weight, next_weight, residual_out, y, codes})
    if (!aligned(p, 16)) return MOE_EINVAL;
  if (!aligned(gate, gate_kind == MOE_GATE_ROW ? dtype_size(gate_dtype) : 16)) return MOE_EINVAL;
  // An output in the place of another, or of an input whose rows it does not cover value
  // for value (other workgroups may not have read those yet).
  for (const void* w : {post_weight, next_weight, gate})
    if (w != nullptr && (residual_out == w || y == w)) return MOE_EINVAL;
  if (residual_out == x && res_dtype == 1) return MOE_EINVAL;
  if (y != nullptr && (y == residual_out || (y == residual && res_dtype == 1))) return MOE_EINVAL;
  auto taken = [&](const void* q) {
    for (const void* p : {x, residual, post_weight, gate, next_weight, residual_out, y})
      if (p != nullptr && p == q) return true;
    return false;
  };
  if (codes != nullptr) {
    if (taken(codes) || taken(scales) || codes == scales) return MOE_EINVAL;
    if (mma_type != MOE_MMA_MXF4_X_MXF4 && mma_type != MOE_MMA_FP8_X_MXF4 && mma_type != MOE_MMA_NVF4_X_NVF4)
      return MOE_EUNSUPPORTED;
    if (mma_type == MOE_MMA_NVF4_X_NVF4 && !nv_scale_ok(g)) return MOE_EINVAL;
  }
  return MOE_OK;
}

}  // namespace moe
