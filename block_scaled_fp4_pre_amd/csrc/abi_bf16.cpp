// C ABI of the bfloat16 operators (declared in include/moe_w4a4.h): linear,
// grouped linear, the experts made of them, and the norm after a block.
// Arguments are checked on the host before any HIP call, as in abi.cpp.
#include <hip/hip_runtime.h>

#include "launch.h"
#include "launch_bf16.h"
#include "moe_w4a4.h"
#include "validate.h"

namespace {

inline int hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_EHIP; }

}  // namespace

extern "C" {

int moe_w4a4_linear_bf16(int64_t num_tokens, int32_t in_features, int32_t out_features, const uint16_t* x,
                         int64_t x_stride, const uint16_t* weight, int32_t function, int32_t gated, int32_t bias_dtype,
                         const void* bias, const float* row_scale, int32_t addend_dtype, const void* addend,
                         int64_t addend_stride, int32_t out_dtype, void* out, int64_t out_stride, void* stream) {
  bool noop = false;
  int st = moe::check_linear_bf16_args(num_tokens, in_features, out_features, x, x_stride, weight, function, gated,
                                       bias_dtype, bias, row_scale, addend_dtype, addend, addend_stride, out_dtype, out,
                                       out_stride, &noop);
  if (st != MOE_OK || noop) return st;
  st = moe::check_device();
  if (st != MOE_OK) return st;
  const moe::Bf16Args a = {x, weight, bias, row_scale, addend, out, nullptr, nullptr, x_stride, addend_stride,
                           out_stride, (int)num_tokens, out_features, in_features, 1, 1, (int)num_tokens, function,
                           bias_dtype == 1, addend_dtype == 1, out_dtype == 1};
  return hip_status(moe::launch_linear_bf16(gated != 0, a, static_cast<hipStream_t>(stream)));
}

int moe_w4a4_grouped_linear_bf16(int32_t num_groups, int64_t num_rows, int32_t in_features, int32_t out_features,
                                 const int32_t* offsets, const uint16_t* x, int64_t x_rows, int64_t x_stride,
                                 const int32_t* rows, int32_t row_divisor, const uint16_t* weight, int32_t function,
                                 int32_t gated, int32_t bias_dtype, const void* bias, const float* row_scale,
                                 int32_t addend_dtype, const void* addend, int64_t addend_stride, int32_t out_dtype,
                                 void* out, int64_t out_stride, void* stream) {
  bool noop = false;
  int st = moe::check_grouped_bf16_args(num_groups, num_rows, in_features, out_features, offsets, x, x_rows, x_stride,
                                        rows, row_divisor, weight, function, gated, bias_dtype, bias, row_scale,
                                        addend_dtype, addend, addend_stride, out_dtype, out, out_stride, &noop);
  if (st != MOE_OK || noop) return st;
  st = moe::check_device();
  if (st != MOE_OK) return st;
  const moe::Bf16Args a = {x, weight, bias, row_scale, addend, out, offsets, rows, x_stride, addend_stride, out_stride,
                           (int)num_rows, out_features, in_features, num_groups, row_divisor, (int)x_rows, function,
                           bias_dtype == 1, addend_dtype == 1, out_dtype == 1};
  return hip_status(moe::launch_linear_bf16(gated != 0, a, static_cast<hipStream_t>(stream)));
}

int moe_w4a4_experts_bf16_query(const moe_w4a4_experts_bf16_cfg* cfg, size_t* workspace_bytes) {
  const int st = moe::check_experts_bf16_cfg(cfg);
  if (st != MOE_OK) return st;
  if (workspace_bytes) *workspace_bytes = (size_t)moe::experts_bf16_layout(cfg).total;
  return MOE_OK;
}

int moe_w4a4_experts_bf16(const moe_w4a4_experts_bf16_cfg* cfg, const uint16_t* w1, const uint16_t* w2,
                          int32_t num_tokens, const uint16_t* x, const int32_t* topk_ids, const float* topk_weights,
                          uint16_t* out, void* workspace, size_t workspace_bytes, void* stream) {
  bool noop = false;
  int st = moe::check_experts_bf16_args(cfg, w1, w2, num_tokens, x, topk_ids, topk_weights, out, workspace,
                                        workspace_bytes, &noop);
  if (st != MOE_OK || noop) return st;
  st = moe::check_device();
  if (st != MOE_OK) return st;
  const moe::ExpertsBf16Layout L = moe::experts_bf16_layout(cfg);
  const int H = cfg->hidden, I = cfg->inter, E = cfg->num_experts, k = cfg->topk, T = num_tokens, R = T * k;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  int32_t* counts = reinterpret_cast<int32_t*>(ws + L.counts);
  int32_t* offsets = reinterpret_cast<int32_t*>(ws + L.offsets);
  int32_t* sorted_rows = reinterpret_cast<int32_t*>(ws + L.sorted_rows);
  int32_t* pos = reinterpret_cast<int32_t*>(ws + L.pos);
  uint16_t* h = reinterpret_cast<uint16_t*>(ws + L.h);
  uint16_t* y = reinterpret_cast<uint16_t*>(ws + L.y);
  hipStream_t s = static_cast<hipStream_t>(stream);
  // one block routes small batches (the pre-dispatch kernel with nothing to quantize)
  st = hip_status(R <= moe::kPredispatchMaxRows
                      ? moe::launch_predispatch(0, nullptr, 0, nullptr, nullptr, nullptr, topk_ids, R, E, counts,
                                                offsets, sorted_rows, pos, 0, nullptr, nullptr, s)
                      : moe::launch_route(topk_ids, R, E, reinterpret_cast<int32_t*>(ws + L.hist), counts, offsets,
                                          sorted_rows, pos, 0, nullptr, nullptr, s));
  if (st != MOE_OK) return st;
  const moe::Bf16Args gate_up = {x, w1, nullptr, nullptr, nullptr, h, offsets, sorted_rows, H, 0, I, R, I, H, E, k, T,
                                 cfg->function, false, false, false};
  st = hip_status(moe::launch_linear_bf16(true, gate_up, s));
  if (st != MOE_OK) return st;
  const moe::Bf16Args down = {h, w2, nullptr, nullptr, nullptr, y, offsets, nullptr, I, 0, H, R, H, I, E, 1, R,
                              MOE_FN_NONE, false, false, false};
  st = hip_status(moe::launch_linear_bf16(false, down, s));
  if (st != MOE_OK) return st;
  return hip_status(moe::launch_combine(y, pos, topk_weights, T, H, k, out, s));
}

int moe_w4a4_post_norm(int32_t mma_type, int32_t res_dtype, int32_t w_dtype, int32_t gate_dtype, int32_t gate_kind,
                       int64_t rows, int32_t cols, const uint16_t* x, const void* residual, const void* post_weight,
                       const void* gate, float scale, const void* next_weight, float eps, float g, void* residual_out,
                       uint16_t* y, uint8_t* codes, uint8_t* scales, void* stream) {
  bool noop = false;
  int st = moe::check_post_norm_args(mma_type, res_dtype, w_dtype, gate_dtype, gate_kind, rows, cols, x, residual,
                                     post_weight, gate, scale, next_weight, eps, g, residual_out, y, codes, scales,
                                     &noop);
  if (st != MOE_OK || noop) return st;
  st = moe::check_device();
  if (st != MOE_OK) return st;
  const int act = codes == nullptr ? -1 : mma_type == MOE_MMA_NVF4_X_NVF4 ? 2 : mma_type == MOE_MMA_FP8_X_MXF4 ? 1 : 0;
  const moe::PostNormArgs a = {x, residual, post_weight, gate, next_weight, residual_out, y, codes, scales, rows, cols,
                               gate_kind, w_dtype == 1, gate_dtype == 1, scale, g, eps, 1.0 / cols};
  return hip_status(moe::launch_post_norm(act, res_dtype == 1, a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
