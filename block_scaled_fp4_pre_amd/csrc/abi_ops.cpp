// C ABI of the operators around the layer (declared in include/moe_w4a4.h):
// norm, router and dense linear.  Arguments are checked on the host before any
// HIP call, as in abi.cpp.
#include <hip/hip_runtime.h>

#include "launch.h"
#include "launch_ops.h"
#include "moe_w4a4.h"
#include "validate.h"

namespace {

inline int hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_EHIP; }

}  // namespace

extern "C" {

int moe_w4a4_add_rmsnorm(int32_t mma_type, int32_t res_dtype, int32_t w_dtype, int64_t rows, int32_t cols,
                         const uint16_t* x, const void* residual, const void* weight, float eps, float g,
                         void* residual_out, uint16_t* y, uint8_t* codes, uint8_t* scales, void* stream) {
  bool noop = false;
  int st = moe::check_norm_args(mma_type, res_dtype, w_dtype, rows, cols, x, residual, weight, eps, g, residual_out, y,
                                codes, scales, &noop);
  if (st != MOE_OK || noop) return st;
  st = moe::check_device();
  if (st != MOE_OK) return st;
  const int act = codes == nullptr ? -1 : mma_type == MOE_MMA_NVF4_X_NVF4 ? 2 : mma_type == MOE_MMA_FP8_X_MXF4 ? 1 : 0;
  return hip_status(moe::launch_add_rmsnorm(act, res_dtype == 1, w_dtype == 1, rows, cols, x, residual, weight, eps, g,
                                            residual_out, y, codes, scales, static_cast<hipStream_t>(stream)));
}

int moe_w4a4_router(int32_t logits_dtype, int32_t scoring, int64_t num_tokens, int32_t num_experts, int32_t topk,
                    int32_t num_groups, int32_t topk_groups, const void* logits, const float* bias,
                    int32_t renormalize, float scale, int32_t* topk_ids, float* topk_weights, void* stream) {
  bool noop = false;
  int st = moe::check_router_args(logits_dtype, scoring, num_tokens, num_experts, topk, num_groups, topk_groups, logits,
                                  bias, scale, topk_ids, topk_weights, &noop);
  if (st != MOE_OK || noop) return st;
  st = moe::check_device();
  if (st != MOE_OK) return st;
  return hip_status(moe::launch_router(logits_dtype == 0, scoring, num_tokens, num_experts, topk, num_groups,
                                       topk_groups, logits, bias, renormalize != 0, scale, topk_ids, topk_weights,
                                       static_cast<hipStream_t>(stream)));
}

int moe_w4a4_linear_query(const moe_w4a4_linear_cfg* cfg, size_t* prepared_bytes, size_t* workspace_bytes) {
  const int st = moe::check_linear_cfg(cfg);
  if (st != MOE_OK) return st;
  const moe::LinearLayout L = moe::linear_layout(cfg);
  if (prepared_bytes) *prepared_bytes = (size_t)L.prepared;
  if (workspace_bytes) *workspace_bytes = (size_t)L.workspace;
  return MOE_OK;
}

int moe_w4a4_linear_prepare(const moe_w4a4_linear_cfg* cfg, const uint8_t* codes, const uint8_t* scales,
                            void* prepared, size_t prepared_bytes, void* stream) {
  int st = moe::check_linear_prepare_args(cfg, codes, scales, prepared, prepared_bytes);
  if (st != MOE_OK) return st;
  st = moe::check_device();
  if (st != MOE_OK) return st;
  const moe::LinearLayout L = moe::linear_layout(cfg);
  uint8_t* base = static_cast<uint8_t*>(prepared);
  return hip_status(moe::launch_linear_prepare(codes, scales, cfg->out_features, cfg->in_features, (int)L.units,
                                               (int)L.steps, base + L.wc, base + L.ws,
                                               static_cast<hipStream_t>(stream)));
}

int moe_w4a4_linear(const moe_w4a4_linear_cfg* cfg, const void* prepared, int32_t num_tokens, const uint16_t* x,
                    const uint8_t* xq, const uint8_t* xsf, const uint16_t* addend, int32_t out_dtype, void* out,
                    void* workspace, size_t workspace_bytes, void* stream) {
  bool noop = false;
  int st = moe::check_linear_args(cfg, prepared, num_tokens, x, xq, xsf, addend, out_dtype, out, workspace,
                                  workspace_bytes, &noop);
  if (st != MOE_OK || noop) return st;
  st = moe::check_device();
  if (st != MOE_OK) return st;
  const moe::LinearLayout L = moe::linear_layout(cfg);
  const bool fp8 = cfg->mma_type == MOE_MMA_FP8_X_MXF4;
  const uint8_t* pw = static_cast<const uint8_t*>(prepared);
  uint8_t* wsp = static_cast<uint8_t*>(workspace);
  hipStream_t s = static_cast<hipStream_t>(stream);
  const moe::LinearArgs a = {pw + L.wc, pw + L.ws, wsp + L.tc, wsp + L.ts, addend, out, num_tokens, cfg->out_features,
                             (int)L.steps, out_dtype == 1};
  const moe::LinearPlan plan = moe::linear_plan(num_tokens, cfg->out_features, (int)L.steps);
  if (plan == moe::kLinearDecode)
    return hip_status(moe::launch_linear_decode(fp8, a, {x, xq, xsf, num_tokens, cfg->in_features}, s));
  st = hip_status(moe::launch_linear_tokens(fp8, x, xq, xsf, num_tokens, cfg->in_features,
                                            moe::linear_token_units(plan, num_tokens), (int)L.steps, wsp + L.tc,
                                            wsp + L.ts, s));
  if (st != MOE_OK) return st;
  return hip_status(plan == moe::kLinearSplit ? moe::launch_linear_split(fp8, a, s)
                                              : moe::launch_linear_tile(fp8, plan, a, s));
}

}  // extern "C"
