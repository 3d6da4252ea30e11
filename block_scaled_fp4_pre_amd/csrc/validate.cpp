// Host-side argument checks and buffer layouts of the C ABI (validate.h).
// The supported configurations, status codes and pointer rules are the ones
// include/moe_w4a4.h documents: the pages' buffer factory ([P3] prhub digest
// of sglang PR "bump sgl-deep-gemm to 0.1.7, MegaMoE uses the mma_type API for
// MXFP4", "Key source snippets": capacity, experts, topk, hidden, inter,
// mma_type, activation="swiglu", group_size=32) made into explicit integers.
#include "validate.h"

namespace moe {
namespace {

inline uint64_t align256(uint64_t x) { return (x + 255) & ~uint64_t(255); }
inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace

int check_cfg(const moe_w4a4_cfg* c) {
  if (c == nullptr) return MOE_EINVAL;
  if (c->hidden <= 0 || c->inter <= 0 || c->num_experts <= 0 || c->topk <= 0 || c->max_tokens < 0)
    return MOE_EINVAL;
  if (c->hidden % 256 != 0 || c->inter % 128 != 0) return MOE_EUNSUPPORTED;
  if (c->hidden > (1 << 16) || c->inter > (1 << 16)) return MOE_EUNSUPPORTED;
  if (c->num_experts > kMaxExperts || c->topk > kMaxTopk) return MOE_EUNSUPPORTED;
  const bool mx = c->mma_type == MOE_MMA_MXF4_X_MXF4 || c->mma_type == MOE_MMA_FP8_X_MXF4;
  const bool nv = c->mma_type == MOE_MMA_NVF4_X_NVF4;
  if (!(mx && c->group_size == 32) && !(nv && c->group_size == 16)) return MOE_EUNSUPPORTED;
  if (c->activation != MOE_ACT_SWIGLU) return MOE_EUNSUPPORTED;
  if (nv && (c->hidden > kNvMaxK || c->inter > kNvMaxK)) return MOE_EUNSUPPORTED;
  if ((int64_t)c->max_tokens * c->topk >= (int64_t)1 << 31) return MOE_EUNSUPPORTED;
  return MOE_OK;
}

PreparedLayout prepared_layout(const moe_w4a4_cfg* c) {
  const uint64_t H = c->hidden, I = c->inter, E = c->num_experts, G = scale_group(c);
  PreparedLayout p{};
  uint64_t off = 0;
  p.w1c = off; off = align256(off + E * 2 * I * H / 2);
  p.w1s = off; off = align256(off + E * 2 * I * H / G);
  p.w2c = off; off = align256(off + E * H * I / 2);
  p.w2s = off; off = align256(off + E * H * I / G);
  p.gsc = off; off = align256(off + (c->mma_type == MOE_MMA_NVF4_X_NVF4 ? (2 * E + 2) * 4 : 0));
  p.total = off + kPreparedTailBytes;
  return p;
}

// Hidden and inter of 512, 1024, 2048 or 4096: K splits into 4 slices of 1,
// 2, 4 or 8 steps of 128, the slice lengths the kernel is built for.
static bool mega_k_ok(int64_t K) { return K >= 512 && K <= kMegaMaxK && (K & (K - 1)) == 0; }

bool mega_shape_ok(const moe_w4a4_cfg* c) {
  return (c->mma_type == MOE_MMA_MXF4_X_MXF4 || c->mma_type == MOE_MMA_FP8_X_MXF4) && mega_k_ok(c->hidden) &&
         mega_k_ok(c->inter);
}

int check_mega_args(const moe_w4a4_cfg* c, int32_t num_tokens) {
  if (!mega_shape_ok(c) || (int64_t)num_tokens * c->topk > kMegaMaxRows) return MOE_EUNSUPPORTED;
  return MOE_OK;
}

moe_w4a4_ws_layout ws_layout(const moe_w4a4_cfg* c) {
  const uint64_t H = c->hidden, I = c->inter, E = c->num_experts, M = c->max_tokens, G = scale_group(c);
  const uint64_t R = M * c->topk;
  const uint64_t nb = (R + kRouteRowsPerBlock - 1) / kRouteRowsPerBlock;
  moe_w4a4_ws_layout L{};
  uint64_t off = 0;
  // First and of one size for every configuration, so that it stays put in
  // the allocation-free forward's scratch, which is laid out per call.
  L.mega = off; off = align256(off + kMegaStateBytes);
  const uint64_t ab = c->mma_type == MOE_MMA_FP8_X_MXF4 ? 2 : 1;   // activation bytes per 2 elements
  L.xq = off; off = align256(off + M * H / 2 * ab);
  L.xsf = off; off = align256(off + M * H / G);
  L.counts = off; off = align256(off + E * 4);
  L.offsets = off; off = align256(off + (E + 1) * 4);
  L.sorted_rows = off; off = align256(off + R * 4);
  L.pos = off; off = align256(off + R * 4);
  L.hist = off; off = align256(off + nb * E * 4);
  L.hq = off; off = align256(off + R * I / 2 * ab);
  L.hsf = off; off = align256(off + R * I / G);
  L.y = off; off = align256(off + R * H * 2);
  L.tiles = off; off = align256(off + (R / 16 + E + 1) * 8);
  L.num_tiles = off; off = align256(off + 4);
  L.xsf_planes = off; off = align256(off + R * H / G);
  L.total = off;
  return L;
}

int check_quantize_args(int32_t src_dtype, const void* src, int64_t rows, int32_t cols, const void* codes,
                        const void* scales, bool* noop) {
  *noop = false;
  if (src_dtype != 0 && src_dtype != 1) return MOE_EUNSUPPORTED;
  if (rows < 0 || cols <= 0) return MOE_EINVAL;
  if (cols % 32 != 0) return MOE_EUNSUPPORTED;
  if (rows == 0) {
    *noop = true;
    return MOE_OK;
  }
  if (src == nullptr || codes == nullptr || scales == nullptr) return MOE_EINVAL;
  if (!aligned(src, 16) || !aligned(codes, 16)) return MOE_EINVAL;
  // one thread per 32-group: the group count must fit the launch's index range
  if (rows > (int64_t)1 << 40 || rows * (int64_t)(cols / 32) >= (int64_t)1 << 40) return MOE_EUNSUPPORTED;
  return MOE_OK;
}

bool nv_scale_ok(float g) { return g >= kNvScaleMin && g <= kNvScaleMax; }   // false for NaN

int check_prepare_args(const moe_w4a4_cfg* cfg, const void* w1_codes, const void* w1_scales,
                       const void* w2_codes, const void* w2_scales, const void* prepared, size_t prepared_bytes) {
  const int st = check_cfg(cfg);
  if (st != MOE_OK) return st;
  if (cfg->mma_type == MOE_MMA_NVF4_X_NVF4) return MOE_EUNSUPPORTED;   // moe_w4a4_prepare_weights_nvfp4
  if (!w1_codes || !w1_scales || !w2_codes || !w2_scales || !prepared) return MOE_EINVAL;
  if (!aligned(w1_codes, 16) || !aligned(w2_codes, 16) || !aligned(prepared, 256)) return MOE_EINVAL;
  if (prepared_bytes < prepared_layout(cfg).total) return MOE_EWORKSPACE;
  return MOE_OK;
}

int check_prepare_nv_args(const moe_w4a4_cfg* cfg, const void* w1_codes, const void* w1_scales,
                          const void* w1_tensor_scales, const void* w2_codes, const void* w2_scales,
                          const void* w2_tensor_scales, float x_tensor_scale, float h_tensor_scale,
                          const void* prepared, size_t prepared_bytes) {
  const int st = check_cfg(cfg);
  if (st != MOE_OK) return st;
  if (cfg->mma_type != MOE_MMA_NVF4_X_NVF4) return MOE_EUNSUPPORTED;   // moe_w4a4_prepare_weights
  if (!w1_codes || !w1_scales || !w1_tensor_scales || !w2_codes || !w2_scales || !w2_tensor_scales || !prepared)
    return MOE_EINVAL;
  if (!aligned(w1_codes, 16) || !aligned(w2_codes, 16) || !aligned(prepared, 256) ||
      !aligned(w1_tensor_scales, 4) || !aligned(w2_tensor_scales, 4))
    return MOE_EINVAL;
  if (!nv_scale_ok(x_tensor_scale) || !nv_scale_ok(h_tensor_scale)) return MOE_EINVAL;
  if (prepared_bytes < prepared_layout(cfg).total) return MOE_EWORKSPACE;
  return MOE_OK;
}

int check_stage_args(const moe_w4a4_cfg* cfg, const void* prepared, int32_t num_tokens, const void* x,
                     const void* topk_ids, const void* topk_weights, const void* out, const void* workspace,
                     size_t workspace_bytes, uint32_t stages, const void* gemm1_acc, bool* noop) {
  *noop = false;
  const int st = check_cfg(cfg);
  if (st != MOE_OK) return st;
  if (num_tokens < 0) return MOE_EINVAL;
  if (num_tokens > cfg->max_tokens) return MOE_ECAPACITY;
  if ((stages & ~uint32_t(MOE_STAGE_ALL)) != 0) return MOE_EINVAL;
  if (num_tokens == 0 || stages == 0) {     // nothing to do; empty tensors may be NULL
    *noop = true;
    return MOE_OK;
  }
  if (workspace == nullptr || !aligned(workspace, 256)) return MOE_EINVAL;
  if (workspace_bytes < ws_layout(cfg).total) return MOE_EWORKSPACE;
  if ((stages & MOE_STAGE_QUANT) && (x == nullptr || !aligned(x, 16))) return MOE_EINVAL;
  if ((stages & MOE_STAGE_ROUTE) && (topk_ids == nullptr || !aligned(topk_ids, 4))) return MOE_EINVAL;
  // the GEMMs read the prepared weights; NVFP4's quantization reads its g_x there too
  const uint32_t need_prepared = MOE_STAGE_GEMM1 | MOE_STAGE_GEMM2 |
                                 (cfg->mma_type == MOE_MMA_NVF4_X_NVF4 ? uint32_t(MOE_STAGE_QUANT) : 0u);
  if ((stages & need_prepared) && (prepared == nullptr || !aligned(prepared, 256))) return MOE_EINVAL;
  if ((stages & MOE_STAGE_COMBINE) &&
      (topk_weights == nullptr || out == nullptr || !aligned(topk_weights, 4) || !aligned(out, 16)))
    return MOE_EINVAL;
  if (gemm1_acc != nullptr && !aligned(gemm1_acc, 16)) return MOE_EINVAL;
  return MOE_OK;
}

int check_norm_args(int32_t mma_type, int32_t res_dtype, int32_t w_dtype, int64_t rows, int32_t cols, const void* x,
                    const void* residual, const void* weight, float eps, float g, const void* residual_out,
                    const void* y, const void* codes, const void* scales, bool* noop) {
  *noop = false;
  if ((res_dtype != 0 && res_dtype != 1) || (w_dtype != 0 && w_dtype != 1)) return MOE_EUNSUPPORTED;
  if (rows < 0 || cols <= 0 || !(eps > 0.0f && eps <= 3.402823466e38f)) return MOE_EINVAL;
  if (cols % 32 != 0 || cols > kNormMaxCols || rows >= (int64_t)1 << 31) return MOE_EUNSUPPORTED;
  if (rows == 0) {
    *noop = true;
    return MOE_OK;
  }
  if (x == nullptr || weight == nullptr || (y == nullptr && codes == nullptr)) return MOE_EINVAL;
  if ((residual == nullptr) != (residual_out == nullptr) || (codes == nullptr) != (scales == nullptr)) return MOE_EINVAL;
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(residual_out, 16) ||
      !aligned(y, 16) || !aligned(codes, 16))
    return MOE_EINVAL;
  // An output in the place of another, or of an input whose rows it does not
  // cover value for value (other workgroups may not have read those yet).
  if (y != nullptr && (y == residual_out || y == weight || (y == residual && res_dtype == 1))) return MOE_EINVAL;
  if (residual_out != nullptr && (residual_out == weight || (residual_out == x && res_dtype == 1))) return MOE_EINVAL;
  auto taken = [&](const void* p) {
    return p != nullptr && (p == x || p == residual || p == weight || p == residual_out || p == y);
  };
  if (taken(codes) || taken(scales) || (codes != nullptr && codes == scales)) return MOE_EINVAL;
  if (codes != nullptr) {
    if (mma_type != MOE_MMA_MXF4_X_MXF4 && mma_type != MOE_MMA_FP8_X_MXF4 && mma_type != MOE_MMA_NVF4_X_NVF4)
      return MOE_EUNSUPPORTED;
    if (mma_type == MOE_MMA_NVF4_X_NVF4 && !nv_scale_ok(g)) return MOE_EINVAL;
  }
  return MOE_OK;
}

int check_router_args(int32_t logits_dtype, int32_t scoring, int64_t num_tokens, int32_t num_experts, int32_t topk,
                      int32_t num_groups, int32_t topk_groups, const void* logits, const void* bias, float scale,
                      const void* topk_ids, const void* topk_weights, bool* noop) {
  *noop = false;
  if (logits_dtype != 0 && logits_dtype != 1) return MOE_EUNSUPPORTED;
  if (scoring != MOE_SCORE_SOFTMAX && scoring != MOE_SCORE_SIGMOID && scoring != MOE_SCORE_SQRTSOFTPLUS)
    return MOE_EUNSUPPORTED;
  if (num_tokens < 0 || num_experts <= 0 || topk <= 0 || num_groups <= 0 || topk_groups <= 0) return MOE_EINVAL;
  if (!(scale >= -3.402823466e38f && scale <= 3.402823466e38f)) return MOE_EINVAL;
  if (num_experts > kMaxExperts || topk > kMaxTopk || num_groups > kRouterMaxGroups) return MOE_EUNSUPPORTED;
  if (num_experts % num_groups != 0 || topk_groups > num_groups ||
      topk > topk_groups * (num_experts / num_groups))
    return MOE_EINVAL;
  if (num_tokens >= ((int64_t)1 << 40) / num_experts) return MOE_EUNSUPPORTED;
  if (num_tokens == 0) {
    *noop = true;
    return MOE_OK;
  }
  if (logits == nullptr || topk_ids == nullptr || topk_weights == nullptr) return MOE_EINVAL;
  if (!aligned(logits, logits_dtype == 0 ? 2 : 4) || !aligned(bias, 4) || !aligned(topk_ids, 4) ||
      !aligned(topk_weights, 4))
    return MOE_EINVAL;
  return MOE_OK;
}

int check_linear_cfg(const moe_w4a4_linear_cfg* c) {
  if (c == nullptr) return MOE_EINVAL;
  if (c->in_features <= 0 || c->out_features <= 0 || c->max_tokens < 0) return MOE_EINVAL;
  if (c->in_features % 32 != 0 || c->in_features > kLinearMaxK || c->out_features > kLinearMaxN ||
      c->max_tokens > kLinearMaxTokens || (int64_t)c->max_tokens * c->out_features > kLinearMaxOut)
    return MOE_EUNSUPPORTED;
  if (c->mma_type != MOE_MMA_MXF4_X_MXF4 && c->mma_type != MOE_MMA_FP8_X_MXF4) return MOE_EUNSUPPORTED;
  return MOE_OK;
}

LinearLayout linear_layout(const moe_w4a4_linear_cfg* c) {
  LinearLayout L{};
  L.steps = (c->in_features + 127) / 128;
  L.units = ((uint64_t)c->out_features + 255) / 256 * 4;
  L.token_units = ((uint64_t)c->max_tokens + 255) / 256 * 4;
  // per unit and step: 4 KiB of packed E2M1 (E4M3: 8 KiB) and 256 B of scales
  const uint64_t tok = c->mma_type == MOE_MMA_FP8_X_MXF4 ? 8192 : 4096;
  L.wc = 0;
  L.ws = L.units * L.steps * 4096;
  L.prepared = L.ws + L.units * L.steps * 256;
  L.tc = 0;
  L.ts = L.token_units * L.steps * tok;
  L.workspace = L.ts + L.token_units * L.steps * 256;
  return L;
}

int check_linear_prepare_args(const moe_w4a4_linear_cfg* cfg, const void* codes, const void* scales,
                              const void* prepared, size_t prepared_bytes) {
  const int st = check_linear_cfg(cfg);
  if (st != MOE_OK) return st;
  if (!codes || !scales || !prepared) return MOE_EINVAL;
  if (!aligned(codes, 16) || !aligned(prepared, 256)) return MOE_EINVAL;
  if (prepared_bytes < linear_layout(cfg).prepared) return MOE_EWORKSPACE;
  return MOE_OK;
}

int check_linear_args(const moe_w4a4_linear_cfg* cfg, const void* prepared, int32_t num_tokens, const void* x,
                      const void* xq, const void* xsf, const void* addend, int32_t out_dtype, const void* out,
                      const void* workspace, size_t workspace_bytes, bool* noop) {
  *noop = false;
  const int st = check_linear_cfg(cfg);
  if (st != MOE_OK) return st;
  if (out_dtype != 0 && out_dtype != 1) return MOE_EUNSUPPORTED;
  if (num_tokens < 0) return MOE_EINVAL;
  if (num_tokens > cfg->max_tokens) return MOE_ECAPACITY;
  if (num_tokens == 0) {
    *noop = true;
    return MOE_OK;
  }
  if (prepared == nullptr || out == nullptr || workspace == nullptr) return MOE_EINVAL;
  if (x != nullptr ? xq != nullptr || xsf != nullptr : xq == nullptr || xsf == nullptr) return MOE_EINVAL;
  if (!aligned(prepared, 256) || !aligned(workspace, 256) || !aligned(x, 16) || !aligned(xq, 16) ||
      !aligned(addend, 16) || !aligned(out, 16))
    return MOE_EINVAL;
  // workgroups read the tokens, the weights and the workspace while others write
  // out; addend's element is read by the lane that writes it, which needs the two
  // to have one type
  if (out == x || out == xq || out == xsf || out == prepared || out == workspace || (out == addend && out_dtype == 1))
    return MOE_EINVAL;
  if (workspace_bytes < linear_layout(cfg).workspace) return MOE_EWORKSPACE;
  return MOE_OK;
}

}  // namespace moe
