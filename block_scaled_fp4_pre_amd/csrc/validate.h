// Host-side argument checks and buffer layouts of the C ABI (moe_w4a4.h).
//
// Plain C++ with no HIP dependency: abi.cpp runs these checks before it makes
// any HIP call, and the CPU tests build this file on its own with the host
// address and undefined-behaviour sanitizers and drive every error path
// through it.  Each check returns MOE_OK or the status code the ABI returns.
#pragma once
#include <stddef.h>
#include <stdint.h>

#include "moe_w4a4.h"

namespace moe {

constexpr int kMaxExperts = 512;
constexpr int kMaxTopk = 16;
constexpr int kRouteRowsPerBlock = 1024;   // rows per block of the multi-block route (per-block histograms)

// NVFP4 (MOE_MMA_NVF4_X_NVF4): token rows per pass of its streaming GEMMs
// with two token tiles, and the longest K (hidden or inter) whose token tile
// (rows * (K/2 code bytes + K/16 scale bytes)) fits a CU's 160 KiB of LDS.
constexpr int kNvStreamRows = 24;
constexpr int kNvMaxK = 12032;
// Range of an NVFP4 tensor scale: every fp32 step of the encoding stays finite.
constexpr float kNvScaleMin = 0x1p-100f;
constexpr float kNvScaleMax = 0x1p100f;

// The single-launch forward (mega.hip): MXFP4 x MXFP4 or fp8xfp4, at most
// kMegaMaxRows routed rows (num_tokens * topk; one thread each in the
// workgroup's own route), hidden and inter each 512, 1024, 2048 or kMegaMaxK
// (each of a work item's 4 waves takes a quarter of K: 1, 2, 4 or 8 steps of
// 128, the slice lengths the kernel is built for).
constexpr int kMegaMaxRows = MOE_MEGA_MAX_ROWS;
constexpr int kMegaMaxK = 4096;
// Ticket counters per work phase of the single-launch forward.
constexpr int kMegaQueues = 16;
// Its state region, the first region of every workspace whatever the
// configuration (so that it stays put in the allocation-free forward's
// scratch): queue, done and error words, one h counter per expert, and one
// combine counter per (token, 64 hidden columns).
constexpr uint64_t kMegaStateBytes = MOE_MEGA_STATE_BYTES;
bool mega_shape_ok(const moe_w4a4_cfg* c);     // c must pass check_cfg
// MOE_OK when the single-launch forward supports cfg and num_tokens (c must
// pass check_cfg), else MOE_EUNSUPPORTED.
int check_mega_args(const moe_w4a4_cfg* c, int32_t num_tokens);

// Bytes after the last region of the prepared weights.  The streaming GEMMs
// keep a ring of up to 4 K steps of weight loads in flight per wave and issue
// the ring's refills past a unit's last step without a branch; for the last
// unit of the last expert those loads (never consumed) read up to 4 steps of
// 16 KiB past the end of the codes, into the following regions and this tail.
constexpr uint64_t kPreparedTailBytes = 64 * 1024;

// Region offsets of the prepared weights (256-byte aligned), tail included in
// total.  gsc: the NVFP4 tensor scales, fp32 [g_w1[E], g_w2[E], g_x, g_h]
// (empty for the MX types).
struct PreparedLayout {
  uint64_t w1c, w1s, w2c, w2s, gsc, total;
};

// Elements per scale byte of cfg's MMA type: 16 for NVFP4, else 32.
inline int scale_group(const moe_w4a4_cfg* c) { return c->mma_type == MOE_MMA_NVF4_X_NVF4 ? 16 : 32; }

int check_cfg(const moe_w4a4_cfg* c);
PreparedLayout prepared_layout(const moe_w4a4_cfg* c);      // c must pass check_cfg
moe_w4a4_ws_layout ws_layout(const moe_w4a4_cfg* c);        // c must pass check_cfg

// Arguments of moe_w4a4_quantize.  *noop is set when there is nothing to
// enqueue (rows == 0) and the call returns MOE_OK.
int check_quantize_args(int32_t src_dtype, const void* src, int64_t rows, int32_t cols, const void* codes,
                        const void* scales, bool* noop);

// An NVFP4 tensor scale passed by value: finite and in [kNvScaleMin, kNvScaleMax].
bool nv_scale_ok(float g);

// Arguments of moe_w4a4_prepare_weights (MX types only).
int check_prepare_args(const moe_w4a4_cfg* cfg, const void* w1_codes, const void* w1_scales,
                       const void* w2_codes, const void* w2_scales, const void* prepared, size_t prepared_bytes);

// Arguments of moe_w4a4_prepare_weights_nvfp4 (NVFP4 configurations only).
int check_prepare_nv_args(const moe_w4a4_cfg* cfg, const void* w1_codes, const void* w1_scales,
                          const void* w1_tensor_scales, const void* w2_codes, const void* w2_scales,
                          const void* w2_tensor_scales, float x_tensor_scale, float h_tensor_scale,
                          const void* prepared, size_t prepared_bytes);

// Arguments of moe_w4a4_run_stages (and so of moe_w4a4_forward, which runs
// every stage).  *noop is set when there is nothing to enqueue (no tokens or
// no stages) and the call returns MOE_OK without looking at any pointer.
int check_stage_args(const moe_w4a4_cfg* cfg, const void* prepared, int32_t num_tokens, const void* x,
                     const void* topk_ids, const void* topk_weights, const void* out, const void* workspace,
                     size_t workspace_bytes, uint32_t stages, const void* gemm1_acc, bool* noop);

// ---- operators around the layer ----
constexpr int kNormMaxCols = 65536;
constexpr int kRouterMaxGroups = 64;      // one lane of a wave each
constexpr int kLinearMaxK = 65536;
constexpr int kLinearMaxN = 1 << 20;
constexpr int kLinearMaxTokens = 1 << 20;
constexpr int64_t kLinearMaxOut = (int64_t)1 << 34;   // tokens * N: the product's launch stays below 2^32 threads

// Arguments of moe_w4a4_add_rmsnorm and moe_w4a4_router; *noop: no rows.
int check_norm_args(int32_t mma_type, int32_t res_dtype, int32_t w_dtype, int64_t rows, int32_t cols, const void* x,
                    const void* residual, const void* weight, float eps, float g, const void* residual_out,
                    const void* y, const void* codes, const void* scales, bool* noop);
int check_router_args(int32_t logits_dtype, int32_t scoring, int64_t num_tokens, int32_t num_experts, int32_t topk,
                      int32_t num_groups, int32_t topk_groups, const void* logits, const void* bias, float scale,
                      const void* topk_ids, const void* topk_weights, bool* noop);

// A linear's tiles (tiles.h, with 4 units = 256 rows a group): weights and
// tokens are padded to whole groups of rows and whole K steps of 128.
struct LinearLayout {
  uint64_t steps;                 // K steps of 128
  uint64_t units;                 // 64-row units of W, a multiple of 4
  uint64_t token_units;           // 64-row units of max_tokens tokens, a multiple of 4
  uint64_t wc, ws, prepared;      // offsets of codes and scales in the prepared weights, and its size
  uint64_t tc, ts, workspace;     // the same of the quantized tokens in the workspace
};
int check_linear_cfg(const moe_w4a4_linear_cfg* c);
LinearLayout linear_layout(const moe_w4a4_linear_cfg* c);   // c must pass check_linear_cfg
int check_linear_prepare_args(const moe_w4a4_linear_cfg* cfg, const void* codes, const void* scales,
                              const void* prepared, size_t prepared_bytes);
int check_linear_args(const moe_w4a4_linear_cfg* cfg, const void* prepared, int32_t num_tokens, const void* x,
                      const void* xq, const void* xsf, const void* addend, int32_t out_dtype, const void* out,
                      const void* workspace, size_t workspace_bytes, bool* noop);

// ---- bfloat16 operators (validate_bf16.cpp) ----
constexpr int kBf16MaxK = 65536;
constexpr int kBf16MaxN = 1 << 20;
constexpr int64_t kBf16MaxRows = (int64_t)1 << 24;
constexpr int64_t kBf16MaxOut = (int64_t)1 << 36;      // rows * N: the products' launches stay below 2^32 threads
constexpr int64_t kBf16MaxGroupCols = (int64_t)1 << 24;  // groups * N: the same
constexpr int64_t kBf16MaxStride = (int64_t)1 << 22;   // elements: a tile's rows are within 32-bit byte offsets

// Arguments of moe_w4a4_linear_bf16, moe_w4a4_grouped_linear_bf16 and
// moe_w4a4_post_norm; *noop: no rows.
int check_linear_bf16_args(int64_t num_tokens, int32_t K, int32_t N, const void* x, int64_t ldx, const void* w,
                           int32_t fn, int32_t gated, int32_t bias_dtype, const void* bias, const void* row_scale,
                           int32_t add_dtype, const void* addend, int64_t lda, int32_t out_dtype, const void* out,
                           int64_t ldo, bool* noop);
int check_grouped_bf16_args(int32_t E, int64_t num_rows, int32_t K, int32_t N, const void* offsets, const void* x,
                            int64_t x_rows, int64_t ldx, const void* rows, int32_t row_divisor, const void* w,
                            int32_t fn, int32_t gated, int32_t bias_dtype, const void* bias, const void* row_scale,
                            int32_t add_dtype, const void* addend, int64_t lda, int32_t out_dtype, const void* out,
                            int64_t ldo, bool* noop);
int check_post_norm_args(int32_t mma_type, int32_t res_dtype, int32_t w_dtype, int32_t gate_dtype, int32_t gate_kind,
                         int64_t rows, int32_t cols, const void* x, const void* residual, const void* post_weight,
                         const void* gate, float scale, const void* next_weight, float eps, float g,
                         const void* residual_out, const void* y, const void* codes, const void* scales, bool* noop);

// Regions of the workspace of moe_w4a4_experts_bf16 (256-byte aligned).
struct ExpertsBf16Layout {
  uint64_t counts, offsets, sorted_rows, pos, hist, h, y, total;
};
int check_experts_bf16_cfg(const moe_w4a4_experts_bf16_cfg* c);
ExpertsBf16Layout experts_bf16_layout(const moe_w4a4_experts_bf16_cfg* c);   // c must pass check_experts_bf16_cfg
int check_experts_bf16_args(const moe_w4a4_experts_bf16_cfg* cfg, const void* w1, const void* w2, int32_t num_tokens,
                            const void* x, const void* topk_ids, const void* topk_weights, const void* out,
                            const void* workspace, size_t workspace_bytes, bool* noop);

}  // namespace moe
