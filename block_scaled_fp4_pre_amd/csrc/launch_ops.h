// Host-side launchers of the operators around the layer (norm, router,
// linear).  Every launcher only enqueues on `stream`; arguments were validated
// by the caller.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

// norm.hip.  act: codes of 0 MXFP4, 1 MXFP8 E4M3, 2 NVFP4 under g, or -1 none.
hipError_t launch_add_rmsnorm(int act, bool res_f32, bool w_f32, int64_t rows, int cols, const uint16_t* x,
                              const void* residual, const void* weight, float eps, float g, void* residual_out,
                              uint16_t* y, uint8_t* codes, uint8_t* scales, hipStream_t stream);

// router.hip
hipError_t launch_router(bool logits_bf16, int scoring, int64_t T, int E, int k, int groups, int keep,
                         const void* logits, const float* bias, bool renormalize, float scale, int32_t* ids,
                         float* weights, hipStream_t stream);

// linear_prepare.hip: canonical MXFP4 weights -> tile order, zeros in the padding.
hipError_t launch_linear_prepare(const uint8_t* codes, const uint8_t* scales, int N, int K, int units, int steps,
                                 uint8_t* p_codes, uint8_t* p_scales, hipStream_t stream);
// Tokens -> the same tile order (units of 64 tokens, fp8: two 1 KiB pieces per
// 16 tokens and step): x quantized, or xq / xsf copied.
hipError_t launch_linear_tokens(bool fp8, const uint16_t* x, const uint8_t* xq, const uint8_t* xsf, int T, int K,
                                int units, int steps, uint8_t* t_codes, uint8_t* t_scales, hipStream_t stream);

// The product over tile-ordered operands.
struct LinearArgs {
  const uint8_t *wc, *ws;      // weights
  const uint8_t *tc, *ts;      // tokens
  const uint16_t* addend;      // or null
  void* out;
  int T, N, steps;
  bool out_f32;
};
// The tokens as the caller gives them: x, or xq and xsf.
struct LinearInput {
  const uint16_t* x;
  const uint8_t *xq, *xsf;
  int T, K;
};

// Which kernel takes a product, from its number of 128 x 128 tiles.  Below 128
// (half the CUs) the split kernel, whose tiles are smaller and whose waves share
// the K steps; from 128 on the tile kernel, with tiles of 256 rows x 128 tokens
// once those give every CU the two workgroups it holds.  Measured with K = 4096
// (split / 128 / 256 rows), MXFP4: 256 x 4096 outputs 8.8 / 13.6 / 21 us, 512 x 4096
// 15.0 / 14.2 / 22, 64 x 32000 18.6 / 15.8 / 22, 2048 x 4096 58 / 23.9 / 25.1, 4096 x 4096
// 119 / 41 / 38; E4M3: 512 x 4096 19.1 / 17.6 / 32, 4096 x 4096 - / 55.7 / 54.7.
// Up to kDecodeMaxTokens tokens and kDecodeMaxSteps K steps: the decode kernel,
// which needs no tokens in tile order.
constexpr int kDecodeMaxTokens = 16, kDecodeMaxSteps = 64;
enum LinearPlan { kLinearDecode, kLinearSplit, kLinearTile128, kLinearTile256 };
inline LinearPlan linear_plan(int T, int N, int steps) {
  if (T <= kDecodeMaxTokens && steps <= kDecodeMaxSteps) return kLinearDecode;
  const int64_t tt = (T + 127) / 128;
  if (tt * ((N + 127) / 128) < 128) return kLinearSplit;
  return tt * ((N + 255) / 256) >= 512 ? kLinearTile256 : kLinearTile128;
}
// Units of 64 tokens that the plan's kernel reads: whole tiles.
inline int linear_token_units(LinearPlan plan, int T) {
  return plan == kLinearSplit ? (T + 63) / 64 : (T + 127) / 128 * 2;
}
hipError_t launch_linear_decode(bool fp8, const LinearArgs& a, const LinearInput& in, hipStream_t stream);   // linear_decode.hip
hipError_t launch_linear_split(bool fp8, const LinearArgs& a, hipStream_t stream);              // linear.hip
hipError_t launch_linear_tile(bool fp8, LinearPlan plan, const LinearArgs& a, hipStream_t stream);   // linear_tile.hip

}  // namespace moe
