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

// Which kernel takes a product.  Measured with K = 4096 and N = 4096 unless said
// otherwise, MXFP4 (E4M3), us of the product's kernel:
//   tokens        split        64 tokens    128 tokens   256 rows
//                              2 groups                  128 tokens
//   128           5.6 (7.4)    9.1 (10.8)   13 (16)      20 (30)
//   256           8.4 (10.6)   9.5 (11.4)   13.6 (16)    21 (30)
//   512           15.2 (18.9)  10.3 (13.0)  14.0 (16.5)  22 (31)
//   1024          26 (35)      18.6 (22.2)  16 (18.6)    22 (32)
//   2048          57 (87)      34 (42)      22.3 (29.5)  25 (35)
//   4096          119 (-)      -            41 (55.7)    37.6 (54.7)
//   64, N 32000   18.6         14.5         15.2         22
//   256, K 16384, N 2048: 13.1 / 23 / 36 / 58
// So, by the number of tiles: the split kernel, whose tiles are smaller and whose
// waves share the K steps, up to 128 tiles of 128 rows x 64 tokens (half the CUs);
// those with two groups of waves up to one a CU; tiles of 128 x 128, two a CU; and
// of 256 rows x 128 tokens once these give every CU its two.
// Up to kDecodeMaxTokens tokens and kDecodeMaxSteps K steps: the decode kernel,
// which needs no tokens in tile order.
constexpr int kDecodeMaxTokens = 16, kDecodeMaxSteps = 64;
enum LinearPlan { kLinearDecode, kLinearSplit, kLinearTile64, kLinearTile128, kLinearTile256 };
inline LinearPlan linear_plan(int T, int N, int steps) {
  if (T <= kDecodeMaxTokens && steps <= kDecodeMaxSteps) return kLinearDecode;
  const int64_t t64 = (T + 63) / 64, t128 = (T + 127) / 128, n128 = (N + 127) / 128, n256 = (N + 255) / 256;
  if (t64 * n128 <= 128) return kLinearSplit;
  if (t64 * n128 <= 256) return kLinearTile64;
  return t128 * n256 >= 512 ? kLinearTile256 : kLinearTile128;
}
// Units of 64 tokens that the plan's kernel reads: whole tiles.
inline int linear_token_units(LinearPlan plan, int T) {
  return plan == kLinearSplit || plan == kLinearTile64 ? (T + 63) / 64 : (T + 127) / 128 * 2;
}
hipError_t launch_linear_decode(bool fp8, const LinearArgs& a, const LinearInput& in, hipStream_t stream);   // linear_decode.hip
hipError_t launch_linear_split(bool fp8, const LinearArgs& a, hipStream_t stream);              // linear.hip
hipError_t launch_linear_tile(bool fp8, LinearPlan plan, const LinearArgs& a, hipStream_t stream);   // linear_tile.hip

}  // namespace moe
