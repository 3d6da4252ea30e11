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
// Few tokens: the decode kernel, which needs no tokens in tile order and so no
// launch before it, but quantizes them in every workgroup.  Passes of one call, us,
// decode against the token kernel and split, MXFP4 (E4M3 within 2 us of these):
//   tokens x K     N 4096        N 8192        N 16384       N 32000
//   1 x 4096       5.8 / 8.9     5.9 / 9.3     7.6 / 9.8     12.2 / 15.5
//   8 x 4096       5.5 / 8.8     7.9 / 9.0     10.3 / 9.9    13.2 / 15.2
//   16 x 2048      6.3 / 9.2     6.9 / 8.8     8.4 / 9.2     10.0 / 11.0
//   16 x 4096      6.9 / 9.0     11.1 / 9.4    12.9 / 10.0   16.1 / 15.6
//   1 x 8192       8.6 / 8.8     -             15.7 / 14.2   -              (N 2048: 6.8 / 8.9)
//   4 x 8192       9.9 / 9.0     -             17.1 / 14.3   -
// So where tokens times K steps are kDecodeMaxWork at most, or there is one block
// of 16 rows a CU; past 32 steps, where a wave holds 8 of them, for one token.
constexpr int kDecodeMaxTokens = 16, kDecodeMaxSteps = 64, kDecodeMaxWork = 256;
enum LinearPlan { kLinearDecode, kLinearSplit, kLinearTile64, kLinearTile128, kLinearTile256 };
inline bool linear_decodes(int T, int N, int steps) {
  const bool a_block_a_cu = N <= 256 * 16;
  if (steps > kDecodeMaxSteps / 2) return T == 1 && steps <= kDecodeMaxSteps && a_block_a_cu;
  return T <= kDecodeMaxTokens && (T * steps <= kDecodeMaxWork || a_block_a_cu);
}
inline LinearPlan linear_plan(int T, int N, int steps) {
  if (linear_decodes(T, N, steps)) return kLinearDecode;
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
