// MXFP8 E4M3 codes by the conversion instruction, for the operators around the
// layer.  gfx950's v_cvt_pk_fp8_f32 rounds to the nearest E4M3 value, ties to
// the even mantissa, keeps the sign and makes subnormals: the rule of e4m3.h,
// with which it agreed on MI355X for 2.2 million fp32 patterns up to 448 (every
// sign, exponent and top 11 mantissa bits, four patterns of the rest), at a fifth
// of the instructions.
#pragma once
#include "quant_group.h"

namespace moe {

// Codes of four values under the block scale 2^e (inv = 2^-e, every |v * inv| <= 448).
__device__ __forceinline__ uint32_t e4m3_cvt4(float v0, float v1, float v2, float v3, float inv) {
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v0 * inv, v1 * inv, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v2 * inv, v3 * inv, lo, true);
}

// E4M3 codes of 32 bf16 values as 16 words (elements 0..15 in lo, 16..31 in
// hi); the return value is the scale byte.
__device__ __forceinline__ uint32_t mx8_cvt_bf16_group(const uint32_t (&w)[16], uint4& lo, uint4& hi) {
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = max(amax, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
  const int e = mx8_scale_exp(amax << 16);
  const float inv = e4m3_exp2(-e);
  uint32_t c[8];
#pragma unroll
  for (int q = 0; q < 8; ++q)
    c[q] = e4m3_cvt4(bf16_to_f32(w[2 * q] & 0xFFFFu), bf16_to_f32(w[2 * q] >> 16), bf16_to_f32(w[2 * q + 1] & 0xFFFFu),
                     bf16_to_f32(w[2 * q + 1] >> 16), inv);
  lo = make_uint4(c[0], c[1], c[2], c[3]);
  hi = make_uint4(c[4], c[5], c[6], c[7]);
  return (uint32_t)(e + 127);
}

}  // namespace moe
