// float32 -> bfloat16 by gfx950's conversion instruction, for the operators around
// the layer.
#pragma once
#include "device_common.h"

namespace moe {

// Two float32 values rounded to bfloat16 (nearest, ties to even; a NaN stays
// one), `lo` in the low half: v_cvt_pk_bf16_f32.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
  typedef float v2f __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f{lo, hi}), v2bf));
}

}  // namespace moe
