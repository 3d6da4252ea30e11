// Pieces shared by the kernels of the dense linear.
#pragma once
#include "device_common.h"
#include "launch_ops.h"
#include "tiles.h"

namespace moe {

// Codes of unit u at K step 0 and the stride to the next step, for operands
// of CB bytes per unit and step (weights and E2M1 tokens 4096, E4M3 8192).
template <int CB>
__device__ __forceinline__ size_t unit_base(int u, int steps) {
  return ((size_t)(u / kGroupUnits) * steps * kGroupUnits + u % kGroupUnits) * CB;
}

// out[t, n..n+3] = v (+ addend), n a multiple of 4; `whole`: N % 4 == 0, so
// that the four are in one row and aligned.
__device__ __forceinline__ void store4(const LinearArgs& a, int t, int n, v4f v, bool whole) {
  const size_t i = (size_t)t * a.N + n;
  const int left = a.N - n;
  if (a.addend != nullptr) {
    if (whole) {
      const uint2 r = *reinterpret_cast<const uint2*>(a.addend + i);
      v[0] += bf16_to_f32(r.x & 0xFFFFu);
      v[1] += bf16_to_f32(r.x >> 16);
      v[2] += bf16_to_f32(r.y & 0xFFFFu);
      v[3] += bf16_to_f32(r.y >> 16);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < left) v[j] += bf16_to_f32(a.addend[i + j]);
    }
  }
  if (a.out_f32) {
    float* o = static_cast<float*>(a.out) + i;
    if (whole) {
      *reinterpret_cast<v4f*>(o) = v;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < left) o[j] = v[j];
    }
  } else {
    uint16_t* o = static_cast<uint16_t*>(a.out) + i;
    if (whole) {
      *reinterpret_cast<uint2*>(o) = make_uint2(f32_to_bf16(v[0]) | (f32_to_bf16(v[1]) << 16),
                                                f32_to_bf16(v[2]) | (f32_to_bf16(v[3]) << 16));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < left) o[j] = (uint16_t)f32_to_bf16(v[j]);
    }
  }
}

}  // namespace moe
