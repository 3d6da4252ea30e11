// Pieces shared by the kernels of the dense linear.
#pragma once
#include "gemm_common.h"
#include "launch_ops.h"
#include "pack_bf16.h"
#include "tiles.h"

namespace moe {

// The block-scaled MFMAs of device_common.h on native vectors: operands that
// live in arrays across a pipelined loop stay in registers only as these.
template <int OA, int OB>
__device__ __forceinline__ v4f mfma_op(const v4u& a, const v4u& b, const v4f& c, int sa, int sb) {
  const v8i av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const v8i bv = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, OA, sa, OB, sb);
}
template <int OA, int OB>
__device__ __forceinline__ v4f mfma_op8(const v4u& a, const v4u& lo, const v4u& hi, const v4f& c, int sa, int sb) {
  const v8i av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const v8i bv = {(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 0, OA, sa, OB, sb);
}

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
      *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < left) o[j] = (uint16_t)pack_bf16(v[j], 0.0f);
    }
  }
}

}  // namespace moe
