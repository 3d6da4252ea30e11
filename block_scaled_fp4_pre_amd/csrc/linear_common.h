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
// E4M3 against E2M1: the instruction cuts each product to a multiple of 2^-13 of the
// largest power of two in its group of eight before it adds them (E2M1 products
// span too few binades to lose a bit).  That is taken as it is: of the bfloat16
// outputs 0.7 % come out one step from a float32 sum's, the error against 64 bits is
// the same 1.66e-3 (16384 x 2048 x 4096 with an addend; float32 outputs: 2.3e-5),
// and keeping the bits would take a second operand and product for the small values.
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

// Vectors at the alignment of one value of `out` (or the addend): rows of any N
// are read and written in whole vectors, which the memory unit takes at any address.
// (One value at a time where N does not keep rows aligned: 11342 x 64 x 14298
// MXFP4 244 against 137 us, 8847 x 64 x 7586 with an addend 208 against 95.)
typedef unsigned int v2u __attribute__((ext_vector_type(2)));
typedef v2u v2u_at2 __attribute__((aligned(2)));
typedef v4u v4u_at2 __attribute__((aligned(2)));
typedef v4f v4f_at4 __attribute__((aligned(4)));

// out[t, n..n+3] = v (+ addend), as far as the row goes.
__device__ __forceinline__ void store4(const LinearArgs& a, int t, int n, v4f v) {
  const size_t i = (size_t)t * a.N + n;
  const int left = a.N - n;
  const bool whole = left >= 4;
  if (a.addend != nullptr) {
    if (whole) {
      const v2u r = *reinterpret_cast<const v2u_at2*>(a.addend + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] += bf16_to_f32(r[j / 2] >> (j % 2 * 16) & 0xFFFFu);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < left) v[j] += bf16_to_f32(a.addend[i + j]);
    }
  }
  if (a.out_f32) {
    float* o = static_cast<float*>(a.out) + i;
    if (whole) {
      *reinterpret_cast<v4f_at4*>(o) = v;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < left) o[j] = v[j];
    }
  } else {
    uint16_t* o = static_cast<uint16_t*>(a.out) + i;
    if (whole) {
      *reinterpret_cast<v2u_at2*>(o) = v2u{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < left) o[j] = (uint16_t)pack_bf16(v[j], 0.0f);
    }
  }
}

}  // namespace moe
