// Pieces of 8 values of a row, shared by the norms (norm.hip, post_norm.hip).
#pragma once
#include "pack_bf16.h"
#include "quant_e4m3.h"

namespace moe {

// The value of lane (l ^ M) of the same quad, M = 1 or 2.
template <int M>
__device__ __forceinline__ uint32_t quad_xor(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, M == 1 ? 0xB1 : 0x4E, 0xF, 0xF, true);
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_to_f32(w[i] & 0xFFFFu);
    f[2 * i + 1] = bf16_to_f32(w[i] >> 16);
  }
}

__device__ __forceinline__ void load_f32x8(const float* p, float (&f)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}

// Sum over the 64 lanes, the same bits in every lane.
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int m = 1; m < kWave; m <<= 1) v += __shfl_xor(v, m);
  return v;
}

// Codes and scales of piece c of a row (8 values of y in bfloat16; `row_piece` is the row's
// first among all) as ACT: 0 MXFP4, 1 MXFP8 E4M3, 2 NVFP4 under the tensor scale g.
// Neighbouring lanes hold neighbouring pieces; every lane calls it, and those with c <
// pieces write.
template <int ACT>
__device__ __forceinline__ void quantize_piece(const uint4& yb, size_t row_piece, int c, int pieces, float g,
                                               uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  // The group's absolute maximum on the bit patterns of the rounded y
  // (bf16 magnitudes order as their low 15 bits).
  const uint32_t yw[4] = {yb.x, yb.y, yb.z, yb.w};
  typedef unsigned short v2u16 __attribute__((ext_vector_type(2)));
  v2u16 m2 = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    m2 = __builtin_elementwise_max(m2, __builtin_bit_cast(v2u16, yw[i] & 0x7FFF7FFFu));
  uint32_t amax = max((uint32_t)m2[0], (uint32_t)m2[1]);
  amax = max(amax, quad_xor<1>(amax));
  if constexpr (ACT != 2) amax = max(amax, quad_xor<2>(amax));
  float n[8];
  unpack8(yb, n);
  const size_t piece = row_piece + c;
  if constexpr (ACT == 1) {
    const int e = mx8_scale_exp(amax << 16);
    const float inv = e4m3_exp2(-e);
    const uint2 q = make_uint2(e4m3_cvt4(n[0], n[1], n[2], n[3], inv), e4m3_cvt4(n[4], n[5], n[6], n[7], inv));
    if (c < pieces) {
      reinterpret_cast<uint2*>(codes)[piece] = q;
      if (c % 4 == 0) scales[piece / 4] = (uint8_t)(e + 127);
    }
  } else if constexpr (ACT == 0) {
    const int e = mx_scale_exp(amax << 16);
    const float sc = exp2_scale(e);
    uint32_t q = e2m1_pack2<0>(0u, n[0], n[1], sc);
    q = e2m1_pack2<1>(q, n[2], n[3], sc);
    q = e2m1_pack2<2>(q, n[4], n[5], sc);
    q = e2m1_pack2<3>(q, n[6], n[7], sc);
    if (c < pieces) {
      reinterpret_cast<uint32_t*>(codes)[piece] = q;
      if (c % 4 == 0) scales[piece / 4] = (uint8_t)(e + 127);
    }
  } else {
    const uint32_t sc = nv_scale_code(__uint_as_float(amax << 16), g);
    const float inv = nv_inv(sc, g);
    uint32_t q = nv_pack2<0>(0u, n[0], n[1], inv);
    q = nv_pack2<1>(q, n[2], n[3], inv);
    q = nv_pack2<2>(q, n[4], n[5], inv);
    q = nv_pack2<3>(q, n[6], n[7], inv);
    if (c < pieces) {
      reinterpret_cast<uint32_t*>(codes)[piece] = q;
      if (c % 2 == 0) scales[piece / 2] = (uint8_t)sc;
    }
  }
}

}  // namespace moe
