// Outputs of the bfloat16 tile kernels, from sums in LDS.
#pragma once
#include "bf16_common.h"

namespace moe {

constexpr int kBand = 8;       // row tiles that take their turn together (launch order of the tiles)

// 8 values in their own type (float32: two vectors), those past `left` zeros.
__device__ __forceinline__ void load8_raw(const void* base, size_t i, bool f32, int left, v4u (&r)[2]) {
  r[0] = r[1] = v4u{0, 0, 0, 0};
  if (f32) {
    const uint32_t* q = static_cast<const uint32_t*>(base) + i;
    if (left >= 8) {
      r[0] = *reinterpret_cast<const v4u_at4*>(q);
      r[1] = *reinterpret_cast<const v4u_at4*>(q + 4);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < left) r[j / 4][j % 4] = q[j];
    }
  } else {
    const uint16_t* q = static_cast<const uint16_t*>(base) + i;
    if (left >= 8) {
      r[0] = *reinterpret_cast<const v4u_at2*>(q);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < left) r[0][j / 2] |= (uint32_t)q[j] << (j % 2 * 16);
    }
  }
}
__device__ __forceinline__ float raw_value(const v4u (&r)[2], bool f32, int j) {
  return f32 ? __uint_as_float(r[j / 4][j % 4]) : bf16_to_f32(r[0][j / 2] >> (j % 2 * 16) & 0xFFFFu);
}

// The outputs of 16 rows from their sums in `mine` (16 x STRIDE bytes of LDS, the wave's own):
// 8 neighbouring ones a lane, so that a store covers a whole run of a row.  f is applied
// in a rolled loop, each lane on the values that it stores (unrolled over a tile, its code
// spilled).  All loads of the rows' addends go out before the first use.  scale: row_scale
// of row row0 - at + lane (a load for each pass cost 98304 x 2048 x 4096 in groups 5 %).
template <int WA, bool GATED>
__device__ __forceinline__ void store_rows(const Bf16Args& p, uint8_t* mine, int n, int row0, int end, int lane,
                                           const v4f (&bias)[2], const v4f (&up_bias)[2], float scale, int at) {
  constexpr int STRIDE = WA * 64 + 16;
  constexpr int LPT = WA * (GATED ? 8 : 16) / 8, TPP = kWave / LPT, IT = 16 / TPP;   // lanes a row, rows a pass, passes
  const int o = lane % LPT * 8;
  const int left = p.N - n, live = left > 0 ? end - row0 : 0;
  uint8_t* place = mine + lane / LPT * STRIDE + (GATED ? o / 16 * 32 + o % 16 : o) * 4;
  v4u add[IT][2];
  if (p.addend != nullptr) {
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int t = i * TPP + lane / LPT;
      load8_raw(p.addend, (size_t)(row0 + t) * p.lda + n, p.add_f32, t < live ? left : 0, add[i]);
    }
  }
  if (GATED || p.fn != MOE_FN_NONE || p.bias != nullptr) {
#pragma unroll 1
    for (int i = 0; i < IT; ++i) {
      v4f* q = reinterpret_cast<v4f*>(place + i * TPP * STRIDE);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        v4f v = apply_function(p.fn, q[h] + bias[h]);
        if constexpr (GATED) v *= q[h + 4] + up_bias[h];
        q[h] = v;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int t = i * TPP + lane / LPT;
    const v4f* q = reinterpret_cast<const v4f*>(place + i * TPP * STRIDE);
    v4f v[2] = {q[0], q[1]};
    if (p.row_scale != nullptr) {
      const float s = __shfl(scale, at + t);
      v[0] *= s;
      v[1] *= s;
    }
    if (p.addend != nullptr) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j / 4][j % 4] += raw_value(add[i], p.add_f32, j);
    }
    if (t >= live) continue;
    const size_t to = (size_t)(row0 + t) * p.ldo + n;
    if (p.out_f32) {
      float* out = static_cast<float*>(p.out) + to;
      if (left >= 8) {
        __builtin_nontemporal_store(v[0], reinterpret_cast<v4f_at4*>(out));
        __builtin_nontemporal_store(v[1], reinterpret_cast<v4f_at4*>(out + 4));
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < left) out[j] = v[j / 4][j % 4];
      }
    } else {
      uint16_t* out = static_cast<uint16_t*>(p.out) + to;
      v4u b;
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = pack_bf16(v[j / 2][j % 2 * 2], v[j / 2][j % 2 * 2 + 1]);
      if (left >= 8) {
        __builtin_nontemporal_store(b, reinterpret_cast<v4u_at2*>(out));
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < left) out[j] = (uint16_t)(b[j / 2] >> (j % 2 * 16));
      }
    }
  }
}

// Biases of the lane's 8 outputs n, n + 1, ... (store_rows).
template <bool GATED>
__device__ __forceinline__ void load_bias(const Bf16Args& p, int group, int n, v4f (&bias)[2], v4f (&up_bias)[2]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) bias[h] = up_bias[h] = v4f{0.f, 0.f, 0.f, 0.f};
  if (p.bias == nullptr) return;
  const size_t at = (size_t)group * (GATED ? 2 : 1) * p.N + n;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    bias[h] = load4_f32(p.bias, at + 4 * h, p.bias_f32, p.N - n - 4 * h);
    if constexpr (GATED) up_bias[h] = load4_f32(p.bias, at + p.N + 4 * h, p.bias_f32, p.N - n - 4 * h);
  }
}

}  // namespace moe
