// Pieces shared by the kernels of the bfloat16 linears: which rows a workgroup
// owns, and what happens to a sum on its way out.
#pragma once
#include "device_common.h"
#include "launch_bf16.h"
#include "moe_w4a4.h"
#include "pack_bf16.h"

namespace moe {

typedef unsigned int v2u __attribute__((ext_vector_type(2)));
typedef unsigned int v4u __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
// Vectors at the alignment of one element: rows of any N are read and written in
// whole vectors, which the memory unit takes at any address.
typedef v2u v2u_at2 __attribute__((aligned(2)));
typedef v4u v4u_at2 __attribute__((aligned(2)));
typedef v4u v4u_at4 __attribute__((aligned(4)));
typedef v4f v4f_at4 __attribute__((aligned(4)));

__device__ __forceinline__ v4f mfma_bf16(const v4u& a, const v4u& b, const v4f& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

// A group and its rows; which of its tiles, of how many.
struct RowTile {
  int group, first, end, tile, tiles;
};

// The groups' tiles, in the order of the groups.  Every wave counts them for itself: a
// lane those of up to 8 consecutive groups (all their offsets in one trip to memory), a
// scan over the lanes says whose a tile is.  Offsets are clamped to the rows there are,
// so that wrong ones give wrong rows but no access outside the tensors.
template <int UNIT>
struct GroupTiles {
  static constexpr int PER = 8;                      // 512 groups
  int per, mine, upto, total, at[PER + 1];
  __device__ __forceinline__ static int count(int first, int end) { return (max(end - first, 0) + UNIT - 1) / UNIT; }
  __device__ __forceinline__ explicit GroupTiles(const Bf16Args& p) {
    const int lane = threadIdx.x & (kWave - 1);
    per = (p.E + kWave - 1) / kWave;
#pragma unroll
    for (int j = 0; j <= PER; ++j) at[j] = j <= per ? p.offsets[min(lane * per + j, p.E)] : 0;
    mine = 0;
#pragma unroll
    for (int j = 0; j <= PER; ++j) {
      at[j] = j <= per ? min(max(at[j], 0), p.T) : at[j - 1];
      if (j > 0) mine += count(at[j - 1], at[j]);
    }
    upto = mine;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const int o = __shfl_up(upto, d, kWave);
      if (lane >= d) upto += o;
    }
    total = __builtin_amdgcn_readlane(upto, kWave - 1);
  }
  // Tile number `tile` < total: its group, the group's rows and tiles, and which of them it is.
  __device__ __forceinline__ RowTile find(int tile) const {
    const int owner = __builtin_ctzll(__ballot(upto > tile));
    int left = tile - __builtin_amdgcn_readlane(upto - mine, owner);
    RowTile t = {0, 0, 0, 0, 0};
    bool found = false;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int first = __builtin_amdgcn_readlane(at[j], owner), end = __builtin_amdgcn_readlane(at[j + 1], owner);
      const int n = count(first, end);
      if (!found && left < n) {
        t = {owner * per + j, first, end, left, n};
        found = true;
      }
      left -= n;
    }
    return t;
  }
};

// The place of a workgroup among `total` items of the groups, or -1.  Workgroups are
// dealt round-robin to the 8 XCDs; each XCD takes runs of 32 items in turn, as many as it
// has CUs, so that items next to each other share operands in its L2 and groups of
// unlike size spread over the XCDs.
constexpr int kRun = 32;
__device__ __forceinline__ int group_item(int total) {
  const int at = blockIdx.x >> 3, L = (at / kRun * 8 + (blockIdx.x & 7)) * kRun + at % kRun;
  return L < total ? L : -1;
}
// Workgroups that cover `total` items so.
inline int64_t group_grid(int64_t total) { return (total + 8 * kRun - 1) / (8 * kRun) * (8 * kRun); }

// Row of x that row i of the product reads (any index gives a row that exists).
__device__ __forceinline__ int source_row(const Bf16Args& p, int i) {
  return p.rows == nullptr ? i : min(max(p.rows[i] / p.row_div, 0), p.x_rows - 1);
}

// v / (1 + 2^(t + r)), r the rounding of t (left out it would cost |t| 2^-24 of a small
// result).  Far out 2^t is taken 2^32 times smaller and 1 is nothing next to it: the
// reciprocal of a power past 2^126 would be flushed to zero where v / 2^t is not.
// (Contraction is off where a product's rounding is known and put back: fused into a later
// sum the product would have another.)
__device__ __forceinline__ float over_one_plus_exp2(float v, float t, float r) {
#pragma clang fp contract(off)
  const bool far = t > 64.0f;
  const float e = __builtin_amdgcn_exp2f(far ? t - 32.0f : t) * fmaf(r, 0.693147181f, 1.0f);
  const float q = v * __builtin_amdgcn_rcpf(far ? e : 1.0f + e);
  return far ? q * 0x1p-32f : q;
}

// silu(v) = v / (1 + e^-v).
__device__ __forceinline__ float silu_f32(float v) {
#pragma clang fp contract(off)
  const float u = fminf(fmaxf(-v, -104.0f), 200.0f), t = u * 1.44269502f;
  return over_one_plus_exp2(v, t, fmaf(u, 1.92596303e-8f, fmaf(u, 1.44269502f, -t)));
}

// gelu(v) = v F(v), F the normal distribution: F(-a) = t 2^(s + r) for a >= 0 with t = 1 /
// (1 + 0.3 a), s = -a^2 / 2 log2(e), and r a polynomial of t - 0.6 (a Chebyshev fit of
// log2(e^(a^2/2) F(-a) / t) over a <= 14.5, within 2^-24) with the roundings of s put back;
// F(a) = 1 - F(-a).  Far out as in over_one_plus_exp2.  (Through erfcf a 128 x 128 tile's
// outputs cost as much as 16 steps of its product.)
__device__ __forceinline__ float gelu_f32(float v) {
#pragma clang fp contract(off)
  const float a = fminf(fabsf(v), 16.0f);
  const float t = __builtin_amdgcn_rcpf(fmaf(a, 0.3f, 1.0f)), u = t - 0.6f;
  float r = 0.207756102f;
  r = fmaf(r, u, -0.20550473f);
  r = fmaf(r, u, -0.287186265f);
  r = fmaf(r, u, 0.323197365f);
  r = fmaf(r, u, 0.318443209f);
  r = fmaf(r, u, -0.400117517f);
  r = fmaf(r, u, -0.509796202f);
  r = fmaf(r, u, 0.537607908f);
  r = fmaf(r, u, 2.2604425f);
  r = fmaf(r, u, -1.9513582f);
  const float h = -0.5f * a, m = h * a, low = fmaf(h, a, -m);          // -a^2 / 2 = m + low
  const float s = m * 1.44269502f;
  r += fmaf(low, 1.44269502f, fmaf(m, 1.92596303e-8f, fmaf(m, 1.44269502f, -s)));
  const bool far = s < -64.0f;
  const float q = t * (__builtin_amdgcn_exp2f(far ? s + 32.0f : s) * __builtin_amdgcn_exp2f(r));
  return v < 0.0f ? (far ? v * q * 0x1p-32f : v * q) : v * (1.0f - (far ? 0.0f : q));
}

// Its tanh form: v (1 + tanh u) / 2 = v / (1 + e^-2u), u = sqrt(2/pi) (v + 0.044715 v^3); the
// exponent in fp64, for a cubic's roundings would be as large as a small result's bits.
__device__ __forceinline__ float gelu_tanh_f32(float v) {
  const double w = v;
  const double t = fmin(fmax(w * fma(w * w, -0.1029432395800235, -2.302208198144325), -150.0), 300.0);
  const float high = (float)t;
  return over_one_plus_exp2(v, high, (float)(t - (double)high));
}

// f of four sums.
__device__ __forceinline__ v4f apply_function(int fn, v4f v) {
  switch (fn) {
    case MOE_FN_RELU:
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = v[j] < 0.0f ? 0.0f : v[j];
      break;
    case MOE_FN_SILU:
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = silu_f32(v[j]);
      break;
    case MOE_FN_GELU:
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = gelu_f32(v[j]);
      break;
    case MOE_FN_GELU_TANH:
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = gelu_tanh_f32(v[j]);
      break;
    default: break;
  }
  return v;
}

__device__ __forceinline__ v4f load4_f32(const void* p, size_t i, bool f32, int left) {
  v4f v = {0.f, 0.f, 0.f, 0.f};
  if (f32) {
    const float* q = static_cast<const float*>(p) + i;
    if (left >= 4) return *reinterpret_cast<const v4f_at4*>(q);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < left) v[j] = q[j];
  } else {
    const uint16_t* q = static_cast<const uint16_t*>(p) + i;
    if (left >= 4) {
      const v2u b = *reinterpret_cast<const v2u_at2*>(q);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = bf16_to_f32(b[j / 2] >> (j % 2 * 16) & 0xFFFFu);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < left) v[j] = bf16_to_f32(q[j]);
    }
  }
  return v;
}

// Four neighbouring outputs of a row from their sums (and, gated, the sums of
// their up rows): bias, f, row scale and addend in fp32, one rounding.  N - n values
// of them exist.
template <bool GATED>
__device__ __forceinline__ void finish4(const Bf16Args& p, int group, int row, int n, v4f v, const v4f& up) {
  const int left = p.N - n;
  if (left <= 0) return;
  const size_t bias_at = (size_t)group * (GATED ? 2 : 1) * p.N + n;
  if (p.bias != nullptr) v += load4_f32(p.bias, bias_at, p.bias_f32, left);
  v = apply_function(p.fn, v);
  if constexpr (GATED) {
    v4f u = up;
    if (p.bias != nullptr) u += load4_f32(p.bias, bias_at + p.N, p.bias_f32, left);
    v *= u;
  }
  if (p.row_scale != nullptr) v *= p.row_scale[row];
  if (p.addend != nullptr) v += load4_f32(p.addend, (size_t)row * p.lda + n, p.add_f32, left);
  if (p.out_f32) {
    float* o = static_cast<float*>(p.out) + (size_t)row * p.ldo + n;
    if (left >= 4) {
      *reinterpret_cast<v4f_at4*>(o) = v;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < left) o[j] = v[j];
    }
  } else {
    uint16_t* o = static_cast<uint16_t*>(p.out) + (size_t)row * p.ldo + n;
    if (left >= 4) {
      *reinterpret_cast<v2u_at2*>(o) = v2u{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < left) o[j] = (uint16_t)pack_bf16(v[j], 0.0f);
    }
  }
}

}  // namespace moe
