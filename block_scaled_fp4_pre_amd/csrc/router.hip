// The router's choice (moe_w4a4_router): per token the scores of its experts,
// the best groups, the top-k experts and their weights.
//
// One wave per token; lane l holds experts l, l + 64, ... (coalesced loads).
// The choice runs on 32-bit keys that order as the floats do (0: not to be
// chosen); a round takes the wave's maximum by a butterfly and the lowest
// expert that has it.  Scores that decide (a bias is added) are computed in
// fp64 and rounded to float32, so that near-equal experts fall the same way as
// in any exact evaluation.
#include "device_common.h"
#include "launch_ops.h"
#include "moe_w4a4.h"

namespace moe {
namespace {

constexpr int kRouterThreads = 256;
constexpr int kRouterRows = kRouterThreads / kWave;

// Float bits -> key: larger float, larger key; -0 and +0 alike; NaN and
// -infinity -> 0.
__device__ __forceinline__ uint32_t order_key(float f) {
  if (!(f > -__builtin_inff())) return 0u;
  const uint32_t b = __float_as_uint(f + 0.0f);
  return (int32_t)b < 0 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {   // of a key that is not 0
  return __uint_as_float((int32_t)k < 0 ? k & 0x7FFFFFFFu : ~k);
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int m = 1; m < kWave; m <<= 1) v = max(v, (uint32_t)__shfl_xor((int)v, m));
  return v;
}
__device__ __forceinline__ uint32_t wave_min(uint32_t v) {
#pragma unroll
  for (int m = 1; m < kWave; m <<= 1) v = min(v, (uint32_t)__shfl_xor((int)v, m));
  return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int m = 1; m < kWave; m <<= 1) v += __shfl_xor(v, m);
  return v;
}

// Orders this wave's LDS writes before its later LDS reads by other lanes.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Score of a logit that can be chosen; softmax before its division.
__device__ __forceinline__ double score64(int scoring, double l, double top) {
  if (scoring == MOE_SCORE_SOFTMAX) return exp(l - top);
  if (scoring == MOE_SCORE_SIGMOID) return 1.0 / (1.0 + exp(-l));
  return sqrt(fmax(l, 0.0) + log1p(exp(-fabs(l))));
}

// EPL: experts per lane.
template <int EPL, bool BF16>
__global__ void __launch_bounds__(kRouterThreads) router_kernel(
    int scoring, int64_t T, int E, int k, int groups, int keep, const void* __restrict__ logits,
    const float* __restrict__ bias, bool renormalize, float scale, int32_t* __restrict__ ids,
    float* __restrict__ weights) {
  __shared__ uint32_t row_keys[kRouterRows][EPL * kWave];
  const int lane = threadIdx.x & (kWave - 1), w = threadIdx.x / kWave;
  const int gs = E / groups;
  for (int64_t t = (int64_t)blockIdx.x * kRouterRows + w; t < T; t += (int64_t)gridDim.x * kRouterRows) {
    float l[EPL];
    uint32_t key[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = i * kWave + lane;
      l[i] = -__builtin_inff();
      if (e < E) {
        if constexpr (BF16)
          l[i] = bf16_to_f32(static_cast<const uint16_t*>(logits)[t * E + e]);
        else
          l[i] = static_cast<const float*>(logits)[t * E + e];
      }
      l[i] = l[i] > 3.402823466e38f ? 3.402823466e38f : l[i];
      key[i] = order_key(l[i]);
    }
    // softmax: the row's maximum and sum
    double top = 0.0, rsum = 1.0;
    if (scoring == MOE_SCORE_SOFTMAX) {
      uint32_t m = key[0];
#pragma unroll
      for (int i = 1; i < EPL; ++i) m = max(m, key[i]);
      m = wave_max(m);
      top = m ? (double)key_value(m) : 0.0;
      double s = 0.0;
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (key[i]) s += exp((double)l[i] - top);
      s = wave_sum(s);
      rsum = m ? s : 1.0;
    }
    if (bias != nullptr) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int e = i * kWave + lane;
        if (key[i]) key[i] = order_key((float)(score64(scoring, (double)l[i], top) / rsum) + bias[e]);
      }
    }
    if (groups > 1) {
      // Ranks of the groups: lanes [g*lpg, (g+1)*lpg) scan group g's keys for
      // its two largest, merge them, and every lane learns the kept groups.
#pragma unroll
      for (int i = 0; i < EPL; ++i) row_keys[w][i * kWave + lane] = key[i];
      wave_lds_fence();
      int lpg = kWave;
      while (lpg * groups > kWave) lpg >>= 1;
      const int g = lane / lpg;
      uint32_t a = 0, b = 0;               // the group's two largest keys, a >= b
      if (g < groups)
        for (int i = lane % lpg; i < gs; i += lpg) {
          const uint32_t v = row_keys[w][g * gs + i];
          b = max(b, min(a, v));
          a = max(a, v);
        }
      for (int m = 1; m < lpg; m <<= 1) {
        const uint32_t a2 = (uint32_t)__shfl_xor((int)a, m), b2 = (uint32_t)__shfl_xor((int)b, m);
        b = max(max(b, b2), min(a, a2));
        a = max(a, a2);
      }
      uint32_t rank = a;
      if (bias != nullptr && b) rank = order_key(key_value(a) + key_value(b));
      int before = 0;                      // groups ahead of this lane's
      for (int j = 0; j < groups; ++j) {
        const uint32_t r = (uint32_t)__shfl((int)rank, j * lpg);
        before += r > rank || (r == rank && j < g) ? 1 : 0;
      }
      const uint64_t kept = __ballot(g < groups && before < keep);
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int e = i * kWave + lane;
        if (e < E && !((kept >> (e / gs * lpg)) & 1)) key[i] = 0;
      }
      wave_lds_fence();
    }
    // k rounds; lane j keeps the winner of round j.
    int mine = -1;
    for (int j = 0; j < k; ++j) {
      uint32_t best = key[0];
      int at = lane;
#pragma unroll
      for (int i = 1; i < EPL; ++i)
        if (key[i] > best) {
          best = key[i];
          at = i * kWave + lane;
        }
      const uint32_t m = wave_max(best);
      if (m == 0) break;
      const uint32_t e = wave_min(best == m ? (uint32_t)at : ~0u);
      if (lane == j) mine = (int)e;
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (i * kWave + lane == (int)e) key[i] = 0;
    }
    double s = 0.0;
    if (mine >= 0) {
      float v;
      if constexpr (BF16)
        v = bf16_to_f32(static_cast<const uint16_t*>(logits)[t * E + mine]);
      else
        v = static_cast<const float*>(logits)[t * E + mine];
      v = v > 3.402823466e38f ? 3.402823466e38f : v;
      s = score64(scoring, (double)v, top) / rsum;
    }
    if (renormalize) {
      double sum = s;                      // lanes >= 16 hold 0
#pragma unroll
      for (int m = 1; m < 16; m <<= 1) sum += __shfl_xor(sum, m);
      s = s / (sum + 1e-20);
    }
    if (lane < k) {
      ids[t * k + lane] = mine;
      weights[t * k + lane] = mine >= 0 ? (float)(s * (double)scale) : 0.0f;
    }
  }
}

}  // namespace

hipError_t launch_router(bool logits_bf16, int scoring, int64_t T, int E, int k, int groups, int keep,
                         const void* logits, const float* bias, bool renormalize, float scale, int32_t* ids,
                         float* weights, hipStream_t stream) {
  const int64_t blocks = (T + kRouterRows - 1) / kRouterRows, most = 1 << 20;   // more tokens: a wave takes several
  const dim3 grid((unsigned)(blocks < most ? blocks : most));
#define MOE_ROUTER(EPL)                                                                                            \
  hipLaunchKernelGGL((logits_bf16 ? router_kernel<EPL, true> : router_kernel<EPL, false>), grid,                   \
                     dim3(kRouterThreads), 0, stream, scoring, T, E, k, groups, keep, logits, bias, renormalize,   \
                     scale, ids, weights)
  if (E <= 64)
    MOE_ROUTER(1);
  else if (E <= 128)
    MOE_ROUTER(2);
  else if (E <= 256)
    MOE_ROUTER(4);
  else
    MOE_ROUTER(8);
#undef MOE_ROUTER
  return hipGetLastError();
}

}  // namespace moe
