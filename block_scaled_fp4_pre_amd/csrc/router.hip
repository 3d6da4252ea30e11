// The router's choice (moe_w4a4_router): per token the scores of its experts,
// the best groups, the top-k experts and their weights.
//
// One wave per token; lane l holds experts l, l + 64, ... (coalesced loads).
// The choice runs on 32-bit keys that order as the floats do (0: not to be
// chosen); a round takes the wave's maximum by six DPP steps and the lowest
// expert that has it.
//
// A bias makes the scores decide, and those are defined as fp64 values rounded to
// float32, so that near-equal experts fall the same way as in any exact
// evaluation.  fp64 exponentials and logarithms of every expert would take most
// of the kernel's time, so the wave first chooses by float32 scores and looks at
// the gaps: where every chosen expert is ahead of the next, and the last kept
// group ahead of the first dropped one, by more than the two kinds of scores can
// differ, the choice is the exact one.  Otherwise (about one token in a thousand
// with random logits) it chooses again by exact scores.
//
// Bound by the latency of one token's chain for few tokens (8 x 256, top-6 with a
// bias: 5.8 us), by instruction issue for many: 16384 x 256 bfloat16 logits, softmax,
// 13.0 us against 1.8 us for their bytes (0.8 more with the chosen logit carried beside its
// key where there is no bias; 32 with fp64 scores and reductions through LDS).
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

// v of the lane that DPP control CTRL names; 0 where there is none.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}
// Lane 63 gathers the wave by shifts of 1, 2, 4, 8 inside rows of 16 and the
// broadcasts of lanes 15 and 31; what comes from outside is 0.
#define MOE_GATHER(op)                                                              \
  op(dpp<0x111>) op(dpp<0x112>) op(dpp<0x114>) op(dpp<0x118>) op(dpp<0x142>) op(dpp<0x143>)
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {   // the same in every lane
#define MOE_OP(f) v = max(v, f(v));
  MOE_GATHER(MOE_OP)
#undef MOE_OP
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ float wave_sum(float v) {
  // (a broadcast adds into the rows behind it only: rows 1 and 3, then 2 and 3)
  v += __uint_as_float(dpp<0x111>(__float_as_uint(v)));
  v += __uint_as_float(dpp<0x112>(__float_as_uint(v)));
  v += __uint_as_float(dpp<0x114>(__float_as_uint(v)));
  v += __uint_as_float(dpp<0x118>(__float_as_uint(v)));
  v += __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), 0x142, 0xA, 0xF, false));
  v += __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), 0x143, 0xC, 0xF, false));
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}
// Sum of lanes 0 to 15.
__device__ __forceinline__ float row_sum(float v) {
  v += __uint_as_float(dpp<0x111>(__float_as_uint(v)));
  v += __uint_as_float(dpp<0x112>(__float_as_uint(v)));
  v += __uint_as_float(dpp<0x114>(__float_as_uint(v)));
  v += __uint_as_float(dpp<0x118>(__float_as_uint(v)));
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 15));
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
__device__ __forceinline__ float score32(int scoring, float l, float top) {
  if (scoring == MOE_SCORE_SOFTMAX) {
    // exp(l - top) with the rounding of the difference put back: half a step of it
    // is 2^-18 from 64 on, far more than the bits of the exponential.
    const float d = l - top, t = d - l, r = (l - (d - t)) - (top + t);   // d + r == l - top
    const float q = expf(d);
    return q > 0.0f ? fmaf(q, r, q) : q;                                 // (d may be -infinity)
  }
  const float e = expf(-fabsf(l));
  if (scoring == MOE_SCORE_SIGMOID) return (l < 0.0f ? e : 1.0f) / (1.0f + e);
  // far below zero log(1 + exp(l)) is exp(l) and would lose its bits there
  return l < -20.0f ? expf(0.5f * l) : sqrtf(fmaxf(l, 0.0f) + log1pf(e));
}
__device__ __noinline__ double score64(int scoring, double l, double top) {
  if (scoring == MOE_SCORE_SOFTMAX) return exp(l - top);
  if (scoring == MOE_SCORE_SIGMOID) return 1.0 / (1.0 + exp(-l));
  return sqrt(fmax(l, 0.0) + log1p(exp(-fabs(l))));
}

__device__ __forceinline__ float load_logit(bool bf16, const void* logits, int64_t i) {
  const float l = bf16 ? bf16_to_f32(static_cast<const uint16_t*>(logits)[i]) : static_cast<const float*>(logits)[i];
  return l > 3.402823466e38f ? 3.402823466e38f : l;
}

// EPL: experts per lane.  BIAS, GROUPS: whether there are any (a token then takes
// a third of the instructions without them).
template <int EPL, int scoring, bool BIAS, bool GROUPS>
__global__ void __launch_bounds__(kRouterThreads) router_kernel(
    bool bf16, int64_t T, int E, int k, int groups, int keep, const void* __restrict__ logits,
    const float* __restrict__ bias, bool renormalize, float scale, int32_t* __restrict__ ids,
    float* __restrict__ weights) {
  __shared__ uint32_t row_keys[GROUPS ? kRouterRows : 1][EPL * kWave];
  const int lane = threadIdx.x & (kWave - 1);
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int gs = GROUPS ? E / groups : E;
  int lpg = kWave;                         // lanes per group: a power of two, all groups in one wave
  if constexpr (GROUPS)
    while (lpg * groups > kWave) lpg >>= 1;
  float b[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) b[i] = BIAS ? bias[min(i * kWave + lane, E - 1)] : 0.0f;
  for (int64_t t = (int64_t)blockIdx.x * kRouterRows + w; t < T; t += (int64_t)gridDim.x * kRouterRows) {
    float l[EPL];
    if (bf16) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) l[i] = load_logit(true, logits, t * E + min(i * kWave + lane, E - 1));
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i) l[i] = load_logit(false, logits, t * E + min(i * kWave + lane, E - 1));
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (i * kWave + lane >= E) l[i] = -__builtin_inff();
    // softmax: the row's maximum and sum
    float top = 0.0f, rsum = 1.0f;
    if constexpr (scoring == MOE_SCORE_SOFTMAX) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < EPL; ++i) m = max(m, order_key(l[i]));
      m = wave_max(m);
      if (m) {
        top = key_value(m);
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
          if (order_key(l[i])) s += expf(l[i] - top);
        rsum = wave_sum(s);
      }
    }
    int mine = -1;                         // lane j: the expert of slot j, and its logit
    float logit = 0.0f;
    for (bool exact = !BIAS;; exact = true) {
      uint32_t key[EPL];
      float unsure = 0.0f;                 // two values further apart than this are in their true order
      if constexpr (!BIAS) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) key[i] = order_key(l[i]);
      } else if (!exact) {
        // In units of 2^-23 of the largest magnitude in play: by the library's
        // bounds (exp 3, log1p 2, sqrt 3, division 2.5 last bits) a float32 score
        // is within 6.5 of the exact one, and the roundings of the scores and of
        // their sums with the bias add 1.5 a side: 16 for the two sides of a
        // comparison.  A softmax's sum is off by 14 at most (exp 3, 14
        // additions 7, the differences' roundings, weighted by the terms, 4) on
        // both sides alike, so this adds 14 times the two scores' difference: 30.
        // A rank of two scores doubles all of it and adds 4 for its own roundings.
        // (Scores below 2^-126: 2^-149 absolute.)
        constexpr float kMargin = scoring == MOE_SCORE_SOFTMAX ? 0x1.1p-18f : 0x1.4p-19f;
        float big = 0.0f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          key[i] = 0;
          if (order_key(l[i])) {
            const float q = score32(scoring, l[i], top);
            const float s = scoring == MOE_SCORE_SOFTMAX ? q / rsum : q, c = s + b[i];
            key[i] = order_key(c);
            if (key[i]) big = fmaxf(big, fmaxf(s, fabsf(c)));
          }
        }
        unsure = __uint_as_float(wave_max(__float_as_uint(big))) * kMargin + 0x1p-140f;
      } else {
        double sum = 1.0;
        if (scoring == MOE_SCORE_SOFTMAX) {
          sum = 0.0;
#pragma unroll 1
          for (int e = lane; e < E; e += kWave) {
            const float v = load_logit(bf16, logits, t * E + e);
            if (order_key(v)) sum += score64(scoring, (double)v, (double)top);
          }
          sum = wave_sum(sum);
        }
#pragma unroll
        for (int i = 0; i < EPL; ++i)
          key[i] = order_key(l[i]) ? order_key((float)(score64(scoring, (double)l[i], (double)top) / sum) + b[i]) : 0u;
      }
      bool sure = true;
      if constexpr (GROUPS) {
        // Ranks of the groups: lanes [g*lpg, (g+1)*lpg) scan group g's keys for
        // its two largest, merge them, and every lane learns the kept groups.
#pragma unroll
        for (int i = 0; i < EPL; ++i) row_keys[w][i * kWave + lane] = key[i];
        wave_lds_fence();
        const int g = lane / lpg;
        uint32_t a = 0, a2 = 0;            // the group's two largest keys, a >= a2
        if (g < groups)
          for (int i = lane % lpg; i < gs; i += lpg) {
            const uint32_t v = row_keys[w][g * gs + i];
            a2 = max(a2, min(a, v));
            a = max(a, v);
          }
        for (int m = 1; m < lpg; m <<= 1) {
          const uint32_t o = (uint32_t)__shfl_xor((int)a, m), o2 = (uint32_t)__shfl_xor((int)a2, m);
          a2 = max(max(a2, o2), min(a, o));
          a = max(a, o);
        }
        uint32_t rank = a;
        if (BIAS && a2) rank = order_key(key_value(a) + key_value(a2));
        int before = 0;                    // groups ahead of this lane's
        for (int j = 0; j < groups; ++j) {
          const uint32_t r = (uint32_t)__builtin_amdgcn_readlane((int)rank, j * lpg);
          before += r > rank || (r == rank && j < g) ? 1 : 0;
        }
        const bool in = g < groups && before < keep;
        const uint64_t kept = __ballot(in);
        if (!exact) {
          // the worst kept group against the best dropped one (a sum of two
          // scores each, so twice the margin)
          const uint32_t worst = ~wave_max(in ? ~rank : 0u), best = wave_max(!in && g < groups ? rank : 0u);
          sure = best == 0 || key_value(worst) - key_value(best) > 2.0f * unsure;
        }
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          const int e = i * kWave + lane;
          if (e < E && !((kept >> (e / gs * lpg)) & 1)) key[i] = 0;
        }
        wave_lds_fence();
      }
      // k rounds; lane j keeps the winner of round j.
      mine = -1;
      float last = 0.0f;
      for (int j = 0; j < k + (exact ? 0 : 1); ++j) {
        uint32_t best = key[0];
        float val = l[0];
        int at = lane;
#pragma unroll
        for (int i = 1; i < EPL; ++i)
          if (key[i] > best) {
            best = key[i];
            if constexpr (BIAS) val = l[i];
            at = i * kWave + lane;
          }
        const uint32_t m = wave_max(best);
        if (m == 0) break;
        if (!exact) {
          if (j > 0 && !(last - key_value(m) > unsure)) sure = false;
          last = key_value(m);
        }
        uint64_t tied = __ballot(best == m);
        int owner = (int)__builtin_ctzll(tied), e = __builtin_amdgcn_readlane(at, owner);
        for (tied &= tied - 1; tied; tied &= tied - 1) {
          const int o = (int)__builtin_ctzll(tied), e2 = __builtin_amdgcn_readlane(at, o);
          if (e2 < e) {
            e = e2;
            owner = o;
          }
        }
        // (without a bias the key is the logit)
        const float v = BIAS ? __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(val), owner))
                             : key_value(m);
        if (j < k && lane == j) {
          mine = e;
          logit = v;
        }
#pragma unroll
        for (int i = 0; i < EPL; ++i)
          if (i * kWave + lane == e) key[i] = 0;
      }
      if (exact || sure) break;
    }
    float s = 0.0f;
    if (mine >= 0) s = scoring == MOE_SCORE_SOFTMAX ? score32(scoring, logit, top) / rsum : score32(scoring, logit, top);
    if (renormalize) s = s / (row_sum(s) + 1e-20f);        // lanes from k on hold 0
    if (lane < k) {
      ids[t * k + lane] = mine;
      weights[t * k + lane] = s * scale;
    }
  }
}

template <int EPL, int SCORING>
hipError_t launch_scoring(bool bf16, int64_t T, int E, int k, int groups, int keep, const void* logits,
                          const float* bias, bool renormalize, float scale, int32_t* ids, float* weights,
                          hipStream_t stream) {
  const int64_t blocks = (T + kRouterRows - 1) / kRouterRows, most = 1 << 20;   // more tokens: a wave takes several
  auto kern = bias != nullptr
                  ? (groups > 1 ? router_kernel<EPL, SCORING, true, true> : router_kernel<EPL, SCORING, true, false>)
                  : (groups > 1 ? router_kernel<EPL, SCORING, false, true> : router_kernel<EPL, SCORING, false, false>);
  hipLaunchKernelGGL(kern, dim3((unsigned)(blocks < most ? blocks : most)), dim3(kRouterThreads), 0, stream, bf16, T, E,
                     k, groups, keep, logits, bias, renormalize, scale, ids, weights);
  return hipGetLastError();
}

template <int EPL>
hipError_t launch_experts(int scoring, bool bf16, int64_t T, int E, int k, int groups, int keep, const void* logits,
                          const float* bias, bool renormalize, float scale, int32_t* ids, float* weights,
                          hipStream_t stream) {
  auto f = scoring == MOE_SCORE_SOFTMAX   ? launch_scoring<EPL, MOE_SCORE_SOFTMAX>
           : scoring == MOE_SCORE_SIGMOID ? launch_scoring<EPL, MOE_SCORE_SIGMOID>
                                          : launch_scoring<EPL, MOE_SCORE_SQRTSOFTPLUS>;
  return f(bf16, T, E, k, groups, keep, logits, bias, renormalize, scale, ids, weights, stream);
}

}  // namespace

hipError_t launch_router(bool logits_bf16, int scoring, int64_t T, int E, int k, int groups, int keep,
                         const void* logits, const float* bias, bool renormalize, float scale, int32_t* ids,
                         float* weights, hipStream_t stream) {
  auto f = E <= 64 ? launch_experts<1> : E <= 128 ? launch_experts<2> : E <= 256 ? launch_experts<4> : launch_experts<8>;
  return f(scoring, logits_bf16, T, E, k, groups, keep, logits, bias, renormalize, scale, ids, weights, stream);
}

}  // namespace moe
