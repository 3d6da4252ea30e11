// The norm after a block with its gate and residual scale, the addition to the residual
// stream, and the norm and quantization before the next block (moe_w4a4_post_norm):
//   z = x * w1 / sqrt(mean(x^2) + eps)   (or x);   h = rnd(r + scale * gate * z);
//   y = bf16(h * w2 / sqrt(mean(h^2) + eps));      codes, scales = Q(y).
//
// Bound by HBM: the row of x and of r stays in registers through both sums, so every
// input is read once and every output written once.  Teams of 64 to 1024 threads and
// pieces of 8 values as in norm.hip, and like there sums, norms and products run in
// fp64 (hidden behind the loads): h has one rounding, the same whatever the order of
// the sums, and the codes behind it are reproducible next to the quantizer's borders.
#include "launch_bf16.h"
#include "moe_w4a4.h"
#include "norm_rows.h"

namespace moe {
namespace {

__device__ __forceinline__ void load8(const void* p, size_t i, bool f32, float (&f)[8]) {
  if (f32)
    load_f32x8(static_cast<const float*>(p) + i, f);
  else
    unpack8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i), f);
}

// 8 values of the residual stream in its own type.
template <bool F32>
struct Stream {
  uint4 b;
  __device__ __forceinline__ void load(const void* p, size_t i) {
    b = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
  }
  __device__ __forceinline__ void store(void* p, size_t i) const {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = b;
  }
  __device__ __forceinline__ void clear() { b = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&f)[8]) const { unpack8(b, f); }
  __device__ __forceinline__ void set(const float (&f)[8]) { b = pack8(f); }
};
template <>
struct Stream<true> {
  float h[8];
  __device__ __forceinline__ void load(const void* p, size_t i) { load_f32x8(static_cast<const float*>(p) + i, h); }
  __device__ __forceinline__ void store(void* p, size_t i) const {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    q[0] = make_float4(h[0], h[1], h[2], h[3]);
    q[1] = make_float4(h[4], h[5], h[6], h[7]);
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = 0.0f;
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = h[i];
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = f[i];
  }
};

// RES_F32: type of the residual stream.  ACT: codes of 0 MXFP4, 1 MXFP8 E4M3, 2 NVFP4,
// or -1 none.  TPR: threads per row, CPL pieces each.
template <bool RES_F32, int ACT, int TPR, int CPL>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) post_norm_kernel(PostNormArgs p) {
  constexpr int THREADS = TPR < 256 ? 256 : TPR;
  constexpr int RPB = THREADS / TPR;
  constexpr int WPR = TPR / kWave;
  __shared__ double part[2][WPR > 1 ? WPR : 1];
  const int t = threadIdx.x % TPR, pieces = p.cols >> 3;
  const double eps = p.eps;
  // The team's sum; two buffers, so that a wave may be a sum ahead of one still reading.
  int flip = 0;
  auto team_sum = [&](double v) {
    v = wave_sum(v);
    if constexpr (WPR > 1) {
      if (t % kWave == 0) part[flip][t / kWave] = v;
      __syncthreads();
      v = 0.0;
#pragma unroll
      for (int i = 0; i < WPR; ++i) v += part[flip][i];
      flip ^= 1;
    }
    return v;
  };
  for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR; row < p.rows; row += (int64_t)gridDim.x * RPB) {
    const size_t base = (size_t)row * p.cols;
    uint4 x[CPL];
    Stream<RES_F32> h[CPL];
#pragma unroll
    for (int j = 0; j < CPL; ++j) {
      const int c = t + j * TPR;
      if (c < pieces) {
        x[j] = *reinterpret_cast<const uint4*>(p.x + base + 8 * c);
        h[j].load(p.residual, base + 8 * c);
      } else {
        x[j] = make_uint4(0, 0, 0, 0);
        h[j].clear();
      }
    }
    double factor = p.scale;
    if (p.gate_kind == MOE_GATE_ROW)
      factor *= p.gate_f32 ? static_cast<const float*>(p.gate)[row]
                           : bf16_to_f32(static_cast<const uint16_t*>(p.gate)[row]);
    if (p.post_weight != nullptr) {
      double ss = 0.0;
#pragma unroll
      for (int j = 0; j < CPL; ++j) {
        float v[8];
        unpack8(x[j], v);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fma((double)v[i], (double)v[i], ss);
      }
      factor /= sqrt(team_sum(ss) / p.cols + eps);
    }
    double ss = 0.0;
#pragma unroll
    for (int j = 0; j < CPL; ++j) {
      const int c = t + j * TPR;
      if (c >= pieces) continue;
      float v[8], r[8], w[8];
      double d[8];
      unpack8(x[j], v);
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] = (double)v[i] * factor;
      if (p.post_weight != nullptr) {
        load8(p.post_weight, 8 * c, p.w_f32, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] *= (double)w[i];
      }
      if (p.gate_kind == MOE_GATE_CHANNEL || p.gate_kind == MOE_GATE_FULL) {
        load8(p.gate, (p.gate_kind == MOE_GATE_FULL ? base : 0) + 8 * c, p.gate_f32, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] *= (double)w[i];
      }
      h[j].get(r);
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i] = (float)((double)r[i] + d[i]);
      h[j].set(r);
      h[j].store(p.residual_out, base + 8 * c);
      h[j].get(r);
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fma((double)r[i], (double)r[i], ss);
    }
    if (p.next_weight == nullptr) continue;
    const double rstd = 1.0 / sqrt(team_sum(ss) / p.cols + eps);
#pragma unroll
    for (int j = 0; j < CPL; ++j) {
      const int c = t + j * TPR;
      float w[8] = {0, 0, 0, 0, 0, 0, 0, 0}, v[8], n[8];
      if (c < pieces) load8(p.next_weight, 8 * c, p.w_f32, w);
      h[j].get(v);
#pragma unroll
      for (int i = 0; i < 8; ++i) n[i] = (float)((double)v[i] * rstd * (double)w[i]);
      const uint4 yb = pack8(n);
      if (p.y != nullptr && c < pieces) *reinterpret_cast<uint4*>(p.y + base + 8 * c) = yb;
      if constexpr (ACT >= 0) quantize_piece<ACT>(yb, (size_t)row * pieces, c, pieces, p.g, p.codes, p.scales);
    }
  }
}

constexpr int64_t kPostMaxBlocks = 1 << 20;   // more rows: a block takes several

template <bool RES_F32, int ACT, int TPR, int CPL>
hipError_t launch_post(const PostNormArgs& a, hipStream_t stream) {
  constexpr int THREADS = TPR < 256 ? 256 : TPR;
  constexpr int RPB = THREADS / TPR;
  const int64_t blocks = (a.rows + RPB - 1) / RPB;
  hipLaunchKernelGGL((post_norm_kernel<RES_F32, ACT, TPR, CPL>),
                     dim3((unsigned)(blocks < kPostMaxBlocks ? blocks : kPostMaxBlocks)), dim3(THREADS), 0, stream, a);
  return hipGetLastError();
}

// The smallest team that holds the row in at most 4 pieces a thread (8 past 32768 values).
template <bool RES_F32, int ACT>
hipError_t launch_post_act(const PostNormArgs& a, hipStream_t stream) {
  if (a.cols <= 512) return launch_post<RES_F32, ACT, 64, 1>(a, stream);
  if (a.cols <= 1024) return launch_post<RES_F32, ACT, 64, 2>(a, stream);
  if (a.cols <= 2048) return launch_post<RES_F32, ACT, 256, 1>(a, stream);
  if (a.cols <= 4096) return launch_post<RES_F32, ACT, 256, 2>(a, stream);
  if (a.cols <= 8192) return launch_post<RES_F32, ACT, 256, 4>(a, stream);
  if (a.cols <= 16384) return launch_post<RES_F32, ACT, 1024, 2>(a, stream);
  if (a.cols <= 32768) return launch_post<RES_F32, ACT, 1024, 4>(a, stream);
  return launch_post<RES_F32, ACT, 1024, 8>(a, stream);
}

template <bool RES_F32>
hipError_t launch_post_res(int act, const PostNormArgs& a, hipStream_t stream) {
  auto f = act == 0 ? launch_post_act<RES_F32, 0> : act == 1 ? launch_post_act<RES_F32, 1>
         : act == 2 ? launch_post_act<RES_F32, 2> : launch_post_act<RES_F32, -1>;
  return f(a, stream);
}

}  // namespace

hipError_t launch_post_norm(int act, bool res_f32, const PostNormArgs& a, hipStream_t stream) {
  return res_f32 ? launch_post_res<true>(act, a, stream) : launch_post_res<false>(act, a, stream);
}

}  // namespace moe
