// Residual addition, root-mean-square norm and quantization of rows
// (moe_w4a4_add_rmsnorm):
//   h = rnd(x + r);  n = h * w / sqrt(mean(h^2) + eps);  y = bf16(n);
//   codes, scales = Q(y), the activation formats of the layer.
//
// Bound by HBM: every input is read once and every output written once; the row
// stays in registers between the sum and the norm, so nothing is read twice.
// A team of 64, 256 or 1024 threads owns a row; a thread holds CPL pieces of
// 8 consecutive values (16-byte loads), so four neighbouring lanes share an
// MX group of 32 (two an NVFP4 block of 16) and exchange its absolute maximum
// by two (one) DPP steps inside their quad.
//
// The squares' sum, the reciprocal root and both products run in fp64 (full
// rate on this chip, hidden behind the loads): the result is then rounded
// the same way whatever the order of the sum, so the codes are reproducible
// next to the quantizer's borders.
#include "launch_ops.h"
#include "quant_e4m3.h"

namespace moe {
namespace {

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
  return make_uint4(f32_to_bf16(f[0]) | (f32_to_bf16(f[1]) << 16), f32_to_bf16(f[2]) | (f32_to_bf16(f[3]) << 16),
                    f32_to_bf16(f[4]) | (f32_to_bf16(f[5]) << 16), f32_to_bf16(f[6]) | (f32_to_bf16(f[7]) << 16));
}

// Sum over the 64 lanes, the same bits in every lane.
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int m = 1; m < kWave; m <<= 1) v += __shfl_xor(v, m);
  return v;
}

// RES: 0 no residual, 1 bfloat16, 2 float32.  TPR: threads per row.
template <int RES, int TPR, int CPL>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) add_rmsnorm_kernel(
    int act, bool w_f32, int64_t rows, int cols, const uint16_t* x, const void* residual,
    const void* __restrict__ weight, double eps, float g, void* residual_out, uint16_t* y,
    uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  constexpr int THREADS = TPR < 256 ? 256 : TPR;
  constexpr int RPB = THREADS / TPR;
  constexpr int WPR = TPR / kWave;
  __shared__ double part[2][WPR > 1 ? WPR : 1];
  const int t = threadIdx.x % TPR, pieces = cols >> 3;
  int flip = 0;
  for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR; row < rows; row += (int64_t)gridDim.x * RPB) {
    const size_t base = (size_t)row * cols;
    float h[CPL][8];
    double ss = 0.0;
#pragma unroll
    for (int j = 0; j < CPL; ++j) {
      const int c = t + j * TPR;
      if (c < pieces) {
        unpack8(reinterpret_cast<const uint4*>(x + base)[c], h[j]);
        if constexpr (RES == 1) {
          float r[8];
          unpack8(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(residual) + base)[c], r);
#pragma unroll
          for (int i = 0; i < 8; ++i) h[j][i] = bf16_to_f32(f32_to_bf16(h[j][i] + r[i]));
        } else if constexpr (RES == 2) {
          float r[8];
          load_f32x8(static_cast<const float*>(residual) + base + 8 * c, r);
#pragma unroll
          for (int i = 0; i < 8; ++i) h[j][i] += r[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[j][i] = 0.0f;
      }
    }
#pragma unroll
    for (int j = 0; j < CPL; ++j) {
      const int c = t + j * TPR;
      if constexpr (RES == 1) {
        if (c < pieces) reinterpret_cast<uint4*>(static_cast<uint16_t*>(residual_out) + base)[c] = pack8(h[j]);
      } else if constexpr (RES == 2) {
        if (c < pieces) {
          float4* p = reinterpret_cast<float4*>(static_cast<float*>(residual_out) + base + 8 * c);
          p[0] = make_float4(h[j][0], h[j][1], h[j][2], h[j][3]);
          p[1] = make_float4(h[j][4], h[j][5], h[j][6], h[j][7]);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fma((double)h[j][i], (double)h[j][i], ss);
    }
    ss = wave_sum(ss);
    if constexpr (WPR > 1) {
      // two buffers: a wave may be a row ahead of one still reading
      if (t % kWave == 0) part[flip][t / kWave] = ss;
      __syncthreads();
      ss = 0.0;
#pragma unroll
      for (int i = 0; i < WPR; ++i) ss += part[flip][i];
      flip ^= 1;
    }
    const double rstd = 1.0 / sqrt(ss / cols + eps);
#pragma unroll
    for (int j = 0; j < CPL; ++j) {
      const int c = t + j * TPR;
      float w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if (c < pieces) {
        if (w_f32)
          load_f32x8(static_cast<const float*>(weight) + 8 * c, w);
        else
          unpack8(static_cast<const uint4*>(weight)[c], w);
      }
      float n[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) n[i] = (float)((double)h[j][i] * rstd * (double)w[i]);
      const uint4 yb = pack8(n);
      if (y != nullptr && c < pieces) reinterpret_cast<uint4*>(y + base)[c] = yb;
      if (act < 0) continue;
      // The group's absolute maximum on the bit patterns of the rounded y
      // (bf16 magnitudes order as their low 15 bits).
      const uint32_t yw[4] = {yb.x, yb.y, yb.z, yb.w};
      uint32_t amax = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) amax = max(amax, max(yw[i] & 0x7FFFu, (yw[i] >> 16) & 0x7FFFu));
      amax = max(amax, quad_xor<1>(amax));
      if (act != 2) amax = max(amax, quad_xor<2>(amax));
      unpack8(yb, n);
      const size_t piece = (size_t)row * pieces + c;   // 8 values each
      if (act == 1) {
        const int e = mx8_scale_exp(amax << 16);
        const float inv = e4m3_exp2(-e);
        const uint2 q = make_uint2(e4m3_cvt4(n[0], n[1], n[2], n[3], inv), e4m3_cvt4(n[4], n[5], n[6], n[7], inv));
        if (c < pieces) {
          reinterpret_cast<uint2*>(codes)[piece] = q;
          if (c % 4 == 0) scales[piece / 4] = (uint8_t)(e + 127);
        }
      } else if (act == 0) {
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
  }
}

constexpr int64_t kNormMaxBlocks = 1 << 20;   // more rows: a block takes several

template <int RES, int TPR, int CPL>
hipError_t launch_norm(int act, bool w_f32, int64_t rows, int cols, const uint16_t* x, const void* residual,
                       const void* weight, float eps, float g, void* residual_out, uint16_t* y, uint8_t* codes,
                       uint8_t* scales, hipStream_t stream) {
  constexpr int THREADS = TPR < 256 ? 256 : TPR;
  constexpr int RPB = THREADS / TPR;
  const int64_t blocks = (rows + RPB - 1) / RPB;
  hipLaunchKernelGGL((add_rmsnorm_kernel<RES, TPR, CPL>), dim3((unsigned)(blocks < kNormMaxBlocks ? blocks : kNormMaxBlocks)),
                     dim3(THREADS), 0, stream, act, w_f32, rows, cols, x, residual, weight, (double)eps, g,
                     residual_out, y, codes, scales);
  return hipGetLastError();
}

template <int RES>
hipError_t launch_norm_res(int act, bool w_f32, int64_t rows, int cols, const uint16_t* x, const void* residual,
                           const void* weight, float eps, float g, void* residual_out, uint16_t* y, uint8_t* codes,
                           uint8_t* scales, hipStream_t stream) {
#define MOE_NORM_ARGS act, w_f32, rows, cols, x, residual, weight, eps, g, residual_out, y, codes, scales, stream
  if (cols <= 512) return launch_norm<RES, 64, 1>(MOE_NORM_ARGS);
  if (cols <= 1024) return launch_norm<RES, 64, 2>(MOE_NORM_ARGS);
  if (cols <= 2048) return launch_norm<RES, 256, 1>(MOE_NORM_ARGS);
  if (cols <= 4096) return launch_norm<RES, 256, 2>(MOE_NORM_ARGS);
  if (cols <= 8192) return launch_norm<RES, 256, 4>(MOE_NORM_ARGS);
  if (cols <= 16384) return launch_norm<RES, 1024, 2>(MOE_NORM_ARGS);
  if (cols <= 32768) return launch_norm<RES, 1024, 4>(MOE_NORM_ARGS);
  return launch_norm<RES, 1024, 8>(MOE_NORM_ARGS);
#undef MOE_NORM_ARGS
}

}  // namespace

hipError_t launch_add_rmsnorm(int act, bool res_f32, bool w_f32, int64_t rows, int cols, const uint16_t* x,
                              const void* residual, const void* weight, float eps, float g, void* residual_out,
                              uint16_t* y, uint8_t* codes, uint8_t* scales, hipStream_t stream) {
  auto f = residual == nullptr ? launch_norm_res<0> : res_f32 ? launch_norm_res<2> : launch_norm_res<1>;
  return f(act, w_f32, rows, cols, x, residual, weight, eps, g, residual_out, y, codes, scales, stream);
}

}  // namespace moe
