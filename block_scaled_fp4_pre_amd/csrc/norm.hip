// Residual addition, root-mean-square norm and quantization of rows
// (moe_w4a4_add_rmsnorm):
//   h = rnd(x + r);  n = h * w / sqrt(mean(h^2) + eps);  y = bf16(n);
//   codes, scales = Q(y), the activation formats of the layer.
//
// Bound by HBM: every input is read once and every output written once; the row
// stays in registers between the sum and the norm, so nothing is read twice.
// A team of 64 to 1024 threads owns a row; a thread holds CPL pieces of
// 8 consecutive values (16-byte loads), so four neighbouring lanes share an
// MX group of 32 (two an NVFP4 block of 16) and exchange its absolute maximum
// by two (one) DPP steps inside their quad.
//
// The squares' sum, the reciprocal root and both products run in fp64 (full
// rate on this chip, hidden behind the loads): the result is then rounded
// the same way whatever the order of the sum, so the codes are reproducible
// next to the quantizer's borders.  16384 x 4096 with residual and E4M3 codes (472
// MB) take 92 us, 5.1 TB/s, the rate of a large copy; 1 x 4096 3.1 us, a launch.
#include "launch_ops.h"
#include "norm_rows.h"

namespace moe {
namespace {

// 8 values of h: as bfloat16 where they are (RES: 0 no residual, 1 bfloat16), in
// float32 with a float32 residual (2).
template <int RES>
struct Held {
  uint4 b;
  __device__ __forceinline__ void load(const uint16_t* x, const void* residual, size_t base, int c) {
    b = reinterpret_cast<const uint4*>(x)[c];
    if constexpr (RES == 1) {
      float f[8], r[8];
      unpack8(b, f);
      unpack8(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(residual) + base)[c], r);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] += r[i];
      b = pack8(f);
    }
  }
  __device__ __forceinline__ void clear() { b = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void store(void* out, size_t base, int c) const {
    reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + base)[c] = b;
  }
  __device__ __forceinline__ void get(float (&f)[8]) const { unpack8(b, f); }
  // The compiler would otherwise keep the fp64 values of the sum until the norm.
  __device__ __forceinline__ void forget() {
#ifdef __HIP_DEVICE_COMPILE__
    asm volatile("" : "+v"(b.x), "+v"(b.y), "+v"(b.z), "+v"(b.w));
#endif
  }
};
template <>
struct Held<2> {
  float h[8];
  __device__ __forceinline__ void load(const uint16_t* x, const void* residual, size_t base, int c) {
    float r[8];
    unpack8(reinterpret_cast<const uint4*>(x)[c], h);
    load_f32x8(static_cast<const float*>(residual) + base + 8 * c, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] += r[i];
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = 0.0f;
  }
  __device__ __forceinline__ void store(void* out, size_t base, int c) const {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(out) + base + 8 * c);
    p[0] = make_float4(h[0], h[1], h[2], h[3]);
    p[1] = make_float4(h[4], h[5], h[6], h[7]);
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = h[i];
  }
  __device__ __forceinline__ void forget() {
#ifdef __HIP_DEVICE_COMPILE__
#pragma unroll
    for (int i = 0; i < 8; ++i) asm volatile("" : "+v"(h[i]));
#endif
  }
};

// RES as above.  ACT: codes of 0 MXFP4, 1 MXFP8 E4M3, 2 NVFP4, or -1 none.  TPR:
// threads per row.
template <int RES, int act, int TPR, int CPL>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) add_rmsnorm_kernel(
    bool w_f32, int64_t rows, int cols, const uint16_t* x, const void* residual,
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
    Held<RES> h[CPL];
#pragma unroll
    for (int j = 0; j < CPL; ++j) {
      const int c = t + j * TPR;
      if (c < pieces)
        h[j].load(x + base, residual, base, c);
      else
        h[j].clear();
    }
    double ss = 0.0;
#pragma unroll
    for (int j = 0; j < CPL; ++j) {
      const int c = t + j * TPR;
      if (RES != 0 && c < pieces) h[j].store(residual_out, base, c);
      float v[8];
      h[j].get(v);
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fma((double)v[i], (double)v[i], ss);
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
    if constexpr (CPL >= 4) {
#pragma unroll
      for (int j = 0; j < CPL; ++j) h[j].forget();
    }
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
      float v[8], n[8];
      h[j].get(v);
#pragma unroll
      for (int i = 0; i < 8; ++i) n[i] = (float)((double)v[i] * rstd * (double)w[i]);
      const uint4 yb = pack8(n);
      if (y != nullptr && c < pieces) reinterpret_cast<uint4*>(y + base)[c] = yb;
      if constexpr (act >= 0) quantize_piece<act>(yb, (size_t)row * pieces, c, pieces, g, codes, scales);
    }
  }
}

constexpr int64_t kNormMaxBlocks = 1 << 20;   // more rows: a block takes several

#define MOE_NORM_PARAMS                                                                                                \
  bool w_f32, int64_t rows, int cols, const uint16_t *x, const void *residual, const void *weight, float eps, float g, \
      void *residual_out, uint16_t *y, uint8_t *codes, uint8_t *scales, hipStream_t stream
#define MOE_NORM_ARGS w_f32, rows, cols, x, residual, weight, eps, g, residual_out, y, codes, scales, stream

template <int RES, int ACT, int TPR, int CPL>
hipError_t launch_norm(MOE_NORM_PARAMS) {
  constexpr int THREADS = TPR < 256 ? 256 : TPR;
  constexpr int RPB = THREADS / TPR;
  const int64_t blocks = (rows + RPB - 1) / RPB;
  hipLaunchKernelGGL((add_rmsnorm_kernel<RES, ACT, TPR, CPL>),
                     dim3((unsigned)(blocks < kNormMaxBlocks ? blocks : kNormMaxBlocks)), dim3(THREADS), 0, stream, w_f32,
                     rows, cols, x, residual, weight, (double)eps, g, residual_out, y, codes, scales);
  return hipGetLastError();
}

// The smallest team that holds the row in at most 4 pieces a thread: a wave up to
// 1024 values (no barrier), 4 waves up to 8192.  Measured with a bfloat16 residual,
// y and E4M3 codes, us (wave / 4 waves / 16 waves): 65536 x 512 64 / 125 / 603,
// 32768 x 1024 59 / 76 / 319, 16384 x 2048 66 / 59 / 178, 16384 x 4096 133 / 111 / 209, 8192 x
// 8192 - / 121 / 129; one row of 2048 3.9 / 2.3 / 3.1, of 4096 6.4 / 2.9 / 3.3, of 8192 - /
// 4.3 / 3.5.  Past 8192 values 8 waves of 4 pieces where there are more rows than CUs:
// more rows are in flight (no residual / bfloat16 / float32 one, y and E4M3 codes, 8
// against 16 waves: 6798 x 9504 100 / 120 / 172 against 110 / 131 / 170, 512 x 16384 11.8 / 12.5
// / 20.1 against 12.6 / 14.3 / 22.0; 64 x 16384 5.6 / 6.2 / 6.9 against 5.1 / 5.8 / 6.9).
template <int RES, int ACT>
hipError_t launch_norm_act(MOE_NORM_PARAMS) {
  if (cols <= 512) return launch_norm<RES, ACT, 64, 1>(MOE_NORM_ARGS);
  if (cols <= 1024) return launch_norm<RES, ACT, 64, 2>(MOE_NORM_ARGS);
  if (cols <= 2048) return launch_norm<RES, ACT, 256, 1>(MOE_NORM_ARGS);
  if (cols <= 4096) return launch_norm<RES, ACT, 256, 2>(MOE_NORM_ARGS);
  if (cols <= 8192) return launch_norm<RES, ACT, 256, 4>(MOE_NORM_ARGS);
  if (cols <= 16384 && rows > 256) return launch_norm<RES, ACT, 512, 4>(MOE_NORM_ARGS);
  if (cols <= 16384) return launch_norm<RES, ACT, 1024, 2>(MOE_NORM_ARGS);
  if (cols <= 32768) return launch_norm<RES, ACT, 1024, 4>(MOE_NORM_ARGS);
  return launch_norm<RES, ACT, 1024, 8>(MOE_NORM_ARGS);
}

template <int RES>
hipError_t launch_norm_res(int act, MOE_NORM_PARAMS) {
  auto f = act == 0 ? launch_norm_act<RES, 0> : act == 1 ? launch_norm_act<RES, 1> : act == 2 ? launch_norm_act<RES, 2>
                                                                                             : launch_norm_act<RES, -1>;
  return f(MOE_NORM_ARGS);
}

}  // namespace

hipError_t launch_add_rmsnorm(int act, bool res_f32, MOE_NORM_PARAMS) {
  auto f = residual == nullptr ? launch_norm_res<0> : res_f32 ? launch_norm_res<2> : launch_norm_res<1>;
  return f(act, MOE_NORM_ARGS);
}
#undef MOE_NORM_ARGS
#undef MOE_NORM_PARAMS

}  // namespace moe
