// Operands of the dense linear in tile order (tiles.h with groups of 4 units =
// 256 rows): weights once at load time, tokens on every call.  One workgroup
// per (64-row unit, K step of 128), wave rb its 16-row block rb: lane l holds
// row l % 16 and the 32-element group l / 16 of the step -- one MX group and
// one MFMA operand slot -- so a token's group is quantized by the lane whose
// 16 bytes it becomes, and every store is a contiguous 1 KiB run per wave.
// Rows past the end and groups past K are written as zeros.
//
// E4M3 tokens take 2 KiB per 16 rows and step, two 1 KiB pieces: the FP8 MFMA
// operand of lane group g is the 16-element chunks g and g + 4 of the step
// (device_common.h), so the two chunks 2g, 2g + 1 of group g go to piece
// g / 2, lane groups 2g % 4 and 2g % 4 + 1.
//
// Both are bound by HBM: one read of the source, one write of the tiles.
#include "launch_ops.h"
#include "quant_e4m3.h"
#include "tiles.h"

namespace moe {
namespace {

// Scale bytes of the four blocks of a unit -> one dword per lane.
__device__ __forceinline__ void store_scales(uint32_t byte, int rb, int lane, uint8_t* dst) {
  __shared__ uint32_t sc[kWave];
  reinterpret_cast<uint8_t*>(sc)[lane * 4 + rb] = (uint8_t)byte;
  __syncthreads();
  if (rb == 0) reinterpret_cast<uint32_t*>(dst)[lane] = sc[lane];
}

__global__ void __launch_bounds__(256) linear_prepare_kernel(const uint8_t* __restrict__ codes,
                                                             const uint8_t* __restrict__ scales, int N, int K, int units,
                                                             int steps, uint8_t* __restrict__ p_codes,
                                                             uint8_t* __restrict__ p_scales) {
  const int u = blockIdx.x / steps, s = blockIdx.x - u * steps;
  const int lane = threadIdx.x & (kWave - 1), rb = threadIdx.x / kWave;
  const int row = u * kUnitRows + rb * 16 + (lane & 15), g = s * 4 + (lane >> 4);
  uint4 c = make_uint4(0, 0, 0, 0);
  uint32_t sc = 0;
  if (row < N && g < K / 32) {
    const size_t i = (size_t)row * (K / 32) + g;
    c = reinterpret_cast<const uint4*>(codes)[i];
    sc = scales[i];
  }
  const size_t chunk = unit_chunk(0, u, s, units, steps);
  reinterpret_cast<uint4*>(p_codes + chunk * kStepCodeBytes)[rb * kWave + lane] = c;
  store_scales(sc, rb, lane, p_scales + chunk * kStepScaleBytes);
}

// SRC_BF16: the tokens are quantized here; else xq and xsf are copied.
template <bool F8, bool SRC_BF16>
__global__ void __launch_bounds__(256) linear_tokens_kernel(const uint16_t* __restrict__ x, const uint8_t* __restrict__ xq,
                                                            const uint8_t* __restrict__ xsf, int T, int K, int units,
                                                            int steps, uint8_t* __restrict__ t_codes,
                                                            uint8_t* __restrict__ t_scales) {
  const int u = blockIdx.x / steps, s = blockIdx.x - u * steps;
  const int lane = threadIdx.x & (kWave - 1), rb = threadIdx.x / kWave;
  const int row = u * kUnitRows + rb * 16 + (lane & 15), kb = lane >> 4, g = s * 4 + kb;
  uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
  uint32_t sc = 0;
  if (row < T && g < K / 32) {
    const size_t i = (size_t)row * (K / 32) + g;
    if constexpr (SRC_BF16) {
      uint32_t w[16];
      load_bf16_words(x, (int64_t)i, w);
      sc = F8 ? mx8_cvt_bf16_group(w, lo, hi) : mx_encode_bf16_group(w, lo);
    } else {
      lo = reinterpret_cast<const uint4*>(xq)[F8 ? 2 * i : i];
      if constexpr (F8) hi = reinterpret_cast<const uint4*>(xq)[2 * i + 1];
      sc = xsf[i];
    }
  }
  const size_t chunk = unit_chunk(0, u, s, units, steps);
  if constexpr (F8) {
    uint4* dst = reinterpret_cast<uint4*>(t_codes + chunk * (2 * kStepCodeBytes)) + rb * 2 * kWave + (kb >> 1) * kWave +
                 (2 * kb % 4) * 16 + (lane & 15);
    dst[0] = lo;
    dst[16] = hi;
  } else {
    reinterpret_cast<uint4*>(t_codes + chunk * kStepCodeBytes)[rb * kWave + lane] = lo;
  }
  store_scales(sc, rb, lane, t_scales + chunk * kStepScaleBytes);
}

}  // namespace

hipError_t launch_linear_prepare(const uint8_t* codes, const uint8_t* scales, int N, int K, int units, int steps,
                                 uint8_t* p_codes, uint8_t* p_scales, hipStream_t stream) {
  hipLaunchKernelGGL(linear_prepare_kernel, dim3((unsigned)(units * steps)), dim3(256), 0, stream, codes, scales, N, K,
                     units, steps, p_codes, p_scales);
  return hipGetLastError();
}

hipError_t launch_linear_tokens(bool fp8, const uint16_t* x, const uint8_t* xq, const uint8_t* xsf, int T, int K,
                                int units, int steps, uint8_t* t_codes, uint8_t* t_scales, hipStream_t stream) {
  auto kern = fp8 ? (x != nullptr ? linear_tokens_kernel<true, true> : linear_tokens_kernel<true, false>)
                  : (x != nullptr ? linear_tokens_kernel<false, true> : linear_tokens_kernel<false, false>);
  hipLaunchKernelGGL(kern, dim3((unsigned)(units * steps)), dim3(256), 0, stream, x, xq, xsf, T, K, units, steps,
                     t_codes, t_scales);
  return hipGetLastError();
}

}  // namespace moe
