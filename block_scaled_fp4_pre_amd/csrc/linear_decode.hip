// The dense linear for few tokens in one launch: every workgroup quantizes the
// tokens itself, so no second kernel has to wait for a first (at these sizes a
// launch costs as much as the product).
//
// Bound by reading the weights once from HBM.  A workgroup of 8 waves quantizes
// the tokens into LDS in MFMA operand order, one 32-element group a thread at a
// time, while its first weights are on their way.  Then it takes one 16-row
// block of the weights after the other: its waves split the K steps (wave w
// takes w, w + 8, ...), each keeping its steps' token operands in registers, and
// their sums meet in LDS, added in wave order.  The next block's weights are
// loaded before this block's sums are exchanged.
//
// 1 x 4096 x 4096 MXFP4: 4.1 us, 2.2 TB/s with the launch in it (a token kernel and
// the split kernel: 7.1); 1 x 4096 x 32000: 12.6 us, 5.5 TB/s; 16 x 2048 x 4096 E4M3
// with addend 5.8.  Quantizing in the lanes that feed the MFMA, each wave its own
// steps, took 5.8 us for one token: straight code for every step, fetched once
// and run once, with one token's four lanes of a wave at work.
#include "linear_common.h"
#include "quant_e4m3.h"

namespace moe {
namespace {

constexpr int kDecodeWaves = 8;
constexpr int kDecodeThreads = 64 * kDecodeWaves;

// Group i = token * (4 * steps) + g of the tokens -> LDS: codes at (step, lane
// (g % 4, token)) -- E4M3: the 16-element chunks 2g and 2g + 1, of which the MFMA
// takes c and c + 4 in lane group c (device_common.h) -- and the scale byte.
// Groups past K are zeros.
template <bool F8>
struct DecodeGroup {
  uint32_t w[16];     // bf16 values, or the codes
  uint32_t sc;
};
template <bool F8>
__device__ __forceinline__ void decode_load(const LinearInput& in, int token, int g, DecodeGroup<F8>& d) {
  const int groups = in.K / 32;
  d.sc = 0;
#pragma unroll
  for (int j = 0; j < 16; ++j) d.w[j] = 0;
  if (token >= in.T || g >= groups) return;
  const size_t i = (size_t)token * groups + g;
  if (in.x != nullptr) {
    load_bf16_words(in.x, (int64_t)i, d.w);
  } else {
    d.sc = in.xsf[i];
#pragma unroll
    for (int h = 0; h < (F8 ? 2 : 1); ++h) {
      const uint4 c = reinterpret_cast<const uint4*>(in.xq)[F8 ? 2 * i + h : i];
      d.w[4 * h] = c.x;
      d.w[4 * h + 1] = c.y;
      d.w[4 * h + 2] = c.z;
      d.w[4 * h + 3] = c.w;
    }
  }
}
template <bool F8>
__device__ __forceinline__ void decode_store(const LinearInput& in, int token, int g, const DecodeGroup<F8>& d,
                                             uint8_t* codes, uint8_t* scales) {
  uint4 lo, hi;
  uint32_t sc;
  if (in.x != nullptr) {
    if constexpr (F8)
      sc = mx8_cvt_bf16_group(d.w, lo, hi);
    else
      sc = mx_encode_bf16_group(d.w, lo);
  } else {
    lo = make_uint4(d.w[0], d.w[1], d.w[2], d.w[3]);
    hi = make_uint4(d.w[4], d.w[5], d.w[6], d.w[7]);
    sc = d.sc;
  }
  const int s = g >> 2, kb = g & 3;
  if constexpr (F8) {
    uint4* c = reinterpret_cast<uint4*>(codes) + s * 2 * kWave + (kb >> 1) * kWave + (2 * kb & 3) * 16 + token;
    c[0] = lo;
    c[16] = hi;
  } else {
    reinterpret_cast<uint4*>(codes)[s * kWave + kb * 16 + token] = lo;
  }
  scales[s * kWave + kb * 16 + token] = (uint8_t)sc;
}

// SPW: K steps per wave, at most.
template <bool F8, int SPW>
__global__ void __launch_bounds__(kDecodeThreads) linear_decode_kernel(LinearArgs p, LinearInput in, int blocks) {
  __shared__ v4f red[2][kDecodeWaves][kWave];
  extern __shared__ __align__(16) uint8_t lds[];        // codes of every step, then scale bytes
  constexpr int TB = F8 ? 2048 : 1024;
  const int lane = threadIdx.x & (kWave - 1), kb = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int S = p.steps;
  uint8_t* scales = lds + S * TB;
  // Workgroups are dealt round-robin to the 8 XCDs: the 4 blocks of a unit,
  // which share their scale dwords, go to one of them.
  const int first = (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3);

  v4u a[SPW];
  uint32_t sa[SPW];
  auto load = [&](int blk) {
    const int u = blk >> 2;
    const uint8_t* wc = p.wc + unit_base<kStepCodeBytes>(u, S) + (blk & 3) * 1024 + lane * 16;
    const uint8_t* ws = p.ws + unit_base<kStepScaleBytes>(u, S) + lane * 4;
#pragma unroll
    for (int i = 0; i < SPW; ++i) {
      const int s = wave + i * kDecodeWaves;
      if (s < S) {
        a[i] = *reinterpret_cast<const v4u*>(wc + (size_t)s * (4 * kStepCodeBytes));
        sa[i] = *reinterpret_cast<const uint32_t*>(ws + (size_t)s * (4 * kStepScaleBytes));
      }
    }
  };
  if (first >= blocks) return;
  load(first);
  // Tokens next to one another in a wave's lanes: groups of one token run along
  // the lanes (coalesced), the LDS writes of 4 lanes go to 4 lane groups.
  const int per = 4 * S, total = in.T * per;
  for (int i = threadIdx.x; i < total; i += 2 * kDecodeThreads) {
    const int i1 = i + kDecodeThreads;
    const int t0 = i / per, t1 = i1 / per;
    DecodeGroup<F8> d0, d1;
    decode_load<F8>(in, t0, i - t0 * per, d0);
    if (i1 < total) decode_load<F8>(in, t1, i1 - t1 * per, d1);
    decode_store<F8>(in, t0, i - t0 * per, d0, lds, scales);
    if (i1 < total) decode_store<F8>(in, t1, i1 - t1 * per, d1, lds, scales);
  }
  __syncthreads();
  // (columns of tokens past the last hold what LDS held: they give outputs
  // that are not stored)
  v4u b[SPW], b2[F8 ? SPW : 1];
  int sb[SPW];
#pragma unroll
  for (int i = 0; i < SPW; ++i) {
    const int s = wave + i * kDecodeWaves;
    if (s < S) {
      b[i] = *reinterpret_cast<const v4u*>(lds + s * TB + lane * 16);
      if constexpr (F8) b2[i] = *reinterpret_cast<const v4u*>(lds + s * TB + 1024 + lane * 16);
      sb[i] = scales[s * kWave + lane];
    }
  }
  int flip = 0;
  for (int blk = first; blk < blocks; blk += gridDim.x) {
    v4f acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < SPW; ++i)
      if (wave + i * kDecodeWaves < S) {
        const int w = (int)(sa[i] >> (8 * (blk & 3)));
        if constexpr (F8)
          acc = mfma_op8<0, 0>(a[i], b[i], b2[i], acc, w, sb[i]);
        else
          acc = mfma_op<0, 0>(a[i], b[i], acc, w, sb[i]);
      }
    if (blk + (int)gridDim.x < blocks) load(blk + gridDim.x);
    red[flip][wave][lane] = acc;
    __syncthreads();
    // One wave adds the partial sums, another each time, so that the others go
    // on; the buffers alternate, so it may be a block behind.
    if (wave == flip) {
      v4f v = red[flip][0][lane];
#pragma unroll
      for (int w = 1; w < kDecodeWaves; ++w) v += red[flip][w][lane];
      const int t = lane & 15, n = blk * 16 + 4 * kb;
      if (t < p.T && n < p.N) store4(p, t, n, v);
    }
    flip ^= 1;
  }
}

template <bool F8, int SPW>
hipError_t launch_decode(const LinearArgs& a, const LinearInput& in, hipStream_t stream) {
  const int blocks = (a.N + 15) / 16;
  const size_t lds = (size_t)a.steps * ((F8 ? 2048 : 1024) + kWave), all = lds + sizeof(v4f) * 2 * kDecodeThreads;
  // No more workgroups than the CUs hold at a time, at most two each: each
  // quantizes the tokens for all its blocks, and one that has to wait for another's
  // LDS would do so after it.
  const int most = 2 * all <= 160 * 1024 ? 512 : 256;
  const int grid = (blocks < most ? blocks + 7 : most) / 8 * 8;
  auto kern = linear_decode_kernel<F8, SPW>;
  if (all > 65536) {
    const hipError_t err = raise_lds_limit(reinterpret_cast<const void*>(kern), kDecodeMaxSteps * (2048 + kWave));
    if (err != hipSuccess) return err;
  }
  hipLaunchKernelGGL(kern, dim3(grid), dim3(kDecodeThreads), lds, stream, a, in, blocks);
  return hipGetLastError();
}

template <bool F8>
hipError_t launch_decode_steps(const LinearArgs& a, const LinearInput& in, hipStream_t stream) {
  static_assert(kDecodeMaxTokens == 16 && kDecodeMaxSteps == 8 * kDecodeWaves, "one token block; the variants below");
  const int spw = (a.steps + kDecodeWaves - 1) / kDecodeWaves;
  if (spw <= 1) return launch_decode<F8, 1>(a, in, stream);
  if (spw <= 2) return launch_decode<F8, 2>(a, in, stream);
  if (spw <= 4) return launch_decode<F8, 4>(a, in, stream);
  return launch_decode<F8, 8>(a, in, stream);
}

}  // namespace

hipError_t launch_linear_decode(bool fp8, const LinearArgs& a, const LinearInput& in, hipStream_t stream) {
  return fp8 ? launch_decode_steps<true>(a, in, stream) : launch_decode_steps<false>(a, in, stream);
}

}  // namespace moe
