// The dense linear's product (moe_w4a4_linear): weight rows are the 16-row
// MFMA A operand, tokens the 16-column B operand, both in tile order, so every
// operand load is one contiguous 1 KiB run per wave straight into registers.
//
// linear_split_kernel: a workgroup of 8 waves owns NR*16 weight rows x NT*16
// tokens; its waves split the K steps (wave w takes w, w + 8, ...), each with
// the whole tile in its accumulators, and their sums meet in LDS, added in wave
// order.  The next step's operands are loaded before this step's product.
// Bound by latency for few tokens (128 x 4096 x 4096 MXFP4 5.6 us, the weights' bytes
// take 1.3) and by the L2s beyond: every tile reads both its operands whole.
#include "linear_common.h"

namespace moe {
namespace {

constexpr int kSplitWaves = 8;

template <bool F8, int NT, int NR>
struct SplitStep {
  v4u a[NR], b[NT], b2[F8 ? NT : 1];
  uint32_t sa, sb;
};

template <int NR, int NT, bool F8, int R, int C>
__device__ __forceinline__ void split_mfma(const SplitStep<F8, NT, NR>& s, v4f (&acc)[NT][NR]) {
  if constexpr (F8)
    acc[C][R] = mfma_op8<R, C>(s.a[R], s.b[C], s.b2[C], acc[C][R], (int)s.sa, (int)s.sb);
  else
    acc[C][R] = mfma_op<R, C>(s.a[R], s.b[C], acc[C][R], (int)s.sa, (int)s.sb);
  if constexpr (R + 1 < NR)
    split_mfma<NR, NT, F8, R + 1, C>(s, acc);
  else if constexpr (C + 1 < NT)
    split_mfma<NR, NT, F8, 0, C + 1>(s, acc);
}

template <bool F8, int NT, int NR>
__global__ void __launch_bounds__(64 * kSplitWaves) linear_split_kernel(LinearArgs p, int row_tiles, int tok_tiles) {
  constexpr int TB = F8 ? 2 * kStepCodeBytes : kStepCodeBytes;   // token code bytes per unit and step
  extern __shared__ __align__(16) uint8_t lds[];
  // Workgroups are dealt round-robin to the 8 XCDs: each XCD gets a run of
  // row tiles with all their token tiles, so its L2 fetches a weight once.
  const int L = (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3);
  if (L >= row_tiles * tok_tiles) return;
  const int rt = L / tok_tiles, tt = L - rt * tok_tiles;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int S = p.steps;
  // First 16-row block of the tile: its unit, and its place among the unit's 4.
  const int wu = rt * NR / 4, wb = rt * NR % 4, tu = tt * NT / 4, tb = tt * NT % 4;
  const uint8_t* wc = p.wc + unit_base<kStepCodeBytes>(wu, S) + wb * 1024 + lane * 16;
  const uint8_t* ws = p.ws + unit_base<kStepScaleBytes>(wu, S) + lane * 4;
  const uint8_t* tc = p.tc + unit_base<TB>(tu, S) + tb * (TB / 4) + lane * 16;
  const uint8_t* ts = p.ts + unit_base<kStepScaleBytes>(tu, S) + lane * 4;

  v4f acc[NT][NR];
#pragma unroll
  for (int c = 0; c < NT; ++c)
#pragma unroll
    for (int r = 0; r < NR; ++r) acc[c][r] = v4f{0.f, 0.f, 0.f, 0.f};

  auto load = [&](int s, SplitStep<F8, NT, NR>& d) {
#pragma unroll
    for (int r = 0; r < NR; ++r)
      d.a[r] = *reinterpret_cast<const v4u*>(wc + (size_t)s * (4 * kStepCodeBytes) + r * 1024);
#pragma unroll
    for (int c = 0; c < NT; ++c) {
      d.b[c] = *reinterpret_cast<const v4u*>(tc + (size_t)s * (4 * TB) + c * (TB / 4));
      if constexpr (F8) d.b2[c] = *reinterpret_cast<const v4u*>(tc + (size_t)s * (4 * TB) + c * (TB / 4) + 1024);
    }
    d.sa = *reinterpret_cast<const uint32_t*>(ws + (size_t)s * (4 * kStepScaleBytes)) >> (8 * wb);
    d.sb = *reinterpret_cast<const uint32_t*>(ts + (size_t)s * (4 * kStepScaleBytes)) >> (8 * tb);
  };
  SplitStep<F8, NT, NR> cur, nxt;
  int s = wave;
  if (s < S) load(s, cur);
  for (; s < S; s += kSplitWaves) {
    if (s + kSplitWaves < S) load(s + kSplitWaves, nxt);
    split_mfma<NR, NT, F8, 0, 0>(cur, acc);
    cur = nxt;
  }

  v4f* red = reinterpret_cast<v4f*>(lds);
#pragma unroll
  for (int c = 0; c < NT; ++c)
#pragma unroll
    for (int r = 0; r < NR; ++r) red[((wave * NT + c) * NR + r) * kWave + lane] = acc[c][r];
  __syncthreads();
  for (int i = threadIdx.x; i < NT * 16 * NR * 4; i += 64 * kSplitWaves) {
    const int t = i / (NR * 4), q = i - t * (NR * 4);
    const int at = ((t / 16) * NR + q / 4) * kWave + (q % 4) * 16 + t % 16;
    v4f v = red[at];
#pragma unroll
    for (int w = 1; w < kSplitWaves; ++w) v += red[w * NT * NR * kWave + at];
    const int tok = tt * NT * 16 + t, n = rt * NR * 16 + 4 * q;
    if (tok < p.T && n < p.N) store4(p, tok, n, v);
  }
}

template <bool F8, int NT, int NR>
hipError_t launch_split(const LinearArgs& a, hipStream_t stream) {
  const int64_t rt = (a.N + NR * 16 - 1) / (NR * 16), tt = (a.T + NT * 16 - 1) / (NT * 16);
  constexpr size_t lds = (size_t)kSplitWaves * NT * NR * 1024;
  static_assert(lds <= 65536, "the default limit");
  hipLaunchKernelGGL((linear_split_kernel<F8, NT, NR>), dim3((unsigned)((rt * tt + 7) / 8 * 8)),
                     dim3(64 * kSplitWaves), lds, stream, a, (int)rt, (int)tt);
  return hipGetLastError();
}

// 16 rows a tile while those of 32 are fewer than the CUs, else 32 (us, K = 4096,
// MXFP4, 16 / 32 / 64 rows: 64 x 4096 5.1 / 5.5 / 7.8, 128 x 4096 6.8 / 5.6 / 7.9, 256 x 4096 10.5
// / 8.4 / 8.5, 64 x 16384 11.0 / 9.0 / 10.2; 32 x 4096 4.4 / 4.6, 32 x 16384 8.5 / 8.3; 16 tokens
// with K = 16384: 1024 rows 8.3 / 8.8, 16384 rows 33.8 / 27.1).
template <bool F8, int NT>
hipError_t launch_split_rows(const LinearArgs& a, hipStream_t stream) {
  const int64_t tiles32 = (int64_t)((a.N + 31) / 32) * ((a.T + NT * 16 - 1) / (NT * 16));
  return tiles32 >= 256 ? launch_split<F8, NT, 2>(a, stream) : launch_split<F8, NT, 1>(a, stream);
}

template <bool F8>
hipError_t launch_linear_type(const LinearArgs& a, hipStream_t stream) {
  if (a.T <= 16) return launch_split_rows<F8, 1>(a, stream);
  if (a.T <= 32) return launch_split_rows<F8, 2>(a, stream);
  return launch_split_rows<F8, 4>(a, stream);
}

}  // namespace

hipError_t launch_linear_split(bool fp8, const LinearArgs& a, hipStream_t stream) {
  return fp8 ? launch_linear_type<true>(a, stream) : launch_linear_type<false>(a, stream);
}

}  // namespace moe
