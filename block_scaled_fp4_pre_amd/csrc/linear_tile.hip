// The dense linear's product for many tokens: both operands go through LDS.
//
// A workgroup of 4 waves (2 x 2) owns 2*WA*16 weight rows x 2*WB*16 tokens, each
// wave a quarter of it: WA x WB MFMA tiles in its accumulators.  Operands are in
// tile order, so a K step of the tile is a contiguous run of 1 KiB pieces, copied
// to LDS as they are by direct-to-LDS loads into a ring of P stages; an operand
// read is lane l's 16 bytes at 16*l, free of bank conflicts.
//
// One barrier a step: a wave passes it when its own DMAs of stage s have landed
// (in-order vmcnt) and its reads of stage s - 1 are done, so after it stage s may
// be read and the buffer of stage s - 1 refilled.  The DMAs are inline assembly:
// the compiler cannot tell the ring's stages apart and would wait for all of them
// before every LDS read.  Reads and DMAs are issued between the step's MFMAs, and
// two workgroups share a CU, so that one's MFMAs cover the other's waits.
//
// KS = 2, for products with too few tiles for that: two groups of 4 waves share a
// tile, each with a ring of its own and every other K step, and exchange half of
// their sums at the end (group 0 finishes the first half of the tokens).
//
// 4096 x 4096 x 4096 MXFP4 take 34.9 us (3.9 PFLOP/s), of which about 10 are the
// first loads and the stores with the matrix cores idle; 16384 x 2048 x 4096 E4M3 120
// us (2.3), with an addend 137: 134 MB each of outputs and addends at copy speed.
// The steps are bound by power: with 256 x 256 outputs a workgroup a step took as
// many cycles on 16 CUs as on 256, but the clock fell from 2.26 to 1.75 GHz (MFMAs
// alone: 2.37 to 1.99).  Such tiles, in 8 waves or in 4 with the accumulators pinned to
// accumulation registers, measured 36.5 and 40 us for MXFP4 4096 x 4096 x 4096 and 134 and
// 143 for E4M3 16384 x 2048 x 4096; reading the next step's operands into registers
// during a step changed nothing at two workgroups a CU.
#include "linear_common.h"

namespace moe {
namespace {

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// The 16 (4) bytes at base + voff of lane l go to LDS byte address lds + 16*l
// (4*l); base and lds are the wave's own (scalar).  M0 carries the LDS address; a
// DMA right after a scalar write of M0 needs one wait state, which the compiler
// cannot insert inside an asm statement.
__device__ __forceinline__ void dma16(const uint8_t* base, int voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(voff), "s"(base), "s"(lds) : "memory", "m0");
}
__device__ __forceinline__ void dma4(const uint8_t* base, int voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1" ::"v"(voff), "s"(base), "s"(lds) : "memory", "m0");
}
#pragma clang diagnostic pop

constexpr int kTileWaves = 4;   // of a group
constexpr int kTileBand = 8;    // row tiles

template <bool F8, int WA, int WB>
struct TileShape {
  static constexpr int WAVES = kTileWaves;
  static constexpr int TB = F8 ? 2048 : 1024;                // token code bytes of a 16-token block and step
  static constexpr int AB = 2 * WA, BB = 2 * WB;             // 16-row blocks of the tile's two sides
  static constexpr int A_CODES = 0, B_CODES = AB * 1024;
  static constexpr int A_SCALES = B_CODES + BB * TB, B_SCALES = A_SCALES + AB / 4 * kStepScaleBytes;
  static constexpr int BYTES = B_SCALES + BB / 4 * kStepScaleBytes;
  static constexpr int AD = AB / WAVES, BD = BB * (TB / 1024) / WAVES;   // code DMAs per wave and stage
  static constexpr int SD = (AB / 4 + BB / 4 + WAVES - 1) / WAVES;       // scale DMAs
  static constexpr int DMAS = AD + BD + SD;
  static constexpr int ROWS = AB * 16, TOKENS = BB * 16;
  static_assert(AD * WAVES == AB && BD * WAVES == BB * (TB / 1024) && AB % 4 == 0 && BB % 4 == 0, "DMA shares");
  static_assert(WA % 4 == 0 && (WB % 4 == 0 || WB == 2), "scale dwords");
};

template <int N>
struct Int {
  static constexpr int value = N;
};
template <int N, int I = 0, class F>
__device__ __forceinline__ void unrolled(F&& f) {
  if constexpr (I < N) {
    f(Int<I>{});
    unrolled<N, I + 1>(f);
  }
}

// The wave's outputs acc[token block][row block] to rows t0.. and columns n0..
// of `out`, G token blocks at a time through `mine` (G*16 x STRIDE bytes of
// LDS), so that every store covers a whole run of a row: V values a lane, 16
// bytes of `out`.  The loads of a pass's addends are all issued before its first
// use (one at a time they cost half the kernel's time at 16384 x 4096 outputs).
// Stores and addend loads are non-temporal: `out` is far larger than an L2, and
// the operands stay there (16384 x 2048 x 4096 MXFP4 104 -> 80 us).  The store loop
// stays rolled: unrolled over the tokens its code took longer to fetch than to
// run.
template <int WA, int WB, int G, bool F32>
__device__ __forceinline__ void tile_store(const LinearArgs& p, const uint8_t* mine, int n0, int t0, int live_tokens,
                                           int lane) {
  constexpr int STRIDE = WA * 16 * 4 + 16;
  constexpr int V = F32 ? 4 : 8, LPT = WA * 16 / V, TPP = kWave / LPT;   // lanes a token, tokens a pass
  constexpr int IT = G * 16 / TPP < 4 ? G * 16 / TPP : 4;                // passes in flight
  static_assert(G * 16 % (IT * TPP) == 0, "whole passes");
  const int n = n0 + lane % LPT * V, tl = lane / LPT;
  const int left = max(0, min(V, p.N - n));
  const bool whole = left == V;
  const int live = left > 0 ? live_tokens : 0;
#pragma unroll 1
  for (int i0 = tl; i0 < G * 16; i0 += IT * TPP) {
    const size_t at = (size_t)(t0 + i0) * p.N + n;
    v4u add[IT];
    if (p.addend != nullptr) {
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        add[i] = v4u{0, 0, 0, 0};
        if (i0 + i * TPP < live) {
          const uint16_t* a = p.addend + at + (size_t)(i * TPP) * p.N;
          if (!whole) {
#pragma unroll
            for (int j = 0; j < V; ++j)
              if (j < left) add[i][j / 2] |= (uint32_t)a[j] << (j % 2 * 16);
          } else if constexpr (F32) {
            const v2u q = __builtin_nontemporal_load(reinterpret_cast<const v2u_at2*>(a));
            add[i][0] = q[0];
            add[i][1] = q[1];
          } else {
            add[i] = __builtin_nontemporal_load(reinterpret_cast<const v4u_at2*>(a));
          }
        }
      }
    }
    v4f v[IT][V / 4];
#pragma unroll
    for (int i = 0; i < IT; ++i)
#pragma unroll
      for (int h = 0; h < V / 4; ++h)
        v[i][h] = *reinterpret_cast<const v4f*>(mine + (i0 + i * TPP) * STRIDE + lane % LPT * (V * 4) + h * 16);
    if (p.addend != nullptr) {
#pragma unroll
      for (int i = 0; i < IT; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) v[i][j / 4][j % 4] += bf16_to_f32(add[i][j / 2] >> (j % 2 * 16) & 0xFFFFu);
    }
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      if (i0 + i * TPP >= live) continue;
      if constexpr (F32) {
        float* o = static_cast<float*>(p.out) + at + (size_t)(i * TPP) * p.N;
        if (whole) {
          __builtin_nontemporal_store(v[i][0], reinterpret_cast<v4f_at4*>(o));
        } else {
#pragma unroll
          for (int j = 0; j < V; ++j)
            if (j < left) o[j] = v[i][0][j];
        }
      } else {
        uint16_t* o = static_cast<uint16_t*>(p.out) + at + (size_t)(i * TPP) * p.N;
        v4u h;
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] = pack_bf16(v[i][j / 2][j % 2 * 2], v[i][j / 2][j % 2 * 2 + 1]);
        if (whole) {
          __builtin_nontemporal_store(h, reinterpret_cast<v4u_at2*>(o));
        } else {
#pragma unroll
          for (int j = 0; j < V; ++j)
            if (j < left) o[j] = (uint16_t)(h[j / 2] >> (j % 2 * 16));
        }
      }
    }
  }
}

template <int WA, int WB, int G>
__device__ __forceinline__ void tile_epilogue(const LinearArgs& p, const v4f (&acc)[WB][WA], uint8_t* mine, int n0,
                                              int t0, int lane) {
  constexpr int STRIDE = WA * 16 * 4 + 16;
  unrolled<WB / G>([&](auto qi) {
    constexpr int q = decltype(qi)::value;
#pragma unroll
    for (int c = 0; c < G; ++c)
#pragma unroll
      for (int r = 0; r < WA; ++r)
        *reinterpret_cast<v4f*>(mine + (c * 16 + (lane & 15)) * STRIDE + (r * 16 + (lane >> 4) * 4) * 4) =
            acc[q * G + c][r];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const int t = t0 + q * G * 16;
    if (p.out_f32)
      tile_store<WA, WB, G, true>(p, mine, n0, t, p.T - t, lane);
    else
      tile_store<WA, WB, G, false>(p, mine, n0, t, p.T - t, lane);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  });
}

template <bool F8, int WA, int WB, int P, int KS>
__global__ void __launch_bounds__(64 * kTileWaves * KS, 2) linear_tile_kernel(LinearArgs p, int row_tiles, int tok_tiles) {
  using S = TileShape<F8, WA, WB>;
  constexpr int TB = S::TB;
  extern __shared__ __align__(16) uint8_t lds[];
  const int group = KS == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / (64 * kTileWaves));
  const uint8_t* ring = lds + group * (P * S::BYTES);
  const uint32_t lbase = (uint32_t)(uintptr_t)ring;
  // Workgroups are dealt round-robin to the 8 XCDs; each XCD gets a run of the
  // order below (a band of 8 row tiles, tokens next), so that the 64 tiles it
  // works on at a time are about 8 x 8 and share their operands in its L2.  (Bands
  // of 4 read the tokens of 16384 x 2048 x 4096 four times instead of twice: E4M3
  // 129 against 120 us; bands of 16 measured as 8.)
  const int L = (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3);
  if (L >= row_tiles * tok_tiles) return;
  const int band = L / (kTileBand * tok_tiles), width = min(kTileBand, row_tiles - band * kTileBand);
  const int in = L - band * kTileBand * tok_tiles, tt = in / width, rt = band * kTileBand + in - tt * width;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave % kTileWaves);   // in its group
  const int wr = wave & 1, wt = wave >> 1;              // the wave's half of the rows, of the tokens
  const int S_ = p.steps;

  const int au = rt * (S::AB / 4), bu = tt * (S::BB / 4);   // first units of the tile
  const uint8_t* ac = p.wc + unit_base<kStepCodeBytes>(au, S_) + wave * S::AD * 1024;
  const uint8_t* bc = p.tc + unit_base<4 * TB>(bu, S_) + wave * S::BD * 1024;
  // scale units of A, then of B, dealt to the waves in turn (a wave past the
  // end copies unit 0 of A again: every wave then has as many DMAs in flight)
  const uint8_t* sc[S::SD];
  int sdst[S::SD];
#pragma unroll
  for (int i = 0; i < S::SD; ++i) {
    const int u = wave + i * S::WAVES < S::AB / 4 + S::BB / 4 ? wave + i * S::WAVES : 0;
    sc[i] = u < S::AB / 4 ? p.ws + unit_base<kStepScaleBytes>(au, S_) + u * kStepScaleBytes
                          : p.ts + unit_base<kStepScaleBytes>(bu, S_) + (u - S::AB / 4) * kStepScaleBytes;
    sdst[i] = S::A_SCALES + u * kStepScaleBytes;
  }

  // DMA i of step s's operands into buffer `buf`.
  auto dma = [&](int s, int buf, int i) {
    const uint32_t b = lbase + (uint32_t)buf * S::BYTES;
    if (i < S::AD)
      dma16(ac + (size_t)s * (4 * kStepCodeBytes) + i * 1024, lane * 16, b + S::A_CODES + (wave * S::AD + i) * 1024);
    else if (i < S::AD + S::BD)
      dma16(bc + (size_t)s * (16 * TB) + (i - S::AD) * 1024, lane * 16,
            b + S::B_CODES + (wave * S::BD + i - S::AD) * 1024);
    else
      dma4(sc[i - S::AD - S::BD] + (size_t)s * (4 * kStepScaleBytes), lane * 4, b + sdst[i - S::AD - S::BD]);
  };
  // Past the last step the DMAs copy the last stage again (out of L2) into a
  // buffer that is not read any more, so that every step has as many in flight.
  // The group's step s is step s * KS + group of the product.
  auto source = [&](int s) { return min(s * KS + group, S_ - 1); };
#pragma unroll 1
  for (int s = 0; s < P - 1; ++s)
    for (int i = 0; i < S::DMAS; ++i) dma(source(s), s, i);

  v4f acc[WB][WA];
#pragma unroll
  for (int c = 0; c < WB; ++c)
#pragma unroll
    for (int r = 0; r < WA; ++r) acc[c][r] = v4f{0.f, 0.f, 0.f, 0.f};
  for (int s = 0, buf = 0; s * KS < S_; ++s) {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(S::DMAS * (P - 2)) : "memory");
    if (KS > 1 && s * KS + group >= S_) break;    // (an odd number of steps: group 1's last)
    const uint8_t* st = ring + buf * S::BYTES;
    const int src = source(s + P - 1), dst = buf == 0 ? P - 1 : buf - 1;
    v4u a[WA], b[WB], b2[F8 ? WB : 1];
    int sa[WA / 4], sb[(WB + 3) / 4];
#pragma unroll
    for (int u = 0; u < WA / 4; ++u)
      sa[u] = *reinterpret_cast<const int*>(st + S::A_SCALES + (wr * (WA / 4) + u) * kStepScaleBytes + lane * 4);
#pragma unroll
    for (int u = 0; u < (WB + 3) / 4; ++u)
      sb[u] = (int)(*reinterpret_cast<const uint32_t*>(st + S::B_SCALES + (wt * WB / 4 + u) * kStepScaleBytes + lane * 4) >>
                    (wt * WB % 4 * 8));      // (two blocks a wave: its half of the dword)
    auto read_b = [&](int c) {
      const uint8_t* q = st + S::B_CODES + (wt * WB + c) * TB + lane * 16;
      b[c] = *reinterpret_cast<const v4u*>(q);
      if constexpr (F8) b2[c] = *reinterpret_cast<const v4u*>(q + 1024);
    };
    read_b(0);
#pragma unroll
    for (int r = 0; r < WA; ++r)
      a[r] = *reinterpret_cast<const v4u*>(st + S::A_CODES + (wr * WA + r) * 1024 + lane * 16);
    unrolled<WA * WB>([&](auto mi) {
      constexpr int m = decltype(mi)::value, c = m / WA, r = m % WA;
      if constexpr (r == 0 && c + 1 < WB) read_b(c + 1);
      if constexpr (F8)
        acc[c][r] = mfma_op8<r % 4, c % 4>(a[r], b[c], b2[c], acc[c][r], sa[r / 4], sb[c / 4]);
      else
        acc[c][r] = mfma_op<r % 4, c % 4>(a[r], b[c], acc[c][r], sa[r / 4], sb[c / 4]);
      unrolled<S::DMAS>([&](auto di) {
        constexpr int i = decltype(di)::value;
        if constexpr (i * (WA * WB) / S::DMAS == m) dma(src, dst, i);
      });
      __builtin_amdgcn_sched_barrier(0);
    });
    buf = buf + 1 == P ? 0 : buf + 1;
  }
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");

  __syncthreads();                          // every wave is done with the rings
  constexpr int STRIDE = WA * 16 * 4 + 16;
  const int n0 = rt * S::ROWS + wr * WA * 16, t0 = tt * S::TOKENS + wt * WB * 16;
  if constexpr (KS == 1) {
    constexpr int G = S::WAVES * 64 * STRIDE <= P * S::BYTES ? 4 : 2;
    static_assert(S::WAVES * G * 16 * STRIDE <= P * S::BYTES, "epilogue staging");
    tile_epilogue<WA, WB, G>(p, acc, lds + wave * G * 16 * STRIDE, n0, t0, lane);
  } else {
    constexpr int HALF = WB / 2;
    static_assert(KS == 2 && 2 * S::WAVES * HALF * WA * 1024 <= KS * P * S::BYTES, "exchange");
    static_assert(2 * S::WAVES * (HALF * WA * 1024 + 16 * STRIDE) <= KS * P * S::BYTES, "epilogue staging");
    v4f* red = reinterpret_cast<v4f*>(lds) + wave * HALF * WA * kWave + lane;
    constexpr int OTHER = S::WAVES * HALF * WA * kWave;
#pragma unroll
    for (int c = 0; c < HALF; ++c)
#pragma unroll
      for (int r = 0; r < WA; ++r) {
        if (group == 0)
          red[(c * WA + r) * kWave] = acc[HALF + c][r];
        else
          red[OTHER + (c * WA + r) * kWave] = acc[c][r];
      }
    __syncthreads();
    v4f fin[HALF][WA];
#pragma unroll
    for (int c = 0; c < HALF; ++c)
#pragma unroll
      for (int r = 0; r < WA; ++r)
        fin[c][r] = group == 0 ? acc[c][r] + red[OTHER + (c * WA + r) * kWave]
                               : red[(c * WA + r) * kWave] + acc[HALF + c][r];
    // staged behind the exchanged sums, which other waves may still read
    tile_epilogue<WA, HALF, 1>(p, fin, lds + 2 * OTHER * sizeof(v4f) + (group * S::WAVES + wave) * 16 * STRIDE, n0,
                               t0 + group * HALF * 16, lane);
  }
}

template <bool F8, int WA, int WB, int P, int KS>
hipError_t launch_tile(const LinearArgs& a, hipStream_t stream) {
  using S = TileShape<F8, WA, WB>;
  const int64_t rt = (a.N + S::ROWS - 1) / S::ROWS, tt = (a.T + S::TOKENS - 1) / S::TOKENS;
  auto kern = linear_tile_kernel<F8, WA, WB, P, KS>;
  const size_t lds = (size_t)KS * P * S::BYTES;
  static_assert(2 * P * S::BYTES <= 160 * 1024, "two rings a CU");
  const hipError_t err = raise_lds_limit(reinterpret_cast<const void*>(kern), lds);
  if (err != hipSuccess) return err;
  hipLaunchKernelGGL(kern, dim3((unsigned)((rt * tt + 7) / 8 * 8)), dim3(64 * S::WAVES * KS), lds, stream, a, (int)rt,
                     (int)tt);
  return hipGetLastError();
}

}  // namespace

// E4M3 tokens double a stage's token bytes: fewer stages, still two rings a CU.
hipError_t launch_linear_tile(bool fp8, LinearPlan plan, const LinearArgs& a, hipStream_t stream) {
  switch (plan) {
    case kLinearTile256: return fp8 ? launch_tile<true, 8, 4, 2, 1>(a, stream) : launch_tile<false, 8, 4, 3, 1>(a, stream);
    case kLinearTile128: return fp8 ? launch_tile<true, 4, 4, 3, 1>(a, stream) : launch_tile<false, 4, 4, 4, 1>(a, stream);
    case kLinearTile64: return fp8 ? launch_tile<true, 4, 2, 4, 2>(a, stream) : launch_tile<false, 4, 2, 4, 2>(a, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace moe
