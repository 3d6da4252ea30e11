// The bfloat16 linears' product for many rows: both operands go through LDS.
//
// A workgroup of WR x WT waves owns WR*WA*16 weight rows x WT*WB*16 rows of x, each wave
// WA x WB MFMA tiles in its accumulators.  A stage holds 64 values (128 bytes) of K of
// every row; 16-byte piece c of row r lies at place c ^ (r % 8), so that the 16 rows of an
// operand read spread over the banks (a copy fills places in order: the lane picks the
// piece instead).
//
// Rings of P stages (P + E of the weights), and the operand registers of half a stage read
// ahead: a step's first half multiplies k 0..31 while it reads k 32..63; then one barrier
// says that the next stages have landed and that these were read; the second half multiplies
// k 32..63 while it reads the next stages' first operands and copies x of step s + P and
// weights of step s + P + E into these ones' places.  The matrix cores do not wait for LDS
// at a step's start.  The copies are inline assembly (tile_dma.h): the compiler cannot tell
// the stages apart and would wait for all of them before every LDS read.
//
// 256 x 256 (2 x 4 waves of 128 x 64; 16384 x 4096 x (2 x 2048) gated 400 us, 1.37 PFLOP/s; 8192^3
// 715 us, 1.54): bound by power, the clock is 1.77 GHz and the MFMAs are busy 75 % of the
// cycles; LDS is read 1536 and written 512 cycles a step of 2048 MFMA cycles, which is why
// smaller tiles are slower for each output.  E = 1: 426 -> 409 us, and 1982 -> 1896 for
// 98304 x 2048 x 4096 in 256 groups, whose weights come from HBM.  64 x 64 (4096 x 4096 x 256 17 us)
// is bound by the L2s' way to LDS, 31 bytes a cycle and CU.
#include "bf16_store.h"
#include "gemm_common.h"
#include "tile_dma.h"

namespace moe {
namespace {

template <int WR, int WT, int WA, int WB, int P, int E>
struct Tile {
  static constexpr int WAVES = WR * WT;
  static constexpr int A = WR * WA * 16, B = WT * WB * 16;   // rows of the two sides
  static constexpr int LDS = ((P + E) * A + P * B) * 128;
  static constexpr int AD = A / 8 / WAVES, BD = B / 8 / WAVES, DMAS = AD + BD;   // copies (8 rows each) a wave and stage
  static constexpr int PER_EU = (LDS > 80 * 1024 ? 1 : 2) * WAVES / 4;   // waves a SIMD
  static_assert(DMAS * P + E * AD <= 63 && E <= 1, "vmcnt");
  static_assert(AD * WAVES * 8 == A && BD * WAVES * 8 == B, "copies");
};

template <int WR, int WT, int WA, int WB, int P, int E, bool ONCE, bool GATED, bool GROUPED>
__global__ void __launch_bounds__(64 * WR * WT, (Tile<WR, WT, WA, WB, P, E>::PER_EU))
    bf16_tile_kernel(Bf16Args p, int row_tiles, int tok_tiles) {
  using S = Tile<WR, WT, WA, WB, P, E>;
  constexpr int COLS = GATED ? S::A / 2 : S::A;              // outputs a row
  extern __shared__ __align__(16) uint8_t lds[];
  int tok_count = tok_tiles, L;
  RowTile t = {0, 0, p.T, 0, 0};
  if constexpr (GROUPED) {
    const GroupTiles<S::B> tiles(p);
    L = group_item(tiles.total * row_tiles);
    if (L < 0) return;
    t = tiles.find(L / row_tiles);
    L -= (L / row_tiles - t.tile) * row_tiles;
    tok_count = t.tiles;
  } else {
    // Workgroups are dealt round-robin to the 8 XCDs; each XCD gets a run.
    L = (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3);
    if (L >= row_tiles * tok_tiles) return;
  }
  // The order (of a group's tiles): a band of row tiles, rows of x next, so that the tiles
  // an XCD works on at a time share their operands in its L2.
  const int band = L / (kBand * tok_count), width = min(kBand, row_tiles - band * kBand);
  const int in = L - band * kBand * tok_count, tt = in / width, rt = band * kBand + in - tt * width;
  t.first += tt * S::B;
  t.end = min(t.end, t.first + S::B);
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wr = wave % WR, wt = wave / WR;
  const int steps = (p.K + 63) / 64, full = p.K / 64;

  // Where the wave's copies read: a scalar base each, and a byte offset a lane.  Rows past
  // the last one read that one again; their sums are not stored.  Gated, blocks of 16 gate
  // rows and of their 16 up rows take turns.
  const int piece = (lane & 7) ^ (lane >> 3);
  const int last = (p.K % 64) / 8 - 1;                        // last piece of the step that K ends in
  const int back = steps > full && piece > last ? (last - piece) * 16 : 0;
  const uint8_t* src[S::DMAS];
  uint32_t off[S::DMAS];
#pragma unroll
  for (int i = 0; i < S::AD; ++i) {
    const int j = (wave * S::AD + i) * 8;                     // first row of the copy in the stage
    const int half = GATED ? j / 16 % 2 : 0;
    const int n = rt * COLS + (GATED ? j / 32 * 16 + j % 16 : j);
    const int first = min(n, p.N - 1), mine = min(n + (lane >> 3), p.N - 1);
    const size_t row = ((size_t)t.group * (GATED ? 2 : 1) + half) * p.N + first;
    src[i] = reinterpret_cast<const uint8_t*>(p.w + row * p.K);
    off[i] = (uint32_t)(mine - first) * p.K * 2 + piece * 16;
  }
#pragma unroll
  for (int i = 0; i < S::BD; ++i) {
    const int m = min(t.first + (wave * S::BD + i) * 8 + (lane >> 3), t.end - 1);
    if (GROUPED && p.rows != nullptr) {
      src[S::AD + i] = reinterpret_cast<const uint8_t*>(p.x);
      off[S::AD + i] = (uint32_t)source_row(p, m) * (uint32_t)(p.ldx * 2) + piece * 16;
    } else {
      src[S::AD + i] = reinterpret_cast<const uint8_t*>(p.x + (size_t)t.first * p.ldx);
      off[S::AD + i] = (uint32_t)(m - t.first) * (uint32_t)(p.ldx * 2) + piece * 16;
    }
  }
  const uint32_t lbase = (uint32_t)(uintptr_t)lds;
  // Past the last step the copies read it again, into a place that is not read any more,
  // so that every step has as many in flight.  Copy i of step s: first those of x.
  auto dma_a = [&](int s, int buf, int i) {
    const int from = min(s, steps - 1);
    const uint32_t o = off[i] + (from == full ? back : 0), to = lbase + buf * (S::A * 128) + (wave * S::AD + i) * 1024;
    if (ONCE)
      dma16_once(src[i] + (size_t)from * 128, (int)o, to);
    else
      dma16(src[i] + (size_t)from * 128, (int)o, to);
  };
  auto dma_b = [&](int s, int buf, int i) {
    const int from = min(s, steps - 1);
    const uint32_t o = off[S::AD + i] + (from == full ? back : 0);
    dma16(src[S::AD + i] + (size_t)from * 128, (int)o,
          lbase + (P + E) * (S::A * 128) + buf * (S::B * 128) + (wave * S::BD + i) * 1024);
  };
#pragma unroll
  for (int s = 0; s < P + E; ++s) {
#pragma unroll
    for (int i = 0; i < S::AD; ++i) dma_a(s, s, i);
    if (s < P) {
#pragma unroll
      for (int i = 0; i < S::BD; ++i) dma_b(s, s, i);
    }
  }

  v4f acc[WB][WA];
#pragma unroll
  for (int c = 0; c < WB; ++c)
#pragma unroll
    for (int r = 0; r < WA; ++r) acc[c][r] = v4f{0.f, 0.f, 0.f, 0.f};
  // The lane's operands: row lane % 16 of a block, piece 4 h + lane / 16 of half h.
  const int at0 = (lane & 15) * 128 + (((lane >> 4) ^ (lane & 7)) * 16);
  const uint8_t* a_ring = lds + wr * WA * 2048;
  const uint8_t* b_ring = lds + (P + E) * (S::A * 128) + wt * WB * 2048;
  v4u a[2][WA], b[2][WB];
  auto read_a = [&](int buf, int h, int r) {
    a[h][r] = *reinterpret_cast<const v4u*>(a_ring + buf * (S::A * 128) + r * 2048 + (at0 ^ (h * 64)));
  };
  auto read_b = [&](int buf, int h, int c) {
    b[h][c] = *reinterpret_cast<const v4u*>(b_ring + buf * (S::B * 128) + c * 2048 + (at0 ^ (h * 64)));
  };
  // Multiplies half H while it reads half 1 - H out of places ra and rb and, with COPY, copies
  // what step s's places are free for.
  auto half = [&](auto hc, int ra, int rb, auto copy, int s, int ca, int cb) {
    constexpr int H = decltype(hc)::value, COPY = decltype(copy)::value, N = WA * WB;
    unrolled<N>([&](auto mi) {
      constexpr int m = decltype(mi)::value, c = m / WA, r = m % WA;
      acc[c][r] = mfma_bf16(a[H][r], b[H][c], acc[c][r]);
      unrolled<WA + WB>([&](auto ri) {
        constexpr int i = decltype(ri)::value;
        if constexpr (i * N / (WA + WB) == m) {
          if constexpr (i < WB)
            read_b(rb, 1 - H, i);
          else
            read_a(ra, 1 - H, i - WB);
        }
      });
      if constexpr (COPY)
        unrolled<S::DMAS>([&](auto di) {
          constexpr int i = decltype(di)::value;
          if constexpr (i * N / S::DMAS == m) {
            if constexpr (i < S::BD)
              dma_b(s + P, cb, i);
            else
              dma_a(s + P + E, ca, i - S::BD);
          }
        });
      __builtin_amdgcn_sched_barrier(0);
    });
  };

  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(S::DMAS * (P - 1) + E * S::AD) : "memory");
#pragma unroll
  for (int c = 0; c < WB; ++c) read_b(0, 0, c);
#pragma unroll
  for (int r = 0; r < WA; ++r) read_a(0, 0, r);
  int ab = 0, bb = 0;
  if (!GROUPED || t.first + wt * WB * 16 < t.end) {
    for (int s = 0; s < full; ++s) {
      const int an = ab + 1 == P + E ? 0 : ab + 1, bn = bb + 1 == P ? 0 : bb + 1;
      half(Int<0>{}, ab, bb, Int<0>{}, 0, 0, 0);
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(S::DMAS * (P - 2) + E * S::AD) : "memory");
      half(Int<1>{}, an, bn, Int<1>{}, s, ab, bb);
      ab = an;
      bb = bn;
    }
  } else {
    // A wave without rows (a group's last tile) copies the weights for the others; the rows
    // of x that it would copy are its own.
    for (int s = 0; s < full; ++s) {
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(S::AD * (P - 2 + E)) : "memory");
#pragma unroll
      for (int i = 0; i < S::AD; ++i) dma_a(s + P + E, ab, i);
      ab = ab + 1 == P + E ? 0 : ab + 1;
      bb = bb + 1 == P ? 0 : bb + 1;
    }
  }
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  if (steps > full) {
    // The step that K ends in: pieces past the end are zeros on both sides (the copies
    // read the last piece again in their place).
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool in = 4 * h + (lane >> 4) <= last;
      const v4u none = {0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < WB; ++c) {
        read_b(bb, h, c);
        b[h][c] = in ? b[h][c] : none;
      }
#pragma unroll
      for (int r = 0; r < WA; ++r) {
        read_a(ab, h, r);
        a[h][r] = in ? a[h][r] : none;
      }
#pragma unroll
      for (int c = 0; c < WB; ++c)
#pragma unroll
        for (int r = 0; r < WA; ++r) acc[c][r] = mfma_bf16(a[h][r], b[h][c], acc[c][r]);
    }
  }

  // The outputs, as many blocks of 16 rows at a time as fit the rings' place.
  __syncthreads();
  constexpr int STRIDE = WA * 64 + 16, OUT = GATED ? WA * 8 : WA * 16;
  constexpr int FIT = S::LDS / (S::WAVES * 16 * STRIDE), PART = FIT >= WB ? WB : FIT >= WB / 2 ? WB / 2 : WB / 4;
  static_assert(PART > 0 && WB % PART == 0 && S::WAVES * PART * 16 * STRIDE <= S::LDS, "staging");
  uint8_t* mine = lds + wave * PART * 16 * STRIDE;
  const int n = rt * COLS + wr * OUT + lane % (OUT / 8) * 8;
  v4f bias[2], up_bias[2];
  load_bias<GATED>(p, t.group, n, bias, up_bias);
  const int row0 = t.first + wt * WB * 16;
#pragma unroll
  for (int h = 0; h < WB / PART; ++h) {
    const int first = row0 + h * PART * 16;
    float scale = 1.0f;                         // of row first + lane
    if (p.row_scale != nullptr) scale = p.row_scale[min(first + lane, t.end - 1)];
#pragma unroll
    for (int c = 0; c < PART; ++c)
#pragma unroll
      for (int r = 0; r < WA; ++r)
        *reinterpret_cast<v4f*>(mine + (c * 16 + (lane & 15)) * STRIDE + (r * 16 + (lane >> 4) * 4) * 4) =
            acc[h * PART + c][r];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll 1
    for (int c = 0; c < PART; ++c) {
      const int row = first + c * 16;
      if (row >= t.end) break;
      store_rows<WA, GATED>(p, mine + c * 16 * STRIDE, n, row, t.end, lane, bias, up_bias, scale, c * 16);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

template <int WR, int WT, int WA, int WB, int P, int E, bool ONCE, bool GATED, bool GROUPED>
hipError_t launch_tile(const Bf16Args& a, hipStream_t stream) {
  using S = Tile<WR, WT, WA, WB, P, E>;
  constexpr int COLS = GATED ? S::A / 2 : S::A;
  const int64_t rt = (a.N + COLS - 1) / COLS;
  const int64_t tt = GROUPED ? a.T / S::B + min(a.E, a.T) : (a.T + S::B - 1) / S::B;
  auto kern = bf16_tile_kernel<WR, WT, WA, WB, P, E, ONCE, GATED, GROUPED>;
  constexpr size_t lds = (size_t)S::LDS;
  const hipError_t err = raise_lds_limit(reinterpret_cast<const void*>(kern), lds);
  if (err != hipSuccess) return err;
  const int64_t grid = GROUPED ? group_grid(rt * tt) : (rt * tt + 7) / 8 * 8;
  hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(64 * S::WAVES), lds, stream, a, (int)rt,
                     (int)tt);
  return hipGetLastError();
}

template <bool GATED, bool GROUPED>
hipError_t launch_tile_plan(Bf16Plan plan, const Bf16Args& a, hipStream_t stream) {
  switch (plan) {
    // (three stages where groups end in the middle of rounds: three workgroups a CU; 37 groups, 1517
    // rows, 1000 to 777: 21.7 -> 18.2 us without an epilogue; 4096 x 4096 x 256 would go from 17.0 to 18.6)
    case kTile64x64: return launch_tile<1, 4, 4, 1, GROUPED ? 3 : 4, 0, false, GATED, GROUPED>(a, stream);
    case kTile128x64: return launch_tile<2, 2, 4, 2, 3, 0, false, GATED, GROUPED>(a, stream);
    case kTile128x128: return launch_tile<2, 2, 4, 4, 3, 0, false, GATED, GROUPED>(a, stream);
    case kTile256x128: return launch_tile<4, 2, 4, 4, 3, 0, false, GATED, GROUPED>(a, stream);
    case kTile256x256: return launch_tile<2, 4, 8, 4, 2, 1, false, GATED, GROUPED>(a, stream);
    default: break;
  }
  if constexpr (GROUPED) {
    if (plan == kTile128x64Once) return launch_tile<2, 2, 4, 2, 3, 0, true, GATED, GROUPED>(a, stream);
    if (plan == kTile256x128Once) return launch_tile<4, 2, 4, 4, 3, 0, true, GATED, GROUPED>(a, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_bf16_tile(Bf16Plan plan, bool gated, const Bf16Args& a, hipStream_t stream) {
  if (a.offsets != nullptr)
    return gated ? launch_tile_plan<true, true>(plan, a, stream) : launch_tile_plan<false, true>(plan, a, stream);
  return gated ? launch_tile_plan<true, false>(plan, a, stream) : launch_tile_plan<false, false>(plan, a, stream);
}

}  // namespace moe
