// The bfloat16 linears' product (moe_w4a4_linear_bf16, _grouped_linear_bf16) for few
// rows: the waves of a workgroup split K and stream their operands through LDS rings of
// their own.
//
// A workgroup of W waves owns NR*16 weight rows (gated: NR*8 gate rows and their NR*8 up
// rows) x XB*8 rows of x; wave w takes the K steps w, w + W, ... of 64 values, each with the
// whole tile in its accumulators, and the sums meet in LDS, added in wave order.  A copy
// brings whole 128-byte lines of 8 rows; 16-byte piece c of row r lies at place c ^ (r % 8),
// so that the 16 rows of an operand read spread over the banks.  P stages of a wave's ring
// are in flight, counted by vmcnt alone: nothing in the loop waits for another wave.
// (Loads straight to registers in the operand's layout touch 16 lines for 64 bytes each: 8 x
// 4096 x 32000 52 us instead of 43 to 46.)
//
// Bound by HBM where the weights come from there: 48 rows of 256 experts, 4096 to 2 x 2048, 199
// us, 6.7 TB/s; two stages of 4 waves a workgroup leave room for five workgroups a CU, whose
// copies cover each other's ends (rings of 4 and 5 stages 253 to 350 us).  Few weights are
// bound by latency: 1 x 4096 x 256 4.5 us, 8 x 4096 to 2 x 2048 7.7.
#include "bf16_common.h"
#include "gemm_common.h"
#include "tile_dma.h"

namespace moe {
namespace {

template <int XB, int NR, int W, int P>
struct Split {
  static constexpr int NT = (XB + 1) / 2;              // 16-row blocks of x
  static constexpr int DMAS = XB + 2 * NR;             // copies of a stage
  static constexpr int BYTES = DMAS * 1024;
  static_assert(DMAS * P <= 63, "vmcnt");
  static constexpr int LDS = W * (P * BYTES > NT * NR * 1024 ? P * BYTES : NT * NR * 1024);
};

template <int XB, int NR, int W, int P, bool ONCE, bool GATED, bool GROUPED>
__global__ void __launch_bounds__(64 * W) bf16_split_kernel(Bf16Args p, int row_tiles, int tok_tiles) {
  using S = Split<XB, NR, W, P>;
  constexpr int NT = S::NT, ROWS = XB * 8;
  extern __shared__ __align__(16) uint8_t lds[];
  constexpr int COLS = GATED ? NR * 8 : NR * 16;     // outputs a row
  int rt;
  RowTile t;
  if constexpr (GROUPED) {
    // a group's tiles with the same weights next to each other
    const GroupTiles<ROWS> tiles(p);
    const int L = group_item(tiles.total * row_tiles);
    if (L < 0) return;
    t = tiles.find(L / row_tiles);
    const int in = L - (L / row_tiles - t.tile) * row_tiles;
    rt = in / t.tiles;
    t.first += (in - rt * t.tiles) * ROWS;
    t.end = min(t.end, t.first + ROWS);
  } else {
    // Workgroups are dealt round-robin to the 8 XCDs: each XCD gets a run of row
    // tiles with all their token tiles, so its L2 fetches a weight once.
    const int L = (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3);
    if (L >= row_tiles * tok_tiles) return;
    rt = L / tok_tiles;
    const int tt = L - rt * tok_tiles;
    t = {0, tt * ROWS, min(p.T, (tt + 1) * ROWS), 0, 1};
  }
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int n0 = rt * COLS;
  const int steps = (p.K + 63) / 64, full = p.K / 64;

  // Where the copies read: a scalar base each, and a byte offset a lane.  Rows past the
  // last one read that one again; their sums are not stored.
  const int piece = (lane & 7) ^ (lane >> 3);
  const int last = (p.K % 64) / 8 - 1;               // last piece of the step that K ends in
  const int back = steps > full && piece > last ? (last - piece) * 16 : 0;
  const uint8_t* src[S::DMAS];
  uint32_t off[S::DMAS];
#pragma unroll
  for (int i = 0; i < 2 * NR; ++i) {
    const int n = n0 + (GATED ? i / 2 * 8 : i * 8);
    const int first = min(n, p.N - 1), mine = min(n + (lane >> 3), p.N - 1);
    const size_t row = GATED ? ((size_t)t.group * 2 + i % 2) * p.N + first : (size_t)t.group * p.N + first;
    src[i] = reinterpret_cast<const uint8_t*>(p.w + row * p.K);
    off[i] = (uint32_t)(mine - first) * p.K * 2 + piece * 16;
  }
#pragma unroll
  for (int i = 0; i < XB; ++i) {
    const int m = min(t.first + i * 8 + (lane >> 3), t.end - 1);
    if (GROUPED && p.rows != nullptr) {
      src[2 * NR + i] = reinterpret_cast<const uint8_t*>(p.x);
      off[2 * NR + i] = (uint32_t)source_row(p, m) * (uint32_t)(p.ldx * 2) + piece * 16;
    } else {
      src[2 * NR + i] = reinterpret_cast<const uint8_t*>(p.x + (size_t)t.first * p.ldx);
      off[2 * NR + i] = (uint32_t)(m - t.first) * (uint32_t)(p.ldx * 2) + piece * 16;
    }
  }
  uint8_t* ring = lds + wave * (P * S::BYTES);
  const uint32_t rbase = (uint32_t)(uintptr_t)ring;
  // Past the last step the copies read it again, so that every step has as many in flight.
  auto copy = [&](int s, int buf) {
    const int from = min(s, steps - 1);
#pragma unroll
    for (int i = 0; i < S::DMAS; ++i) {
      const uint8_t* at = src[i] + (size_t)from * 128;
      const int o = (int)(off[i] + (from == full ? back : 0));
      const uint32_t to = rbase + buf * S::BYTES + i * 1024;
      if (ONCE && i < 2 * NR)
        dma16_once(at, o, to);
      else
        dma16(at, o, to);
    }
  };

  v4f acc[NT][NR];
#pragma unroll
  for (int c = 0; c < NT; ++c)
#pragma unroll
    for (int r = 0; r < NR; ++r) acc[c][r] = v4f{0.f, 0.f, 0.f, 0.f};
  // The lane's operands: row lane % 16 of a block (x of 8 rows: lane % 8), piece 4 h + lane / 16.
  const int at0 = (lane & 15) * 128 + (((lane >> 4) ^ (lane & 7)) * 16);
  const int x0 = XB == 1 ? at0 & 1023 : at0;
  if (wave < steps) {
#pragma unroll
    for (int d = 0; d < P; ++d) copy(wave + d * W, d);
    for (int s = wave, buf = 0; s < steps; s += W) {
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"(S::DMAS * (P - 1)) : "memory");
      const uint8_t* st = ring + buf * S::BYTES;
      v4u a[NR][2], b[NT][2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int r = 0; r < NR; ++r) a[r][h] = *reinterpret_cast<const v4u*>(st + r * 2048 + (at0 ^ (h * 64)));
#pragma unroll
        for (int c = 0; c < NT; ++c) b[c][h] = *reinterpret_cast<const v4u*>(st + NR * 2048 + c * 2048 + (x0 ^ (h * 64)));
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");     // read: the place may be filled again
      copy(s + P * W, buf);
      if (s == full) {
        // The step that K ends in: pieces past the end are zeros on both sides (the copies read
        // the last piece again in their place).
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const bool in = 4 * h + (lane >> 4) <= last;
          const v4u none = {0, 0, 0, 0};
#pragma unroll
          for (int r = 0; r < NR; ++r) a[r][h] = in ? a[r][h] : none;
#pragma unroll
          for (int c = 0; c < NT; ++c) b[c][h] = in ? b[c][h] : none;
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int c = 0; c < NT; ++c)
#pragma unroll
          for (int r = 0; r < NR; ++r) acc[c][r] = mfma_bf16(a[r][h], b[c][h], acc[c][r]);
      buf = buf + 1 == P ? 0 : buf + 1;
    }
  }
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  __syncthreads();                                   // every wave is done with its ring

  v4f* red = reinterpret_cast<v4f*>(lds);
#pragma unroll
  for (int c = 0; c < NT; ++c)
#pragma unroll
    for (int r = 0; r < NR; ++r) red[((wave * NT + c) * NR + r) * kWave + lane] = acc[c][r];
  __syncthreads();
  auto sum = [&](int at) {
    v4f v = red[at];
#pragma unroll
    for (int w = 1; w < W; ++w) v += red[w * NT * NR * kWave + at];
    return v;
  };
  for (int q = threadIdx.x; q < ROWS * (COLS / 4); q += 64 * W) {
    const int tok = q / (COLS / 4), c4 = q - tok * (COLS / 4);
    const int row = t.first + tok;
    if (row >= t.end) continue;
    if constexpr (GATED) {
      // quad c4 of the tile's gates: block c4 / 2, lanes 16 (c4 % 2) and on; its up rows 32 lanes further
      const int at = ((tok / 16) * NR + c4 / 2) * kWave + (c4 % 2) * 16 + tok % 16;
      finish4<true>(p, t.group, row, n0 + 4 * c4, sum(at), sum(at + 32));
    } else {
      const int at = ((tok / 16) * NR + c4 / 4) * kWave + (c4 % 4) * 16 + tok % 16;
      finish4<false>(p, t.group, row, n0 + 4 * c4, sum(at), v4f{});
    }
  }
}

template <int XB, int NR, int W, int P, bool ONCE, bool GATED, bool GROUPED>
hipError_t launch_split(const Bf16Args& a, hipStream_t stream) {
  using S = Split<XB, NR, W, P>;
  constexpr int COLS = GATED ? NR * 8 : NR * 16, ROWS = XB * 8;
  const int64_t rt = (a.N + COLS - 1) / COLS;
  const int64_t tt = GROUPED ? a.T / ROWS + min(a.E, a.T) : (a.T + ROWS - 1) / ROWS;
  auto kern = bf16_split_kernel<XB, NR, W, P, ONCE, GATED, GROUPED>;
  if (S::LDS > 65536) {
    const hipError_t err = raise_lds_limit(reinterpret_cast<const void*>(kern), S::LDS);
    if (err != hipSuccess) return err;
  }
  const int64_t grid = GROUPED ? group_grid(rt * tt) : (rt * tt + 7) / 8 * 8;
  hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(64 * W), S::LDS, stream, a, (int)rt, (int)tt);
  return hipGetLastError();
}

template <bool GATED, bool GROUPED>
hipError_t launch_split_plan(Bf16Plan plan, const Bf16Args& a, hipStream_t stream) {
  switch (plan) {
    case kSplit16x8: return launch_split<1, 1, 4, 2, false, GATED, GROUPED>(a, stream);
    case kSplit16x8Wide: return launch_split<1, 1, 8, 2, false, GATED, GROUPED>(a, stream);
    case kSplit16x16: return launch_split<2, 1, 4, 2, false, GATED, GROUPED>(a, stream);
    case kSplit16x32: return launch_split<4, 1, 4, 2, false, GATED, GROUPED>(a, stream);
    case kSplit32x32: return launch_split<4, 2, 4, 2, false, GATED, GROUPED>(a, stream);
    case kSplit32x64: return launch_split<8, 2, 4, 2, false, GATED, GROUPED>(a, stream);
    case kSplit16x8Once: return launch_split<1, 1, 4, 2, true, GATED, GROUPED>(a, stream);
    case kSplit32x16Once: return launch_split<2, 2, 4, 2, true, GATED, GROUPED>(a, stream);
    case kSplit32x32Once: return launch_split<4, 2, 4, 2, true, GATED, GROUPED>(a, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_bf16_split(Bf16Plan plan, bool gated, const Bf16Args& a, hipStream_t stream) {
  if (a.offsets != nullptr)
    return gated ? launch_split_plan<true, true>(plan, a, stream) : launch_split_plan<false, true>(plan, a, stream);
  return gated ? launch_split_plan<true, false>(plan, a, stream) : launch_split_plan<false, false>(plan, a, stream);
}

}  // namespace moe
