// The bfloat16 linears' product (moe_w4a4_linear_bf16, _grouped_linear_bf16) for few
// rows: weight rows are the 16-row MFMA A operand, x rows the 16-column B operand,
// both straight from memory to registers.
//
// A workgroup of 8 waves owns NR*16 weight rows x NT*16 rows of x (gated: NR*8 gate
// rows and their NR*8 up rows); the waves split K in steps of 64 (wave w takes w, w + 8,
// ...), each with the whole tile in its accumulators, and their sums meet in LDS, added
// in wave order.  A dot product's terms may come in any order as long as both operands
// agree, so a lane's two 16-byte loads of a step are neighbours: k = 16 g + 8 j with g =
// lane / 16, MFMA j = 0, 1, and a step covers a whole 128-byte line of every row.
// The loads of step s + 1 are issued before the products of step s.
#include "bf16_common.h"
#include "gemm_common.h"

namespace moe {
namespace {

constexpr int kSplitWaves = 8;

template <int NT, int NR>
struct SplitStep {
  v4u a[NR][2], b[NT][2];
};

template <int NT, int NR, bool GATED, bool GROUPED>
__global__ void __launch_bounds__(64 * kSplitWaves) bf16_split_kernel(Bf16Args p, int row_tiles, int tok_tiles) {
  extern __shared__ __align__(16) uint8_t lds[];
  constexpr int COLS = GATED ? NR * 8 : NR * 16;     // outputs a row
  // Workgroups are dealt round-robin to the 8 XCDs: each XCD gets a run of the order
  // below, a group's or token tile's rows of the weights next to each other.
  int rt, tt;
  RowTile t;
  if constexpr (GROUPED) {
    const GroupTiles tiles(p, NT * 16);
    const int per = (tiles.total * row_tiles + 7) / 8, at = blockIdx.x >> 3, L = (blockIdx.x & 7) * per + at;
    if (at >= per || L >= tiles.total * row_tiles) return;
    tt = L / row_tiles;
    rt = L - tt * row_tiles;
    t = tiles.find(p, NT * 16, tt);
  } else {
    const int L = (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3);
    if (L >= row_tiles * tok_tiles) return;
    rt = L / tok_tiles;
    tt = L - rt * tok_tiles;
    t = {0, tt * NT * 16, min(p.T, (tt + 1) * NT * 16)};
  }
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int i = lane & 15, g = lane >> 4;
  const int n0 = rt * COLS;

  // Rows past the last one read that one again; their sums are not stored.
  const uint16_t *wp[NR], *xp[NT];
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    const int n = min(n0 + (GATED ? r * 8 + (i & 7) : r * 16 + i), p.N - 1);
    const size_t row = GATED ? ((size_t)t.group * 2 + (i >> 3)) * p.N + n : (size_t)t.group * p.N + n;
    wp[r] = p.w + row * p.K + g * 16;
  }
#pragma unroll
  for (int c = 0; c < NT; ++c) xp[c] = p.x + (size_t)source_row(p, min(t.first + c * 16 + i, t.end - 1)) * p.ldx + g * 16;

  v4f acc[NT][NR];
#pragma unroll
  for (int c = 0; c < NT; ++c)
#pragma unroll
    for (int r = 0; r < NR; ++r) acc[c][r] = v4f{0.f, 0.f, 0.f, 0.f};

  auto load = [&](int s, SplitStep<NT, NR>& d) {
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int j = 0; j < 2; ++j) d.a[r][j] = *reinterpret_cast<const v4u*>(wp[r] + (size_t)s * 64 + j * 8);
#pragma unroll
    for (int c = 0; c < NT; ++c)
#pragma unroll
      for (int j = 0; j < 2; ++j) d.b[c][j] = *reinterpret_cast<const v4u*>(xp[c] + (size_t)s * 64 + j * 8);
  };
  // The step that K ends in: pieces of 8 past the end are zeros on both sides.
  auto load_last = [&](int s, SplitStep<NT, NR>& d) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const bool in = s * 64 + g * 16 + j * 8 < p.K;
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        d.a[r][j] = v4u{0, 0, 0, 0};
        if (in) d.a[r][j] = *reinterpret_cast<const v4u*>(wp[r] + (size_t)s * 64 + j * 8);
      }
#pragma unroll
      for (int c = 0; c < NT; ++c) {
        d.b[c][j] = v4u{0, 0, 0, 0};
        if (in) d.b[c][j] = *reinterpret_cast<const v4u*>(xp[c] + (size_t)s * 64 + j * 8);
      }
    }
  };
  auto product = [&](const SplitStep<NT, NR>& d) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int c = 0; c < NT; ++c)
#pragma unroll
        for (int r = 0; r < NR; ++r) acc[c][r] = mfma_bf16(d.a[r][j], d.b[c][j], acc[c][r]);
  };
  const int full = p.K / 64;
  SplitStep<NT, NR> cur, nxt;
  int s = wave;
  if (s < full) load(s, cur);
  for (; s < full; s += kSplitWaves) {
    if (s + kSplitWaves < full) load(s + kSplitWaves, nxt);
    product(cur);
    cur = nxt;
  }
  if (p.K % 64 != 0 && full % kSplitWaves == wave) {
    load_last(full, cur);
    product(cur);
  }

  v4f* red = reinterpret_cast<v4f*>(lds);
#pragma unroll
  for (int c = 0; c < NT; ++c)
#pragma unroll
    for (int r = 0; r < NR; ++r) red[((wave * NT + c) * NR + r) * kWave + lane] = acc[c][r];
  __syncthreads();
  auto sum = [&](int at) {
    v4f v = red[at];
#pragma unroll
    for (int w = 1; w < kSplitWaves; ++w) v += red[w * NT * NR * kWave + at];
    return v;
  };
  for (int q = threadIdx.x; q < NT * 16 * (COLS / 4); q += 64 * kSplitWaves) {
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

template <int NT, int NR, bool GATED, bool GROUPED>
hipError_t launch_split(const Bf16Args& a, hipStream_t stream) {
  constexpr int COLS = GATED ? NR * 8 : NR * 16, ROWS = NT * 16;
  const int64_t rt = (a.N + COLS - 1) / COLS;
  const int64_t tt = GROUPED ? a.T / ROWS + min(a.E, a.T) : (a.T + ROWS - 1) / ROWS;
  constexpr size_t lds = (size_t)kSplitWaves * NT * NR * 1024;
  auto kern = bf16_split_kernel<NT, NR, GATED, GROUPED>;
  if (lds > 65536) {
    const hipError_t err = raise_lds_limit(reinterpret_cast<const void*>(kern), lds);
    if (err != hipSuccess) return err;
  }
  hipLaunchKernelGGL(kern, dim3((unsigned)((rt * tt + 7) / 8 * 8)), dim3(64 * kSplitWaves), lds, stream, a, (int)rt,
                     (int)tt);
  return hipGetLastError();
}

template <bool GATED, bool GROUPED>
hipError_t launch_rows(const Bf16Args& a, hipStream_t stream) {
  const int rows = GROUPED ? (a.T + a.E - 1) / a.E : a.T;
  if (rows <= 16) return launch_split<1, 1, GATED, GROUPED>(a, stream);
  if (rows <= 32) return launch_split<2, 2, GATED, GROUPED>(a, stream);
  return launch_split<4, 4, GATED, GROUPED>(a, stream);
}

}  // namespace

hipError_t launch_bf16_split(bool gated, const Bf16Args& a, hipStream_t stream) {
  if (a.offsets != nullptr) return gated ? launch_rows<true, true>(a, stream) : launch_rows<false, true>(a, stream);
  return gated ? launch_rows<true, false>(a, stream) : launch_rows<false, false>(a, stream);
}

}  // namespace moe
