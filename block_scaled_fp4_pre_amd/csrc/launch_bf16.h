// Host-side launchers of the bfloat16 operators (linear, grouped linear, norm
// after a block).  Every launcher only enqueues on `stream`; arguments were
// validated by the caller.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

// One product out = addend + row_scale * f(x W^T + bias), dense (offsets null) or
// grouped: rows [offsets[e], offsets[e + 1]) belong to group e, whose weights and
// bias are the e-th.  Gated: W has 2N rows, f(gate) * up.
struct Bf16Args {
  const uint16_t* x;
  const uint16_t* w;           // [E][N or 2N][K]
  const void* bias;            // [E][N or 2N] or null
  const float* row_scale;      // [T] or null
  const void* addend;          // or null
  void* out;
  const int32_t* offsets;      // [E + 1], grouped
  const int32_t* rows;         // x row of row i: rows[i] / row_div; null: i
  int64_t ldx, lda, ldo;       // elements from row to row
  int T, N, K, E, row_div, x_rows;
  int fn;                      // MOE_FN_*
  bool bias_f32, add_f32, out_f32;
};

// Which kernel takes a product: tiles of weight rows x rows of x, of the split kernel
// (bf16_split.hip) or the tile kernel (bf16_tile.hip); Once: weights read past the caches.
enum Bf16Plan {
  kSplit16x8, kSplit16x8Wide, kSplit16x16, kSplit16x32, kSplit32x32, kSplit32x64,
  kSplit16x8Once, kSplit32x16Once, kSplit32x32Once,
  kTile64x64, kTile128x64, kTile128x128, kTile256x128, kTile256x256, kTile128x64Once, kTile256x128Once
};
// 128 MiB of weights and more, and few rows for each: the time is the weights' way from HBM.
// Read once, past the caches, they come at 6.9-7.0 TB/s instead of 6.1-6.3 (48 rows of 256
// experts, 4096 to 2 x 2048: 214 against 240 us).  The caches hold 256 MB: a call repeated on weights
// of up to that is faster through them, one whose weights others have pushed out is slower.  us
// through the caches / past them, repeated; then behind a pass that writes 1 GiB:
//   8 x 4096 x 8000 (63 MiB, left to the caches)   11.5 / 11.2    27 / 16
//   8 x 4096 x 16300 (127 MiB, left to them)       20.5 / 26      62 / 32
//   8 x 4096 x 16500 (129 MiB, past them)          22 / 28-31     66 / 34
//   8 x 4096 x 24000 (188 MiB, past them)          29 / 32        70 / 36
//   8 x 4096 x 32000 (250 MiB, past them)          38 / 46       106 / 49
// (8 x 4096 to 2 x 2048, 33 MB, repeated: 7.6 / 8.4.)  Groups count as far as the rows go, whatever
// the offsets say (the host does not see them), and their rows are taken to be alike: 512 rows of 256
// experts, 4096 to 2 x 2048, take 1243 us where each has two, and 242 where one has all, whose weights
// 64 tiles of rows read each for themselves (128 x 64 once: 1401 and 47).  Measured by the mean
// rows of a group, 256 groups, us, 4096 to 2 x 2048 (2048 to 4096):
//   rows   16 x 8       32 x 16      32 x 32      128 x 64     256 x 128    256 x 128    256 x 256
//          split once   split once   split once   tile once    tile once    tile         tile
//   4      1320 (673)   1235 (631)   1261 (707)   1365 (700)   1390 (735)   1502 (778)   1591 (817)
//   8      1893 (977)   1295 (679)   1310 (754)   1395 (722)   1418 (764)   1513 (785)   1608 (836)
//   16     2999 (1532)  1868 (996)   1377 (840)   1408 (753)   1416 (786)   1539 (805)   1640 (860)
//   32     -            -            2233 (1278)  1464 (797)   1460 (826)   1564 (831)   1676 (892)
//   48     -            -            3080 (-)     1507 (-)     1492 (-)     1589 (-)     1716 (-)
//   64     -            -            -            1986 (1093)  1545 (881)   1634 (875)   1700 (927)
//   96     -            -            -            2566 (1424)  1623 (914)   1709 (914)   1764 (947)
//   128    -            -            -            3242 (1790)  2102 (1098)  1792 (938)   1815 (971)
//   192    -            -            -            -            2680 (1323)  2219 (1229)  2084 (1115)
inline bool bf16_once(const Bf16Args& a, bool gated, int64_t groups) {
  return groups * a.N * a.K * (gated ? 4 : 2) >= (int64_t)128 << 20;
}
// Everything else by the time of a round, 256 tiles: `step` us for every 64 values of K (from
// products with K = 4096) and `ends` us for the rest (from 16384 x 64 x 4096); the least of
// rounds * (steps * step + ends).  Measured us, the rule's choice first: 512 x 4096 x 4096 128 x
// 64 23.0, 64 x 64 25.5, 128 x 128 28.6; 200 x 4096 x 4096 64 x 64 16.9, 32 x 64 21.9, 128 x 64 21.9; 96 x
// 4096 x 4096 32 x 64 12.0, 32 x 32 14.1, 64 x 64 15.9; 48 x 4096 x 4096 32 x 32 9.3, 16 x 32 10.6; 1024 x
// 4096 x 4096 128 x 128 32.6, 128 x 64 40; 2048 x 4096 x 4096 256 x 128 55, 128 x 128 58, 256 x 256 71;
// 4096 x 2048 x 4096 256 x 256 57, 256 x 128 63; 4096 x 4096 x 256 64 x 64 17.1, 128 x 64 21.7, 32 x 64
// 41.7; 4096 x 256 x 4096 256 x 256 15.7, 256 x 128 17.2, 128 x 64 21.9; 1000 x 64 x 1000 64 x 64 4.2, 128 x
// 64 4.8, 32 x 32 5.5; 37 groups, 1517 rows, 1000 to 777, 64 x 64 18.6, 128 x 64 20.8, 128 x 128 26.1, 32 x 64 33.
// (The products of K = 4096 had their weights in the caches, as a repeated call has.)
struct Bf16Tile {
  Bf16Plan plan;
  int w, t;              // weight rows, rows of x
  double step, ends;     // us
};
constexpr Bf16Tile kBf16Tiles[] = {
    {kSplit16x8, 16, 8, 0.055, 0.25},   {kSplit16x16, 16, 16, 0.06, 0.35},  {kSplit16x32, 16, 32, 0.10, 0.55},
    {kSplit32x32, 32, 32, 0.115, 0.85}, {kSplit32x64, 32, 64, 0.155, 1.5},  {kTile64x64, 64, 64, 0.225, 1.3},
    {kTile128x64, 128, 64, 0.33, 1.8},  {kTile128x128, 128, 128, 0.47, 4.5}, {kTile256x128, 256, 128, 0.86, 5.7},
    {kTile256x256, 256, 256, 1.65, 9.5}};
inline Bf16Plan bf16_plan(bool gated, const Bf16Args& a) {
  const int64_t cols = gated ? 2 * (int64_t)a.N : a.N, groups = a.offsets == nullptr ? 1 : a.E < a.T ? a.E : a.T;
  const int64_t mean = (a.T + groups - 1) / groups;
  const bool grouped = a.offsets != nullptr;
  if (bf16_once(a, gated, groups)) {
    if (mean <= 2 || (!grouped && mean <= 8)) return kSplit16x8Once;
    if (mean <= 8 || (!grouped && mean <= 16)) return kSplit32x16Once;
    if (mean <= 16 || (!grouped && mean <= 32)) return kSplit32x32Once;
    if (grouped && mean <= 48) return kTile128x64Once;
    if (grouped && mean <= 96) return kTile256x128Once;
    if (grouped && mean <= 160) return kTile256x128;
    if (grouped) return kTile256x256;
  }
  Bf16Plan best = kTile256x256;
  double least = 1e30;
  for (const Bf16Tile& c : kBf16Tiles) {
    // (of every group's last tile half is taken to be empty)
    const double tok = grouped && groups > 1 ? (double)a.T / c.t + 0.5 * groups : (double)((a.T + c.t - 1) / c.t);
    double rounds = tok * (double)((cols + c.w - 1) / c.w) / 256;
    // (a CU holds several of the small ones: they do not wait for a round to end)
    if (rounds < 1 || (c.w * c.t >= 32 * 64 && c.plan != kTile64x64)) rounds = __builtin_ceil(rounds);
    const double time = ((a.K + 63) / 64 * c.step + c.ends) * rounds;
    if (time < least) {
      least = time;
      best = c.plan;
    }
  }
  // Few weight rows: 8 waves a tile take its K in half the steps (1 x 4096 x 256 4.1 against 4.5 us, 8 x
  // 4096 x 2048 4.9 against 5.7, 1 x 4096 x 4096 7.3 against 7.1).  Nothing else is asked: groups of a row
  // each take them too, 16 of 4096 to 512 in the same time (12.6 us), 64 of 512 to 256 7.9 against 7.1, 512 of
  // 8 to 256 76 against 41.
  if (best == kSplit16x8 && cols <= 16 * 192) return kSplit16x8Wide;
  return best;
}
hipError_t launch_bf16_split(Bf16Plan plan, bool gated, const Bf16Args& a, hipStream_t stream);   // bf16_split.hip
hipError_t launch_bf16_tile(Bf16Plan plan, bool gated, const Bf16Args& a, hipStream_t stream);    // bf16_tile.hip
inline hipError_t launch_linear_bf16(bool gated, const Bf16Args& a, hipStream_t stream) {
  const Bf16Plan plan = bf16_plan(gated, a);
  return plan < kTile64x64 ? launch_bf16_split(plan, gated, a, stream) : launch_bf16_tile(plan, gated, a, stream);
}

// post_norm.hip.  act as for launch_add_rmsnorm; gate_kind: MOE_GATE_*.
struct PostNormArgs {
  const uint16_t* x;
  const void *residual, *post_weight, *gate, *next_weight;
  void* residual_out;
  uint16_t* y;
  uint8_t *codes, *scales;
  int64_t rows;
  int cols, gate_kind;
  bool w_f32, gate_f32;
  float scale, g;
  double eps, per_col;   // per_col = 1 / cols
};
hipError_t launch_post_norm(int act, bool res_f32, const PostNormArgs& a, hipStream_t stream);

}  // namespace moe
