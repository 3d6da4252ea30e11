// The bfloat16 linears' product for many rows: both operands go through LDS.
//
// A workgroup of WR x WT waves owns WR*WA*16 weight rows x WT*WB*16 rows of x, each wave
// WA x WB MFMA tiles in its accumulators.  A stage holds 64 values (128 bytes) of K of
// every row; 16-byte piece c of row r lies at place c ^ (r % 8), so that the 16 rows of an
// operand read spread over the banks (a copy fills places in order: the lane picks the
// piece instead).
//
// Two stages, and the operand registers of half a stage read ahead: a step's first half
// multiplies k 0..31 while it reads k 32..63; then one barrier says that the next stage has
// landed and that this one was read; the second half multiplies k 32..63 while it reads
// the next stage's first operands and copies the stage after that into this one's place.
// Every copy has a whole step to land, and the matrix cores do not wait for LDS at a
// step's start.  The copies are inline assembly (tile_dma.h): the compiler cannot tell the
// stages apart and would wait for all of them before every LDS read.
#include "bf16_common.h"
#include "gemm_common.h"
#include "tile_dma.h"

namespace moe {
namespace {

constexpr int kBand = 8;       // row tiles

template <int WR, int WT, int WA, int WB>
struct Tile {
  static constexpr int WAVES = WR * WT;
  static constexpr int A = WR * WA * 16, B = WT * WB * 16;   // rows of the two sides
  static constexpr int BYTES = (A + B) * 128;                // of a stage
  static constexpr int AD = A / 8 / WAVES, BD = B / 8 / WAVES, DMAS = AD + BD;   // copies (8 rows each) a wave and stage
  static_assert(AD * WAVES * 8 == A && BD * WAVES * 8 == B, "copies");
};

// 8 values in their own type (float32: two vectors), those past `left` zeros.
__device__ __forceinline__ void load8_raw(const void* base, size_t i, bool f32, int left, v4u (&r)[2]) {
  r[0] = r[1] = v4u{0, 0, 0, 0};
  if (f32) {
    const uint32_t* q = static_cast<const uint32_t*>(base) + i;
    if (left >= 8) {
      r[0] = *reinterpret_cast<const v4u_at4*>(q);
      r[1] = *reinterpret_cast<const v4u_at4*>(q + 4);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < left) r[j / 4][j % 4] = q[j];
    }
  } else {
    const uint16_t* q = static_cast<const uint16_t*>(base) + i;
    if (left >= 8) {
      r[0] = *reinterpret_cast<const v4u_at2*>(q);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < left) r[0][j / 2] |= (uint32_t)q[j] << (j % 2 * 16);
    }
  }
}
__device__ __forceinline__ float raw_value(const v4u (&r)[2], bool f32, int j) {
  return f32 ? __uint_as_float(r[j / 4][j % 4]) : bf16_to_f32(r[0][j / 2] >> (j % 2 * 16) & 0xFFFFu);
}

// The outputs of 16 rows from their sums in `mine` (16 x STRIDE bytes of LDS, the wave's own):
// 8 neighbouring ones a lane, so that a store covers a whole run of a row.  All loads
// of the rows' addends go out before the first use; f is applied in a rolled loop, each
// lane on the values that it stores (unrolled over a tile, its code spilled).
template <int WA, bool GATED>
__device__ __forceinline__ void store_rows(const Bf16Args& p, uint8_t* mine, int n, int row0, int end, int lane,
                                           const v4f (&bias)[2], const v4f (&up_bias)[2]) {
  constexpr int STRIDE = WA * 64 + 16;
  constexpr int LPT = WA * (GATED ? 8 : 16) / 8, TPP = kWave / LPT, IT = 16 / TPP;   // lanes a row, rows a pass, passes
  const int o = lane % LPT * 8;
  const int left = p.N - n, live = left > 0 ? end - row0 : 0;
  uint8_t* at = mine + lane / LPT * STRIDE + (GATED ? o / 16 * 32 + o % 16 : o) * 4;
  v4u add[IT][2];
  if (p.addend != nullptr) {
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int t = i * TPP + lane / LPT;
      load8_raw(p.addend, (size_t)(row0 + t) * p.lda + n, p.add_f32, t < live ? left : 0, add[i]);
    }
  }
  if (GATED || p.fn != MOE_FN_NONE || p.bias != nullptr || p.row_scale != nullptr) {
#pragma unroll 1
    for (int i = 0; i < IT; ++i) {
      v4f* q = reinterpret_cast<v4f*>(at + i * TPP * STRIDE);
      const int t = i * TPP + lane / LPT;
      const float scale = p.row_scale != nullptr && t < live ? p.row_scale[row0 + t] : 1.0f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        v4f v = apply_function(p.fn, q[h] + bias[h]);
        if constexpr (GATED) v *= q[h + 4] + up_bias[h];
        q[h] = v * scale;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int t = i * TPP + lane / LPT;
    if (t >= live) continue;
    const v4f* q = reinterpret_cast<const v4f*>(at + i * TPP * STRIDE);
    v4f v[2] = {q[0], q[1]};
    if (p.addend != nullptr) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j / 4][j % 4] += raw_value(add[i], p.add_f32, j);
    }
    const size_t to = (size_t)(row0 + t) * p.ldo + n;
    if (p.out_f32) {
      float* out = static_cast<float*>(p.out) + to;
      if (left >= 8) {
        __builtin_nontemporal_store(v[0], reinterpret_cast<v4f_at4*>(out));
        __builtin_nontemporal_store(v[1], reinterpret_cast<v4f_at4*>(out + 4));
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < left) out[j] = v[j / 4][j % 4];
      }
    } else {
      uint16_t* out = static_cast<uint16_t*>(p.out) + to;
      v4u b;
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = pack_bf16(v[j / 2][j % 2 * 2], v[j / 2][j % 2 * 2 + 1]);
      if (left >= 8) {
        __builtin_nontemporal_store(b, reinterpret_cast<v4u_at2*>(out));
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < left) out[j] = (uint16_t)(b[j / 2] >> (j % 2 * 16));
      }
    }
  }
}

template <int WR, int WT, int WA, int WB, bool GATED, bool GROUPED>
__global__ void __launch_bounds__(64 * WR * WT, 2) bf16_tile_kernel(Bf16Args p, int row_tiles, int tok_tiles) {
  using S = Tile<WR, WT, WA, WB>;
  constexpr int COLS = GATED ? S::A / 2 : S::A;              // outputs a row
  extern __shared__ __align__(16) uint8_t lds[];
  int rt, tt;
  RowTile t;
  if constexpr (GROUPED) {
    const GroupTiles tiles(p, S::B);
    const int per = (tiles.total * row_tiles + 7) / 8, at = blockIdx.x >> 3, L = (blockIdx.x & 7) * per + at;
    if (at >= per || L >= tiles.total * row_tiles) return;
    tt = L / row_tiles;
    rt = L - tt * row_tiles;
    t = tiles.find(p, S::B, tt);
  } else {
    // Workgroups are dealt round-robin to the 8 XCDs; each XCD gets a run of the order
    // below (a band of row tiles, rows of x next), so that the tiles it works on at a
    // time share their operands in its L2.
    const int L = (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3);
    if (L >= row_tiles * tok_tiles) return;
    const int band = L / (kBand * tok_tiles), width = min(kBand, row_tiles - band * kBand);
    const int in = L - band * kBand * tok_tiles;
    tt = in / width;
    rt = band * kBand + in - tt * width;
    t = {0, tt * S::B, min(p.T, (tt + 1) * S::B)};
  }
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
  // so that every step has as many in flight.
  auto dma = [&](int s, int buf, int i) {
    const int from = min(s, steps - 1);
    const uint32_t o = off[i] + (from == full ? back : 0);
    const uint32_t to = lbase + buf * S::BYTES + (i < S::AD ? (wave * S::AD + i) * 1024
                                                            : S::A * 128 + (wave * S::BD + i - S::AD) * 1024);
    dma16(src[i] + (size_t)from * 128, (int)o, to);
  };
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int i = 0; i < S::DMAS; ++i) dma(s, s, i);

  v4f acc[WB][WA];
#pragma unroll
  for (int c = 0; c < WB; ++c)
#pragma unroll
    for (int r = 0; r < WA; ++r) acc[c][r] = v4f{0.f, 0.f, 0.f, 0.f};
  // The lane's operands: row lane % 16 of a block, piece 4 h + lane / 16 of half h.
  const int at0 = (lane & 15) * 128 + (((lane >> 4) ^ (lane & 7)) * 16);
  const int a_at = wr * WA * 2048, b_at = S::A * 128 + wt * WB * 2048;
  v4u a[2][WA], b[2][WB];
  auto read_a = [&](const uint8_t* st, int h, int r) {
    a[h][r] = *reinterpret_cast<const v4u*>(st + a_at + r * 2048 + (at0 ^ (h * 64)));
  };
  auto read_b = [&](const uint8_t* st, int h, int c) {
    b[h][c] = *reinterpret_cast<const v4u*>(st + b_at + c * 2048 + (at0 ^ (h * 64)));
  };
  // Multiplies half H while it reads half 1 - H out of `st` and, with COPY, copies step s.
  auto half = [&](auto hc, const uint8_t* st, auto copy, int s, int buf) {
    constexpr int H = decltype(hc)::value, COPY = decltype(copy)::value, N = WA * WB;
    unrolled<N>([&](auto mi) {
      constexpr int m = decltype(mi)::value, c = m / WA, r = m % WA;
      acc[c][r] = mfma_bf16(a[H][r], b[H][c], acc[c][r]);
      unrolled<WA + WB>([&](auto ri) {
        constexpr int i = decltype(ri)::value;
        if constexpr (i * N / (WA + WB) == m) {
          if constexpr (i < WB)
            read_b(st, 1 - H, i);
          else
            read_a(st, 1 - H, i - WB);
        }
      });
      if constexpr (COPY)
        unrolled<S::DMAS>([&](auto di) {
          constexpr int i = decltype(di)::value;
          if constexpr (i * N / S::DMAS == m) dma(s, buf, i);
        });
      __builtin_amdgcn_sched_barrier(0);
    });
  };

  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(S::DMAS) : "memory");
#pragma unroll
  for (int c = 0; c < WB; ++c) read_b(lds, 0, c);
#pragma unroll
  for (int r = 0; r < WA; ++r) read_a(lds, 0, r);
  for (int s = 0; s < full; ++s) {
    const uint8_t* st = lds + (s & 1) * S::BYTES;
    half(Int<0>{}, st, Int<0>{}, 0, 0);
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    half(Int<1>{}, lds + (1 - (s & 1)) * S::BYTES, Int<1>{}, s + 2, s & 1);
  }
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  if (steps > full) {
    // The step that K ends in: pieces past the end are zeros on both sides (the copies
    // read the last piece again in their place).
    const uint8_t* st = lds + (full & 1) * S::BYTES;
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool in = 4 * h + (lane >> 4) <= last;
      const v4u none = {0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < WB; ++c) {
        read_b(st, h, c);
        b[h][c] = in ? b[h][c] : none;
      }
#pragma unroll
      for (int r = 0; r < WA; ++r) {
        read_a(st, h, r);
        a[h][r] = in ? a[h][r] : none;
      }
#pragma unroll
      for (int c = 0; c < WB; ++c)
#pragma unroll
        for (int r = 0; r < WA; ++r) acc[c][r] = mfma_bf16(a[h][r], b[h][c], acc[c][r]);
    }
  }

  // 16 rows at a time through the wave's part of the stages' place.
  __syncthreads();
  constexpr int STRIDE = WA * 64 + 16, OUT = GATED ? WA * 8 : WA * 16;
  static_assert(S::WAVES * 16 * STRIDE <= 2 * S::BYTES, "staging");
  uint8_t* mine = lds + wave * 16 * STRIDE;
  const int n = rt * COLS + wr * OUT + lane % (OUT / 8) * 8;
  v4f bias[2] = {}, up_bias[2] = {};
  if (p.bias != nullptr) {
    const size_t at = (size_t)t.group * (GATED ? 2 : 1) * p.N + n;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      bias[h] = load4_f32(p.bias, at + 4 * h, p.bias_f32, p.N - n - 4 * h);
      if constexpr (GATED) up_bias[h] = load4_f32(p.bias, at + p.N + 4 * h, p.bias_f32, p.N - n - 4 * h);
    }
  }
  unrolled<WB>([&](auto ci) {
    constexpr int c = decltype(ci)::value;
#pragma unroll
    for (int r = 0; r < WA; ++r)
      *reinterpret_cast<v4f*>(mine + (lane & 15) * STRIDE + (r * 16 + (lane >> 4) * 4) * 4) = acc[c][r];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    store_rows<WA, GATED>(p, mine, n, t.first + (wt * WB + c) * 16, t.end, lane, bias, up_bias);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  });
}

template <int WR, int WT, int WA, int WB, bool GATED, bool GROUPED>
hipError_t launch_tile(const Bf16Args& a, hipStream_t stream) {
  using S = Tile<WR, WT, WA, WB>;
  constexpr int COLS = GATED ? S::A / 2 : S::A;
  const int64_t rt = (a.N + COLS - 1) / COLS;
  const int64_t tt = GROUPED ? a.T / S::B + min(a.E, a.T) : (a.T + S::B - 1) / S::B;
  auto kern = bf16_tile_kernel<WR, WT, WA, WB, GATED, GROUPED>;
  constexpr size_t lds = 2 * (size_t)S::BYTES;
  const hipError_t err = raise_lds_limit(reinterpret_cast<const void*>(kern), lds);
  if (err != hipSuccess) return err;
  hipLaunchKernelGGL(kern, dim3((unsigned)((rt * tt + 7) / 8 * 8)), dim3(64 * S::WAVES), lds, stream, a, (int)rt,
                     (int)tt);
  return hipGetLastError();
}

template <bool GATED, bool GROUPED>
hipError_t launch_size(const Bf16Args& a, hipStream_t stream) {
  const int64_t cols = GATED ? 2 * (int64_t)a.N : a.N;
  const int64_t rows = GROUPED ? (a.T + a.E - 1) / a.E : a.T;
  const int64_t big = (cols + 255) / 256 * ((rows + 255) / 256) * (GROUPED ? a.E : 1);
  if (rows > 192 && big >= 256) return launch_tile<2, 4, 8, 4, GATED, GROUPED>(a, stream);
  return launch_tile<2, 2, 4, 4, GATED, GROUPED>(a, stream);
}

}  // namespace

hipError_t launch_bf16_tile(bool gated, const Bf16Args& a, hipStream_t stream) {
  if (a.offsets != nullptr) return gated ? launch_size<true, true>(a, stream) : launch_size<false, true>(a, stream);
  return gated ? launch_size<true, false>(a, stream) : launch_size<false, false>(a, stream);
}

}  // namespace moe
