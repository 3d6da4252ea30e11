// The norm after a block with its gate and residual scale, the addition to the residual
// stream, and the norm and quantization before the next block (moe_w4a4_post_norm):
//   z = x * w1 / sqrt(mean(x^2) + eps)   (or x);   h = rnd(r + scale * gate * z);
//   y = bf16(h * w2 / sqrt(mean(h^2) + eps));      codes, scales = Q(y).
//
// Bound by HBM: the row of x and of r stays in registers through both sums, so every
// input is read once and every output written once.  Teams of 64 to 1024 threads and
// pieces of 8 values as in norm.hip, and like there sums, norms and products run in
// fp64 (hidden behind the loads): h has one rounding, the same whatever the order of
// the sums, and the codes behind it are reproducible next to the quantizer's borders.
// 16384 x 4096 with E4M3 codes (472 MB) take 104 us, 4.5 TB/s (91 at a copy's rate): the fp64
// conversions, 7 a value, are what the loads do not hide (without the first norm 96 us).
#include "launch_bf16.h"
#include "moe_w4a4.h"
#include "norm_rows.h"

namespace moe {
namespace {

__device__ __forceinline__ void load8(const void* p, size_t i, bool f32, float (&f)[8]) {
  if (f32)
    load_f32x8(static_cast<const float*>(p) + i, f);
  else
    unpack8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i), f);
}

// 8 values of the residual stream in its own type.
template <bool F32>
struct Stream {
  uint4 b;
  __device__ __forceinline__ void load(const void* p, size_t i) {
    b = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
  }
  __device__ __forceinline__ void store(void* p, size_t i) const {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = b;
  }
  __device__ __forceinline__ void clear() { b = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&f)[8]) const { unpack8(b, f); }
  __device__ __forceinline__ void set(const float (&f)[8]) { b = pack8(f); }
};
template <>
struct Stream<true> {
  float h[8];
  __device__ __forceinline__ void load(const void* p, size_t i) { load_f32x8(static_cast<const float*>(p) + i, h); }
  __device__ __forceinline__ void store(void* p, size_t i) const {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    q[0] = make_float4(h[0], h[1], h[2], h[3]);
    q[1] = make_float4(h[4], h[5], h[6], h[7]);
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = 0.0f;
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = h[i];
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = f[i];
  }
};

// h += factor * gate * w1 * x for piece c of the row that begins at `base`.
template <bool F32>
__device__ __forceinline__ void add_step(const PostNormArgs& p, const uint4& x, Stream<F32>& h, double factor, size_t base,
                                         int c) {
  float v[8], r[8], w[8];
  double d[8];
  unpack8(x, v);
#pragma unroll
  for (int i = 0; i < 8; ++i) d[i] = (double)v[i] * factor;
  if (p.post_weight != nullptr) {
    load8(p.post_weight, 8 * c, p.w_f32, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) d[i] *= (double)w[i];
  }
  if (p.gate_kind == MOE_GATE_CHANNEL || p.gate_kind == MOE_GATE_FULL) {
    load8(p.gate, (p.gate_kind == MOE_GATE_FULL ? base : 0) + 8 * c, p.gate_f32, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) d[i] *= (double)w[i];
  }
  h.get(r);
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = (float)((double)r[i] + d[i]);
  h.set(r);
}

// y of piece c.
template <bool F32>
__device__ __forceinline__ uint4 normed(const PostNormArgs& p, const Stream<F32>& h, double rstd, int c, bool live) {
  float w[8] = {0, 0, 0, 0, 0, 0, 0, 0}, v[8], n[8];
  if (live) load8(p.next_weight, 8 * c, p.w_f32, w);
  h.get(v);
#pragma unroll
  for (int i = 0; i < 8; ++i) n[i] = (float)((double)v[i] * rstd * (double)w[i]);
  return pack8(n);
}

// The sum of the wave's 64 lanes: within quads, halves and rows of 16, then from row to
// row, by lane moves of the vector unit (wave_sum's go through LDS).
template <int CTRL, int ROWS>
__device__ __forceinline__ double lanes_moved(double v) {
  const uint2 b = __builtin_bit_cast(uint2, v);
  return __builtin_bit_cast(double, make_uint2((uint32_t)__builtin_amdgcn_update_dpp(0, (int)b.x, CTRL, ROWS, 0xF, false),
                                               (uint32_t)__builtin_amdgcn_update_dpp(0, (int)b.y, CTRL, ROWS, 0xF, false)));
}
__device__ __forceinline__ double lanes_sum(double v) {
  v += lanes_moved<0xB1, 0xF>(v);      // lane ^ 1
  v += lanes_moved<0x4E, 0xF>(v);      // lane ^ 2
  v += lanes_moved<0x141, 0xF>(v);     // the other half of 8, mirrored
  v += lanes_moved<0x140, 0xF>(v);     // the other half of 16, mirrored
  v += lanes_moved<0x142, 0xA>(v);     // rows 1 and 3: the last lane of the row before
  v += lanes_moved<0x143, 0xC>(v);     // rows 2 and 3: lane 31
  const uint2 b = __builtin_bit_cast(uint2, v);
  return __builtin_bit_cast(double, make_uint2((uint32_t)__builtin_amdgcn_readlane((int)b.x, 63),
                                               (uint32_t)__builtin_amdgcn_readlane((int)b.y, 63)));
}

// 1 / sqrt(v): the instruction's estimate and three steps of Newton's, to the last bits
// of fp64 (a division by a square root takes every wave about 600 cycles more, twice a row).
// Of infinity 0, as a division has it: a step would make 0 * infinity of it, and a row's finite
// values NaN.
__device__ __forceinline__ double inverse_root(double v) {
  const double estimate = __builtin_amdgcn_rsq(v);
  double y = estimate;
#pragma unroll
  for (int i = 0; i < 3; ++i) y = fma(0.5 * y, fma(-v * y, y, 1.0), y);
  return estimate == 0.0 ? 0.0 : y;
}

// The row's factor before its norm: scale, and a gate of rows.
__device__ __forceinline__ double row_factor(const PostNormArgs& p, int64_t row) {
  if (p.gate_kind != MOE_GATE_ROW) return p.scale;
  return (double)p.scale * (p.gate_f32 ? static_cast<const float*>(p.gate)[row]
                                       : bf16_to_f32(static_cast<const uint16_t*>(p.gate)[row]));
}

// RES_F32: type of the residual stream.  ACT: codes of 0 MXFP4, 1 MXFP8 E4M3, 2 NVFP4,
// or -1 none.  TPR: threads per row, CPL pieces each.
template <bool RES_F32, int ACT, int TPR, int CPL>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) post_norm_kernel(PostNormArgs p) {
  constexpr int THREADS = TPR < 256 ? 256 : TPR;
  constexpr int RPB = THREADS / TPR;
  constexpr int WPR = TPR / kWave;
  __shared__ double part[2][WPR > 1 ? WPR : 1];
  const int t = threadIdx.x % TPR, pieces = p.cols >> 3;
  // The team's sum; two buffers, so that a wave may be a sum ahead of one still reading.
  int flip = 0;
  auto team_sum = [&](double v) {
    v = lanes_sum(v);
    if constexpr (WPR > 1) {
      if (t % kWave == 0) part[flip][t / kWave] = v;
      __syncthreads();
      v = 0.0;
#pragma unroll
      for (int i = 0; i < WPR; ++i) v += part[flip][i];
      flip ^= 1;
    }
    return v;
  };
  for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR; row < p.rows; row += (int64_t)gridDim.x * RPB) {
    const size_t base = (size_t)row * p.cols;
    uint4 x[CPL];
    Stream<RES_F32> h[CPL];
#pragma unroll
    for (int j = 0; j < CPL; ++j) {
      const int c = t + j * TPR;
      if (c < pieces) {
        x[j] = *reinterpret_cast<const uint4*>(p.x + base + 8 * c);
        h[j].load(p.residual, base + 8 * c);
      } else {
        x[j] = make_uint4(0, 0, 0, 0);
        h[j].clear();
      }
    }
    double factor = row_factor(p, row);
    if (p.post_weight != nullptr) {
      double ss = 0.0;
#pragma unroll
      for (int j = 0; j < CPL; ++j) {
        float v[8];
        unpack8(x[j], v);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fma((double)v[i], (double)v[i], ss);
      }
      factor *= inverse_root(fma(team_sum(ss), p.per_col, p.eps));
    }
    double ss = 0.0;
#pragma unroll
    for (int j = 0; j < CPL; ++j) {
      const int c = t + j * TPR;
      if (c >= pieces) continue;
      float r[8];
      add_step(p, x[j], h[j], factor, base, c);
      h[j].store(p.residual_out, base + 8 * c);
      h[j].get(r);
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fma((double)r[i], (double)r[i], ss);
    }
    if (p.next_weight != nullptr) {
      const double rstd = inverse_root(fma(team_sum(ss), p.per_col, p.eps));
#pragma unroll
      for (int j = 0; j < CPL; ++j) {
        const int c = t + j * TPR;
        const uint4 yb = normed(p, h[j], rstd, c, c < pieces);
        if (p.y != nullptr && c < pieces) *reinterpret_cast<uint4*>(p.y + base + 8 * c) = yb;
        if constexpr (ACT >= 0) quantize_piece<ACT>(yb, (size_t)row * pieces, c, pieces, p.g, p.codes, p.scales);
      }
    }
  }
}

// Rows too long for registers: x, the residual and h come out of the caches again.
// A thread reads and writes its own pieces only.
constexpr int kLongThreads = 1024;
template <bool RES_F32, int ACT>
__global__ void __launch_bounds__(kLongThreads) post_norm_long_kernel(PostNormArgs p) {
  __shared__ double part[2][kLongThreads / kWave];
  const int t = threadIdx.x, pieces = p.cols >> 3;
  int flip = 0;
  auto block_sum = [&](double v) {
    v = lanes_sum(v);
    if (t % kWave == 0) part[flip][t / kWave] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int i = 0; i < kLongThreads / kWave; ++i) v += part[flip][i];
    flip ^= 1;
    return v;
  };
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const size_t base = (size_t)row * p.cols;
    double factor = row_factor(p, row);
    if (p.post_weight != nullptr) {
      double ss = 0.0;
#pragma unroll 4
      for (int c = t; c < pieces; c += kLongThreads) {
        float v[8];
        unpack8(*reinterpret_cast<const uint4*>(p.x + base + 8 * c), v);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fma((double)v[i], (double)v[i], ss);
      }
      factor *= inverse_root(fma(block_sum(ss), p.per_col, p.eps));
    }
    double ss = 0.0;
    for (int c = t; c < pieces; c += kLongThreads) {
      Stream<RES_F32> h;
      float r[8];
      h.load(p.residual, base + 8 * c);
      add_step(p, *reinterpret_cast<const uint4*>(p.x + base + 8 * c), h, factor, base, c);
      h.store(p.residual_out, base + 8 * c);
      h.get(r);
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fma((double)r[i], (double)r[i], ss);
    }
    if (p.next_weight == nullptr) continue;
    const double rstd = inverse_root(fma(block_sum(ss), p.per_col, p.eps));
    // (every lane of a wave takes part in each piece's quantization)
    for (int c0 = 0; c0 < pieces; c0 += kLongThreads) {
      const int c = c0 + t;
      Stream<RES_F32> h;
      h.clear();
      if (c < pieces) h.load(p.residual_out, base + 8 * c);
      const uint4 yb = normed(p, h, rstd, c, c < pieces);
      if (p.y != nullptr && c < pieces) *reinterpret_cast<uint4*>(p.y + base + 8 * c) = yb;
      if constexpr (ACT >= 0) quantize_piece<ACT>(yb, (size_t)row * pieces, c, pieces, p.g, p.codes, p.scales);
    }
  }
}

// Workgroups of 1024 threads, one a CU at a time, take several rows each (4096 x 16384
// 167 -> 149 us); smaller ones do not gain from it (65536 x 512 75 -> 91).
template <int TPR>
constexpr int64_t kPostBlocks = TPR == 1024 ? 512 : 1 << 20;

template <bool RES_F32, int ACT, int TPR, int CPL>
hipError_t launch_post(const PostNormArgs& a, hipStream_t stream) {
  constexpr int THREADS = TPR < 256 ? 256 : TPR;
  constexpr int RPB = THREADS / TPR;
  const int64_t blocks = (a.rows + RPB - 1) / RPB;
  hipLaunchKernelGGL((post_norm_kernel<RES_F32, ACT, TPR, CPL>),
                     dim3((unsigned)(blocks < kPostBlocks<TPR> ? blocks : kPostBlocks<TPR>)), dim3(THREADS), 0, stream, a);
  return hipGetLastError();
}

// Teams of a wave up to 1024 values, of 4 waves up to 4096, of 8 where every row has a CU of
// its own (1 x 4096 4.4 -> 3.8 us, 64 x 4096 4.9 -> 4.0; 16384 x 4096 128 -> 152) and up to 8192
// (1 x 8192 6.2 -> 5.0, 8192 x 8192 145 -> 130 against 4 waves of 4 pieces; 16 waves 146).
// Past 16384 values the registers do not hold the row (4 pieces of 1024 threads spilled):
// 1000 x 32768 106 -> 93 us (float32 stream 140 -> 126), 500 x 65536 with 8 pieces 363 -> 130.
template <bool RES_F32, int ACT>
hipError_t launch_post_act(const PostNormArgs& a, hipStream_t stream) {
  if (a.cols <= 512) return launch_post<RES_F32, ACT, 64, 1>(a, stream);
  if (a.cols <= 1024) return launch_post<RES_F32, ACT, 64, 2>(a, stream);
  if (a.cols <= 2048) return launch_post<RES_F32, ACT, 256, 1>(a, stream);
  if (a.cols <= 4096 && a.rows <= 256) return launch_post<RES_F32, ACT, 512, 1>(a, stream);
  if (a.cols <= 4096) return launch_post<RES_F32, ACT, 256, 2>(a, stream);
  if (a.cols <= 8192) return launch_post<RES_F32, ACT, 512, 2>(a, stream);
  if (a.cols <= 16384) return launch_post<RES_F32, ACT, 1024, 2>(a, stream);
  const int64_t blocks = a.rows < kPostBlocks<kLongThreads> ? a.rows : kPostBlocks<kLongThreads>;
  hipLaunchKernelGGL((post_norm_long_kernel<RES_F32, ACT>), dim3((unsigned)blocks), dim3(kLongThreads), 0, stream, a);
  return hipGetLastError();
}

template <bool RES_F32>
hipError_t launch_post_res(int act, const PostNormArgs& a, hipStream_t stream) {
  auto f = act == 0 ? launch_post_act<RES_F32, 0> : act == 1 ? launch_post_act<RES_F32, 1>
         : act == 2 ? launch_post_act<RES_F32, 2> : launch_post_act<RES_F32, -1>;
  return f(a, stream);
}

}  // namespace

hipError_t launch_post_norm(int act, bool res_f32, const PostNormArgs& a, hipStream_t stream) {
  return res_f32 ? launch_post_res<true>(act, a, stream) : launch_post_res<false>(act, a, stream);
}

}  // namespace moe
