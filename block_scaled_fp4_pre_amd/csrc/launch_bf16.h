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

hipError_t launch_bf16_split(bool gated, const Bf16Args& a, hipStream_t stream);   // bf16_split.hip
hipError_t launch_bf16_tile(bool gated, const Bf16Args& a, hipStream_t stream);    // bf16_tile.hip
inline hipError_t launch_linear_bf16(bool gated, const Bf16Args& a, hipStream_t stream) {
  const int64_t rows = a.offsets != nullptr ? (a.T + a.E - 1) / a.E : a.T;
  return rows > 64 ? launch_bf16_tile(gated, a, stream) : launch_bf16_split(gated, a, stream);
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
  float scale, eps, g;
};
hipError_t launch_post_norm(int act, bool res_f32, const PostNormArgs& a, hipStream_t stream);

}  // namespace moe
