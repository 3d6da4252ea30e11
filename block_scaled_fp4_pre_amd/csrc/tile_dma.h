// Pieces shared by the tile kernels that keep rings of direct-to-LDS copies in flight
// (linear_tile.hip, bf16_tile.hip).
#pragma once
#include "device_common.h"

namespace moe {

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// The 16 (4) bytes at base + voff of lane l go to LDS byte address lds + 16*l
// (4*l); base and lds are the wave's own (scalar).  M0 carries the LDS address; a
// DMA right after a scalar write of M0 needs one wait state, which the compiler
// cannot insert inside an asm statement.
__device__ __forceinline__ void dma16(const uint8_t* base, int voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(voff), "s"(base), "s"(lds) : "memory", "m0");
}
// The same for bytes that are read once: past the caches as far as they let it.
__device__ __forceinline__ void dma16_once(const uint8_t* base, int voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1 nt" ::"v"(voff), "s"(base), "s"(lds) : "memory", "m0");
}
__device__ __forceinline__ void dma4(const uint8_t* base, int voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1" ::"v"(voff), "s"(base), "s"(lds) : "memory", "m0");
}
#pragma clang diagnostic pop

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

}  // namespace moe
