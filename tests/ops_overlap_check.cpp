// Buffers of the operators around the layer that share an address where they may
// not, and those that may (block_scaled_fp4_pre_amd/csrc/validate.cpp), built for
// the host by tests/test_abi_ops_cpu.py.  Prints a line per failed expectation
// and "<cases> cases, <n> failed".
#include <stdint.h>
#include <stdio.h>

#include "validate.h"

namespace {

int g_cases = 0, g_fail = 0;

void expect(int got, int want, const char* what) {
  ++g_cases;
  if (got != want) {
    ++g_fail;
    printf("FAIL %s: got %d want %d\n", what, got, want);
  }
}

const void* P(uintptr_t a) { return reinterpret_cast<const void*>(a); }

struct Norm {
  int32_t mma = MOE_MMA_FP8_X_MXF4, res = 0, w = 0;
  const void *x = P(0x100000), *residual = P(0x200000), *weight = P(0x300000), *residual_out = P(0x400000),
             *y = P(0x500000), *codes = P(0x600000), *scales = P(0x700000);
  int operator()() {
    bool noop = false;
    return moe::check_norm_args(mma, res, w, 4, 64, x, residual, weight, 1e-6f, 1.0f, residual_out, y, codes, scales,
                                &noop);
  }
};
#define NORM(set, want) do { Norm a; set; expect(a(), want, "norm: " #set); } while (0)

void norm() {
  NORM(a.scales = a.codes, MOE_EINVAL);
  NORM(a.scales = a.y, MOE_EINVAL);
  NORM(a.scales = a.residual_out, MOE_EINVAL);
  NORM(a.scales = a.x, MOE_EINVAL);
  NORM(a.scales = a.residual, MOE_EINVAL);
  NORM(a.scales = a.weight, MOE_EINVAL);
  NORM(a.codes = a.weight, MOE_EINVAL);
  NORM(a.codes = a.y, MOE_EINVAL);
  NORM(a.y = a.weight, MOE_EINVAL);
  NORM(a.y = a.weight; a.w = 1, MOE_EINVAL);
  NORM(a.residual_out = a.weight, MOE_EINVAL);
  // a float32 row lies over two bfloat16 ones
  NORM(a.residual_out = a.x; a.res = 1, MOE_EINVAL);
  NORM(a.y = a.residual; a.res = 1, MOE_EINVAL);
  NORM(a.y = a.residual; a.res = 1; a.codes = a.scales = nullptr, MOE_EINVAL);
  // element by element in place: one thread reads what it writes
  NORM(a.residual_out = a.x, MOE_OK);
  NORM(a.residual_out = a.residual, MOE_OK);
  NORM(a.residual_out = a.residual; a.res = 1, MOE_OK);
  NORM(a.y = a.x, MOE_OK);
  NORM(a.y = a.residual, MOE_OK);
  NORM(a.x = a.residual, MOE_OK);
  // no scales, no residual: nothing to compare with
  NORM(a.codes = a.scales = nullptr, MOE_OK);
  NORM(a.y = nullptr; a.residual = a.residual_out = nullptr, MOE_OK);
}

struct Linear {
  moe_w4a4_linear_cfg c{96, 100, 70, MOE_MMA_MXF4_X_MXF4};
  const void *prepared = P(0x1000000), *x = nullptr, *xq = P(0x2000000), *xsf = P(0x3000000), *addend = nullptr,
             *out = P(0x5000000), *workspace = P(0x6000000);
  int operator()() {
    bool noop = false;
    return moe::check_linear_args(&c, prepared, 70, x, xq, xsf, addend, 0, out, workspace, (size_t)1 << 30, &noop);
  }
};
#define LINEAR(set, want) do { Linear a; set; expect(a(), want, "linear: " #set); } while (0)

void linear() {
  LINEAR(, MOE_OK);
  LINEAR(a.out = a.xq, MOE_EINVAL);
  LINEAR(a.out = a.xsf, MOE_EINVAL);
  LINEAR(a.out = a.prepared, MOE_EINVAL);
  LINEAR(a.out = a.workspace, MOE_EINVAL);
  LINEAR(a.x = a.out; a.xq = a.xsf = nullptr, MOE_EINVAL);
  LINEAR(a.addend = a.out, MOE_OK);
}

}  // namespace

int main(int argc, char** argv) {
  if (argc > 1 && argv[1][0] == 'l')
    linear();
  else
    norm();
  printf("%d cases, %d failed\n", g_cases, g_fail);
  return g_fail != 0;
}
