// Every argument check of the operators around the layer (norm, router,
// linear; block_scaled_fp4_pre_amd/csrc/validate.cpp), built for the host under
// the address and undefined-behaviour sanitizers by tests/test_abi_ops_cpu.py.
// Prints a line per failed expectation and "<cases> cases, <n> failed".
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "validate.h"

namespace {

int g_cases = 0, g_fail = 0;

void expect(int got, int want, int line) {
  ++g_cases;
  if (got != want) {
    ++g_fail;
    printf("FAIL line %d: got %d want %d\n", line, got, want);
  }
}
#define EXPECT(call, want) expect((call), (want), __LINE__)

const void* P(uintptr_t a) { return reinterpret_cast<const void*>(a); }
const void* const A = P(uintptr_t(1) << 20);

struct Norm {
  int32_t mma = MOE_MMA_FP8_X_MXF4, res = 0, w = 0;
  int64_t rows = 4;
  int32_t cols = 64;
  const void *x = P(0x100000), *residual = P(0x200000), *weight = P(0x300000);
  float eps = 1e-6f, g = 1.0f;
  const void *residual_out = P(0x400000), *y = P(0x500000), *codes = P(0x600000), *scales = P(0x700000);
  bool noop = false;
  int operator()() {
    return moe::check_norm_args(mma, res, w, rows, cols, x, residual, weight, eps, g, residual_out, y, codes, scales,
                                &noop);
  }
};
#define NORM(set, want) do { Norm a; set; EXPECT(a(), want); } while (0)

void norm() {
  NORM(, MOE_OK);
  NORM(a.res = 2, MOE_EUNSUPPORTED);
  NORM(a.w = -1, MOE_EUNSUPPORTED);
  NORM(a.rows = -1, MOE_EINVAL);
  NORM(a.rows = (int64_t)1 << 31, MOE_EUNSUPPORTED);
  NORM(a.cols = 0, MOE_EINVAL);
  NORM(a.cols = 48, MOE_EUNSUPPORTED);
  NORM(a.cols = 65536, MOE_OK);
  NORM(a.cols = 65568, MOE_EUNSUPPORTED);
  NORM(a.eps = 0.0f, MOE_EINVAL);
  NORM(a.eps = -1.0f, MOE_EINVAL);
  NORM(a.eps = NAN, MOE_EINVAL);
  NORM(a.eps = INFINITY, MOE_EINVAL);
  NORM(a.x = nullptr, MOE_EINVAL);
  NORM(a.weight = nullptr, MOE_EINVAL);
  NORM(a.residual = nullptr, MOE_EINVAL);
  NORM(a.residual_out = nullptr, MOE_EINVAL);
  NORM(a.residual = a.residual_out = nullptr, MOE_OK);
  NORM(a.scales = nullptr, MOE_EINVAL);
  NORM(a.codes = nullptr, MOE_EINVAL);
  NORM(a.codes = a.scales = nullptr, MOE_OK);
  NORM(a.codes = a.scales = nullptr; a.mma = 99, MOE_OK);
  NORM(a.y = nullptr, MOE_OK);
  NORM(a.y = a.codes = a.scales = nullptr, MOE_EINVAL);
  NORM(a.mma = 3, MOE_EUNSUPPORTED);
  NORM(a.mma = MOE_MMA_NVF4_X_NVF4, MOE_OK);
  NORM(a.mma = MOE_MMA_NVF4_X_NVF4; a.g = 0.0f, MOE_EINVAL);
  NORM(a.mma = MOE_MMA_NVF4_X_NVF4; a.g = NAN, MOE_EINVAL);
  NORM(a.x = P(0x100008), MOE_EINVAL);
  NORM(a.residual = P(0x100008), MOE_EINVAL);
  NORM(a.weight = P(0x100004), MOE_EINVAL);
  NORM(a.residual_out = P(0x100002), MOE_EINVAL);
  NORM(a.y = P(0x100008), MOE_EINVAL);
  NORM(a.codes = P(0x100001), MOE_EINVAL);
  NORM(a.scales = P(0x100001), MOE_OK);
  NORM(a.residual_out = a.residual; a.y = a.x, MOE_OK);      // in place
  NORM(a.residual_out = a.x, MOE_OK);
  NORM(a.y = a.residual_out, MOE_EINVAL);
  NORM(a.codes = a.y, MOE_EINVAL);
  NORM(a.codes = a.x, MOE_EINVAL);
  NORM(a.codes = a.residual_out, MOE_EINVAL);
  NORM(a.rows = 0; a.x = a.weight = a.y = a.codes = nullptr, MOE_OK);
  Norm z;
  z.rows = 0;
  z();
  EXPECT(z.noop, 1);
}

struct Router {
  int32_t dtype = 1, scoring = MOE_SCORE_SIGMOID;
  int64_t tokens = 4;
  int32_t experts = 64, topk = 6, groups = 8, keep = 4;
  const void *logits = A, *bias = A;
  float scale = 1.0f;
  const void *ids = A, *weights = A;
  bool noop = false;
  int operator()() {
    return moe::check_router_args(dtype, scoring, tokens, experts, topk, groups, keep, logits, bias, scale, ids, weights,
                                  &noop);
  }
};
#define ROUTER(set, want) do { Router a; set; EXPECT(a(), want); } while (0)

void router() {
  ROUTER(, MOE_OK);
  ROUTER(a.dtype = 2, MOE_EUNSUPPORTED);
  ROUTER(a.scoring = 3, MOE_EUNSUPPORTED);
  ROUTER(a.scoring = -1, MOE_EUNSUPPORTED);
  ROUTER(a.tokens = -1, MOE_EINVAL);
  ROUTER(a.tokens = (int64_t)1 << 40, MOE_EUNSUPPORTED);
  ROUTER(a.experts = 0, MOE_EINVAL);
  ROUTER(a.experts = 520, MOE_EUNSUPPORTED);
  ROUTER(a.experts = 512, MOE_OK);
  ROUTER(a.topk = 0, MOE_EINVAL);
  ROUTER(a.topk = 17, MOE_EUNSUPPORTED);
  ROUTER(a.groups = 0, MOE_EINVAL);
  ROUTER(a.groups = 7, MOE_EINVAL);
  ROUTER(a.groups = 128; a.experts = 256, MOE_EUNSUPPORTED);
  ROUTER(a.groups = 64; a.keep = 6, MOE_OK);
  ROUTER(a.groups = 64; a.keep = 5, MOE_EINVAL);           // five experts for six slots
  ROUTER(a.keep = 0, MOE_EINVAL);
  ROUTER(a.keep = 9, MOE_EINVAL);
  ROUTER(a.scale = NAN, MOE_EINVAL);
  ROUTER(a.scale = INFINITY, MOE_EINVAL);
  ROUTER(a.scale = -INFINITY, MOE_EINVAL);
  ROUTER(a.scale = -2.5f, MOE_OK);
  ROUTER(a.logits = nullptr, MOE_EINVAL);
  ROUTER(a.ids = nullptr, MOE_EINVAL);
  ROUTER(a.weights = nullptr, MOE_EINVAL);
  ROUTER(a.bias = nullptr, MOE_OK);
  ROUTER(a.logits = P(0x100002), MOE_EINVAL);
  ROUTER(a.logits = P(0x100002); a.dtype = 0, MOE_OK);
  ROUTER(a.logits = P(0x100001); a.dtype = 0, MOE_EINVAL);
  ROUTER(a.bias = P(0x100002), MOE_EINVAL);
  ROUTER(a.ids = P(0x100001), MOE_EINVAL);
  ROUTER(a.weights = P(0x100002), MOE_EINVAL);
  ROUTER(a.tokens = 0; a.logits = a.ids = a.weights = nullptr, MOE_OK);
}

moe_w4a4_linear_cfg cfg() { return moe_w4a4_linear_cfg{96, 100, 70, MOE_MMA_MXF4_X_MXF4}; }
#define CFG(set, want) do { moe_w4a4_linear_cfg c = cfg(); set; EXPECT(moe::check_linear_cfg(&c), want); } while (0)

struct Linear {
  moe_w4a4_linear_cfg c = cfg();
  const void* prepared = A;
  int32_t tokens = 70;
  const void *x = A, *xq = nullptr, *xsf = nullptr, *addend = nullptr;
  int32_t dtype = 0;
  const void *out = P(0x800000), *workspace = A;
  size_t bytes = (size_t)1 << 30;
  bool noop = false;
  int operator()() {
    return moe::check_linear_args(&c, prepared, tokens, x, xq, xsf, addend, dtype, out, workspace, bytes, &noop);
  }
};
#define LINEAR(set, want) do { Linear a; set; EXPECT(a(), want); } while (0)

void linear() {
  EXPECT(moe::check_linear_cfg(nullptr), MOE_EINVAL);
  CFG(, MOE_OK);
  CFG(c.in_features = 0, MOE_EINVAL);
  CFG(c.in_features = 48, MOE_EUNSUPPORTED);
  CFG(c.in_features = 65536, MOE_OK);
  CFG(c.in_features = 65568, MOE_EUNSUPPORTED);
  CFG(c.out_features = 0, MOE_EINVAL);
  CFG(c.out_features = 1, MOE_OK);
  CFG(c.out_features = (1 << 20) + 1, MOE_EUNSUPPORTED);
  CFG(c.max_tokens = -1, MOE_EINVAL);
  CFG(c.max_tokens = 0, MOE_OK);
  CFG(c.max_tokens = (1 << 20) + 1, MOE_EUNSUPPORTED);
  CFG(c.max_tokens = 1 << 20; c.out_features = 1 << 14, MOE_OK);
  CFG(c.max_tokens = 1 << 20; c.out_features = (1 << 14) + 1, MOE_EUNSUPPORTED);
  CFG(c.mma_type = MOE_MMA_FP8_X_MXF4, MOE_OK);
  CFG(c.mma_type = MOE_MMA_NVF4_X_NVF4, MOE_EUNSUPPORTED);
  CFG(c.mma_type = 9, MOE_EUNSUPPORTED);

  moe_w4a4_linear_cfg c = cfg();                            // 1 K step, 4 units of rows and of tokens
  moe::LinearLayout L = moe::linear_layout(&c);
  EXPECT(L.prepared == 4 * (4096 + 256) && L.workspace == 4 * (4096 + 256) && L.steps == 1, 1);
  c.mma_type = MOE_MMA_FP8_X_MXF4;
  L = moe::linear_layout(&c);
  EXPECT(L.prepared == 4 * (4096 + 256) && L.workspace == 4 * (8192 + 256), 1);
  c.in_features = 65536; c.out_features = 1 << 20; c.max_tokens = 0;
  L = moe::linear_layout(&c);
  EXPECT(L.prepared == ((uint64_t)1 << 20) * 65536 / 32 * 17 && L.workspace == 0, 1);

  c = cfg();
  const size_t need = (size_t)moe::linear_layout(&c).prepared;
  EXPECT(moe::check_linear_prepare_args(&c, A, A, A, need), MOE_OK);
  EXPECT(moe::check_linear_prepare_args(&c, A, A, A, need - 1), MOE_EWORKSPACE);
  EXPECT(moe::check_linear_prepare_args(&c, nullptr, A, A, need), MOE_EINVAL);
  EXPECT(moe::check_linear_prepare_args(&c, A, nullptr, A, need), MOE_EINVAL);
  EXPECT(moe::check_linear_prepare_args(&c, A, A, nullptr, need), MOE_EINVAL);
  EXPECT(moe::check_linear_prepare_args(&c, P(0x100008), A, A, need), MOE_EINVAL);
  EXPECT(moe::check_linear_prepare_args(&c, A, P(0x100001), A, need), MOE_OK);
  EXPECT(moe::check_linear_prepare_args(&c, A, A, P(0x100080), need), MOE_EINVAL);
  EXPECT(moe::check_linear_prepare_args(nullptr, A, A, A, need), MOE_EINVAL);

  LINEAR(, MOE_OK);
  LINEAR(a.tokens = 71, MOE_ECAPACITY);
  LINEAR(a.tokens = -1, MOE_EINVAL);
  LINEAR(a.tokens = 0; a.prepared = a.x = a.out = a.workspace = nullptr; a.bytes = 0, MOE_OK);
  LINEAR(a.x = nullptr, MOE_EINVAL);
  LINEAR(a.xq = A, MOE_EINVAL);
  LINEAR(a.xsf = A, MOE_EINVAL);
  LINEAR(a.x = nullptr; a.xq = A, MOE_EINVAL);
  LINEAR(a.x = nullptr; a.xsf = A, MOE_EINVAL);
  LINEAR(a.x = nullptr; a.xq = a.xsf = A, MOE_OK);
  LINEAR(a.x = nullptr; a.xq = A; a.xsf = P(0x100001), MOE_OK);
  LINEAR(a.x = nullptr; a.xq = P(0x100008); a.xsf = A, MOE_EINVAL);
  LINEAR(a.x = P(0x100002), MOE_EINVAL);
  LINEAR(a.addend = A, MOE_OK);
  LINEAR(a.addend = P(0x100008), MOE_EINVAL);
  LINEAR(a.dtype = 1, MOE_OK);
  LINEAR(a.dtype = 2, MOE_EUNSUPPORTED);
  LINEAR(a.out = nullptr, MOE_EINVAL);
  LINEAR(a.out = P(0x100008), MOE_EINVAL);
  LINEAR(a.prepared = nullptr, MOE_EINVAL);
  LINEAR(a.prepared = P(0x100010), MOE_EINVAL);
  LINEAR(a.workspace = nullptr, MOE_EINVAL);
  LINEAR(a.workspace = P(0x100010), MOE_EINVAL);
  LINEAR(a.bytes = (size_t)moe::linear_layout(&a.c).workspace, MOE_OK);
  LINEAR(a.bytes = (size_t)moe::linear_layout(&a.c).workspace - 1, MOE_EWORKSPACE);
  LINEAR(a.c.mma_type = MOE_MMA_NVF4_X_NVF4, MOE_EUNSUPPORTED);
  const void* const B = P(uintptr_t(1) << 21);             // overlaps
  LINEAR(a.x = B; a.out = B, MOE_EINVAL);
  LINEAR(a.x = nullptr; a.xq = B; a.xsf = A; a.out = B, MOE_EINVAL);
  LINEAR(a.addend = B; a.out = B, MOE_OK);
  LINEAR(a.addend = B; a.out = B; a.dtype = 1, MOE_EINVAL);
}

}  // namespace

int main() {
  norm();
  router();
  linear();
  printf("%d cases, %d failed\n", g_cases, g_fail);
  return g_fail != 0;
}
