// Every argument check of the bfloat16 operators (linear, grouped linear, experts, norm
// after a block; block_scaled_fp4_pre_amd/csrc/validate_bf16.cpp), built for the host under the
// address and undefined-behaviour sanitizers by tests/test_abi_bf16_cpu.py.
// Prints a line per failed expectation and "<cases> cases, <n> failed".
#include <math.h>
#include <stdio.h>

#include "validate.h"

namespace {

int g_cases = 0, g_fail = 0;
void expect(int got, int want, const char* what, int line) {
  ++g_cases;
  if (got != want) {
    ++g_fail;
    printf("FAIL line %d: %s: got %d want %d\n", line, what, got, want);
  }
}
const void* P(uintptr_t a) { return reinterpret_cast<const void*>(a); }

struct Linear {
  int64_t T = 4;
  int32_t K = 64, N = 30;
  const void* x = P(0x100000);
  int64_t ldx = 64;
  const void* w = P(0x200000);
  int32_t fn = MOE_FN_SILU, gated = 1, bias_t = 1;
  const void *bias = P(0x300000), *scale = P(0x400000);
  int32_t add_t = 0;
  const void* add = P(0x500000);
  int64_t lda = 30;
  int32_t out_t = 0;
  const void* out = P(0x600000);
  int64_t ldo = 30;
  bool noop = false;
  int operator()() {
    return moe::check_linear_bf16_args(T, K, N, x, ldx, w, fn, gated, bias_t, bias, scale, add_t, add, lda, out_t, out,
                                       ldo, &noop);
  }
};
struct Grouped : Linear {
  int32_t E = 3;
  const void* offsets = P(0x700000);
  int64_t x_rows = 4;
  const void* rows = nullptr;
  int32_t div = 1;
  int operator()() {
    return moe::check_grouped_bf16_args(E, T, K, N, offsets, x, x_rows, ldx, rows, div, w, fn, gated, bias_t, bias, scale,
                                        add_t, add, lda, out_t, out, ldo, &noop);
  }
};
struct Experts {
  moe_w4a4_experts_bf16_cfg c{64, 32, 8, 2, 16, MOE_FN_SILU};
  int32_t T = 4;
  const void *w1 = P(0x100000), *w2 = P(0x200000), *x = P(0x300000), *ids = P(0x400000), *tw = P(0x500000),
             *out = P(0x600000), *ws = P(0x700000);
  size_t bytes = (size_t)1 << 30;
  bool noop = false;
  int operator()() {
    return moe::check_experts_bf16_args(&c, w1, w2, T, x, ids, tw, out, ws, bytes, &noop);
  }
};
struct Post {
  int32_t mma = MOE_MMA_FP8_X_MXF4, res = 0, w = 0, gate_t = 0, kind = MOE_GATE_FULL;
  int64_t rows = 4;
  int32_t cols = 64;
  const void *x = P(0x100000), *r = P(0x200000), *pw = P(0x300000), *gate = P(0x400000);
  float scale = 1.0f;
  const void* nw = P(0x500000);
  float eps = 1e-6f, g = 1.0f;
  const void *ro = P(0x600000), *y = P(0x700000), *codes = P(0x800000), *scales = P(0x900000);
  bool noop = false;
  int operator()() {
    return moe::check_post_norm_args(mma, res, w, gate_t, kind, rows, cols, x, r, pw, gate, scale, nw, eps, g, ro, y,
                                     codes, scales, &noop);
  }
};
#define CASE(T, set, want) do { T a; set; expect(a(), want, #T ": " #set, __LINE__); } while (0)
#define NOOP(T, set) do { T a; set; expect(a(), MOE_OK, #T ": " #set, __LINE__); expect(a.noop, 1, #T " noop: " #set, __LINE__); } while (0)

template <class L>
void product() {
  CASE(L, , MOE_OK);
  CASE(L, a.bias = a.scale = a.add = nullptr, MOE_OK);
  CASE(L, a.add = nullptr; a.lda = 0, MOE_OK);
  CASE(L, a.T = -1, MOE_EINVAL);
  CASE(L, a.K = 0, MOE_EINVAL);
  CASE(L, a.K = -8, MOE_EINVAL);
  CASE(L, a.N = 0, MOE_EINVAL);
  CASE(L, a.K = 60, MOE_EUNSUPPORTED);
  CASE(L, a.K = 65544; a.ldx = 65544, MOE_EUNSUPPORTED);
  CASE(L, a.K = 65536; a.ldx = 65536, MOE_OK);
  CASE(L, a.N = (1 << 20) + 1; a.ldo = a.lda = 1 << 21, MOE_EUNSUPPORTED);
  CASE(L, a.fn = 5, MOE_EUNSUPPORTED);
  CASE(L, a.fn = -1, MOE_EUNSUPPORTED);
  CASE(L, a.gated = 2, MOE_EUNSUPPORTED);
  CASE(L, a.bias_t = 2, MOE_EUNSUPPORTED);
  CASE(L, a.add_t = -1, MOE_EUNSUPPORTED);
  CASE(L, a.out_t = 2, MOE_EUNSUPPORTED);
  CASE(L, a.x = nullptr, MOE_EINVAL);
  CASE(L, a.w = nullptr, MOE_EINVAL);
  CASE(L, a.out = nullptr, MOE_EINVAL);
  CASE(L, a.x = P(0x100008), MOE_EINVAL);
  CASE(L, a.w = P(0x200008), MOE_EINVAL);
  CASE(L, a.out = P(0x600001), MOE_EINVAL);
  CASE(L, a.out = P(0x600002), MOE_OK);
  CASE(L, a.out = P(0x600002); a.out_t = 1, MOE_EINVAL);
  CASE(L, a.bias = P(0x300002), MOE_EINVAL);
  CASE(L, a.bias = P(0x300002); a.bias_t = 0, MOE_OK);
  CASE(L, a.scale = P(0x400002), MOE_EINVAL);
  CASE(L, a.add = P(0x500001), MOE_EINVAL);
  CASE(L, a.ldx = 63, MOE_EINVAL);
  CASE(L, a.ldx = 65, MOE_EUNSUPPORTED);
  CASE(L, a.ldx = 72, MOE_OK);
  CASE(L, a.ldo = 29, MOE_EINVAL);
  CASE(L, a.ldo = 31, MOE_OK);
  CASE(L, a.lda = 29, MOE_EINVAL);
  CASE(L, a.ldx = (1 << 22) + 8, MOE_EUNSUPPORTED);
  CASE(L, a.ldo = (1 << 22) + 1, MOE_EUNSUPPORTED);
  CASE(L, a.lda = (1 << 22) + 1, MOE_EUNSUPPORTED);
  CASE(L, a.out = a.x, MOE_EINVAL);
  CASE(L, a.out = a.w, MOE_EINVAL);
  CASE(L, a.out = a.bias, MOE_EINVAL);
  CASE(L, a.out = a.scale, MOE_EINVAL);
  CASE(L, a.out = a.add, MOE_OK);
  CASE(L, a.out = a.add; a.out_t = 1, MOE_EINVAL);
  CASE(L, a.out = a.add; a.ldo = 32, MOE_EINVAL);
  NOOP(L, a.T = 0);
  NOOP(L, a.T = 0; a.x = a.w = a.out = nullptr);
}

void post() {
  CASE(Post, , MOE_OK);
  CASE(Post, a.res = 2, MOE_EUNSUPPORTED);
  CASE(Post, a.w = 2, MOE_EUNSUPPORTED);
  CASE(Post, a.gate_t = 2, MOE_EUNSUPPORTED);
  CASE(Post, a.kind = 4, MOE_EUNSUPPORTED);
  CASE(Post, a.kind = -1, MOE_EUNSUPPORTED);
  CASE(Post, a.rows = -1, MOE_EINVAL);
  CASE(Post, a.rows = (int64_t)1 << 31, MOE_EUNSUPPORTED);
  CASE(Post, a.cols = 0, MOE_EINVAL);
  CASE(Post, a.cols = 48, MOE_EUNSUPPORTED);
  CASE(Post, a.cols = 65568, MOE_EUNSUPPORTED);
  CASE(Post, a.eps = 0.0f, MOE_EINVAL);
  CASE(Post, a.eps = NAN, MOE_EINVAL);
  CASE(Post, a.scale = INFINITY, MOE_EINVAL);
  CASE(Post, a.scale = NAN, MOE_EINVAL);
  CASE(Post, a.scale = -2.0f, MOE_OK);
  CASE(Post, a.x = nullptr, MOE_EINVAL);
  CASE(Post, a.r = nullptr, MOE_EINVAL);
  CASE(Post, a.ro = nullptr, MOE_EINVAL);
  CASE(Post, a.pw = nullptr, MOE_OK);
  CASE(Post, a.gate = nullptr, MOE_EINVAL);
  CASE(Post, a.kind = MOE_GATE_NONE, MOE_EINVAL);
  CASE(Post, a.kind = MOE_GATE_NONE; a.gate = nullptr, MOE_OK);
  CASE(Post, a.nw = nullptr, MOE_EINVAL);
  CASE(Post, a.nw = a.y = a.codes = a.scales = nullptr, MOE_OK);
  CASE(Post, a.y = a.codes = a.scales = nullptr, MOE_EINVAL);
  CASE(Post, a.codes = nullptr, MOE_EINVAL);
  CASE(Post, a.scales = nullptr, MOE_EINVAL);
  CASE(Post, a.codes = a.scales = nullptr, MOE_OK);
  CASE(Post, a.y = nullptr, MOE_OK);
  CASE(Post, a.x = P(0x100008), MOE_EINVAL);
  CASE(Post, a.r = P(0x200008), MOE_EINVAL);
  CASE(Post, a.pw = P(0x300008), MOE_EINVAL);
  CASE(Post, a.nw = P(0x500008), MOE_EINVAL);
  CASE(Post, a.ro = P(0x600008), MOE_EINVAL);
  CASE(Post, a.y = P(0x700008), MOE_EINVAL);
  CASE(Post, a.codes = P(0x800008), MOE_EINVAL);
  CASE(Post, a.scales = P(0x900001), MOE_OK);
  CASE(Post, a.gate = P(0x400002), MOE_EINVAL);
  CASE(Post, a.gate = P(0x400002); a.kind = MOE_GATE_ROW, MOE_OK);
  CASE(Post, a.gate = P(0x400002); a.kind = MOE_GATE_ROW; a.gate_t = 1, MOE_EINVAL);
  CASE(Post, a.gate = P(0x400002); a.kind = MOE_GATE_CHANNEL, MOE_EINVAL);
  CASE(Post, a.ro = a.r, MOE_OK);
  CASE(Post, a.ro = a.x, MOE_OK);
  CASE(Post, a.ro = a.x; a.res = 1, MOE_EINVAL);
  CASE(Post, a.ro = a.pw, MOE_EINVAL);
  CASE(Post, a.ro = a.nw, MOE_EINVAL);
  CASE(Post, a.ro = a.gate, MOE_EINVAL);
  CASE(Post, a.y = a.x, MOE_OK);
  CASE(Post, a.y = a.r, MOE_OK);
  CASE(Post, a.y = a.r; a.res = 1, MOE_EINVAL);
  CASE(Post, a.y = a.ro, MOE_EINVAL);
  CASE(Post, a.y = a.pw, MOE_EINVAL);
  CASE(Post, a.y = a.nw, MOE_EINVAL);
  CASE(Post, a.y = a.gate, MOE_EINVAL);
  CASE(Post, a.ro = a.y = a.x, MOE_EINVAL);
  for (int i = 0; i < 7; ++i) {
    Post a;
    const void* p[] = {a.x, a.r, a.pw, a.gate, a.nw, a.ro, a.y};
    a.codes = p[i];
    expect(a(), MOE_EINVAL, "codes in another's place", i);
    a = Post();
    a.scales = p[i];
    expect(a(), MOE_EINVAL, "scales in another's place", i);
  }
  CASE(Post, a.codes = a.scales, MOE_EINVAL);
  CASE(Post, a.mma = 3, MOE_EUNSUPPORTED);
  CASE(Post, a.mma = 3; a.codes = a.scales = nullptr, MOE_OK);
  CASE(Post, a.mma = MOE_MMA_NVF4_X_NVF4; a.g = 0.0f, MOE_EINVAL);
  CASE(Post, a.mma = MOE_MMA_NVF4_X_NVF4, MOE_OK);
  NOOP(Post, a.rows = 0);
  NOOP(Post, a.rows = 0; a.x = a.r = a.ro = nullptr);
}

}  // namespace

int main() {
  product<Linear>();
  product<Grouped>();
  CASE(Linear, a.T = 1 << 24, MOE_OK);
  CASE(Linear, a.T = (1 << 24) + 1, MOE_EUNSUPPORTED);
  CASE(Linear, a.T = 1 << 20; a.N = (1 << 16) + 1; a.ldo = a.lda = a.N, MOE_EUNSUPPORTED);
  CASE(Grouped, a.E = 0, MOE_EINVAL);
  CASE(Grouped, a.E = 513, MOE_EUNSUPPORTED);
  CASE(Grouped, a.E = 512, MOE_OK);
  CASE(Grouped, a.E = 512; a.N = a.ldo = a.lda = 32769, MOE_EUNSUPPORTED);
  CASE(Grouped, a.div = 0, MOE_EINVAL);
  CASE(Grouped, a.offsets = nullptr, MOE_EINVAL);
  CASE(Grouped, a.offsets = P(0x700002), MOE_EINVAL);
  CASE(Grouped, a.x_rows = 3, MOE_EINVAL);
  CASE(Grouped, a.x_rows = 0, MOE_EINVAL);
  CASE(Grouped, a.x_rows = 0; a.T = 0, MOE_OK);
  CASE(Grouped, a.x_rows = 2; a.rows = P(0x800000), MOE_OK);
  CASE(Grouped, a.x_rows = 2; a.rows = P(0x800002), MOE_EINVAL);
  CASE(Grouped, a.x_rows = 1 << 24; a.rows = P(0x800000); a.ldx = 128, MOE_EUNSUPPORTED);
  CASE(Grouped, a.x_rows = (1 << 24) - 1; a.rows = P(0x800000); a.ldx = 128, MOE_OK);
  CASE(Grouped, a.x_rows = 1 << 24; a.ldx = 128, MOE_OK);
  CASE(Grouped, a.x_rows = (1 << 24) + 1, MOE_EUNSUPPORTED);
  CASE(Grouped, a.out = a.offsets, MOE_EINVAL);
  CASE(Grouped, a.rows = a.out, MOE_EINVAL);

  CASE(Experts, , MOE_OK);
  CASE(Experts, a.c.hidden = 60, MOE_EUNSUPPORTED);
  CASE(Experts, a.c.inter = 20, MOE_EUNSUPPORTED);
  CASE(Experts, a.c.hidden = 0, MOE_EINVAL);
  CASE(Experts, a.c.num_experts = 513, MOE_EUNSUPPORTED);
  CASE(Experts, a.c.topk = 17, MOE_EUNSUPPORTED);
  CASE(Experts, a.c.topk = 0, MOE_EINVAL);
  CASE(Experts, a.c.max_tokens = -1, MOE_EINVAL);
  CASE(Experts, a.c.max_tokens = (1 << 23) + 1, MOE_EUNSUPPORTED);
  CASE(Experts, a.c.hidden = 65536; a.c.max_tokens = 32768, MOE_EUNSUPPORTED);
  CASE(Experts, a.c.hidden = 65536; a.c.num_experts = 257, MOE_EUNSUPPORTED);
  CASE(Experts, a.c.function = 5, MOE_EUNSUPPORTED);
  CASE(Experts, a.T = -1, MOE_EINVAL);
  CASE(Experts, a.T = 17, MOE_ECAPACITY);
  NOOP(Experts, a.T = 0; a.w1 = a.x = a.ws = nullptr);
  CASE(Experts, a.w1 = nullptr, MOE_EINVAL);
  CASE(Experts, a.w2 = P(0x200008), MOE_EINVAL);
  CASE(Experts, a.x = nullptr, MOE_EINVAL);
  CASE(Experts, a.ids = P(0x400002), MOE_EINVAL);
  CASE(Experts, a.tw = nullptr, MOE_EINVAL);
  CASE(Experts, a.out = P(0x600008), MOE_EINVAL);
  CASE(Experts, a.out = a.x, MOE_OK);
  CASE(Experts, a.out = a.w1, MOE_EINVAL);
  CASE(Experts, a.out = a.tw, MOE_EINVAL);
  CASE(Experts, a.ws = a.out, MOE_EINVAL);
  CASE(Experts, a.ws = a.x, MOE_EINVAL);
  CASE(Experts, a.ws = P(0x700080), MOE_EINVAL);
  CASE(Experts, a.bytes = moe::experts_bf16_layout(&a.c).total - 1, MOE_EWORKSPACE);
  CASE(Experts, a.bytes = moe::experts_bf16_layout(&a.c).total, MOE_OK);
  post();
  printf("%d cases, %d failed\n", g_cases, g_fail);
  return g_fail != 0;
}
