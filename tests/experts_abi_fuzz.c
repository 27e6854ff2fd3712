/* Random and limit-value arguments through the host side of the bf16 expert products, the gradient clipping and the single-token products.
 * No call may reach a launch: entry points that launch always miss a pointer or the workspace, and
 * the driver checks that none of them is accepted. */
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "moe_nvfp4.h"

static uint64_t s = 88172645463325252ull;
static uint64_t next(void) {
  s ^= s << 13;
  s ^= s >> 7;
  s ^= s << 17;
  return s;
}
static int64_t size64(void) {
  static const int64_t limits[] = {0, 1, -1, 15, 16, 127, 128, 129, 256, 384, 1024, 1025, 65536, 65537, 1 << 20, (1 << 20) + 16,
                                   2147483647, 2147483648ll, -2147483648ll, 1ll << 40, 9223372036854775807ll,
                                   (-9223372036854775807ll - 1)};
  switch (next() % 4) {
    case 0: return limits[next() % (sizeof limits / sizeof *limits)];
    case 1: return (int64_t)(next() % 4096) * 16;
    case 2: return (int64_t)(next() % 70000);
    default: return (int64_t)next();
  }
}
static int32_t size32(void) { return (int32_t)size64(); }
static void *ptr(void) { return next() % 8 ? (void *)0x1000 : NULL; }

#define REFUSED(call)                            \
  do {                                           \
    if ((call) == MOE_OK) {                      \
      printf("accepted: line %d\n", __LINE__);   \
      return 1;                                  \
    }                                            \
  } while (0)

int main(int argc, char **argv) {
  const long n = argc > 1 ? atol(argv[1]) : 1000;
  size_t seen = 0;
  for (long i = 0; i < n; i++) {
    moe_gemm_bf16_args g;
    memset(&g, 0, sizeof g);
    g.A = ptr(), g.A_rows = ptr(), g.rows_A = size64(), g.B = ptr(), g.expert_offsets = ptr(), g.E = size32(), g.N = size32();
    g.K = size32(), g.epilogue = next() % 4 ? (int)(next() % 6) : size32(), g.B_layout = next() % 4 ? (int)(next() % 3) : size32();
    g.R = size64(), g.D = ptr(), g.Z = ptr();
    seen += moe_grouped_gemm_bf16_can_implement(&g) == MOE_OK;
    g.B = NULL;
    REFUSED(moe_grouped_gemm_bf16(&g, 0));
    moe_wgrad_bf16_args w;
    memset(&w, 0, sizeof w);
    w.Y = ptr(), w.X = ptr(), w.X_rows = ptr(), w.rows_X = size64(), w.expert_offsets = ptr(), w.E = size32(), w.N = size32();
    w.K = size32(), w.D_dtype = size32(), w.R = size64(), w.D = ptr();
    seen += moe_grouped_wgrad_bf16_can_implement(&w) == MOE_OK;
    w.D = NULL;
    REFUSED(moe_grouped_wgrad_bf16(&w, 0));
    moe_gemv_args v;
    memset(&v, 0, sizeof v);
    v.T = next() % 2 ? (int)(next() % 100) : size32(), v.k = next() % 2 ? (int)(next() % 34) : size32();
    v.x = ptr(), v.rows_x = next() % 2 ? v.T : next() % 2 ? (int64_t)v.T * v.k : size64(), v.B = ptr(), v.B_sf = ptr(), v.B_gs = ptr();
    v.ids = ptr(), v.topk_w = ptr(), v.E = size32(), v.N = size32(), v.K = size32(), v.epilogue = (int)(next() % 6), v.B_layout = (int)(next() % 3);
    v.D = ptr();
    seen += moe_gemv_nvfp4_can_implement(&v) == MOE_OK;
    if (v.T == 0) v.T = -1;
    v.D = NULL;
    REFUSED(moe_gemv_nvfp4(&v, 0));
    moe_tensor t[8];
    memset(t, 0, sizeof t);
    const int count = next() % 4 ? (int)(next() % 9) : -(int)(next() % 3);
    for (int j = 0; j < 8; j++) {
      t[j].src = next() % 8 ? (void *)(0x1000 + next() % 4 * 2) : NULL, t[j].dst = ptr(), t[j].n = next() % 2 ? (int64_t)(next() % 100000) : size64();
      t[j].dtype = next() % 8 ? (int)(next() % 2) : size32();
    }
    const size_t ws = moe_grad_norm_workspace(t, count);
    seen += ws != 0;
    REFUSED(moe_grad_norm(t, count, ptr(), (void *)0x1000, ws ? ws - 1 : 0, 0));
    REFUSED(moe_grad_clip(t, count, NULL, 1.0f, 0));
  }
  printf("ok %zu\n", seen);
  return 0;
}
