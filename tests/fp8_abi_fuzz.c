/* Random and limit-value arguments through the host side of the FP8 and balance-loss entry points.
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
    int64_t rows = size64();
    REFUSED(moe_quantize_fp8(NULL, size32(), rows ? rows : 1, size64(), ptr(), ptr(), 0));
    REFUSED(moe_quantize_fp8_weights(NULL, size32(), size32(), size32(), size32(), ptr(), ptr(), ptr(), ptr(), 0));
    REFUSED(moe_quantize_fp8_tokens(ptr(), size32(), size64(), ptr(), NULL, size32(), size64(), size64(), ptr(), ptr(), 0));
    seen += (size_t)moe_fp8_token_blocks(size64(), size32());
    moe_gemm_fp8_args g;
    memset(&g, 0, sizeof g);
    g.A = ptr(), g.A_sf = ptr(), g.A_rows = ptr(), g.rows_A = size64(), g.B = ptr(), g.B_sf = ptr(), g.expert_offsets = ptr();
    g.E = size32(), g.N = size32(), g.K = size32(), g.epilogue = size32(), g.R = size64(), g.D = ptr(), g.D_sf = ptr();
    seen += moe_grouped_gemm_fp8_can_implement(&g) == MOE_OK;
    g.B = NULL;
    REFUSED(moe_grouped_gemm_fp8(&g, 0));
    moe_wgrad_fp8_args w;
    memset(&w, 0, sizeof w);
    w.Y = ptr(), w.Y_sf = ptr(), w.X = ptr(), w.X_sf = ptr(), w.expert_offsets = ptr(), w.E = size32(), w.N = size32();
    w.K = size32(), w.D_dtype = size32(), w.R = size64(), w.D = ptr();
    seen += moe_grouped_wgrad_fp8_can_implement(&w) == MOE_OK;
    w.D = NULL;
    REFUSED(moe_grouped_wgrad_fp8(&w, 0));
    const int T = size32(), E = size32(), k = size32(), S = size32();
    const size_t ws = moe_balance_loss_workspace(T, E, k, S);
    seen += ws != 0;
    REFUSED(moe_balance_loss(ptr(), ptr(), T, E, k, ptr(), S, ptr(), ptr(), ptr(), ptr(), ptr(), ws ? ws - 1 : 0, 0));
    REFUSED(moe_balance_loss_backward(ptr(), T, E, ptr(), S, ptr(), NULL, ptr(), ptr(), ptr(), ptr(), k, ptr(), 0));
  }
  printf("ok %zu\n", seen);
  return 0;
}
