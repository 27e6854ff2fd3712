// Host side of the FP8 and balance-loss entry points declared in moe_nvfp4.h: argument
// validation (before any HIP call) and the launches on the caller's stream.  No entry point
// allocates, synchronises or throws.
#include "balance_loss.hpp"
#include "fp8_gemm.hpp"
#include "fp8_round.hpp"
#include "groups.hpp"

namespace moe {
namespace {

// A launch has fewer than 2^32 threads, all here at most 256 for each item counted below.  Row
// numbers, and the rows past a tile's end, stay in 31 bits.
constexpr int64_t kMaxItems = (int64_t(1) << 24) - 8;
constexpr int64_t kMaxRows = int64_t(1) << 30;
constexpr int64_t kMaxRowBlocks = int64_t(1) << 28;   // of the row quantiser: 16 threads each
constexpr int kMaxTokens = 1 << 26;                   // of the balance term: 32 threads each
constexpr int kMaxFp8Dim = 1 << 20;   // N, K, C: byte offsets inside a tile stay in 32 bits

bool known_dtype(int d) { return d == MOE_DTYPE_BF16 || d == MOE_DTYPE_F32; }
int64_t blocks_of(int64_t n) { return (n + kFp8Block - 1) / kFp8Block; }

// Sizes that both products share.
moe_status check_product(int32_t E, int32_t N, int32_t K, int64_t R) {
  if (E < 1 || E > 1024 || N < 1 || K < 1 || R < 0 || R >= int64_t(1) << 31) return MOE_ERR_SHAPE;
  if (R > kMaxRows || N % 16 != 0 || K % 16 != 0 || N > kMaxFp8Dim || K > kMaxFp8Dim) return MOE_ERR_UNSUPPORTED;
  // one expert's operand is addressed through a 32-bit range-checked descriptor
  if (static_cast<int64_t>(N) * K > kMaxPackedBufBytes) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int epilogue_of(const moe_gemm_fp8_args *a) { return a->epilogue & ~MOE_SUMS_WHOLE; }

moe_status check_gemm_fp8(const moe_gemm_fp8_args *a, bool need_pointers) {
  if (a == nullptr) return MOE_ERR_NULL;
  const moe_status st = check_product(a->E, a->N, a->K, a->R);
  if (st != MOE_OK) return st;
  if (a->rows_A < 0 || (a->R > 0 && a->rows_A < 1)) return MOE_ERR_SHAPE;
  const int epilogue = epilogue_of(a);
  if (epilogue != MOE_EPI_NONE && epilogue != MOE_EPI_SWIGLU_FP8) return MOE_ERR_UNSUPPORTED;
  if (epilogue == MOE_EPI_SWIGLU_FP8 && a->N % (2 * kFp8Block) != 0) return MOE_ERR_UNSUPPORTED;
  // without a gather map row p of A is permuted row p; with one, all of A sits behind one descriptor
  if (a->A_rows == nullptr && a->rows_A < a->R) return MOE_ERR_SHAPE;
  if (a->A_rows != nullptr && a->rows_A > kMaxPackedBufBytes / a->K) return MOE_ERR_UNSUPPORTED;
  // the tiles of large calls: 64 x 128 by 256 threads, or more elements per thread
  if (groups::max_chunks(a->R, a->E, 64) * blocks_of(a->N) >= kMaxItems) return MOE_ERR_UNSUPPORTED;
  if (need_pointers) {
    if (!a->B || !a->B_sf || !a->expert_offsets) return MOE_ERR_NULL;
    if (a->R > 0 && (!a->A || !a->A_sf || !a->D)) return MOE_ERR_NULL;
    if (epilogue == MOE_EPI_SWIGLU_FP8 && a->R > 0 && !a->D_sf) return MOE_ERR_NULL;
  }
  return MOE_OK;
}

moe_status check_wgrad_fp8(const moe_wgrad_fp8_args *a) {
  if (a == nullptr) return MOE_ERR_NULL;
  const moe_status st = check_product(a->E, a->N, a->K, a->R);
  if (st != MOE_OK) return st;
  if (!known_dtype(a->D_dtype)) return MOE_ERR_UNSUPPORTED;
  if (a->E * blocks_of(a->N) * blocks_of(a->K) >= kMaxItems) return MOE_ERR_UNSUPPORTED;
  if (!a->expert_offsets || !a->D) return MOE_ERR_NULL;
  if (a->R > 0 && (!a->Y || !a->Y_sf || !a->X || !a->X_sf)) return MOE_ERR_NULL;
  return MOE_OK;
}

moe_status check_balance(int T, int E, int k, bool has_offsets, int S) {
  if (T < 0 || E < 1 || E > 1024 || k < 1 || k > 32 || k > E || S < 1 || S > 65536) return MOE_ERR_SHAPE;
  if (T > kMaxTokens || static_cast<int64_t>(T) * k >= int64_t(1) << 31) return MOE_ERR_SHAPE;
  if (!has_offsets && S != 1) return MOE_ERR_NULL;
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_quantize_fp8(const void *x, int x_dtype, int64_t rows, int64_t C, uint8_t *q, float *sf,
                            hipStream_t stream) {
  if (rows < 0 || C < 16 || C % 16 != 0) return MOE_ERR_SHAPE;
  if (!known_dtype(x_dtype)) return MOE_ERR_UNSUPPORTED;
  if (C > kMaxFp8Dim || (rows > 0 && blocks_of(C) > (kMaxRowBlocks - 1) / rows)) return MOE_ERR_UNSUPPORTED;
  if (rows > 0 && (!x || !q || !sf)) return MOE_ERR_NULL;
  return launch_status(launch_quantize_fp8(x, x_dtype, rows, static_cast<int>(C), q, sf, stream));
}

moe_status moe_quantize_fp8_weights(const void *w, int w_dtype, int E, int N, int K, uint8_t *q, float *sf, uint8_t *qt,
                                    float *sft, hipStream_t stream) {
  if (E < 1 || E > 1024 || N < 1 || K < 1) return MOE_ERR_SHAPE;
  if (!known_dtype(w_dtype) || N % 16 != 0 || K % 16 != 0 || N > kMaxFp8Dim || K > kMaxFp8Dim) return MOE_ERR_UNSUPPORTED;
  if (E * blocks_of(N) * blocks_of(K) >= kMaxItems) return MOE_ERR_UNSUPPORTED;
  if (!w || !q || !sf || (qt == nullptr) != (sft == nullptr)) return MOE_ERR_NULL;
  return launch_status(launch_quantize_fp8_weights(w, w_dtype, E, N, K, q, sf, qt, sft, stream));
}

int64_t moe_fp8_token_blocks(int64_t R, int E) {
  if (R < 0 || R > kMaxRows || E < 1 || E > 1024) return 0;
  return groups::max_chunks(R, E, kFp8Block);
}

moe_status moe_quantize_fp8_tokens(const void *x, int x_dtype, int64_t rows_x, const int32_t *rows,
                                   const int32_t *expert_offsets, int E, int64_t R, int64_t C, uint8_t *q, float *sf,
                                   hipStream_t stream) {
  if (E < 1 || E > 1024 || R < 0 || R >= int64_t(1) << 31 || C < 16 || C % 16 != 0 || rows_x < 0) return MOE_ERR_SHAPE;
  if (R > 0 && (rows_x < 1 || (rows == nullptr && rows_x < R))) return MOE_ERR_SHAPE;
  if (!known_dtype(x_dtype) || C > kMaxFp8Dim || R > kMaxRows) return MOE_ERR_UNSUPPORTED;
  if (groups::max_chunks(R, E, kFp8Block) * blocks_of(C) >= kMaxItems) return MOE_ERR_UNSUPPORTED;
  if (!expert_offsets || (R > 0 && (!x || !q || !sf))) return MOE_ERR_NULL;
  return launch_status(launch_quantize_fp8_tokens(x, x_dtype, rows_x, rows, expert_offsets, E, R, static_cast<int>(C), q,
                                                  sf, stream));
}

moe_status moe_grouped_gemm_fp8_can_implement(const moe_gemm_fp8_args *args) { return check_gemm_fp8(args, true); }

moe_status moe_grouped_gemm_fp8(const moe_gemm_fp8_args *args, hipStream_t stream) {
  const moe_status st = check_gemm_fp8(args, true);
  if (st != MOE_OK) return st;
  fp8::GemmParams p = {};
  p.A = args->A;
  p.A_sf = args->A_sf;
  p.A_rows = args->A_rows;
  p.rows_A = args->rows_A;
  p.B = args->B;
  p.B_sf = args->B_sf;
  p.offsets = args->expert_offsets;
  p.E = args->E;
  p.N = args->N;
  p.K = args->K;
  p.R = static_cast<int>(args->R);
  p.D = args->D;
  p.D_sf = args->D_sf;
  return launch_status(fp8::launch_gemm(p, epilogue_of(args) == MOE_EPI_SWIGLU_FP8, (args->epilogue & MOE_SUMS_WHOLE) != 0, stream));
}

moe_status moe_grouped_wgrad_fp8_can_implement(const moe_wgrad_fp8_args *args) { return check_wgrad_fp8(args); }

moe_status moe_grouped_wgrad_fp8(const moe_wgrad_fp8_args *args, hipStream_t stream) {
  const moe_status st = check_wgrad_fp8(args);
  if (st != MOE_OK) return st;
  fp8::WgradParams p = {};
  p.Y = args->Y;
  p.X = args->X;
  p.Y_sf = args->Y_sf;
  p.X_sf = args->X_sf;
  p.offsets = args->expert_offsets;
  p.E = args->E;
  p.N = args->N;
  p.K = args->K;
  p.R = static_cast<int>(args->R);
  p.blocks = static_cast<int>(groups::max_chunks(args->R, args->E, kFp8Block));
  p.D = args->D;
  return launch_status(fp8::launch_wgrad(p, args->D_dtype == MOE_DTYPE_BF16, stream));
}

size_t moe_balance_loss_workspace(int T, int E, int k, int S) {
  if (check_balance(T, E, k, true, S) != MOE_OK) return 0;
  return balance::loss_ws_bytes(T, E, S);
}

moe_status moe_balance_loss(const float *logits, const int32_t *topk_ids, int T, int E, int k, const int32_t *seq_offsets,
                            int S, const uint8_t *token_mask, int32_t *counts, float *coef, float *loss, void *ws,
                            size_t ws_bytes, hipStream_t stream) {
  const moe_status st = check_balance(T, E, k, seq_offsets != nullptr, S);
  if (st != MOE_OK) return st;
  if (!counts || !coef || !loss || (T > 0 && (!logits || !topk_ids))) return MOE_ERR_NULL;
  if (!ws || reinterpret_cast<uintptr_t>(ws) % 16 != 0 || ws_bytes < balance::loss_ws_bytes(T, E, S)) return MOE_ERR_WORKSPACE;
  balance::LossParams p = {};
  p.logits = logits;
  p.ids = topk_ids;
  p.seq_offsets = seq_offsets;
  p.mask = token_mask;
  p.T = T;
  p.E = E;
  p.k = k;
  p.S = S;
  p.counts = counts;
  p.coef = coef;
  p.loss = loss;
  return launch_status(balance::launch_loss(p, ws, stream));
}

moe_status moe_balance_loss_backward(const float *logits, int T, int E, const int32_t *seq_offsets, int S,
                                     const uint8_t *token_mask, const float *coef, const float *grad_loss,
                                     const int32_t *topk_ids, const float *topk_w, const float *d_topk_w, int k,
                                     float *dlogits, hipStream_t stream) {
  const moe_status st = check_balance(T, E, d_topk_w ? k : 1, seq_offsets != nullptr, S);
  if (st != MOE_OK) return st;
  if (!coef || !grad_loss || (T > 0 && (!logits || !dlogits))) return MOE_ERR_NULL;
  if (d_topk_w && T > 0 && (!topk_ids || !topk_w)) return MOE_ERR_NULL;
  balance::GradParams p = {};
  p.logits = logits;
  p.seq_offsets = seq_offsets;
  p.mask = token_mask;
  p.T = T;
  p.E = E;
  p.k = k;
  p.S = S;
  p.coef = coef;
  p.grad_loss = grad_loss;
  p.ids = topk_ids;
  p.topk_w = topk_w;
  p.d_topk_w = d_topk_w;
  p.dlogits = dlogits;
  return launch_status(balance::launch_backward(p, stream));
}

}  // extern "C"
