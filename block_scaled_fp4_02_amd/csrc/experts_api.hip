// Host side of the bf16 expert products, the gradient clipping and the single-token products declared in
// moe_nvfp4.h: argument validation (before any HIP call) and the launches on the caller's stream.  No
// entry point allocates, synchronises or throws.
#include "bf16_gemm.hpp"
#include "gemv_nvfp4.hpp"
#include "grad_clip.hpp"
#include "groups.hpp"

#include <math.h>

#include <algorithm>

namespace moe {
namespace {

// A launch has fewer than 2^32 threads, here at most 256 for each item counted below.  Row numbers,
// and the rows past a tile's end, stay in 31 bits.
constexpr int64_t kMaxItems = (int64_t(1) << 24) - 8;
constexpr int64_t kMaxRows = int64_t(1) << 30;
constexpr int kMaxDim = 1 << 20;                          // N, K: byte offsets inside a tile stay in 32 bits
constexpr int64_t kMaxOperand = kMaxPackedBufBytes / 2;   // elements behind one 32-bit range-checked descriptor

bool known_dtype(int d) { return d == MOE_DTYPE_BF16 || d == MOE_DTYPE_F32; }
int64_t blocks_of(int64_t n) { return (n + 127) / 128; }

// Sizes that both products share.
moe_status check_product(int32_t E, int32_t N, int32_t K, int64_t R) {
  if (E < 1 || E > 1024 || N < 1 || K < 1 || R < 0 || R >= int64_t(1) << 31) return MOE_ERR_SHAPE;
  if (R > kMaxRows || N % 8 != 0 || K % 8 != 0 || N > kMaxDim || K > kMaxDim) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status check_gemm_bf16(const moe_gemm_bf16_args *a) {
  if (a == nullptr) return MOE_ERR_NULL;
  const moe_status st = check_product(a->E, a->N, a->K, a->R);
  if (st != MOE_OK) return st;
  if (static_cast<int64_t>(a->N) * a->K > kMaxOperand) return MOE_ERR_UNSUPPORTED;
  if (a->rows_A < 0 || (a->R > 0 && a->rows_A < 1)) return MOE_ERR_SHAPE;
  if (a->B_layout != MOE_LAYOUT_ROWMAJOR && a->B_layout != MOE_LAYOUT_TRANSPOSED) return MOE_ERR_UNSUPPORTED;
  switch (a->epilogue) {
    case MOE_EPI_NONE:
      break;
    case MOE_EPI_SWIGLU:
      if (a->B_layout != MOE_LAYOUT_ROWMAJOR || a->N % 16 != 0) return MOE_ERR_UNSUPPORTED;
      break;
    case MOE_EPI_SWIGLU_BACKWARD:
      if (a->B_layout != MOE_LAYOUT_TRANSPOSED) return MOE_ERR_UNSUPPORTED;
      break;
    default:
      return MOE_ERR_UNSUPPORTED;
  }
  // without a gather map row p of A is permuted row p; with one, all of A sits behind one descriptor
  if (a->A_rows == nullptr && a->rows_A < a->R) return MOE_ERR_SHAPE;
  if (a->A_rows != nullptr && a->rows_A > kMaxOperand / a->K) return MOE_ERR_UNSUPPORTED;
  // the smallest tiles: 16 rows by 8 columns are only taken for up to 256 of them, then 32 by 128 of 256 threads
  if (groups::max_chunks(a->R, a->E, 32) * blocks_of(a->N) >= kMaxItems) return MOE_ERR_UNSUPPORTED;
  if (!a->B || !a->expert_offsets) return MOE_ERR_NULL;
  if (a->R > 0 && (!a->A || !a->D)) return MOE_ERR_NULL;
  if (a->epilogue == MOE_EPI_SWIGLU_BACKWARD && a->R > 0 && !a->Z) return MOE_ERR_NULL;
  return MOE_OK;
}

moe_status check_wgrad_bf16(const moe_wgrad_bf16_args *a) {
  if (a == nullptr) return MOE_ERR_NULL;
  const moe_status st = check_product(a->E, a->N, a->K, a->R);
  if (st != MOE_OK) return st;
  if (!known_dtype(a->D_dtype)) return MOE_ERR_UNSUPPORTED;
  if (a->rows_X < 0 || (a->R > 0 && a->rows_X < 1)) return MOE_ERR_SHAPE;
  if (a->X_rows == nullptr && a->rows_X < a->R) return MOE_ERR_SHAPE;
  if (a->X_rows != nullptr && a->rows_X > kMaxOperand / a->K) return MOE_ERR_UNSUPPORTED;
  if (a->E * blocks_of(a->N) * blocks_of(a->K) >= kMaxItems) return MOE_ERR_UNSUPPORTED;
  if (!a->expert_offsets || !a->D) return MOE_ERR_NULL;
  if (a->R > 0 && (!a->Y || !a->X)) return MOE_ERR_NULL;
  return MOE_OK;
}

// Every tensor of the list, its dst too where only the norm is asked for: one list serves both calls.
moe_status check_tensors(const moe_tensor *tensors, int count) {
  if (count < 0 || count > 1 << 20) return MOE_ERR_SHAPE;
  if (count > 0 && tensors == nullptr) return MOE_ERR_NULL;
  int64_t total = 0;
  for (int i = 0; i < count; i++) {
    const moe_tensor &t = tensors[i];
    if (t.n < 0 || t.n > int64_t(1) << 37) return MOE_ERR_SHAPE;
    if (!known_dtype(t.dtype)) return MOE_ERR_UNSUPPORTED;
    if (t.n > 0 && !t.src) return MOE_ERR_NULL;
    const uintptr_t align = t.dtype == MOE_DTYPE_BF16 ? 2 : 4;
    if ((reinterpret_cast<uintptr_t>(t.src) | reinterpret_cast<uintptr_t>(t.dst)) % align != 0) return MOE_ERR_UNSUPPORTED;
    total += t.n;
    if (total > int64_t(1) << 37) return MOE_ERR_SHAPE;
  }
  return MOE_OK;
}

struct Range {
  uint64_t start, end;   // of bytes; the end's low bit (elements have at least two bytes): written
};

// Whether nothing that clipping writes overlaps another range that is read or written, but a src that it
// replaces.  scratch: 4 words a tensor.
bool written_apart(const moe_tensor *tensors, int count, uint64_t *scratch) {
  auto each_range = [&](auto take) {
    for (int i = 0; i < count; i++) {
      const moe_tensor &t = tensors[i];
      if (t.n == 0) continue;
      const uint64_t src = reinterpret_cast<uint64_t>(t.src), dst = t.dst ? reinterpret_cast<uint64_t>(t.dst) : src;
      const uint64_t bytes = static_cast<uint64_t>(t.n) * (t.dtype == MOE_DTYPE_BF16 ? 2 : 4);
      take(dst, dst + bytes, 1);
      if (src != dst) take(src, src + bytes, 0);
    }
  };
  // ranges are all apart where each end, in order, is no further than the next start, in order
  uint64_t *const starts = scratch, *const ends = scratch + 2 * static_cast<int64_t>(count);
  int64_t n = 0;
  each_range([&](uint64_t start, uint64_t end, int) {
    starts[n] = start;
    ends[n++] = end;
  });
  std::sort(starts, starts + n);
  std::sort(ends, ends + n);
  bool apart = true;
  for (int64_t i = 1; i < n; i++) apart &= ends[i - 1] <= starts[i];
  if (apart) return true;
  // what is only read may overlap: each range against those that start before it
  Range *const ranges = reinterpret_cast<Range *>(scratch);
  n = 0;
  each_range([&](uint64_t start, uint64_t end, int write) { ranges[n++] = {start, end | write}; });
  std::sort(ranges, ranges + n, [](const Range &a, const Range &b) { return a.start < b.start; });
  uint64_t any_end = 0, written_end = 0;
  for (int64_t i = 0; i < n; i++) {
    const uint64_t end = ranges[i].end & ~uint64_t(1);
    const bool write = ranges[i].end & 1;
    if (ranges[i].start < (write ? any_end : written_end)) return false;
    any_end = std::max(any_end, end);
    if (write) written_end = std::max(written_end, end);
  }
  return true;
}

moe_status check_gemv(const moe_gemv_args *a) {
  if (a == nullptr) return MOE_ERR_NULL;
  if (a->T < 0 || a->T > 4096 || a->k < 1 || a->k > 32 || a->E < 1 || a->E > 65536 || a->N < 1 || a->K < 1) return MOE_ERR_SHAPE;
  if (a->ids == nullptr && a->k != 1) return MOE_ERR_SHAPE;
  if (a->rows_x != a->T && a->rows_x != static_cast<int64_t>(a->T) * a->k) return MOE_ERR_SHAPE;
  if (a->N > kMaxDim || a->K > kMaxDim || a->N % 16 != 0 || a->K % 32 != 0) return MOE_ERR_UNSUPPORTED;
  if (a->B_layout != MOE_LAYOUT_ROWMAJOR && a->B_layout != MOE_LAYOUT_PACKED) return MOE_ERR_UNSUPPORTED;
  if (a->B_layout == MOE_LAYOUT_PACKED && a->K % 256 != 0) return MOE_ERR_UNSUPPORTED;
  if (a->epilogue != MOE_EPI_NONE && a->epilogue != MOE_EPI_SWIGLU && a->epilogue != MOE_EPI_FINALIZE) return MOE_ERR_UNSUPPORTED;
  if (a->epilogue == MOE_EPI_SWIGLU && a->N % 32 != 0) return MOE_ERR_UNSUPPORTED;
  if (a->T > 0 && (!a->x || !a->B || !a->B_gs || !a->D)) return MOE_ERR_NULL;
  if (a->T > 0 && a->B_layout == MOE_LAYOUT_ROWMAJOR && !a->B_sf) return MOE_ERR_NULL;
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_grouped_gemm_bf16_can_implement(const moe_gemm_bf16_args *args) { return check_gemm_bf16(args); }

moe_status moe_grouped_gemm_bf16(const moe_gemm_bf16_args *args, hipStream_t stream) {
  const moe_status st = check_gemm_bf16(args);
  if (st != MOE_OK) return st;
  bf16::GemmParams p = {};
  p.A = args->A;
  p.A_rows = args->A_rows;
  p.rows_A = args->rows_A;
  p.B = args->B;
  p.offsets = args->expert_offsets;
  p.E = args->E;
  p.N = args->N;
  p.K = args->K;
  p.R = static_cast<int>(args->R);
  p.D = args->D;
  p.Z = args->epilogue == MOE_EPI_NONE ? nullptr : args->Z;
  const bf16::Epilogue epilogue = args->epilogue == MOE_EPI_NONE     ? bf16::kPlain
                                  : args->epilogue == MOE_EPI_SWIGLU ? bf16::kGated
                                                                     : bf16::kGatedBackward;
  return launch_status(bf16::launch_gemm(p, epilogue, args->B_layout == MOE_LAYOUT_TRANSPOSED, stream));
}

moe_status moe_grouped_wgrad_bf16_can_implement(const moe_wgrad_bf16_args *args) { return check_wgrad_bf16(args); }

moe_status moe_grouped_wgrad_bf16(const moe_wgrad_bf16_args *args, hipStream_t stream) {
  const moe_status st = check_wgrad_bf16(args);
  if (st != MOE_OK) return st;
  bf16::WgradParams p = {};
  p.Y = args->Y;
  p.X = args->X;
  p.X_rows = args->R > 0 ? args->X_rows : nullptr;
  p.rows_X = args->rows_X;
  p.offsets = args->expert_offsets;
  p.E = args->E;
  p.N = args->N;
  p.K = args->K;
  p.R = static_cast<int>(args->R);
  p.D = args->D;
  return launch_status(bf16::launch_wgrad(p, args->D_dtype == MOE_DTYPE_BF16, stream));
}

size_t moe_grad_norm_workspace(const moe_tensor *tensors, int count) {
  return check_tensors(tensors, count) == MOE_OK ? grad::norm_ws_bytes(tensors, count) : 0;
}

moe_status moe_grad_norm(const moe_tensor *tensors, int count, float *norm, void *ws, size_t ws_bytes, hipStream_t stream) {
  const moe_status st = check_tensors(tensors, count);
  if (st != MOE_OK) return st;
  if (!norm) return MOE_ERR_NULL;
  if (!ws || reinterpret_cast<uintptr_t>(ws) % 16 != 0 || ws_bytes < grad::norm_ws_bytes(tensors, count)) return MOE_ERR_WORKSPACE;
  return launch_status(grad::launch_norm(tensors, count, norm, ws, stream));
}

moe_status moe_grad_clip(const moe_tensor *tensors, int count, const float *norm, float max_norm, hipStream_t stream) {
  const moe_status st = check_tensors(tensors, count);
  if (st != MOE_OK) return st;
  if (!(max_norm >= 0.0f)) return MOE_ERR_SHAPE;
  if (!norm) return MOE_ERR_NULL;
  return launch_status(grad::launch_clip(tensors, count, norm, max_norm, stream));
}

moe_status moe_grad_clip_can_implement(const moe_tensor *tensors, int count, uint64_t *scratch) {
  const moe_status st = check_tensors(tensors, count);
  if (st != MOE_OK) return st;
  if (count > 0 && !scratch) return MOE_ERR_NULL;
  return written_apart(tensors, count, scratch) ? MOE_OK : MOE_ERR_UNSUPPORTED;
}

moe_status moe_gemv_nvfp4_can_implement(const moe_gemv_args *args) { return check_gemv(args); }

moe_status moe_gemv_nvfp4(const moe_gemv_args *args, hipStream_t stream) {
  const moe_status st = check_gemv(args);
  if (st != MOE_OK) return st;
  gemv::Params p = {};
  p.x = args->x;
  p.B = args->B;
  p.B_sf = args->B_sf;
  p.B_gs = args->B_gs;
  p.ids = args->ids;
  p.topk_w = args->topk_w;
  p.T = args->T;
  p.k = args->k;
  p.E = args->E;
  p.N = args->N;
  p.K = args->K;
  p.per_pair = args->k > 1 && args->rows_x != args->T;
  p.D = args->D;
  const gemv::Epilogue epilogue = args->epilogue == MOE_EPI_NONE     ? gemv::kPlain
                                  : args->epilogue == MOE_EPI_SWIGLU ? gemv::kGated
                                                                     : gemv::kWeighted;
  return launch_status(gemv::launch(p, epilogue, args->B_layout == MOE_LAYOUT_PACKED, stream));
}

}  // extern "C"
