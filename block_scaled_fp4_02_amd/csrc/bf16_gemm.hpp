// Parameters and launchers of the bf16 grouped products (not part of the ABI).
#pragma once

#include "bf16_tiles.hpp"
#include "common.hpp"

namespace moe {
namespace bf16 {

struct GemmParams {
  const uint16_t *A;        // [rows_A, K]
  const int32_t *A_rows;    // [R] or NULL
  int64_t rows_A;
  const uint16_t *B;        // [E, N, K], transposed: [E, K, N]
  const int32_t *offsets;   // [E + 1]
  int E, N, K, R;
  uint16_t *D;              // [R, N], gated: [R, N / 2], gated backward: [R, 2 N]
  uint16_t *Z;              // gated: out [R, N] or NULL, gated backward: in [R, 2 N]
  int n_tiles;              // set by the launcher, with:
  bool stream_weights;      // the weights are too many to stay cached from one call to the next
};

struct WgradParams {
  const uint16_t *Y, *X;    // [R, N], [rows_X, K]
  const int32_t *X_rows;    // [R] or NULL
  int64_t rows_X;
  const int32_t *offsets;
  int E, N, K, R;
  void *D;                  // [E, N, K]
};

hipError_t launch_gemm(GemmParams p, Epilogue epilogue, bool transposed, hipStream_t stream);
hipError_t launch_wgrad(const WgradParams &p, bool bf16, hipStream_t stream);

}  // namespace bf16
}  // namespace moe
