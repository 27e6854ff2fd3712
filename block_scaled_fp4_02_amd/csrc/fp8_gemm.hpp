// Parameters and launchers of the FP8 grouped products (not part of the ABI).
#pragma once

#include "common.hpp"

namespace moe {
namespace fp8 {

struct GemmParams {
  const uint8_t *A;         // [rows_A, K]
  const float *A_sf;        // [rows_A, ceil(K / 128)]
  const int32_t *A_rows;    // [R] or NULL
  int64_t rows_A;
  const uint8_t *B;         // [E, N, K]
  const float *B_sf;        // [E, ceil(N / 128), ceil(K / 128)]
  const int32_t *offsets;   // [E + 1]
  int E, N, K, R;
  void *D;
  float *D_sf;
  int n_tiles;              // set by the launcher, with:
  bool stream_weights;      // the weights are too many to stay cached from one call to the next
};

struct WgradParams {
  const uint8_t *Y, *X;     // [blocks, N, 128], [blocks, K, 128]
  const float *Y_sf, *X_sf; // [blocks, N], [blocks, K]
  const int32_t *offsets;
  int E, N, K, R;
  int blocks;
  void *D;                  // [E, N, K]
};

hipError_t launch_gemm(GemmParams p, bool swiglu, bool whole, hipStream_t stream);
hipError_t launch_wgrad(const WgradParams &p, bool bf16, hipStream_t stream);

}  // namespace fp8

hipError_t launch_quantize_fp8(const void *x, int x_dtype, int64_t rows, int C, uint8_t *q, float *sf, hipStream_t stream);
hipError_t launch_quantize_fp8_weights(const void *w, int w_dtype, int E, int N, int K, uint8_t *q, float *sf, uint8_t *qt,
                                       float *sft, hipStream_t stream);
hipError_t launch_quantize_fp8_tokens(const void *x, int x_dtype, int64_t rows_x, const int32_t *rows,
                                      const int32_t *offsets, int E, int64_t R, int C, uint8_t *q, float *sf,
                                      hipStream_t stream);

}  // namespace moe
