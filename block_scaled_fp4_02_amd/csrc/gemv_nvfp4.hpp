// Parameters and launcher of the products of single tokens with NVFP4 weights (not part of the ABI).
#pragma once

#include "common.hpp"

namespace moe {
namespace gemv {

enum Epilogue { kPlain, kGated, kWeighted };

struct Params {
  const uint16_t *x;        // [T, K], or with per_pair [T * k, K]
  const uint8_t *B, *B_sf;  // row-major NVFP4, or (B_sf unused) the packed layout
  const float *B_gs;        // [E]
  const int32_t *ids;       // [T, k], or NULL: expert 0 (k = 1)
  const float *topk_w;      // kWeighted: [T, k], or NULL: 1
  int T, k, E, N, K;
  bool per_pair;
  uint16_t *D;
};

hipError_t launch(const Params &p, Epilogue epilogue, bool packed, hipStream_t stream);

}  // namespace gemv
}  // namespace moe
