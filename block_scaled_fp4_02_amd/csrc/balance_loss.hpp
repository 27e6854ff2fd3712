// Parameters and launchers of the balance loss (not part of the ABI).
#pragma once

#include "common.hpp"

namespace moe {
namespace balance {

struct LossParams {
  const float *logits;          // [T, E]
  const int32_t *ids;           // [T, k]
  const int32_t *seq_offsets;   // [S + 1] or NULL (S = 1)
  const uint8_t *mask;          // [T] or NULL
  int T, E, k, S;
  int32_t *counts;              // [S, E]
  float *coef;                  // [S, E]
  float *loss;
  // workspace, laid out by the launcher
  int chunks, chunk;            // partial rows, and the most tokens of one
  uint32_t *ticket;
  double *part_loss;            // one per workgroup of the second kernel
  int32_t *part_kept;           // [chunks]
  int32_t *part_count;          // [chunks, E]
  float *part_sum;              // [chunks, E]
};

struct GradParams {
  const float *logits;
  const int32_t *seq_offsets;
  const uint8_t *mask;
  int T, E, k, S;
  const float *coef, *grad_loss;
  const int32_t *ids;           // with d_topk_w
  const float *topk_w, *d_topk_w;
  float *dlogits;
};

size_t loss_ws_bytes(int T, int E, int S);
hipError_t launch_loss(LossParams p, void *ws, hipStream_t stream);
hipError_t launch_backward(const GradParams &p, hipStream_t stream);

}  // namespace balance
}  // namespace moe
