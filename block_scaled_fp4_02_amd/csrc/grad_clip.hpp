// Launchers of the global gradient norm and its clipping (not part of the ABI).
#pragma once

#include "common.hpp"

namespace moe {
namespace grad {

size_t norm_ws_bytes(const moe_tensor *tensors, int count);
hipError_t launch_norm(const moe_tensor *tensors, int count, float *norm, void *ws, hipStream_t stream);
hipError_t launch_clip(const moe_tensor *tensors, int count, const float *norm, float max_norm, hipStream_t stream);

}  // namespace grad
}  // namespace moe
