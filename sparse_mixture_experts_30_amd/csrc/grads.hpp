// Host launchers of the global gradient norm and clipping (grads.hip).
#pragma once

#include "moe_internal.hpp"

namespace moe {

// Gradients in host arrays of n; out may be null where nothing is scaled.
// Fewer than 2^31 chunks of 4 KiB in all.
struct GradList {
  int n;
  const void* const* grad;
  void* const* out;
  const int64_t* count;
  const uint8_t* bf16;
};

size_t grad_norm_ws_bytes(const GradList& l);
hipError_t launch_grad_norm(const GradList& l, double* part, float* norm, hipStream_t s);
// norm_given: norm is read and part not used.
hipError_t launch_clip(const GradList& l, double* part, float* norm, bool norm_given,
                       float max_norm, hipStream_t s);

}  // namespace moe
