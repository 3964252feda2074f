// Host launchers of the feed-forward block of dense layers (dense.hip).
#pragma once

#include "moe_internal.hpp"

namespace moe {

// Whether every product fits one launch and the kernels' 32-bit offsets.
bool dense_fits(int64_t T, int64_t H, int64_t I);
// Bytes of `part`, the partial sums of products whose k range is split, of the
// forward's or the backward's products.
size_t dense_part_bytes(int64_t T, int64_t H, int64_t I, bool backward);
// h = silu(g) u of [g u] = x W13^T; gu [T, 2 I] and h [T, I] may be null.
hipError_t launch_dense_gate_up(const uint16_t* x, const uint16_t* w13, int64_t T, int H, int I,
                                float* gu, uint16_t* h, float* part, hipStream_t s);
// y = h W2^T.
hipError_t launch_dense_down(const uint16_t* h, const uint16_t* w2, int64_t T, int H, int I,
                             uint16_t* y, float* part, hipStream_t s);
// da [T, 2 I] and h [T, I] are scratch; dx may be null.
hipError_t launch_dense_backward(const uint16_t* x, const uint16_t* w13, const uint16_t* w2,
                                 const float* gu, const uint16_t* dy, int64_t T, int H, int I,
                                 uint16_t* da, uint16_t* h, uint16_t* dx, uint16_t* dw13,
                                 uint16_t* dw2, float* part, hipStream_t s);

}  // namespace moe
