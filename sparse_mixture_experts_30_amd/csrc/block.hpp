// Host launchers of the operators around the layer: residual add + RMS norm,
// sorted token rows, and the expert FFNs on 4-bit weights.
#pragma once

#include "moe_internal.hpp"

namespace moe {

// Threads that a launch may have along one grid dimension.
constexpr int64_t kMaxGridThreads = 0xffffffffLL;

// Expert FFNs on packed 4-bit weights with group scales (ffn_int4.hip);
// group is 128 or 32.  No tile list.  A matrix is packed by a thread per 16
// bytes of packed4_bytes and quantised by a thread per 8 values, in one launch
// each.
size_t packed4_bytes(bool gate_up, int64_t experts, int n, int kd, int group);
hipError_t launch_pack_int4(bool gate_up, int group, const uint8_t* codes, const uint16_t* scales,
                            void* dst, int64_t experts, int n, int kd, hipStream_t s);
hipError_t launch_quantize_int4(int group, const uint16_t* src, int64_t rows, int kd,
                                uint8_t* codes, uint16_t* scales, hipStream_t s);
hipError_t launch_ffn_int4(const FfnDims& d, int group, const uint16_t* x, const int32_t* perm,
                           const int32_t* offsets, const void* w13p, const void* w2p,
                           const void* ws13p, const void* ws2p, uint16_t* h, uint16_t* y,
                           uint16_t* ys, hipStream_t s);

// Residual add + RMS norm and its backward (norm.hip).  The forward has a
// workgroup per row, for at most add_rmsnorm_max_rows rows.
int64_t add_rmsnorm_max_rows(int H, bool bf16);
hipError_t launch_add_rmsnorm(const void* x, const void* residual, const float* weight, float eps,
                              int64_t rows, int H, bool bf16, void* sum, void* y, uint8_t* yq,
                              float* ys, bool pow2, hipStream_t s);
size_t rmsnorm_backward_ws_bytes(int64_t rows, int H);
hipError_t launch_add_rmsnorm_backward(const void* sum, const float* weight, float eps,
                                       const void* dy, const void* dsum, int64_t rows, int H,
                                       bool bf16, void* dx, float* dweight, float* part,
                                       hipStream_t s);

// Sorted token rows and the gradients of the two ends (dispatch.hip): a
// workgroup per token, for at most dispatch_max_tokens tokens.
int64_t dispatch_max_tokens(int64_t row_bytes);
hipError_t launch_dispatch(const void* x, int64_t row_bytes, const float* xs, int n_scales,
                           const int32_t* pos, int64_t T, int K, void* rows, float* rows_s,
                           hipStream_t s);
hipError_t launch_dispatch_backward(const void* drows, const void* dx_add, const int32_t* pos,
                                    int64_t T, int H, int K, bool bf16, void* dx, hipStream_t s);
hipError_t launch_combine_backward(const void* dout, const void* y, const int32_t* pos,
                                   const float* w, int64_t T, int H, int K, bool bf16, void* dy,
                                   float* dw, hipStream_t s);

}  // namespace moe
