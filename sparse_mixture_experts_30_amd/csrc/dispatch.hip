// Token rows sorted by expert, and the gradients of that and of the weighted
// combine (page "从 1024 块 GPU 到 558 万美元：拆解 DeepSeek-V3 的算法-系统协同设计",
// section 2.3: tokens go to their experts in sorted order and the results
// come back to their tokens).  With p = pos[t, k], the sorted row of token
// t's slot k:
//   dispatch           rows[p] = x[t]
//   dispatch backward  dx[t] = dx_add[t] + sum_k drows[p]
//   combine backward   dy[p] = w[t,k] dout[t],  dw[t,k] = <dout[t], y[p]>
// A position outside [0, T*K) is a slot without a row (a dropped token): it
// is neither read nor written, and its dw is 0.  One workgroup per token, so
// a token's row is read once and its K rows are whole rows.
#include "rows_device.hpp"

namespace moe {

namespace {

constexpr int kDispatchThreads = 256;
constexpr int kMaxK = 64;

__device__ __forceinline__ void load_slots(const int32_t* __restrict__ pos, int64_t t, int K,
                                           int64_t N, int32_t* sp) {
  if (threadIdx.x < K) {
    const int32_t p = pos[t * K + threadIdx.x];
    sp[threadIdx.x] = (p >= 0 && p < N) ? p : -1;
  }
  __syncthreads();
}

// Rows of n16 16-byte units, and (scales not null) of n4 4-byte scales.
__global__ void __launch_bounds__(kDispatchThreads)
dispatch_kernel(const u32x4* __restrict__ x, int n16, const float* __restrict__ xs, int n4,
                const int32_t* __restrict__ pos, int K, int64_t N, u32x4* __restrict__ rows,
                float* __restrict__ rows_s) {
  __shared__ int32_t sp[kMaxK];
  const int64_t t = blockIdx.x;
  load_slots(pos, t, K, N, sp);
  for (int c = threadIdx.x; c < n16; c += kDispatchThreads) {
    const u32x4 v = x[t * n16 + c];
    for (int k = 0; k < K; ++k)
      if (sp[k] >= 0) rows[(int64_t)sp[k] * n16 + c] = v;
  }
  if (!xs) return;
  for (int c = threadIdx.x; c < n4; c += kDispatchThreads) {
    const float v = xs[t * n4 + c];
    for (int k = 0; k < K; ++k)
      if (sp[k] >= 0) rows_s[(int64_t)sp[k] * n4 + c] = v;
  }
}

template <typename IO>
__global__ void __launch_bounds__(kDispatchThreads)
dispatch_backward_kernel(const IO* __restrict__ drows, const IO* dx_add,
                         const int32_t* __restrict__ pos, int H, int K, int64_t N, IO* dx) {
  __shared__ int32_t sp[kMaxK];
  const int64_t t = blockIdx.x;
  load_slots(pos, t, K, N, sp);
  for (int c = threadIdx.x * kChunk; c < H; c += kDispatchThreads * kChunk) {
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (dx_add) load_chunk(dx_add + t * H + c, acc);
    for (int k = 0; k < K; ++k) {
      if (sp[k] < 0) continue;
      float r[8];
      load_chunk(drows + (int64_t)sp[k] * H + c, r);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] += r[j];
    }
    store_chunk(dx + t * H + c, acc);
  }
}

template <typename IO>
__global__ void __launch_bounds__(kDispatchThreads)
combine_backward_kernel(const IO* __restrict__ dout, const IO* y, const int32_t* __restrict__ pos,
                        const float* __restrict__ w, int H, int K, int64_t N, IO* dy,
                        float* __restrict__ dw) {
  __shared__ int32_t sp[kMaxK];
  __shared__ float red[kDispatchThreads / 64];
  const int64_t t = blockIdx.x;
  load_slots(pos, t, K, N, sp);
  for (int k = 0; k < K; ++k) {
    float part = 0.0f;
    if (sp[k] >= 0) {
      const float wk = w[t * K + k];
      const int64_t row = (int64_t)sp[k] * H;
      for (int c = threadIdx.x * kChunk; c < H; c += kDispatchThreads * kChunk) {
        float d[8], yv[8];
        load_chunk(dout + t * H + c, d);
        load_chunk(y + row + c, yv);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          part = fmaf(d[j], yv[j], part);
          d[j] *= wk;
        }
        store_chunk(dy + row + c, d);
      }
    }
    const float s = workgroup_sum<kDispatchThreads>(part, red);
    if (threadIdx.x == 0) dw[t * K + k] = s;
  }
}

}  // namespace

hipError_t launch_dispatch(const void* x, int64_t row_bytes, const float* xs, int n_scales,
                           const int32_t* pos, int64_t T, int K, void* rows, float* rows_s,
                           hipStream_t s) {
  MOE_TIMED_LAUNCH(s, "dispatch_kernel",
    hipLaunchKernelGGL(dispatch_kernel, dim3((unsigned)T), dim3(kDispatchThreads), 0, s,
                       (const u32x4*)x, (int)(row_bytes / 16), xs, n_scales, pos, K, T * K,
                       (u32x4*)rows, rows_s));
  return hipGetLastError();
}

hipError_t launch_dispatch_backward(const void* drows, const void* dx_add, const int32_t* pos,
                                    int64_t T, int H, int K, bool bf16, void* dx, hipStream_t s) {
  if (bf16)
    MOE_TIMED_LAUNCH(s, "dispatch_backward_kernel",
      hipLaunchKernelGGL(dispatch_backward_kernel<uint16_t>, dim3((unsigned)T),
                         dim3(kDispatchThreads), 0, s, (const uint16_t*)drows,
                         (const uint16_t*)dx_add, pos, H, K, T * K, (uint16_t*)dx));
  else
    MOE_TIMED_LAUNCH(s, "dispatch_backward_kernel",
      hipLaunchKernelGGL(dispatch_backward_kernel<float>, dim3((unsigned)T),
                         dim3(kDispatchThreads), 0, s, (const float*)drows, (const float*)dx_add,
                         pos, H, K, T * K, (float*)dx));
  return hipGetLastError();
}

hipError_t launch_combine_backward(const void* dout, const void* y, const int32_t* pos,
                                   const float* w, int64_t T, int H, int K, bool bf16, void* dy,
                                   float* dw, hipStream_t s) {
  if (bf16)
    MOE_TIMED_LAUNCH(s, "combine_backward_kernel",
      hipLaunchKernelGGL(combine_backward_kernel<uint16_t>, dim3((unsigned)T),
                         dim3(kDispatchThreads), 0, s, (const uint16_t*)dout, (const uint16_t*)y,
                         pos, w, H, K, T * K, (uint16_t*)dy, dw));
  else
    MOE_TIMED_LAUNCH(s, "combine_backward_kernel",
      hipLaunchKernelGGL(combine_backward_kernel<float>, dim3((unsigned)T),
                         dim3(kDispatchThreads), 0, s, (const float*)dout, (const float*)y, pos, w,
                         H, K, T * K, (float*)dy, dw));
  return hipGetLastError();
}

}  // namespace moe
