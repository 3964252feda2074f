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
#include "block.hpp"
#include "rows_device.hpp"

#include <algorithm>

namespace moe {

namespace {

constexpr int kMaxThreads = 1024;
constexpr int kMaxK = 64;
constexpr int kBatch = 8;   // expert rows whose loads are issued together

__device__ __forceinline__ void load_slots(const int32_t* __restrict__ pos, int64_t t, int K,
                                           int64_t N, int32_t* sp) {
  if (threadIdx.x < K) {   // every workgroup has at least kMaxK threads
    const int32_t p = pos[t * K + threadIdx.x];
    sp[threadIdx.x] = (p >= 0 && p < N) ? p : -1;
  }
  __syncthreads();
}

// Rows of n16 16-byte units, and (scales not null) of n4 4-byte scales.
template <bool kNt>
__global__ void __launch_bounds__(kMaxThreads)
dispatch_kernel(const u32x4* __restrict__ x, int n16, const float* __restrict__ xs, int n4,
                const int32_t* __restrict__ pos, int K, int64_t N, u32x4* __restrict__ rows,
                float* __restrict__ rows_s) {
  __shared__ int32_t sp[kMaxK];
  const int64_t t = blockIdx.x;
  load_slots(pos, t, K, N, sp);
  for (int c = threadIdx.x; c < n16; c += blockDim.x) {
    const u32x4 v = x[t * n16 + c];
    for (int k = 0; k < K; ++k)
      if (sp[k] >= 0) store16<kNt>(&rows[(int64_t)sp[k] * n16 + c], v);
  }
  if (!xs) return;
  for (int c = threadIdx.x; c < n4; c += blockDim.x) {
    const float v = xs[t * n4 + c];
    for (int k = 0; k < K; ++k)
      if (sp[k] >= 0) rows_s[(int64_t)sp[k] * n4 + c] = v;
  }
}

template <typename IO, bool kNt>
__global__ void __launch_bounds__(kMaxThreads)
dispatch_backward_kernel(const IO* __restrict__ drows, const IO* dx_add,
                         const int32_t* __restrict__ pos, int H, int K, int64_t N, IO* dx) {
  __shared__ int32_t sp[kMaxK];
  const int64_t t = blockIdx.x;
  load_slots(pos, t, K, N, sp);
  constexpr int W = kWidth<IO>;
  for (int c = threadIdx.x * W; c < H; c += blockDim.x * W) {
    float acc[W];
#pragma unroll
    for (int j = 0; j < W; ++j) acc[j] = 0.0f;
    if (dx_add) load_chunk(dx_add + t * H + c, acc);
    for (int k0 = 0; k0 < K; k0 += kBatch) {
      RawChunk<IO> v[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
        if (k0 + b < K && sp[k0 + b] >= 0) v[b].template load<kNt>(drows + (int64_t)sp[k0 + b] * H + c);
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (k0 + b >= K || sp[k0 + b] < 0) continue;
        float r[W];
        v[b].to(r);
#pragma unroll
        for (int j = 0; j < W; ++j) acc[j] += r[j];
      }
    }
    store_chunk(dx + t * H + c, acc);
  }
}

template <typename IO, bool kNt>
__global__ void __launch_bounds__(kMaxThreads)
combine_backward_kernel(const IO* __restrict__ dout, const IO* y, const int32_t* __restrict__ pos,
                        const float* __restrict__ w, int H, int K, int64_t N, IO* dy,
                        float* __restrict__ dw) {
  __shared__ int32_t sp[kMaxK];
  __shared__ float sw[kMaxK], red[kMaxK][kMaxThreads / 64];
  const int64_t t = blockIdx.x;
  constexpr int W = kWidth<IO>;
  if (threadIdx.x < K) sw[threadIdx.x] = w[t * K + threadIdx.x];
  load_slots(pos, t, K, N, sp);
  for (int k0 = 0; k0 < K; k0 += kBatch) {
    float part[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) part[b] = 0.0f;
    for (int c = threadIdx.x * W; c < H; c += blockDim.x * W) {
      RawChunk<IO> v[kBatch];
      float d[W];
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
        if (k0 + b < K && sp[k0 + b] >= 0) v[b].template load<kNt>(y + (int64_t)sp[k0 + b] * H + c);
      load_chunk(dout + t * H + c, d);
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (k0 + b >= K || sp[k0 + b] < 0) continue;
        float yv[W], g[W];
        v[b].to(yv);
        const float wk = sw[k0 + b];
#pragma unroll
        for (int j = 0; j < W; ++j) {
          part[b] = fmaf(d[j], yv[j], part[b]);
          g[j] = d[j] * wk;
        }
        store_chunk<kNt>(dy + (int64_t)sp[k0 + b] * H + c, g);
      }
    }
    // The wave's sums: in each of two steps a lane keeps half of its values
    // and hands the other half over; the two left are summed over the rows of
    // 16 lanes.  The order is fixed.
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int n = kBatch / 2, off = 32; n >= 2; n >>= 1, off >>= 1)
#pragma unroll
      for (int b = 0; b < n; ++b) {
        const bool high = lane & off;
        const float keep = high ? part[b + n] : part[b], give = high ? part[b] : part[b + n];
        part[b] = keep + __shfl_xor(give, off, 64);
      }
    const int k = k0 + (lane >> 4 & 1) * 2 + (lane >> 5) * 4;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      part[b] = row_sum(part[b]);
      if ((lane & 15) == 0 && k + b < K) red[k + b][threadIdx.x >> 6] = part[b];
    }
  }
  __syncthreads();
  if (threadIdx.x < K) {
    float s = 0.0f;
    for (int i = 0; i < (int)(blockDim.x >> 6); ++i) s += red[threadIdx.x][i];
    dw[t * K + threadIdx.x] = s;
  }
}

}  // namespace

// Sorted rows past this size are read and written non-temporally: they leave
// the last-level cache before a next kernel could read them there.  Measured
// at H = 7168, K = 8, bf16, cached -> non-temporal: the calls by themselves
// 29 -> 24 us (dispatch) and 56 -> 51 us (combine backward) at 117 MB, 107 ->
// 93 and 210 -> 196 us at 470 MB; followed by a kernel that reads the rows 28
// -> 35 and 46 -> 52 us at 59 MB, 53 -> 54 and 80 -> 81 us at 117 MB, 246 ->
// 210 and 321 -> 311 us at 470 MB.
constexpr int64_t kStreamBytes = (int64_t)128 << 20;

// Threads per token: as many as the row has pieces, so that a row is one
// round trip; with more tokens than CUs at most eight waves, so that several
// tokens share a CU.  Combine backward at H = 7168, K = 8, bf16, with 896 / 512
// / 256 threads: T = 32 9.7 / 11.2 / 16.8 us, T = 512 34.7 / 29.6 / 31.8,
// T = 1024 64.4 / 55.5 / 56.1, T = 4096 198.5 / 197.4 / 200.6.
constexpr int64_t kCus = 256;
int row_threads(int64_t T, int64_t pieces) {
  return (int)std::min<int64_t>((pieces + 63) / 64 * 64, T > kCus ? 512 : kMaxThreads);
}

// From kCus + 1 tokens on the workgroups have one size.
int64_t dispatch_max_tokens(int64_t row_bytes) {
  return kMaxGridThreads / row_threads(kCus + 1, row_bytes / 16);
}

hipError_t launch_dispatch(const void* x, int64_t row_bytes, const float* xs, int n_scales,
                           const int32_t* pos, int64_t T, int K, void* rows, float* rows_s,
                           hipStream_t s) {
  auto* kernel = T * K * row_bytes > kStreamBytes ? dispatch_kernel<true> : dispatch_kernel<false>;
  MOE_TIMED_LAUNCH(s, "dispatch_kernel",
    hipLaunchKernelGGL(kernel, dim3((unsigned)T), dim3(row_threads(T, row_bytes / 16)), 0, s, (const u32x4*)x,
                       (int)(row_bytes / 16), xs, n_scales, pos, K, T * K, (u32x4*)rows, rows_s));
  return hipGetLastError();
}

template <typename IO>
static hipError_t dispatch_backward(const void* drows, const void* dx_add, const int32_t* pos,
                                    int64_t T, int H, int K, void* dx, hipStream_t s) {
  auto* kernel = T * K * H * (int64_t)sizeof(IO) > kStreamBytes ? dispatch_backward_kernel<IO, true>
                                                                : dispatch_backward_kernel<IO, false>;
  MOE_TIMED_LAUNCH(s, "dispatch_backward_kernel",
    hipLaunchKernelGGL(kernel, dim3((unsigned)T), dim3(row_threads(T, H / kWidth<IO>)), 0, s, (const IO*)drows,
                       (const IO*)dx_add, pos, H, K, T * K, (IO*)dx));
  return hipGetLastError();
}

hipError_t launch_dispatch_backward(const void* drows, const void* dx_add, const int32_t* pos,
                                    int64_t T, int H, int K, bool bf16, void* dx, hipStream_t s) {
  return bf16 ? dispatch_backward<uint16_t>(drows, dx_add, pos, T, H, K, dx, s)
              : dispatch_backward<float>(drows, dx_add, pos, T, H, K, dx, s);
}

template <typename IO>
static hipError_t combine_backward(const void* dout, const void* y, const int32_t* pos,
                                   const float* w, int64_t T, int H, int K, void* dy, float* dw,
                                   hipStream_t s) {
  auto* kernel = T * K * H * (int64_t)sizeof(IO) > kStreamBytes ? combine_backward_kernel<IO, true>
                                                                : combine_backward_kernel<IO, false>;
  MOE_TIMED_LAUNCH(s, "combine_backward_kernel",
    hipLaunchKernelGGL(kernel, dim3((unsigned)T), dim3(row_threads(T, H / kWidth<IO>)), 0, s, (const IO*)dout,
                       (const IO*)y, pos, w, H, K, T * K, (IO*)dy, dw));
  return hipGetLastError();
}

hipError_t launch_combine_backward(const void* dout, const void* y, const int32_t* pos,
                                   const float* w, int64_t T, int H, int K, bool bf16, void* dy,
                                   float* dw, hipStream_t s) {
  return bf16 ? combine_backward<uint16_t>(dout, y, pos, w, T, H, K, dy, dw, s)
              : combine_backward<float>(dout, y, pos, w, T, H, K, dy, dw, s);
}

}  // namespace moe
