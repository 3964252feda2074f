// Residual add and RMS norm in front of the layer, and its backward.
//
//   r = x + residual  (rounded to the activation type: the stream as stored),
//   y = r * rstd * w,   rstd = 1 / sqrt(mean(r^2) + eps),
// and for FP8 experts the same y per 1x128 tile in e4m3: scale a / 448 (or
// the smallest power of two not below it) with a = max |y| of the tile.  The
// tile is quantised from the fp32 y, not from its bf16 rounding: one rounding
// instead of two.
// Backward, with g = dy * w and n = r * rstd:
//   dr = rstd * (g - n * mean(g * n)) + dsum,   dw = sum over rows of dy * n.
// Sums are fp32 in a fixed order.
#include "fp8_device.hpp"
#include "rows_device.hpp"

#include <algorithm>

namespace moe {

namespace {

constexpr int kNormThreads = 256;

// fp32 -> e4m3fn bits as f32_to_e4m3, with NaN kept NaN.
__device__ __forceinline__ uint32_t e4m3_code(float v) {
  return v != v ? 0x7Fu : f32_to_e4m3(v);
}

// e4m3 codes of the 8 values v (one chunk; 16 consecutive lanes hold a tile)
// and the tile's scale.  All 16 lanes of the tile call this.
__device__ __forceinline__ uint2 quant_chunk(const float (&v)[8], bool pow2, float& scale) {
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[j]));
#pragma unroll
  for (int off = 8; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
  float inv;
  if (pow2)
    tile_scale_pow2(m, scale, inv);
  else
    tile_scale(m, scale, inv);
  uint32_t lo = 0, hi = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) lo |= e4m3_code(v[j] * inv) << (8 * j);
#pragma unroll
  for (int j = 0; j < 4; ++j) hi |= e4m3_code(v[4 + j] * inv) << (8 * j);
  return make_uint2(lo, hi);
}

template <typename IO>
__device__ __forceinline__ void add_chunk(const IO* x, const IO* residual, float (&r)[8]) {
  load_chunk(x, r);
  if (!residual) return;
  float b[8];
  load_chunk(residual, b);
#pragma unroll
  for (int j = 0; j < 8; ++j) r[j] = as_stored<IO>(r[j] + b[j]);
}

// One workgroup per row, two passes over it.
// sum may be x or residual itself: a thread rewrites only chunks that it
// alone reads, after reading them.
template <typename IO>
__global__ void __launch_bounds__(kNormThreads)
add_rmsnorm_kernel(const IO* x, const IO* residual, const float* __restrict__ weight, float eps,
                   int H, IO* sum, IO* y, uint8_t* __restrict__ yq, float* __restrict__ ys,
                   bool pow2) {
  __shared__ float red[kNormThreads / 64];
  const int64_t row = (int64_t)blockIdx.x * H;
  const int nc = H / kChunk;
  float ss = 0.0f;
  for (int c = threadIdx.x; c < nc; c += kNormThreads) {
    float r[8];
    add_chunk(x + row + c * 8, residual ? residual + row + c * 8 : nullptr, r);
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(r[j], r[j], ss);
  }
  const float rstd = 1.0f / sqrtf(workgroup_sum<kNormThreads>(ss, red) / (float)H + eps);
  for (int c = threadIdx.x; c < nc; c += kNormThreads) {
    float r[8], w[8];
    add_chunk(x + row + c * 8, residual ? residual + row + c * 8 : nullptr, r);
    load_chunk(weight + c * 8, w);
    if (sum) store_chunk(sum + row + c * 8, r);
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = r[j] * rstd * w[j];
    if (y) store_chunk(y + row + c * 8, r);
    if (yq) {
      float scale;
      *reinterpret_cast<uint2*>(yq + row + c * 8) = quant_chunk(r, pow2, scale);
      if ((c & 15) == 0) ys[(row >> 7) + (c >> 4)] = scale;
    }
  }
}

// Workgroup b takes rows b, b + gridDim.x, ...; its share of dw is kept in
// its row of `part` [gridDim.x][H].
template <typename IO>
__global__ void __launch_bounds__(kNormThreads)
add_rmsnorm_backward_kernel(const IO* __restrict__ sum, const float* __restrict__ weight,
                            float eps, const IO* dy, const IO* dsum, int64_t rows, int H, IO* dx,
                            float* __restrict__ part) {
  __shared__ float red[kNormThreads / 64];
  const int nc = H / kChunk;
  float* mine = part + (int64_t)blockIdx.x * H;
  for (int64_t t = blockIdx.x; t < rows; t += gridDim.x) {
    const int64_t row = t * H;
    float ss = 0.0f, dot = 0.0f;
    for (int c = threadIdx.x; c < nc; c += kNormThreads) {
      float r[8], g[8], w[8];
      load_chunk(sum + row + c * 8, r);
      load_chunk(dy + row + c * 8, g);
      load_chunk(weight + c * 8, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        ss = fmaf(r[j], r[j], ss);
        dot = fmaf(g[j] * w[j], r[j], dot);
      }
    }
    ss = workgroup_sum<kNormThreads>(ss, red);
    dot = workgroup_sum<kNormThreads>(dot, red);
    const float rstd = 1.0f / sqrtf(ss / (float)H + eps);
    const float mean = dot * rstd / (float)H;   // mean(g * n)
    for (int c = threadIdx.x; c < nc; c += kNormThreads) {
      float r[8], g[8], w[8], a[8], d[8];
      load_chunk(sum + row + c * 8, r);
      load_chunk(dy + row + c * 8, g);
      load_chunk(weight + c * 8, w);
      if (dsum) load_chunk(dsum + row + c * 8, d);
      if (t != blockIdx.x) load_chunk(mine + c * 8, a);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float n = r[j] * rstd;
        a[j] = (t != blockIdx.x ? a[j] : 0.0f) + g[j] * n;
        r[j] = rstd * (g[j] * w[j] - n * mean) + (dsum ? d[j] : 0.0f);
      }
      store_chunk(mine + c * 8, a);
      store_chunk(dx + row + c * 8, r);
    }
  }
}

// dw[h] = sum of part[b][h] over b in order; zeros for nparts = 0.
__global__ void __launch_bounds__(kNormThreads)
rmsnorm_dweight_kernel(const float* __restrict__ part, int nparts, int H,
                       float* __restrict__ dweight) {
  const int h = blockIdx.x * kNormThreads + threadIdx.x;
  if (h >= H) return;
  float a = 0.0f;
  for (int b = 0; b < nparts; ++b) a += part[(int64_t)b * H + h];
  dweight[h] = a;
}

constexpr int64_t kNormParts = 512;   // row sums of dw kept apart at most

}  // namespace

size_t rmsnorm_backward_ws_bytes(int64_t rows, int H) {
  return ((size_t)std::min(rows, kNormParts) * H * sizeof(float) + 255) / 256 * 256;
}

template <typename IO>
static hipError_t add_rmsnorm(const void* x, const void* residual, const float* weight, float eps,
                              int64_t rows, int H, void* sum, void* y, uint8_t* yq, float* ys,
                              bool pow2, hipStream_t s) {
  MOE_TIMED_LAUNCH(s, "add_rmsnorm_kernel",
    hipLaunchKernelGGL(add_rmsnorm_kernel<IO>, dim3((unsigned)rows), dim3(kNormThreads), 0, s,
                       (const IO*)x, (const IO*)residual, weight, eps, H, (IO*)sum, (IO*)y, yq, ys,
                       pow2));
  return hipGetLastError();
}

hipError_t launch_add_rmsnorm(const void* x, const void* residual, const float* weight, float eps,
                              int64_t rows, int H, bool bf16, void* sum, void* y, uint8_t* yq,
                              float* ys, bool pow2, hipStream_t s) {
  return bf16 ? add_rmsnorm<uint16_t>(x, residual, weight, eps, rows, H, sum, y, yq, ys, pow2, s)
              : add_rmsnorm<float>(x, residual, weight, eps, rows, H, sum, y, yq, ys, pow2, s);
}

template <typename IO>
static hipError_t add_rmsnorm_backward(const void* sum, const float* weight, float eps,
                                       const void* dy, const void* dsum, int64_t rows, int H,
                                       void* dx, float* dweight, float* part, hipStream_t s) {
  const int64_t parts = std::min(rows, kNormParts);
  if (parts) {
    MOE_TIMED_LAUNCH(s, "add_rmsnorm_backward_kernel",
      hipLaunchKernelGGL(add_rmsnorm_backward_kernel<IO>, dim3((unsigned)parts),
                         dim3(kNormThreads), 0, s, (const IO*)sum, weight, eps, (const IO*)dy,
                         (const IO*)dsum, rows, H, (IO*)dx, part));
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  MOE_TIMED_LAUNCH(s, "rmsnorm_dweight_kernel",
    hipLaunchKernelGGL(rmsnorm_dweight_kernel, dim3((H + kNormThreads - 1) / kNormThreads),
                       dim3(kNormThreads), 0, s, part, (int)parts, H, dweight));
  return hipGetLastError();
}

hipError_t launch_add_rmsnorm_backward(const void* sum, const float* weight, float eps,
                                       const void* dy, const void* dsum, int64_t rows, int H,
                                       bool bf16, void* dx, float* dweight, float* part,
                                       hipStream_t s) {
  return bf16 ? add_rmsnorm_backward<uint16_t>(sum, weight, eps, dy, dsum, rows, H, dx, dweight,
                                               part, s)
              : add_rmsnorm_backward<float>(sum, weight, eps, dy, dsum, rows, H, dx, dweight, part,
                                            s);
}

}  // namespace moe
