// Global norm over many gradients, and clipping to it (gfx950).
//   norm = sqrt(sum over all of g^2),  out = g min(1, max_norm / (norm + 1e-6)).
// Squares are summed in 64 bits, which the vector units have at half the rate
// of fp32, far above what memory delivers: no range is lost to overflow and
// the order of the sums does not show.  Bound by memory: one read for the
// norm, one read and one write for the scaling.
//
// The gradients are cut into chunks of equal size that start on 16-byte
// addresses (the first takes what lies before the first such address), a
// workgroup takes every gridDim'th chunk.  The table of gradients travels as
// a kernel argument, so nothing is copied to the device and a call can be
// captured; lists longer than a table take several launches.
#include "grads.hpp"

#include <math.h>

#include <algorithm>

namespace moe {

namespace {

constexpr int kTable = 96;            // gradients a launch (the argument stays under 4 KiB)
constexpr int kGradThreads = 256;
constexpr int kGradBlocks = 2048;     // workgroups a launch at most, and partial sums

struct Table {
  const void* g[kTable];
  void* out[kTable];
  int64_t n[kTable];
  int32_t first[kTable + 1];   // first chunk of each gradient, then their number
  uint8_t bf16[kTable];
  int32_t count;
  int32_t chunk;               // bytes
};

// Values before the first 16-byte address.
__host__ __device__ inline int64_t head_of(const void* p, int64_t n, int size) {
  const int64_t h = (int64_t)((16 - ((uintptr_t)p & 15)) & 15) / size;
  return h < n ? h : n;
}

// Calls f(gradient, first value, end) for every chunk of this workgroup.
template <class F>
__device__ __forceinline__ void for_chunks(const Table& t, F f) {
  const int total = t.first[t.count];
  for (int c = blockIdx.x; c < total; c += gridDim.x) {
    int lo = 0, hi = t.count - 1;   // the gradient that holds chunk c
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (t.first[mid] <= c) lo = mid;
      else hi = mid - 1;
    }
    const int size = t.bf16[lo] ? 2 : 4, per = t.chunk / size;
    const int64_t n = t.n[lo], head = head_of(t.g[lo], n, size), k = c - t.first[lo];
    const int64_t a = k ? head + k * per : 0, b = min(n, head + (k + 1) * per);
    f(lo, a, b);
  }
}

template <typename IO>
__device__ __forceinline__ float value(IO v) {
  if constexpr (sizeof(IO) == 2) return bf16_bits_to_f32(v);
  else return v;
}

template <typename IO>
__device__ __forceinline__ double squares(const IO* g, int64_t a, int64_t b) {
  constexpr int W = 16 / sizeof(IO);
  double s = 0.0;
  const int64_t va = a + head_of(g + a, b - a, sizeof(IO));
  if (a + threadIdx.x < va) {
    const double v = value(g[a + threadIdx.x]);
    s = v * v;
  }
  const int64_t nv = (b - va) / W;
  const u32x4* p = reinterpret_cast<const u32x4*>(g + va);
  for (int64_t i = threadIdx.x; i < nv; i += kGradThreads) {
    const u32x4 q = p[i];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (sizeof(IO) == 2) {
        const double x = __uint_as_float(q[j] << 16), y = __uint_as_float(q[j] & 0xFFFF0000u);
        s = fma(x, x, s);
        s = fma(y, y, s);
      } else {
        const double x = __uint_as_float(q[j]);
        s = fma(x, x, s);
      }
    }
  }
  for (int64_t i = va + nv * W + threadIdx.x; i < b; i += kGradThreads) {
    const double v = value(g[i]);
    s = fma(v, v, s);
  }
  return s;
}

// Sum over the workgroup in a fixed order, for thread 0.
__device__ __forceinline__ double workgroup_sum(double s) {
  __shared__ double red[kGradThreads / 64];
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) s += __shfl_xor(s, off, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  double r = 0.0;
  for (int i = 0; i < kGradThreads / 64; ++i) r += red[i];
  return r;
}

__global__ void __launch_bounds__(kGradThreads)
grad_squares_kernel(Table t, double* __restrict__ part) {
  double s = 0.0;
  for_chunks(t, [&](int i, int64_t a, int64_t b) {
    s += t.bf16[i] ? squares((const uint16_t*)t.g[i], a, b) : squares((const float*)t.g[i], a, b);
  });
  s = workgroup_sum(s);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

__global__ void __launch_bounds__(kGradThreads)
grad_norm_kernel(const double* __restrict__ part, int64_t n, float* __restrict__ norm) {
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += kGradThreads) s += part[i];
  s = workgroup_sum(s);
  if (threadIdx.x == 0) *norm = (float)sqrt(s);
}

template <typename IO>
__device__ __forceinline__ void scale(const IO* g, IO* out, int64_t a, int64_t b, float f) {
  constexpr int W = 16 / sizeof(IO);
  auto one = [&](int64_t i) {
    const float v = value(g[i]) * f;
    if constexpr (sizeof(IO) == 2) out[i] = (uint16_t)f32_to_bf16_bits(v);
    else out[i] = v;
  };
  if (((uintptr_t)g ^ (uintptr_t)out) & 15) {   // no common 16-byte address
    for (int64_t i = a + threadIdx.x; i < b; i += kGradThreads) one(i);
    return;
  }
  const int64_t va = a + head_of(g + a, b - a, sizeof(IO));
  if (a + threadIdx.x < va) one(a + threadIdx.x);
  const int64_t nv = (b - va) / W;
  const u32x4* p = reinterpret_cast<const u32x4*>(g + va);
  u32x4* o = reinterpret_cast<u32x4*>(out + va);
  for (int64_t i = threadIdx.x; i < nv; i += kGradThreads) {
    const u32x4 q = p[i];
    u32x4 r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (sizeof(IO) == 2)
        r[j] = pack_bf16x2(__uint_as_float(q[j] << 16) * f, __uint_as_float(q[j] & 0xFFFF0000u) * f);
      else
        r[j] = __float_as_uint(__uint_as_float(q[j]) * f);
    }
    o[i] = r;
  }
  for (int64_t i = va + nv * W + threadIdx.x; i < b; i += kGradThreads) one(i);
}

__global__ void __launch_bounds__(kGradThreads)
grad_scale_kernel(Table t, const float* __restrict__ norm, float max_norm) {
  const float n = *norm;
  // A norm that is not finite says nothing about the scale: the gradients stay
  // as they are, for the caller to skip the step.
  const float f = isfinite(n) ? fminf(1.0f, max_norm / (n + 1e-6f)) : 1.0f;
  for_chunks(t, [&](int i, int64_t a, int64_t b) {
    if (f == 1.0f && t.g[i] == t.out[i]) return;
    if (t.bf16[i]) scale((const uint16_t*)t.g[i], (uint16_t*)t.out[i], a, b, f);
    else scale((const float*)t.g[i], (float*)t.out[i], a, b, f);
  });
}

// Bytes of a chunk: 64 KiB, or less where the workgroups would not be busy.
int chunk_bytes(const GradList& l) {
  int64_t bytes = 0;
  for (int i = 0; i < l.n; ++i) bytes += l.count[i] * (l.bf16[i] ? 2 : 4);
  int c = 1 << 16;
  while (c > 4096 && bytes / c < kGradBlocks) c /= 2;
  return c;
}

// The table of gradients [i0, i0 + count) and its number of workgroups.
unsigned fill(const GradList& l, int i0, int chunk, Table& t) {
  t.count = std::min(kTable, l.n - i0);
  t.chunk = chunk;
  int64_t c = 0;
  for (int j = 0; j < t.count; ++j) {
    const int i = i0 + j, size = l.bf16[i] ? 2 : 4;
    t.g[j] = l.grad[i];
    t.out[j] = l.out ? l.out[i] : nullptr;
    t.n[j] = l.count[i];
    t.bf16[j] = l.bf16[i];
    t.first[j] = (int32_t)c;
    const int64_t rest = l.count[i] - head_of(l.grad[i], l.count[i], size), per = chunk / size;
    c += l.count[i] ? std::max<int64_t>(1, (rest + per - 1) / per) : 0;
  }
  t.first[t.count] = (int32_t)c;
  return (unsigned)std::min<int64_t>(c, kGradBlocks);
}

}  // namespace

size_t grad_norm_ws_bytes(int n) {
  return (size_t)((n + kTable - 1) / kTable) * kGradBlocks * sizeof(double);
}

hipError_t launch_grad_norm(const GradList& l, double* part, float* norm, hipStream_t s) {
  const int chunk = chunk_bytes(l);
  int64_t used = 0;
  for (int i = 0; i < l.n; i += kTable) {
    Table t;
    const unsigned grid = fill(l, i, chunk, t);
    if (!grid) continue;
    MOE_TIMED_LAUNCH(s, "grad_squares_kernel",
      hipLaunchKernelGGL(grad_squares_kernel, dim3(grid), dim3(kGradThreads), 0, s, t, part + used));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    used += grid;
  }
  MOE_TIMED_LAUNCH(s, "grad_norm_kernel",
    hipLaunchKernelGGL(grad_norm_kernel, dim3(1), dim3(kGradThreads), 0, s, part, used, norm));
  return hipGetLastError();
}

hipError_t launch_grad_scale(const GradList& l, const float* norm, float max_norm, hipStream_t s) {
  const int chunk = chunk_bytes(l);
  for (int i = 0; i < l.n; i += kTable) {
    Table t;
    const unsigned grid = fill(l, i, chunk, t);
    if (!grid) continue;
    MOE_TIMED_LAUNCH(s, "grad_scale_kernel",
      hipLaunchKernelGGL(grad_scale_kernel, dim3(grid), dim3(kGradThreads), 0, s, t, norm,
                         max_norm));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moe
