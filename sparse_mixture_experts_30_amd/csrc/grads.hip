// Global norm over many gradients, and clipping to it (gfx950).
//   norm = sqrt(sum over all of g^2),  out = g min(1, max_norm / (norm + 1e-6)).
// Squares are summed in 64 bits, which the vector units have at half the rate
// of fp32, far above what memory delivers: no square and no sum overflows and
// the order of the sums does not show.  The norm itself is an fp32 number, which
// the caller has and the factor is made from: above 3.4e38 it is infinite, and
// counts as not finite.  Bound by memory: one read for the norm, one read and
// one write for the scaling.
//
// Gradients that lie one behind the other, like their outputs, count as one (the
// pieces of flat buffers; one run per type is watched).  They are cut into
// chunks of equal size that start on 16-byte addresses (the first takes what
// lies before the first such address); a workgroup takes every gridDim'th
// chunk, the scaling from the last one on, which the caches still hold.  The
// table of gradients travels as a kernel argument, so nothing is copied to the
// device and a call can be captured; lists longer than a table take several
// launches.  With one table the scaling's workgroups each join the partial sums
// themselves (a launch less, 4 us), with several a kernel does it between.
#include "grads.hpp"

#include <math.h>

#include <algorithm>

namespace moe {

namespace {

constexpr int kTable = 168;           // runs a launch (the argument stays under 4 KiB)
constexpr int kGradThreads = 256;
constexpr int kGradBlocks = 2048;     // workgroups a launch at most, and partial sums
constexpr int64_t kMostValues = 1 << 30;   // of one run
// The scaling passes the caches by: it is the gradients' last reader here and
// its stores would push out what it still has to read (76 MB 52 -> 44 us, 300 MB
// 182 -> 149).  The norm does so from a size on of which the caches keep nothing
// for the scaling (600 MB 312 us without, 327 with; 2.9 GB 1551 and 1523).
constexpr double kStreamBytes = 1e9;

struct Run {
  const char* g;
  char* out;
  uint32_t n;       // values, and 2^31 for bf16
  int32_t first;    // first chunk
};
struct Table {
  Run run[kTable];
  int32_t count;
  int32_t chunks;
  int32_t chunk;    // bytes
};

// Values before the first 16-byte address.
__host__ __device__ inline int64_t head_of(const void* p, int64_t n, int size) {
  const int64_t h = (int64_t)((16 - ((uintptr_t)p & 15)) & 15) / size;
  return h < n ? h : n;
}

// Calls f(run, whether it is bf16, first value, end) for every chunk of this
// workgroup; kBack: from the last chunk on.
template <bool kBack, class F>
__device__ __forceinline__ void for_chunks(const Table& t, F f) {
  for (int b = blockIdx.x; b < t.chunks; b += gridDim.x) {
    const int c = kBack ? t.chunks - 1 - b : b;
    int lo = 0, hi = t.count - 1;   // the run that holds chunk c
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (t.run[mid].first <= c) lo = mid;
      else hi = mid - 1;
    }
    const Run r = t.run[lo];
    const bool bf16 = r.n >> 31;
    const int size = bf16 ? 2 : 4;
    const int64_t n = r.n & 0x7fffffffu, per = t.chunk / size, head = head_of(r.g, n, size),
                  k = c - r.first;
    f(r, bf16, k ? head + k * per : 0, min(n, head + (k + 1) * per));
  }
}

template <typename IO>
__device__ __forceinline__ float value(IO v) {
  if constexpr (sizeof(IO) == 2) return bf16_bits_to_f32(v);
  else return v;
}

template <bool kNt, typename IO>
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
    const u32x4 q = kNt ? __builtin_nontemporal_load(p + i) : p[i];
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

// Sum over the workgroup in a fixed order.
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

template <bool kNt>
__global__ void __launch_bounds__(kGradThreads)
grad_squares_kernel(Table t, double* __restrict__ part) {
  double s = 0.0;
  for_chunks<false>(t, [&](const Run& r, bool bf16, int64_t a, int64_t b) {
    s += bf16 ? squares<kNt>((const uint16_t*)r.g, a, b)
              : squares<kNt>((const float*)r.g, a, b);
  });
  s = workgroup_sum(s);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// The norm of n partial sums, the same in every workgroup that asks.
__device__ __forceinline__ float joined_norm(const double* __restrict__ part, int64_t n) {
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += kGradThreads) s += part[i];
  return (float)sqrt(workgroup_sum(s));
}

__global__ void __launch_bounds__(kGradThreads)
grad_norm_kernel(const double* __restrict__ part, int64_t n, float* __restrict__ norm) {
  const float v = joined_norm(part, n);
  if (threadIdx.x == 0) *norm = v;
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
    const u32x4 q = __builtin_nontemporal_load(p + i);
    u32x4 r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (sizeof(IO) == 2)
        r[j] = pack_bf16x2(__uint_as_float(q[j] << 16) * f, __uint_as_float(q[j] & 0xFFFF0000u) * f);
      else
        r[j] = __float_as_uint(__uint_as_float(q[j]) * f);
    }
    __builtin_nontemporal_store(r, o + i);
  }
  for (int64_t i = va + nv * W + threadIdx.x; i < b; i += kGradThreads) one(i);
}

// parts > 0: the norm is joined here from that many partial sums, and written;
// else it is read.
__global__ void __launch_bounds__(kGradThreads)
grad_scale_kernel(Table t, const double* __restrict__ part, int parts, float* __restrict__ norm,
                  float max_norm) {
  const float n = parts ? joined_norm(part, parts) : *norm;
  if (parts && blockIdx.x == 0 && threadIdx.x == 0) *norm = n;
  // A norm that is not finite says nothing about the scale: the gradients stay
  // as they are, for the caller to skip the step.
  const float f = isfinite(n) ? fminf(1.0f, max_norm / (n + 1e-6f)) : 1.0f;
  for_chunks<true>(t, [&](const Run& r, bool bf16, int64_t a, int64_t b) {
    if (f == 1.0f && r.g == r.out) return;
    if (bf16) scale((const uint16_t*)r.g, (uint16_t*)r.out, a, b, f);
    else scale((const float*)r.g, (float*)r.out, a, b, f);
  });
}

// The tables of a list, one after another: next() fills one and returns its
// number of workgroups, 0 at the end.
class Tables {
 public:
  Tables(const GradList& l) : l_(l) {
    for (int i = 0; i < l.n; ++i) bytes_ += (double)l.count[i] * (l.bf16[i] ? 2 : 4);
    // Whole turns of the workgroups, of at most 64 KiB a chunk.
    const double turn = (double)kGradBlocks * 65536, turns = std::max(1.0, ceil(bytes_ / turn));
    chunk_ = (int)std::max(1.0, ceil(bytes_ / (kGradBlocks * turns) / 4096)) * 4096;
  }
  double bytes() const { return bytes_; }
  unsigned next(Table& t) {
    t.count = 0;
    t.chunk = chunk_;
    int open[2] = {-1, -1};   // the last run of each type
    for (; i_ < l_.n; ++i_, at_ = 0) {
      const int size = l_.bf16[i_] ? 2 : 4;
      while (at_ < l_.count[i_]) {
        const char* g = (const char*)l_.grad[i_] + at_ * size;
        char* out = l_.out ? (char*)l_.out[i_] + at_ * size : nullptr;
        int& o = open[l_.bf16[i_]];
        const int64_t has = o >= 0 ? (int64_t)(t.run[o].n & 0x7fffffffu) : kMostValues;
        if (has < kMostValues && t.run[o].g + has * size == g &&
            (!out || t.run[o].out + has * size == out)) {
          const int64_t n = std::min(l_.count[i_] - at_, kMostValues - has);
          t.run[o].n += (uint32_t)n;
          at_ += n;
          continue;
        }
        if (t.count == kTable) return close(t);
        o = t.count++;
        const int64_t n = std::min(l_.count[i_] - at_, kMostValues);
        t.run[o] = {g, out, (uint32_t)n | (l_.bf16[i_] ? 0x80000000u : 0u), 0};
        at_ += n;
      }
    }
    return close(t);
  }

 private:
  unsigned close(Table& t) const {
    int64_t c = 0;
    for (int j = 0; j < t.count; ++j) {
      Run& r = t.run[j];
      const int size = r.n >> 31 ? 2 : 4;
      const int64_t n = r.n & 0x7fffffffu, per = chunk_ / size;
      r.first = (int32_t)c;
      c += std::max<int64_t>(1, (n - head_of(r.g, n, size) + per - 1) / per);
    }
    t.chunks = (int32_t)c;
    return (unsigned)std::min<int64_t>(c, kGradBlocks);
  }
  const GradList& l_;
  int i_ = 0;
  int64_t at_ = 0;
  double bytes_ = 0;
  int chunk_;
};

hipError_t launch_squares(const GradList& l, double* part, int64_t* parts, int* tables,
                          hipStream_t s) {
  Tables tables_of(l);
  Table t;
  *parts = 0;
  *tables = 0;
  while (const unsigned grid = tables_of.next(t)) {
    MOE_TIMED_LAUNCH(s, "grad_squares_kernel",
      hipLaunchKernelGGL((tables_of.bytes() > kStreamBytes ? grad_squares_kernel<true>
                                                           : grad_squares_kernel<false>),
                         dim3(grid), dim3(kGradThreads), 0, s, t, part + *parts));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    *parts += grid;
    ++*tables;
  }
  return hipSuccess;
}

hipError_t launch_norm(const double* part, int64_t parts, float* norm, hipStream_t s) {
  MOE_TIMED_LAUNCH(s, "grad_norm_kernel",
    hipLaunchKernelGGL(grad_norm_kernel, dim3(1), dim3(kGradThreads), 0, s, part, parts, norm));
  return hipGetLastError();
}

}  // namespace

size_t grad_norm_ws_bytes(const GradList& l) {
  // A table holds kTable runs or more gradients, of kMostValues each at most.
  int64_t runs = 0;
  for (int i = 0; i < l.n; ++i) runs += (l.count[i] + kMostValues - 1) / kMostValues;
  return (size_t)(runs / kTable + 1) * kGradBlocks * sizeof(double);
}

hipError_t launch_grad_norm(const GradList& l, double* part, float* norm, hipStream_t s) {
  int64_t parts;
  int tables;
  const hipError_t e = launch_squares(l, part, &parts, &tables, s);
  return e != hipSuccess ? e : launch_norm(part, parts, norm, s);
}

hipError_t launch_clip(const GradList& l, double* part, float* norm, bool norm_given,
                       float max_norm, hipStream_t s) {
  int64_t parts = 0;
  int tables = 0;
  hipError_t e;
  if (!norm_given) {
    e = launch_squares(l, part, &parts, &tables, s);
    if (e == hipSuccess && tables != 1) e = launch_norm(part, parts, norm, s);
    if (e != hipSuccess) return e;
    if (tables != 1) parts = 0;
  }
  Tables tables_of(l);
  Table t;
  while (const unsigned grid = tables_of.next(t)) {
    MOE_TIMED_LAUNCH(s, "grad_scale_kernel",
      hipLaunchKernelGGL(grad_scale_kernel, dim3(grid), dim3(kGradThreads), 0, s, t, part,
                         (int)parts, norm, max_norm));
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moe
