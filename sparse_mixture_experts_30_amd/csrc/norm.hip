// Residual add and RMS norm in front of the layer, and its backward.
//
//   r = x + residual  (rounded to the activation type: the stream as stored),
//   y = r * rstd * w,   rstd = 1 / sqrt(mean(r^2) + eps),
// and for FP8 experts the same y per 1x128 tile in e4m3: scale a / 448 (or
// the smallest power of two not below it) with a = max |y| of the tile.  The
// tile is quantised from the fp32 y, not from its bf16 rounding: one rounding
// instead of two.  Codes are y times 448 / a rather than y over the scale, one
// multiplication a value: a code at a rounding boundary can differ by a step.
// Backward, with g = dy * w and n = r * rstd:
//   dr = rstd * (g - n * mean(g * n)) + dsum,   dw = sum over rows of dy * n.
// Sums are fp32 in a fixed order.
#include "block.hpp"
#include "rows_device.hpp"

#include <algorithm>

namespace moe {

namespace {

// e4m3fn codes of four values: round to nearest even, saturated at 448, NaN
// kept NaN (the conversion itself would make a value past 448 NaN).
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  auto sat = [](float v) { return v != v ? v : __builtin_amdgcn_fmed3f(v, -448.0f, 448.0f); };
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(sat(a), sat(b), 0, false);
  r = __builtin_amdgcn_cvt_pk_fp8_f32(sat(c), sat(d), r, true);
  return (uint32_t)r;
}

// The tile scales of fp8_device.hpp without 64-bit arithmetic, which is most
// of a decode batch's time here: a / 448 and 448 / a in fp32 are the rounded
// 64-bit quotients (a quotient of two 24-bit numbers rounds the same through
// 53 bits), and the smallest power of two >= a / 448 = a / (1.75 2^8) follows
// from a's exponent and from whether its mantissa exceeds 1.75.
__device__ __forceinline__ void row_tile_scale(float amax, bool pow2, float& scale, float& inv) {
  if (!(amax > 0.0f)) {
    scale = 1.0f;
    inv = 0.0f;
  } else if (pow2) {
    const uint32_t u = __float_as_uint(amax);
    const int x = (int)(u >> 23);   // 255: infinity
    const int e = x == 255 ? 127 : max(x - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0), -126);
    scale = __uint_as_float((uint32_t)(e + 127) << 23);
    inv = __uint_as_float((uint32_t)(127 - e) << 23);
  } else {
    scale = amax / 448.0f;
    inv = 448.0f / amax;
  }
}

// e4m3 codes of the 8 values v (one chunk; 16 consecutive lanes hold a tile)
// and the tile's scale.  All 16 lanes of the tile call this; v is scratch.
__device__ __forceinline__ uint2 quant_chunk(float (&v)[8], bool pow2, float& scale) {
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[j]));
  m = row_max(m);   // the tile's 16 lanes are a row
  float inv;
  row_tile_scale(m, pow2, scale, inv);
  if (m < 0x1p-119f && m > 0.0f && !pow2) {
    // 448 / m is past fp32 (its infinity times a zero of the tile is NaN): the
    // values are lifted by 2^64 first, exactly.  A scale that rounds to 0
    // makes the tile one of zeros.
    inv = 448.0f / (m * 0x1p64f);
    if (scale == 0.0f) {
      scale = 1.0f;
      inv = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= 0x1p64f;
  }
  return make_uint2(e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                    e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
}

// r = x + residual of one chunk, rounded as the stream stores it.
template <typename IO>
__device__ __forceinline__ void add_chunk(const RawChunk<IO>& x, bool has_residual,
                                          const RawChunk<IO>& residual, float (&r)[kWidth<IO>]) {
  x.to(r);
  if (!has_residual) return;
  float b[kWidth<IO>];
  residual.to(b);
#pragma unroll
  for (int j = 0; j < kWidth<IO>; ++j) r[j] = as_stored<IO>(r[j] + b[j]);
}

// Sums over the workgroup of N values per thread in a fixed order, one
// barrier; every thread gets them.  red holds N * 16 floats that the previous
// call does not use (calls alternate halves).
template <int N>
__device__ __forceinline__ void workgroup_sums(float (&v)[N], float* red) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  const int waves = blockDim.x >> 6, lane = threadIdx.x & 63;
  if (waves == 1) return;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) red[16 * i + (threadIdx.x >> 6)] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i)
    v[i] = lane_value(row_sum(lane < waves ? red[16 * i + lane] : 0.0f), 0);   // waves <= 16
}

// One workgroup per row.  A row of up to NC * blockDim.x chunks stays in
// registers between the sum of squares and the output (NC > 0); longer rows
// (NC = 0) are read twice.
// sum may be x or residual itself: a thread rewrites only chunks that it
// alone reads, after reading them.
// kNt: x, residual and sum pass the caches by (see kStreamBytes).
template <typename IO, int NC, bool kNt>
__global__ void __launch_bounds__(1024)
add_rmsnorm_kernel(const IO* x, const IO* residual, const float* __restrict__ weight, float eps,
                   int H, IO* sum, IO* y, uint8_t* __restrict__ yq, float* __restrict__ ys,
                   bool pow2) {
  __shared__ float red[16];
  const int64_t row = (int64_t)blockIdx.x * H;
  constexpr int W = kWidth<IO>;
  const int nc = H / W;
  auto finish = [&](int c, float (&r)[W], const float (&w)[W], float rstd) {
    if (sum) store_chunk<kNt>(sum + row + c * W, r);
#pragma unroll
    for (int j = 0; j < W; ++j) r[j] = r[j] * rstd * w[j];
    if (y) store_chunk(y + row + c * W, r);
    if constexpr (W == 8) {   // bf16
      if (yq) {
        float scale;
        *reinterpret_cast<uint2*>(yq + row + c * 8) = quant_chunk(r, pow2, scale);
        if ((c & 15) == 0) ys[(row >> 7) + (c >> 4)] = scale;
      }
    }
  };
  auto load = [&](int c, float (&r)[W]) {
    RawChunk<IO> a, b{};
    a.load(x + row + c * W);
    if (residual) b.load(residual + row + c * W);
    add_chunk(a, residual != nullptr, b, r);
  };
  float ss[1] = {0.0f};
  if constexpr (NC > 0) {
    RawChunk<IO> a[NC], b[NC];
    float r[NC][W], w[NC][W];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      if (c < nc) a[i].template load<kNt>(x + row + c * W);
    }
    if (residual) {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c < nc) b[i].template load<kNt>(residual + row + c * W);
      }
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      if (c < nc) load_f32(weight + c * W, w[i]);
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      if (c >= nc) break;
      add_chunk(a[i], residual != nullptr, b[i], r[i]);
#pragma unroll
      for (int j = 0; j < W; ++j) ss[0] = fmaf(r[i][j], r[i][j], ss[0]);
    }
    workgroup_sums(ss, red);
    const float rstd = 1.0f / sqrtf(ss[0] / (float)H + eps);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      if (c < nc) finish(c, r[i], w[i], rstd);
    }
  } else {
    float r[W];
    for (int c = threadIdx.x; c < nc; c += blockDim.x) {
      load(c, r);
#pragma unroll
      for (int j = 0; j < W; ++j) ss[0] = fmaf(r[j], r[j], ss[0]);
    }
    workgroup_sums(ss, red);
    const float rstd = 1.0f / sqrtf(ss[0] / (float)H + eps);
    for (int c = threadIdx.x; c < nc; c += blockDim.x) {
      float w[W];
      load(c, r);
      load_f32(weight + c * W, w);
      finish(c, r, w, rstd);
    }
  }
}

// Workgroup b takes rows b, b + gridDim.x, ... and writes its share of dw to
// its row of `part` [gridDim.x][H].  Rows of up to NC * blockDim.x chunks
// (NC > 0): each thread keeps its columns' weight and dw in registers, reads
// every value once, and has the next row's loads in flight during the sums.
// Longer rows (NC = 0) are read twice and dw is kept in `part`.
// kNt: the rows read pass the caches by (see kStreamBytes).
template <typename IO, int NC, bool kNt>
__global__ void __launch_bounds__(1024)
add_rmsnorm_backward_kernel(const IO* __restrict__ sum, const float* __restrict__ weight,
                            float eps, const IO* dy, const IO* dsum, int64_t rows, int H, IO* dx,
                            float* __restrict__ part) {
  __shared__ float red[2][32];
  constexpr int W = kWidth<IO>;
  const int nc = H / W;
  float* mine = part + (int64_t)blockIdx.x * H;
  int turn = 0;
  if constexpr (NC > 0) {
    float w[NC][W], dw[NC][W];
    RawChunk<IO> r[NC], g[NC], nr[NC], ng[NC];
    auto fetch = [&](int64_t t) {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c >= nc) break;
        nr[i].template load<kNt>(sum + t * H + c * W);
        ng[i].template load<kNt>(dy + t * H + c * W);
      }
    };
    fetch(blockIdx.x);   // the grid has at most `rows` workgroups
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      if (c < nc) load_f32(weight + c * W, w[i]);
#pragma unroll
      for (int j = 0; j < W; ++j) dw[i][j] = 0.0f;
    }
    for (int64_t t = blockIdx.x; t < rows; t += gridDim.x, turn ^= 1) {
      float sums[2] = {0.0f, 0.0f};   // r^2, g w r
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        r[i] = nr[i];
        g[i] = ng[i];
      }
      RawChunk<IO> d[NC];
      if (dsum) {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          const int c = threadIdx.x + i * blockDim.x;
          if (c < nc) d[i].template load<kNt>(dsum + t * H + c * W);
        }
      }
      if (t + gridDim.x < rows) fetch(t + gridDim.x);
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c >= nc) break;
        float rv[W], gv[W];
        r[i].to(rv);
        g[i].to(gv);
#pragma unroll
        for (int j = 0; j < W; ++j) {
          sums[0] = fmaf(rv[j], rv[j], sums[0]);
          sums[1] = fmaf(gv[j] * w[i][j], rv[j], sums[1]);
        }
      }
      workgroup_sums(sums, red[turn]);
      const float rstd = 1.0f / sqrtf(sums[0] / (float)H + eps);
      const float mean = sums[1] * rstd / (float)H;   // mean(g * n)
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c >= nc) break;
        float rv[W], gv[W], dv[W];
        r[i].to(rv);
        g[i].to(gv);
        if (dsum) d[i].to(dv);
#pragma unroll
        for (int j = 0; j < W; ++j) {
          const float n = rv[j] * rstd;
          dw[i][j] = fmaf(gv[j], n, dw[i][j]);
          rv[j] = rstd * (gv[j] * w[i][j] - n * mean) + (dsum ? dv[j] : 0.0f);
        }
        store_chunk(dx + t * H + c * W, rv);
      }
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      if (c < nc) store_f32(mine + c * W, dw[i]);
    }
  } else {
    for (int64_t t = blockIdx.x; t < rows; t += gridDim.x, turn ^= 1) {
      const int64_t row = t * H;
      float sums[2] = {0.0f, 0.0f};   // r^2, g w r
      for (int c = threadIdx.x; c < nc; c += blockDim.x) {
        float r[W], g[W], w[W];
        load_chunk(sum + row + c * W, r);
        load_chunk(dy + row + c * W, g);
        load_f32(weight + c * W, w);
#pragma unroll
        for (int j = 0; j < W; ++j) {
          sums[0] = fmaf(r[j], r[j], sums[0]);
          sums[1] = fmaf(g[j] * w[j], r[j], sums[1]);
        }
      }
      workgroup_sums(sums, red[turn]);
      const float rstd = 1.0f / sqrtf(sums[0] / (float)H + eps);
      const float mean = sums[1] * rstd / (float)H;
      for (int c = threadIdx.x; c < nc; c += blockDim.x) {
        float r[W], g[W], w[W], a[W], d[W];
        load_chunk(sum + row + c * W, r);
        load_chunk(dy + row + c * W, g);
        load_f32(weight + c * W, w);
        if (dsum) load_chunk(dsum + row + c * W, d);
        if (t != blockIdx.x) load_f32(mine + c * W, a);
#pragma unroll
        for (int j = 0; j < W; ++j) {
          const float n = r[j] * rstd;
          a[j] = fmaf(g[j], n, t != blockIdx.x ? a[j] : 0.0f);
          r[j] = rstd * (g[j] * w[j] - n * mean) + (dsum ? d[j] : 0.0f);
        }
        store_f32(mine + c * W, a);
        store_chunk(dx + row + c * W, r);
      }
    }
  }
}

// dw[h] = sum of part[b][h] over b; zeros for nparts = 0.  A workgroup takes
// 32 columns (one 128-byte line of every part): thread (q, slice) sums the
// parts slice, slice + 32, ... of columns 4q..4q+3, and the 32 slices are
// joined through LDS in a fixed order.
constexpr int kDwCols = 32, kDwSlices = 32;
__global__ void __launch_bounds__(256)
rmsnorm_dweight_kernel(const float* __restrict__ part, int nparts, int H,
                       float* __restrict__ dweight) {
  __shared__ f32x4 lds[kDwSlices][kDwCols / 4 + 1];
  const int q = threadIdx.x & 7, slice = threadIdx.x >> 3;
  const int h = blockIdx.x * kDwCols + q * 4;   // H is a multiple of 64
  f32x4 a = {0.f, 0.f, 0.f, 0.f};
  constexpr int B = 8;   // parts whose loads are issued together
  for (int b0 = slice; b0 < nparts; b0 += B * kDwSlices) {
    f32x4 v[B];
#pragma unroll
    for (int u = 0; u < B; ++u) {
      const int b = b0 + u * kDwSlices;
      v[u] = (f32x4){0.f, 0.f, 0.f, 0.f};
      if (b < nparts) v[u] = *reinterpret_cast<const f32x4*>(part + (int64_t)b * H + h);
    }
#pragma unroll
    for (int u = 0; u < B; ++u) a += v[u];
  }
  lds[slice][q] = a;
  __syncthreads();
  if (slice >= 4) return;
  // thread (q, slice): column quad q, sums 8 slices each, then lane shuffles
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int u = 0; u < kDwSlices / 4; ++u) s += lds[slice * (kDwSlices / 4) + u][q];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    s[j] += __shfl_xor(s[j], 8, 64);
    s[j] += __shfl_xor(s[j], 16, 64);
  }
  if (slice == 0) *reinterpret_cast<f32x4*>(dweight + h) = s;
}

// Chunks of a row that a thread of the forward holds in registers: two, four
// from 2048 chunks on, none (the row is read twice) past 4096.
int norm_held(int chunks) { return chunks > 4096 ? 0 : chunks > 2048 ? 4 : 2; }

// Threads of a workgroup for rows of `chunks` held as nc chunks a thread (as
// four if none are held).
int norm_threads(int chunks, int nc) {
  const int n = nc ? nc : 4;
  return std::min(1024, (chunks + 64 * n - 1) / (64 * n) * 64);
}

// Row sums of dw kept apart at most: two workgroups per CU (256 instead of 512
// take 61 us instead of 55 at T = 4096, H = 7168).
constexpr int64_t kNormParts = 512;

// Arrays of rows past this size are read (and the sum written)
// non-temporally.  Measured at H = 7168, bf16, cached -> non-temporal: forward
// 12.7 -> 13.4 us at 15 MB an array, 26.4 -> 25.0 at 29 MB, 46.5 -> 42.7 at
// 59 MB; backward 20.2 -> 23.1, 32.2 -> 30.7, 53.9 -> 48.7 us.  With a kernel
// before that writes x or dy and one after that reads y or dx the three stay
// within 1% of each other from 29 MB on (95.0 -> 94.3 and 100.3 -> 100.7 us at
// 59 MB).
constexpr int64_t kStreamBytes = 24000000;

}  // namespace

size_t rmsnorm_backward_ws_bytes(int64_t rows, int H) {
  return ((size_t)std::min(rows, kNormParts) * H * sizeof(float) + 255) / 256 * 256;
}

template <typename IO, int NC, bool kNt>
static void add_rmsnorm(const void* x, const void* residual, const float* weight, float eps,
                        int64_t rows, int H, void* sum, void* y, uint8_t* yq, float* ys,
                        bool pow2, hipStream_t s) {
  MOE_TIMED_LAUNCH(s, "add_rmsnorm_kernel",
    hipLaunchKernelGGL((add_rmsnorm_kernel<IO, NC, kNt>), dim3((unsigned)rows),
                       dim3(norm_threads(H / kWidth<IO>, NC)), 0, s, (const IO*)x,
                       (const IO*)residual, weight, eps, H, (IO*)sum, (IO*)y, yq, ys, pow2));
}

template <typename IO>
static hipError_t add_rmsnorm(const void* x, const void* residual, const float* weight, float eps,
                              int64_t rows, int H, void* sum, void* y, uint8_t* yq, float* ys,
                              bool pow2, hipStream_t s) {
  const int held = norm_held(H / kWidth<IO>);
  auto* run = held == 0   ? add_rmsnorm<IO, 0, false>
              : held == 4 ? add_rmsnorm<IO, 4, false>
              : rows * H * (int64_t)sizeof(IO) > kStreamBytes ? add_rmsnorm<IO, 2, true>
                                                              : add_rmsnorm<IO, 2, false>;
  run(x, residual, weight, eps, rows, H, sum, y, yq, ys, pow2, s);
  return hipGetLastError();
}

int64_t add_rmsnorm_max_rows(int H, bool bf16) {
  const int chunks = H / (bf16 ? kWidth<uint16_t> : kWidth<float>);
  return kMaxGridThreads / norm_threads(chunks, norm_held(chunks));
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
    // Two chunks a thread; wider rows leave no registers for a thread's share
    // of dw.
    constexpr int NC = 2;
    const int chunks = H / kWidth<IO>;
    const bool wide = chunks > 1024 * NC;
    auto* kernel = wide ? add_rmsnorm_backward_kernel<IO, 0, false>
                   : rows * H * (int64_t)sizeof(IO) > kStreamBytes
                       ? add_rmsnorm_backward_kernel<IO, NC, true>
                       : add_rmsnorm_backward_kernel<IO, NC, false>;
    MOE_TIMED_LAUNCH(s, "add_rmsnorm_backward_kernel",
      hipLaunchKernelGGL(kernel, dim3((unsigned)parts), dim3(norm_threads(chunks, wide ? 0 : NC)),
                         0, s, (const IO*)sum, weight, eps, (const IO*)dy, (const IO*)dsum, rows, H,
                         (IO*)dx, part));
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  MOE_TIMED_LAUNCH(s, "rmsnorm_dweight_kernel",
    hipLaunchKernelGGL(rmsnorm_dweight_kernel, dim3(H / kDwCols), dim3(256), 0, s, part,
                       (int)parts, H, dweight));
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
