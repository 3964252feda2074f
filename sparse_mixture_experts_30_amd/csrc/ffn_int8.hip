// Expert FFNs in 8-bit integers (gfx950), for serving: activations with one
// scale per token row, weights with one scale per output channel,
//   q[t][k] = round(127 x[t][k] / max_k |x[t][k]|),  s[t] = max / 127,
//   y[t][n] = s[t] c[n] sum_k q[t][k] w[n][k],
// the sums in 32-bit integers over the whole k (exact: |sum| <= 127^2 k, so k
// up to 131072).  h = silu(g) u is kept in fp32 between the two products and
// quantised per row like x: rounding it to bf16 first would move a tenth of
// its codes by a step (five times the error of the bf16 outputs).
//
// Layout (pack_int8): per output tile (64 h columns of gate and up together,
// or 128 output rows of the down projection) and 128-k step one block of 16
// KiB: eight fragments of 16 rows, each two 1 KiB halves of 64 k, lane l of a
// half holding row l % 16, k = 64 half + 16 (l / 16) + 0..15.  Fragments 0, 1
// and 4, 5 of a gate/up tile are gate rows of its first and second 32 columns,
// 2, 3 and 6, 7 the up rows of the same.
#include "block.hpp"
#include "gemm_device.hpp"
#include "items_device.hpp"
#include "rows_device.hpp"

#include <algorithm>

namespace moe {

namespace {

typedef int i32x16 __attribute__((ext_vector_type(16)));

constexpr int kThreads8 = 256;
constexpr int kStepK = 128;          // k per packed step
constexpr int kFrags = 8;            // 16-row fragments per tile
constexpr int kUnits = kFrags * 128; // 16-byte units of a step block

struct Int8Args : ItemArgs {
  const int8_t* a_r;            // rows of codes, row length kdim
  const int8_t* a_s;
  const float* as_r;            // row scales
  const float* as_s;
  const int32_t* perm;          // gate/up: routed A row = perm[j] / K
  int kdim_r, kdim_s;
  const u32x4* b_r;             // packed routed weights
  int nt_r;                     // output tiles per routed expert
  const u32x4* b_s;
  int nt_s;
  const float* bs_r;            // channel scales [E][channels]
  const float* bs_s;
  int ncol_r, ncol_s;           // h columns (gate/up) or output columns
  void* c_r;                    // fp32 h or bf16 y, row length ncol
  void* c_s;
};

__device__ __forceinline__ i32x4 mfma_i8(u32x4 a, u32x4 b, i32x4 c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a),
                                               __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}

__device__ __forceinline__ float swiglu(float g, float u) { return g / (1.0f + __expf(-g)) * u; }

// ---------------------------------------------------------------- few rows
// A tile of at most 16 rows and one packed output tile; the four waves take a
// quarter of the k steps each, their integer sums are joined through LDS.
constexpr int kFewRows = 16;
constexpr int kFewWaves = 4;

template <bool kGateUp, bool kStream>
__device__ __forceinline__ void int8_few_tile(const Int8Args& p, int* lds, const Item& it) {
  const bool sh = it.g == p.E;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int lr = lane & 15, lq = lane >> 4;
  const int kdim = sh ? p.kdim_s : p.kdim_r, nsteps = kdim / kStepK;
  const int s0 = nsteps * wave / kFewWaves, s1 = nsteps * (wave + 1) / kFewWaves;
  const u32x4* bw = (sh ? p.b_s : p.b_r + (int64_t)it.g * p.nt_r * nsteps * kUnits) +
                    (int64_t)it.ntile * nsteps * kUnits + lane;
  u32x4 rb[kFrags][2], ra[2];
  auto load_w = [&](int step) {
    const u32x4* src = bw + (int64_t)step * kUnits;
#pragma unroll
    for (int b = 0; b < kFrags; ++b)
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const u32x4* q = src + (b * 2 + f) * 64;
        rb[b][f] = kStream ? __builtin_nontemporal_load(q) : *q;
      }
  };
  if (s0 < s1) load_w(s0);
  // This lane's row (past the end the first one; those results are not stored).
  const int rr = lr < it.nrows ? lr : 0;
  const int arow = (!sh && kGateUp) ? p.perm[it.row0 + rr] / p.K : it.row0 + rr;
  const int8_t* ap = (sh ? p.a_s : p.a_r) + (int64_t)arow * kdim + lq * 16;
  auto load_a = [&](int step) {
#pragma unroll
    for (int f = 0; f < 2; ++f)
      ra[f] = *reinterpret_cast<const u32x4*>(ap + step * kStepK + f * 64);
  };
  if (s0 < s1) load_a(s0);
  i32x4 acc[kFrags];
#pragma unroll
  for (int b = 0; b < kFrags; ++b) acc[b] = (i32x4){0, 0, 0, 0};
  auto compute = [&]() {
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int b = 0; b < kFrags; ++b) acc[b] = mfma_i8(ra[f], rb[b][f], acc[b]);
  };
  int s = s0;
  for (; s + 1 < s1; ++s) {
    compute();
    load_w(s + 1);
    load_a(s + 1);
  }
  if (s < s1) compute();

  // [wave][frag][row 16][col 16]
#pragma unroll
  for (int b = 0; b < kFrags; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      lds[((wave * kFrags + b) * 16 + 4 * lq + i) * 16 + lr] = acc[b][i];
  __syncthreads();
  const int row = tid >> 4;   // 16 threads a row
  if (row >= it.nrows) return;
  const int64_t crow = it.row0 + row;
  const int64_t srow = (!sh && kGateUp) ? p.perm[crow] / p.K : crow;
  const float as = (sh ? p.as_s : p.as_r)[srow];
  const int ncol = sh ? p.ncol_s : p.ncol_r;
  const float* bs = sh ? p.bs_s : p.bs_r + (int64_t)it.g * (kGateUp ? 2 : 1) * ncol;
  // Four neighbouring sums of fragment b from column col, scaled.
  auto joined = [&](int b, int col, const float* scale) {
    i32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < kFewWaves; ++w)
      v += *reinterpret_cast<const i32x4*>(lds + ((w * kFrags + b) * 16 + row) * 16 + col);
    const f32x4 c = *reinterpret_cast<const f32x4*>(scale);
    f32x4 r;
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j] = (float)v[j] * (as * c[j]);
    return r;
  };
  if (kGateUp) {
    const int col = (tid & 15) * 4, b = (col >> 5) * 4 + (col >> 4 & 1), n = it.ntile * 64 + col;
    const f32x4 gv = joined(b, col & 15, bs + n), uv = joined(b + 2, col & 15, bs + ncol + n);
    f32x4 h;
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = swiglu(gv[j], uv[j]);
    *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(sh ? p.c_s : p.c_r) + crow * ncol + n) = h;
  } else {
    const int col = (tid & 15) * 8, b = col >> 4, n = it.ntile * 128 + col;
    const f32x4 v = joined(b, col & 15, bs + n), w = joined(b, (col & 15) + 4, bs + n + 4);
    *reinterpret_cast<u32x4*>(reinterpret_cast<uint16_t*>(sh ? p.c_s : p.c_r) + crow * ncol + n) =
        (u32x4){pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(w[0], w[1]),
                pack_bf16x2(w[2], w[3])};
  }
}

template <bool kGateUp>
__global__ void __launch_bounds__(kThreads8) grouped_gemm_int8_few(Int8Args p) {
  __shared__ __align__(16) int lds[kFewWaves * kFrags * 256];
  Item it;
  if (!find_item<kFewRows>(p, it)) return;
  if (it.ntile >= (it.g == p.E ? p.nt_s : p.nt_r)) return;
  // A weight tile that only this row tile reads is not kept in cache.
  if (it.alone)
    int8_few_tile<kGateUp, true>(p, lds, it);
  else
    int8_few_tile<kGateUp, false>(p, lds, it);
}

// --------------------------------------------------------------- many rows
// A tile of at most 128 rows and two packed output tiles, four waves of all rows
// x 64 columns, two workgroups a CU.  Each weight goes straight to the registers
// of the one wave that multiplies it, its load started two steps ahead; the rows
// pass through three LDS stages that loads from memory fill directly.  The waits
// for a slice's weights are the compiler's, which counts the 14 loads of weights
// behind them but not the rows' loads to LDS in between (inline assembly): with
// four row blocks the newest 14 loads of both kinds may be under way, 1.2 steps.
// Waits for the weights alone (22 and 21 loads behind) were not measured.
// Bound by HBM up to about 128 rows an expert: T = 4096 (H = 7168, I = 2048,
// top-8 of 256) 2.83 ms
// with both quantisers, 4.2 TB/s of weights and rows counted once; the kernels
// themselves move 5.0 (experts of several tiles, rows read by more than one XCD).
// A step of a workgroup takes 1.2 us, about what its matrix instructions, its LDS
// reads and its loads take one after another.  Tiles of 256 rows, one workgroup a
// CU: 4.06 ms; both operands through LDS, eight waves in step: 3.04; the step's
// loads behind its matrix instructions instead of among them: 2.96.
constexpr int kManyRows = 128;

// Place of 16-byte chunk c of row r among a step's rows of eight chunks.
__device__ __forceinline__ int token_chunk(int r, int c) {
  return r * 8 + (c ^ (r & 7) ^ (r >> 3 & 3));
}

template <bool kGateUp, int kMI, bool kStream>
__device__ __forceinline__ void int8_many_tile(const Int8Args& p, u32x4* lds, const Item& it) {
  constexpr int kStage = kMI * 32 * 8;   // pieces of a step's rows
  const bool sh = it.g == p.E;
  const int tid = threadIdx.x, lane = tid & 63, lr = lane & 31, lh = lane >> 5;
  const int wave = (int)scalar(tid >> 6);
  const int kdim = sh ? p.kdim_s : p.kdim_r, nsteps = kdim / kStepK;
  const int nt = sh ? p.nt_s : p.nt_r;
  // An odd number of packed tiles leaves the last pair's second half to no
  // one: its waves repeat the first half and store nothing.
  const int tile = it.ntile * 2 + (wave >> 1);
  const bool mine = tile < nt;
  // Fragments 4 (wave & 1) + 2 j and + 2 j + 1 are the wave's column block j (gate
  // and up, or 32 columns each).
  const u32x4* bw = (sh ? p.b_s : p.b_r + (int64_t)it.g * nt * nsteps * kUnits) +
                    (int64_t)(mine ? tile : tile - 1) * nsteps * kUnits;
  const int bl = ((wave & 1) * 4 + (lr >> 4)) * 128 + lh * 16 + (lr & 15);
  u32x4 rb[2][2][4];   // [slot][column block][k slice of 32]
  auto load_w = [&](int slot, int step, int t) {
    // Past the last step one piece for all lanes (the last step again came from
    // memory a second time, an eighth of the down projection's weights).
    const u32x4* src = bw + (step < nsteps ? step * kUnits + bl : 0);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const u32x4* q = src + j * 256 + (t >> 1) * 64 + (t & 1) * 32;
      rb[slot][j][t] = kStream ? __builtin_nontemporal_load(q) : *q;
    }
  };
  // Rows tid / 8 + 32 i; past the end the first row again (not stored).
  const char* src_a[kMI];
#pragma unroll
  for (int i = 0; i < kMI; ++i) {
    const int r = (tid >> 3) + 32 * i, rr = r < it.nrows ? r : 0;
    const int arow = (!sh && kGateUp) ? p.perm[it.row0 + rr] / p.K : it.row0 + rr;
    src_a[i] = reinterpret_cast<const char*>(sh ? p.a_s : p.a_r) + (int64_t)arow * kdim +
               (token_chunk(r, tid & 7) - r * 8) * 16;
  }
  const uint32_t lds_at = lds_address(lds) + wave * 1024;
  auto load_a = [&](int stage, int step, int i) {
    load_global_to_lds(src_a[i] + min(step, nsteps - 1) * kStepK,
                       lds_at + (stage * kStage + i * 256) * 16);
  };

  i32x16 acc[kMI][2];
#pragma unroll
  for (int i = 0; i < kMI; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0;
  // Slice t of step s in its stage: behind its MFMAs the loads of the rows' pass t
  // and of the slice's weights of step s + 2 are started, into the stage that
  // step s - 1 has read and into the registers that the slice has.
  auto slice = [&](const i32x4 (&a)[kMI], int stage, int slot, int t, int s) {
#pragma unroll
    for (int i = 0; i < kMI; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(
            a[i], __builtin_bit_cast(i32x4, rb[slot][j][t]), acc[i][j], 0, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
    if (t < kMI) load_a((stage + 2) % 3, s + 2, t);
    load_w(slot, s + 2, t);
    __builtin_amdgcn_sched_barrier(0);
  };
  // Loads behind the last of a step's rows: the weights of its slices from there
  // on, then a whole step's.
  constexpr int kAhead = 2 * (5 - kMI) + 8 + kMI;
  auto one = [&](int stage, int slot, int s) {
    const u32x4* l = lds + stage * kStage;
    i32x4 a[2][kMI];   // a slice's rows are read while the one before is multiplied
    auto read = [&](int t) {
#pragma unroll
      for (int i = 0; i < kMI; ++i)
        a[t & 1][i] = __builtin_bit_cast(i32x4, l[token_chunk(i * 32 + lr, 2 * t + lh)]);
    };
    wait_and_meet<kAhead>();
    read(0);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if (t < 3) read(t + 1);
      __builtin_amdgcn_sched_barrier(0);
      slice(a[t & 1], stage, slot, t, s);
    }
  };
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if (t < kMI) load_a(s, s, t);
      load_w(s, s, t);
      __builtin_amdgcn_sched_barrier(0);
    }
  // Left by breaks: where a path joins that skips a step the compiler takes the
  // weights for just loaded and waits for all.
  for (int s = 0;;) {
    one(0, 0, s);
    if (++s >= nsteps) break;
    one(1, 1, s);
    if (++s >= nsteps) break;
    one(2, 0, s);
    if (++s >= nsteps) break;
    one(0, 1, s);
    if (++s >= nsteps) break;
    one(1, 0, s);
    if (++s >= nsteps) break;
    one(2, 1, s);
    if (++s >= nsteps) break;
  }
  wait_and_meet<0>();   // the stages are free
  if (!mine) return;    // the whole wave; nothing waits behind this

  const int ncol = sh ? p.ncol_s : p.ncol_r;
  const float* as = sh ? p.as_s : p.as_r;
  const float* bs = sh ? p.bs_s : p.bs_r + (int64_t)it.g * (kGateUp ? 2 : 1) * ncol;
  f32x16 v[kMI][2];
#pragma unroll
  for (int i = 0; i < kMI; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) v[i][j][q] = (float)acc[i][j][q];
  float* l = reinterpret_cast<float*>(lds) + wave * (32 * 64);
  auto scaled = [&](float (&x)[8], float s, const float* c) {
    const f32x4 c0 = *reinterpret_cast<const f32x4*>(c),
                c1 = *reinterpret_cast<const f32x4*>(c + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[j] *= s * c0[j];
      x[4 + j] *= s * c1[j];
    }
  };
  if constexpr (kGateUp) {
    const int col0 = tile * 64 + (wave & 1) * 32;
    wave_rows<true>(l, v, [&](int row, int c, float (&g)[8], float (&u)[8]) {
      if (row >= it.nrows) return;
      const int col = col0 + c;
      const int64_t crow = it.row0 + row;
      const float s = as[sh ? crow : p.perm[crow] / p.K];
      scaled(g, s, bs + col);
      scaled(u, s, bs + ncol + col);
      f32x4* o = reinterpret_cast<f32x4*>(reinterpret_cast<float*>(sh ? p.c_s : p.c_r) +
                                          crow * ncol + col);
#pragma unroll
      for (int j = 0; j < 2; ++j)
        o[j] = (f32x4){swiglu(g[4 * j], u[4 * j]), swiglu(g[4 * j + 1], u[4 * j + 1]),
                       swiglu(g[4 * j + 2], u[4 * j + 2]), swiglu(g[4 * j + 3], u[4 * j + 3])};
    });
  } else {
    const int col0 = tile * 128 + (wave & 1) * 64;
    wave_rows<false>(l, v, [&](int row, int c, float (&x)[8]) {
      if (row >= it.nrows) return;
      const int col = col0 + c;
      const int64_t crow = it.row0 + row;
      scaled(x, as[crow], bs + col);
      *reinterpret_cast<u32x4*>(reinterpret_cast<uint16_t*>(sh ? p.c_s : p.c_r) + crow * ncol +
                                col) = pack_bf16x8(x);
    });
  }
}

template <bool kGateUp>
__global__ void __launch_bounds__(kThreads8, 2) grouped_gemm_int8_many(Int8Args p) {
  __shared__ u32x4 lds[3 * kManyRows * 8];
  Item it;
  if (!find_item<kManyRows>(p, it)) return;
  if (2 * it.ntile >= (it.g == p.E ? p.nt_s : p.nt_r)) return;
  const int blocks = (it.nrows + 31) >> 5;
#define MOE_INT8_CASE(n)                                               \
  if (blocks == n) {                                                   \
    if (it.alone) int8_many_tile<kGateUp, n, true>(p, lds, it);        \
    else int8_many_tile<kGateUp, n, false>(p, lds, it);                \
  }
  MOE_INT8_CASE(1)
  MOE_INT8_CASE(2)
  MOE_INT8_CASE(3)
  MOE_INT8_CASE(4)
#undef MOE_INT8_CASE
}

// ---------------------------------------------------------------- quantising
// Codes and scale of one row of kIn (bf16 or fp32) values: a workgroup a row.
// 127 x is exact for bf16 and its quotient by the maximum, if not a tie, is
// at least 2^-9 from one, so the code is that of the exact quotient, ties to
// even.  A row with a NaN or an infinity gets the scale NaN, a row of zeros
// codes 0 and the scale 1.  Rows of up to 8192 values stay in registers.  The
// first rows have cols values, rows from rows1 on (h's, behind the routed ones)
// cols2; h is not read again and passes the caches by.
template <typename IO>
__global__ void __launch_bounds__(256)
quantize_rows_int8_kernel(const IO* __restrict__ x, int64_t rows1, int cols1, int cols2,
                          int8_t* __restrict__ q, float* __restrict__ scale) {
  constexpr int kKeep = 4;
  __shared__ uint32_t red[4];
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  const int cols = row < rows1 ? cols1 : cols2;
  const int64_t at = row < rows1 ? row * cols1 : rows1 * cols1 + (row - rows1) * cols2;
  const IO* xr = x + at;
  const int chunks = cols / 8;
  auto load = [&](int c, float* v) {
    if constexpr (sizeof(IO) == 2) {
      const u32x4 p = *reinterpret_cast<const u32x4*>(xr + c * 8);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = __uint_as_float(p[j] << 16);
        v[2 * j + 1] = __uint_as_float(p[j] & 0xFFFF0000u);
      }
    } else {
      const f32x4* p = reinterpret_cast<const f32x4*>(xr + c * 8);
      const f32x4 a = __builtin_nontemporal_load(p), b = __builtin_nontemporal_load(p + 1);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = a[j];
        v[4 + j] = b[j];
      }
    }
  };
  float keep[kKeep][8];
  uint32_t m = 0;   // bits of the largest magnitude: NaN above infinity above the rest
  auto track = [&](const float* v) {
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
  };
#pragma unroll
  for (int i = 0; i < kKeep; ++i)
    if (tid + i * 256 < chunks) {
      load(tid + i * 256, keep[i]);
      track(keep[i]);
    }
  for (int c = tid + kKeep * 256; c < chunks; c += 256) {
    float v[8];
    load(c, v);
    track(v);
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, off, 64));
  if ((tid & 63) == 0) red[tid >> 6] = m;
  __syncthreads();
  m = max(max(red[0], red[1]), max(red[2], red[3]));
  const bool bad = m >= 0x7F800000u;
  const float a = __uint_as_float(m);
  // 127 x must stay finite
  const float lift = a > 0x1p120f ? 0x1p-16f : 1.0f, d = a * lift;
  auto store = [&](int c, const float* v) {
    uint32_t w[2] = {0, 0};
    if (!bad && m != 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float r = __builtin_rintf(v[j] * lift * 127.0f / d);
        w[j >> 2] |= ((uint32_t)(int)fminf(fmaxf(r, -127.0f), 127.0f) & 0xFFu) << (8 * (j & 3));
      }
    }
    *reinterpret_cast<uint2*>(q + at + c * 8) = make_uint2(w[0], w[1]);
  };
#pragma unroll
  for (int i = 0; i < kKeep; ++i)
    if (tid + i * 256 < chunks) store(tid + i * 256, keep[i]);
  for (int c = tid + kKeep * 256; c < chunks; c += 256) {
    float v[8];
    load(c, v);
    store(c, v);
  }
  if (tid == 0) scale[row] = bad ? __uint_as_float(0x7FC00000u) : m == 0 ? 1.0f : a / 127.0f;
}

// One thread per 16-byte piece of the packed matrix.
__global__ void __launch_bounds__(256)
pack_int8_kernel(bool gate_up, const int8_t* __restrict__ codes, u32x4* __restrict__ dst,
                 int64_t units, int n, int kd, int nt) {
  const int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (u >= units) return;
  const int nsteps = kd / kStepK;
  const int lane = (int)(u & 63), f = (int)(u >> 6 & 1), b = (int)(u >> 7 & 7);
  const int64_t blk = u / kUnits;
  const int step = (int)(blk % nsteps);
  const int64_t et = blk / nsteps;
  const int tile = (int)(et % nt);
  const int64_t e = et / nt, rows = gate_up ? 2 * (int64_t)n : n;
  const int r = lane & 15;
  const int64_t row = gate_up ? (b & 2 ? n : 0) + (int64_t)tile * 64 + (b >> 2) * 32 + (b & 1) * 16 + r
                              : (int64_t)tile * 128 + b * 16 + r;
  dst[u] = *reinterpret_cast<const u32x4*>(codes + (e * rows + row) * kd + step * kStepK + f * 64 +
                                           16 * (lane >> 4));
}

// Rows of an M-tile, which name the kernel: the few-row kernel up to kFewAverage
// rows per expert on average, and where the tall tiles would be too few
// workgroups (its own split k over four waves and are shorter).  Measured few /
// many at H = 7168, I = 2048, E = 256, K = 8: T = 384 (12 rows an expert) 1.84 /
// 1.88 ms, T = 512 1.94 / 1.93, T = 700 2.24 / 1.98.  By tall workgroups x rows an
// expert: 92 x 50 34 / 46 us, 114 x 100 34 / 44, 156 x 500 34 / 42, 160 x 32 67 / 64,
// 288 x 16 143 / 128, 368 x 250 207 / 137, 540 x 47 117 / 101.
// The choice is the whole layer's, whichever of its groups the launch computes.
// The shared expert's T rows do not count beside routed ones, which costs layers
// with few experts a token: E = 256, K = 1, T = 3000 (12 rows an expert) 2.23 ms,
// all in tall tiles 1.93; with Is = 18432 5.50 and 2.94.
constexpr int kFewAverage = 14;
constexpr int64_t kTallGrid = 256, kTallWork = 100000;
int tile_rows(FfnDims d) {
  d.groups = kGroupsAll;
  const int64_t tall = ffn_grid_mtiles(d, kManyRows) * (std::max(d.I, d.Is) / 128);
  if (d.T <= kFewRows || (d.N && d.N <= (int64_t)kFewAverage * d.E) ||
      (tall < kTallGrid && tall * (d.N ? d.N : d.T) < kTallWork * (d.N ? d.E : 1)))
    return kFewRows;
  return kManyRows;
}

// nt: packed tiles of the group with the most of them.
template <bool kGateUp>
hipError_t launch_gemm(Int8Args a, int rows, int64_t mtiles, int nt, hipStream_t s) {
  a.ntn = rows == kFewRows ? nt : (nt + 1) / 2;
  const int64_t work = mtiles * a.ntn;
  if (work > kMaxGridThreads / kThreads8 - kXcdGrid) return hipErrorInvalidValue;
  const dim3 grid(xcd_grid(work));
  if (rows == kFewRows)
    MOE_TIMED_LAUNCH(s, kGateUp ? "grouped_gemm_int8_few<true>" : "grouped_gemm_int8_few<false>",
      hipLaunchKernelGGL((grouped_gemm_int8_few<kGateUp>), grid, dim3(kThreads8), 0, s, a));
  else
    MOE_TIMED_LAUNCH(s, kGateUp ? "grouped_gemm_int8_many<true>" : "grouped_gemm_int8_many<false>",
      hipLaunchKernelGGL((grouped_gemm_int8_many<kGateUp>), grid, dim3(kThreads8), 0, s, a));
  return hipGetLastError();
}

}  // namespace

size_t packed_int8_bytes(bool gate_up, int64_t experts, int n, int kd) {
  const int64_t nt = gate_up ? n / 64 : n / 128;
  return (size_t)(experts * nt * (kd / kStepK) * kUnits) * sizeof(u32x4);
}

hipError_t launch_pack_int8(bool gate_up, const int8_t* codes, void* dst, int64_t experts, int n,
                            int kd, hipStream_t s) {
  const int64_t units = (int64_t)(packed_int8_bytes(gate_up, experts, n, kd) / sizeof(u32x4));
  MOE_TIMED_LAUNCH(s, "pack_int8_kernel",
    hipLaunchKernelGGL(pack_int8_kernel, dim3((unsigned)((units + 255) / 256)), dim3(256), 0, s,
                       gate_up, codes, (u32x4*)dst, units, n, kd, gate_up ? n / 64 : n / 128));
  return hipGetLastError();
}

hipError_t launch_quantize_rows_int8(const uint16_t* x, int64_t rows, int cols, int8_t* q,
                                     float* scale, hipStream_t s) {
  if (rows > quantize_rows_int8_max()) return hipErrorInvalidValue;
  MOE_TIMED_LAUNCH(s, "quantize_rows_int8_kernel",
    hipLaunchKernelGGL(quantize_rows_int8_kernel<uint16_t>, dim3((unsigned)rows), dim3(256), 0, s,
                       x, rows, cols, 0, q, scale));
  return hipGetLastError();
}

hipError_t launch_ffn_int8(const FfnDims& d, const int8_t* xq, const float* xs,
                           const int32_t* perm, const int32_t* offsets, const void* w13p,
                           const float* w13s, const void* w2p, const float* w2s,
                           const void* ws13p, const float* ws13s, const void* ws2p,
                           const float* ws2s, float* h, int8_t* hq, float* hs, uint16_t* y,
                           uint16_t* ys, hipStream_t s) {
  const int rows = tile_rows(d);
  const int64_t mt = ffn_grid_mtiles(d, rows);
  const bool routed = d.groups & kGroupRouted, shared = (d.groups & kGroupShared) && d.Is > 0;
  Int8Args a{};
  a.offsets = offsets;
  a.routed = routed;
  a.per = (d.E + kWave - 1) / kWave;
  a.shared_rows = shared ? (int)d.T : 0;
  a.E = d.E;
  a.K = d.K;
  a.a_r = a.a_s = xq;
  a.as_r = a.as_s = xs;
  a.perm = perm;
  a.kdim_r = a.kdim_s = d.H;
  a.b_r = (const u32x4*)w13p;
  a.b_s = (const u32x4*)ws13p;
  a.nt_r = d.I / 64;
  a.nt_s = d.Is / 64;
  a.bs_r = w13s;
  a.bs_s = ws13s;
  a.ncol_r = d.I;
  a.ncol_s = d.Is;
  a.c_r = h;
  a.c_s = h + d.N * d.I;
  hipError_t e = launch_gemm<true>(a, rows, mt, std::max(a.nt_r, a.nt_s), s);
  if (e != hipSuccess) return e;

  int8_t* hq_s = hq + d.N * d.I;
  float* hs_s = hs + d.N;
  // The routed rows and the shared expert's lie one behind the other; either may
  // be another launch's.
  const int64_t first = routed ? 0 : d.N, end = d.N + (shared ? d.T : 0);
  if (end - first > quantize_rows_int8_max()) return hipErrorInvalidValue;
  if (end > first) {
    MOE_TIMED_LAUNCH(s, "quantize_rows_int8_kernel<h>",
      hipLaunchKernelGGL(quantize_rows_int8_kernel<float>, dim3((unsigned)(end - first)),
                         dim3(256), 0, s, h + first * d.I, d.N - first, d.I, d.Is,
                         hq + first * d.I, hs + first));
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }

  a.nt_r = a.nt_s = d.H / 128;
  a.a_r = hq;
  a.a_s = hq_s;
  a.as_r = hs;
  a.as_s = hs_s;
  a.kdim_r = d.I;
  a.kdim_s = d.Is;
  a.b_r = (const u32x4*)w2p;
  a.b_s = (const u32x4*)ws2p;
  a.bs_r = w2s;
  a.bs_s = ws2s;
  a.ncol_r = a.ncol_s = d.H;
  a.c_r = y;
  a.c_s = ys;
  return launch_gemm<false>(a, rows, mt, a.nt_r, s);
}

}  // namespace moe
