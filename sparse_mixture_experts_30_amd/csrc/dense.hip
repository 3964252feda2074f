// The SwiGLU feed-forward block of a layer without routed experts, and its
// backward, on bf16 MFMA (row-major bf16 weights, fp32 accumulation):
//   [g; u] = W13 x,  h = silu(g) u,  y = W2 h;
//   dh = dy W2,  dg = dh u silu'(g),  du = dh silu(g),
//   dx = [dg du] W13,  dW2 = dy^T h,  dW13 = [dg du]^T x.
// Six matrix products, two fused epilogues (the activation behind [g; u], its
// derivative behind dh).  Every operand is read as it lies: the products
// that contract over tokens or over a weight's rows read it through the
// LDS's transposing loads.  g and u are kept in fp32 for the backward: in
// bf16 they would save 2.8% of a training step's time and double the error of
// [dg du] (gradients 3.5e-3 from 64 bits instead of 2.4e-3, of which their own
// rounding is 1.7e-3).  h and [dg du] are rounded to bf16 as operands of the
// products that follow.
#include "dense.hpp"
#include "gemm_device.hpp"
#include "rows_device.hpp"

#include <math.h>

#include <algorithm>

namespace moe {

namespace {

enum : int { EPI_STORE = 0, EPI_SWIGLU = 1, EPI_DSWIGLU = 2 };

struct DenseArgs {
  const char* a;         // A and B as Operand, from row / column 0
  int64_t lda;
  const char* b;
  int64_t ldb;
  int64_t M, N, K;       // EPI_SWIGLU: N = I, the columns of h
  uint16_t* c;           // EPI_STORE: [M, N]; else h [M, I] (may be null)
  float* gu;             // [M, 2 I]: written (EPI_SWIGLU; may be null) or read (EPI_DSWIGLU)
  uint16_t* da;          // EPI_DSWIGLU: [M, 2 I]
  float* part;           // sums of each k range [splits][M][N, EPI_SWIGLU: 2 N]
  int mt, nt, splits;
};

__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<f32x4*>(p)[0] = (f32x4){v[0], v[1], v[2], v[3]};
  reinterpret_cast<f32x4*>(p)[1] = (f32x4){v[4], v[5], v[6], v[7]};
}

// What becomes of eight neighbouring sums (EPI_SWIGLU: of g and of u) from
// (row, col) on.
__device__ __forceinline__ void epi_store(const DenseArgs& p, int64_t row, int64_t col,
                                          const float (&v)[8]) {
  *reinterpret_cast<u32x4*>(p.c + row * p.N + col) = pack_bf16x8(v);
}
__device__ __forceinline__ void epi_swiglu(const DenseArgs& p, int64_t row, int64_t col,
                                           const float (&g)[8], const float (&u)[8]) {
  if (p.gu) {
    float* o = p.gu + row * 2 * p.N + col;
    store8(o, g);
    store8(o + p.N, u);
  }
  if (p.c) {
    float h[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = g[j] / (1.0f + __expf(-g[j])) * u[j];
    *reinterpret_cast<u32x4*>(p.c + row * p.N + col) = pack_bf16x8(h);
  }
}
struct GateUp {   // g and u of eight columns
  f32x4 g[2], u[2];
  __device__ __forceinline__ void load(const DenseArgs& p, int64_t row, int64_t col) {
    const float* at = p.gu + row * 2 * p.N + col;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      g[i] = reinterpret_cast<const f32x4*>(at)[i];
      u[i] = reinterpret_cast<const f32x4*>(at + p.N)[i];
    }
  }
};
__device__ __forceinline__ void epi_dswiglu(const DenseArgs& p, int64_t row, int64_t col,
                                            const float (&dh)[8], const GateUp& v) {
  float dg[8], du[8], h[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float g = v.g[j >> 2][j & 3], u = v.u[j >> 2][j & 3];
    const float s = 1.0f / (1.0f + __expf(-g)), gs = g * s;
    dg[j] = dh[j] * u * (s + gs * (1.0f - s));
    du[j] = dh[j] * gs;
    h[j] = gs * u;
  }
  uint16_t* dp = p.da + row * 2 * p.N + col;
  *reinterpret_cast<u32x4*>(dp) = pack_bf16x8(dg);
  *reinterpret_cast<u32x4*>(dp + p.N) = pack_bf16x8(du);
  *reinterpret_cast<u32x4*>(p.c + row * p.N + col) = pack_bf16x8(h);
}

// Tile and k range of workgroup b of `grid`.  Each XCD takes one contiguous part of the
// tiles, in groups of kGroupM tiles down by all across, column by column: the 32
// workgroups that run on an XCD together are then 8 x 4 tiles that share
// operands in its L2.
constexpr int kGroupM = 8;
__device__ __forceinline__ bool tile_of(const DenseArgs& p, int b, int grid, int& m, int& n,
                                        int& split) {
  const int w = xcd_contiguous(b, grid);
  const int tiles = p.mt * p.nt;
  if (w >= tiles * p.splits) return false;
  split = w / tiles;
  const int t = w - split * tiles;
  const int per = kGroupM * p.nt, g = t / per, l = t % per;
  const int rows = min(p.mt - g * kGroupM, kGroupM);
  m = g * kGroupM + l % rows;
  n = l / rows;
  return true;
}

// Tiles of 256 x 256, 128 x 128 or 64 x 128, of kM / 2 x 64 a wave; A in three LDS
// stages, B in two.
constexpr int cols_of(int m) { return m == 256 ? 256 : 128; }
template <int kM, int kOpA, int kOpB>
using DenseTile = GemmTile<kM, cols_of(kM), 2, cols_of(kM) / 64, 3, 2, kOpA, kOpB>;

template <int kM, int kOpA, int kOpB, int kEpi>
__device__ __forceinline__ void dense_tile(const DenseArgs& p, u32x4* lds, int b, int grid) {
  typedef DenseTile<kM, kOpA, kOpB> Tile;
  constexpr int kN = cols_of(kM);
  int m, n, split;
  if (!tile_of(p, b, grid, m, n, split)) return;
  constexpr int kNh = kEpi == EPI_SWIGLU ? kN / 2 : kN;   // output columns of a tile
  const int64_t m0 = (int64_t)m * kM, n0 = (int64_t)n * kNh;
  Operand A, B;
  A.ld = p.lda;
  B.ld = p.ldb;
  A.to2 = 0;
  A.p = kOpA == OP_COL ? p.a : p.a + m0 * p.lda;
  A.rows = kOpA == OP_COL ? p.K : p.M - m0;
  if (kOpB == OP_COL) {
    B.p = p.b;
    B.to2 = 0;
    B.rows = p.K;
  } else {
    B.p = p.b + n0 * p.ldb;
    B.to2 = p.N * p.ldb;
    B.rows = p.N - n0;
  }
  const int steps = (int)((p.K + kGemmBK - 1) / kGemmBK);
  // EPI_DSWIGLU: g and u of 32 rows are loaded together, each piece as soon as the
  // one of the 32 rows before is used, the first before the sums: one by one they
  // would each wait for memory.  Past the edge the last value again.
  GateUp gu[4];
  auto load_gu = [&](int i, int t) {
    const int lane = threadIdx.x & 63, w = Tile::wave();
    gu[t].load(p, min(m0 + Tile::row0(w) + i * 32 + t * 8 + (lane >> 3), p.M - 1),
               min(n0 + Tile::col0(w) + (lane & 7) * 8, p.N - 8));
  };
  constexpr bool kEarly = kEpi == EPI_DSWIGLU && kM < 256;   // registers for it
  if (kEarly && p.splits == 1) {
#pragma unroll
    for (int t = 0; t < 4; ++t) load_gu(0, t);
  }
  f32x16 acc[Tile::kMI][Tile::kNJ];
  Tile::run(lds, A, (int)m0, B, (int)n0, (int)((int64_t)steps * split / p.splits),
            (int)((int64_t)steps * (split + 1) / p.splits), acc);

  // The operands are read for the last time: the waves share their LDS out.
  const int w = Tile::wave();
  float* l = reinterpret_cast<float*>(lds) + w * (32 * 64);
  const int64_t row0 = m0 + Tile::row0(w);
  const int64_t col0 = n0 + (kEpi == EPI_SWIGLU ? Tile::col0(w) / 2 : Tile::col0(w));
  auto keep = [&](int64_t at, const float (&v)[8]) { store8(p.part + at, v); };
  if constexpr (kEpi == EPI_SWIGLU) {
    wave_rows<true>(l, acc, [&](int r, int c, const float (&g)[8], const float (&u)[8]) {
      const int64_t row = row0 + r, col = col0 + c;
      if (row >= p.M || col >= p.N) return;
      if (p.splits > 1) {
        const int64_t at = (split * p.M + row) * 2 * p.N + col;
        keep(at, g);
        keep(at + p.N, u);
      } else {
        epi_swiglu(p, row, col, g, u);
      }
    });
  } else if (kEpi == EPI_STORE || p.splits > 1) {
    wave_rows<false>(l, acc, [&](int r, int c, const float (&v)[8]) {
      const int64_t row = row0 + r, col = col0 + c;
      if (row >= p.M || col >= p.N) return;
      if (p.splits > 1) keep((split * p.M + row) * p.N + col, v);
      else epi_store(p, row, col, v);
    });
  } else {
    if (!kEarly) {
#pragma unroll
      for (int t = 0; t < 4; ++t) load_gu(0, t);
    }
#pragma unroll
    for (int i = 0; i < Tile::kMI; ++i) {
      int t = 0;
      f32x16(&block)[1][Tile::kNJ] = reinterpret_cast<f32x16(&)[1][Tile::kNJ]>(acc[i]);
      wave_rows<false>(l, block, [&](int r, int c, const float (&dh)[8]) {
        const int64_t row = row0 + i * 32 + r, col = col0 + c;
        if (row < p.M && col < p.N) epi_dswiglu(p, row, col, dh, gu[t]);
        if (i + 1 < Tile::kMI) load_gu(i + 1, t);
        ++t;
      });
    }
  }
}

template <int kM, int kOpA, int kOpB, int kEpi>
__global__ void __launch_bounds__(2 * cols_of(kM), 2) dense_gemm(DenseArgs p) {
  __shared__ u32x4 lds[DenseTile<kM, kOpA, kOpB>::kPieces];
  dense_tile<kM, kOpA, kOpB, kEpi>(p, lds, (int)blockIdx.x, (int)gridDim.x);
}

// Three products that do not wait for each other as one launch of 128 x 128 tiles:
// dx = [dg du] W13 first (its workgroups take longest), dW13 and dW2.  dx_end and
// dw13_end: workgroups up to the end of the first and the second.
struct DenseGradArgs {
  DenseArgs dx, dw13, dw2;
  int dx_end, dw13_end;
};
__global__ void __launch_bounds__(256, 2) dense_gemm_grads(DenseGradArgs a) {
  __shared__ u32x4 lds[DenseTile<128, OP_COL, OP_COL>::kPieces];
  const int b = (int)blockIdx.x;
  if (b < a.dx_end) {
    dense_tile<128, OP_ROW, OP_COL, EPI_STORE>(a.dx, lds, b, a.dx_end);
  } else {
    // Field by field: a reference to one of the two would put both in LDS.
    const bool w2 = b >= a.dw13_end;
    DenseArgs p{};
    p.a = w2 ? a.dw2.a : a.dw13.a;
    p.lda = w2 ? a.dw2.lda : a.dw13.lda;
    p.b = w2 ? a.dw2.b : a.dw13.b;
    p.ldb = w2 ? a.dw2.ldb : a.dw13.ldb;
    p.M = w2 ? a.dw2.M : a.dw13.M;
    p.N = w2 ? a.dw2.N : a.dw13.N;
    p.K = a.dw13.K;
    p.c = w2 ? a.dw2.c : a.dw13.c;
    p.part = w2 ? a.dw2.part : a.dw13.part;
    p.mt = w2 ? a.dw2.mt : a.dw13.mt;
    p.nt = w2 ? a.dw2.nt : a.dw13.nt;
    p.splits = w2 ? a.dw2.splits : a.dw13.splits;
    dense_tile<128, OP_COL, OP_COL, EPI_STORE>(p, lds, b - (w2 ? a.dw13_end : a.dx_end),
                                               (w2 ? (int)gridDim.x - a.dw13_end
                                                   : a.dw13_end - a.dx_end));
  }
}

// The k ranges' sums joined in their order, eight columns a thread.  Bound by
// latency: four ranges under way at a time and workgroups of 256 take 1 us longer
// (T = 16, H = 2048, I = 5632: block 32.7 instead of 30.7 us).
constexpr int kJoinThreads = 128;
template <int kEpi>
__global__ void __launch_bounds__(kJoinThreads) dense_join(DenseArgs p) {
  const int64_t i = ((int64_t)blockIdx.x * kJoinThreads + threadIdx.x) * 8;
  if (i >= p.M * p.N) return;
  const int64_t row = i / p.N, col = i % p.N;
  constexpr int kParts = kEpi == EPI_SWIGLU ? 2 : 1;
  const int64_t all = p.M * p.N * kParts;
  float v[kParts][8];
#pragma unroll
  for (int h = 0; h < kParts; ++h) {
    const float* src = p.part + (row * kParts + h) * p.N + col;
    f32x4 a = {0.f, 0.f, 0.f, 0.f}, b = a;
    for (int s = 0; s < p.splits; s += 8) {   // eight ranges' loads under way at a time
      f32x4 x[8], y[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float* at = src + min(s + q, p.splits - 1) * all;
        x[q] = *reinterpret_cast<const f32x4*>(at);
        y[q] = *reinterpret_cast<const f32x4*>(at + 4);
      }
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (s + q < p.splits) {
          a += x[q];
          b += y[q];
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[h][j] = a[j];
      v[h][4 + j] = b[j];
    }
  }
  if constexpr (kEpi == EPI_SWIGLU) epi_swiglu(p, row, col, v[0], v[1]);
  else if constexpr (kEpi == EPI_STORE) epi_store(p, row, col, v[0]);
  else {
    GateUp gu;
    gu.load(p, row, col);
    epi_dswiglu(p, row, col, v[0], gu);
  }
}

// Tile height and k ranges of an M x n product (n rows of B, so 2 I for the gate and
// up projections) over K, by estimated time.  Measured, a step of 64 k: a tile
// of 256 takes 1.45 us with every CU at work (1.1 with few); tiles of 128 share
// a CU by twos, 1.1 us both or 0.55 one alone (bound by loading 60 GB/s a CU),
// 0.75 one alone with operands that no other tile reads, from HBM; tiles of 64
// rows 0.85 and 0.42.  Ranges of k make more workgroups of a small product and
// cost a pass over their sums.
//   T = 1, H = 7168, I = 18432, gate and up projections in 1 / 3 / 4 / 6 ranges
//   about 117 / 99 / 108 / 107 us and 9 for the join, down projection 3 / 4 / 6 / 8
//   ranges 86 / 66 / 55 / 52; as tiles of 256 151 and 330.  T = 32: gate and up
//   121 / 105 / 115 / 117.  T = 300, H = 2048, I = 5632: tiles of 128 in 1 / 2 / 4
//   ranges 36 / 35 / 41, of 256 53; T = 1500 1 / 2 ranges 138 / 186, of 256 190.
//   T = 4096, H = 7168: of 256 1660.
// The derivative's epilogue moves 230 KB a tile of 128, 6 us: tiles of 64 rows,
// on twice as many CUs, take half of that (T = 333, H = 1024, I = 2752: 19 instead
// of 24 us, T = 700, H = 2048, I = 5632: 39 of 46; T = 1500, H = 1024: 39 against 35).
// The other products gain less than 1 us from them.
// More than kMostParts workgroups' sums are never kept apart (a plan for which that
// would pay was estimated 2.5% faster at best), which bounds the workspace.
constexpr int kMostSplits = 16, kMostParts = 1024;
constexpr size_t kMostPartBytes = (size_t)kMostParts * 128 * 128 * 4;
struct Plan {
  int rows, splits;   // of a tile, of k
};
Plan plan_of(int64_t M, int64_t n, int64_t K, bool derivative = false) {
  constexpr double kCus = 256, kFill = 5.0, kJoin = 3.0;   // us
  constexpr double kHbm = 5.3e6, kSums = 5e6;              // bytes / us
  const double steps = (double)((K + kGemmBK - 1) / kGemmBK);
  auto tiles = [&](int64_t rows) {
    const int64_t cols = cols_of((int)rows);
    return (double)((M + rows - 1) / rows) * ((n + cols - 1) / cols);
  };
  // The time of `work` tiles, `slots` at once, `one` alone on a CU, `all` with
  // every slot taken, per step; `turn` what start and end of a tile add.
  auto turns = [&](double work, double slots, double per, double one, double all, double turn) {
    const double full = floor(work / slots), rest = work - full * slots;
    const double last = slots > kCus ? (rest <= kCus ? one : all)
                                     : one + (all - one) * rest / slots;
    return full * (per * all + turn) + (rest > 0 ? per * last + turn : 0) + kFill;
  };
  const double least_us = 2.0 * ((double)M + (double)n) * (double)K / kHbm + kFill;
  const double end = derivative ? 6.0 : 1.0, alone = M <= 256 ? 0.75 : 0.55;
  Plan best{256, 1};
  double least = 1e300;
  auto consider = [&](int rows, int splits, double t) {
    if (std::max(t, least_us) < least) {
      least = std::max(t, least_us);
      best = {rows, splits};
    }
  };
  consider(256, 1, turns(tiles(256), kCus, steps, 1.1, 1.45, 5.0 + end));
  consider(128, 1, turns(tiles(128), 2 * kCus, steps, alone, 1.1, end));
  if (derivative) consider(64, 1, turns(tiles(64), 2 * kCus, steps, alone * 0.77, 0.85, end / 2));
  // At least two steps a range: one without any would leave its sums unset.
  for (int s = 2; s <= kMostSplits && steps >= 2 * s && tiles(128) * s <= kMostParts; ++s)
    consider(128, s, turns(tiles(128) * s, 2 * kCus, ceil(steps / s), alone, 1.1, 1.0) + kJoin +
                         (8.0 * s + (derivative ? 14 : 0)) * (double)M * (double)n / kSums);
  return best;
}
// Room for the sums of any plan of up to this size: a workspace for the largest
// batch does for the smaller ones too, which may take more ranges.
size_t part_bytes(int64_t M, int64_t n, int64_t K) {
  const int64_t splits = std::min<int64_t>(kMostSplits, (K + kGemmBK - 1) / kGemmBK / 2);
  if (splits < 2) return 0;
  return (size_t)std::min((double)splits * M * n * 4, (double)kMostPartBytes);
}

// Workgroups of a product in tiles of `rows` and `splits` k ranges.
int64_t workgroups(DenseArgs& a, int64_t n, int rows, int splits) {
  a.mt = (int)((a.M + rows - 1) / rows);
  a.nt = (int)((n + cols_of(rows) - 1) / cols_of(rows));
  a.splits = splits;
  return ((int64_t)a.mt * a.nt * splits + kNumXcd - 1) / kNumXcd * kNumXcd;
}

template <int kEpi>
hipError_t launch_join(const DenseArgs& a, hipStream_t s) {
  if (a.splits == 1) return hipSuccess;
  MOE_TIMED_LAUNCH(s, "dense_join",
    hipLaunchKernelGGL(dense_join<kEpi>,
                       dim3((unsigned)((a.M * a.N / 8 + kJoinThreads - 1) / kJoinThreads)),
                       dim3(kJoinThreads), 0, s, a));
  return hipGetLastError();
}

template <int kOpA, int kOpB, int kEpi>
hipError_t launch_gemm(DenseArgs a, const char* name, hipStream_t s) {
  const int64_t n = kEpi == EPI_SWIGLU ? 2 * a.N : a.N;
  const Plan q = plan_of(a.M, n, a.K, kEpi == EPI_DSWIGLU);
  const unsigned grid = (unsigned)workgroups(a, n, q.rows, q.splits);
  if (grid == 0) return hipSuccess;
  MOE_TIMED_LAUNCH(s, name,
    if (q.rows == 256)
      hipLaunchKernelGGL((dense_gemm<256, kOpA, kOpB, kEpi>), dim3(grid), dim3(512), 0, s, a);
    else if (kEpi == EPI_DSWIGLU && q.rows == 64)
      hipLaunchKernelGGL((dense_gemm<kEpi == EPI_DSWIGLU ? 64 : 128, kOpA, kOpB, kEpi>), dim3(grid),
                         dim3(256), 0, s, a);
    else
      hipLaunchKernelGGL((dense_gemm<128, kOpA, kOpB, kEpi>), dim3(grid), dim3(256), 0, s, a));
  const hipError_t e = hipGetLastError();
  return e != hipSuccess ? e : launch_join<kEpi>(a, s);
}

// dx, dW13 and dW2 as one launch if each would take tiles of 128 by itself and
// their sums by k ranges fit the workspace: their last turns then overlap.  k
// ranges such that no workgroup has more than its share of all steps.  With
// `behind`, dx waits for the other two in a launch of its own; its k ranges and
// theirs are the same then, also where no dx is wanted (c null).
bool launch_grads(DenseArgs dx, DenseArgs dw13, DenseArgs dw2, bool behind, hipStream_t s,
                  hipError_t& e) {
  constexpr int64_t kShortest = 8;   // steps of a k range, about what a join costs
  DenseArgs* const all[] = {&dx, &dw13, &dw2};
  int64_t work = 0;
  for (DenseArgs* a : all) {
    if (plan_of(a->M, a->N, a->K).rows == 256) return false;
    work += (a->M + 127) / 128 * ((a->N + 127) / 128) * ((a->K + kGemmBK - 1) / kGemmBK);
  }
  const int64_t share = std::max(kShortest, work / 512);
  int64_t grid = 0, end[3], parts = 0;
  float* part = dx.part;
  for (int i = 0; i < 3; ++i) {
    DenseArgs& a = *all[i];
    const int64_t steps = (a.K + kGemmBK - 1) / kGemmBK;
    const int splits = (int)std::max<int64_t>(
        1, std::min({(int64_t)kMostSplits, steps / 2, (steps + share - 1) / share}));
    end[i] = grid += workgroups(a, a.N, 128, splits);
    a.part = part;
    if (splits > 1) {
      parts += (int64_t)a.mt * a.nt * splits;
      part += a.M * a.N * splits;
    }
  }
  if (parts > kMostParts || grid > (1 << 22)) return false;
  e = hipSuccess;
  auto launch = [&](bool with_dx, bool with_dw) {
    const int xs = with_dx ? (int)end[0] : 0, ws = with_dw ? (int)(grid - end[0]) : 0;
    if (xs + ws == 0 || e != hipSuccess) return;
    DenseGradArgs g{dx, dw13, dw2, xs, xs + (int)(end[1] - end[0])};
    MOE_TIMED_LAUNCH(s, "dense_gemm<gradients>",
      hipLaunchKernelGGL(dense_gemm_grads, dim3((unsigned)(xs + ws)), dim3(256), 0, s, g));
    e = hipGetLastError();
  };
  launch(dx.c && !behind, true);
  launch(dx.c && behind, false);
  for (DenseArgs* a : all)
    if (e == hipSuccess && a->c) e = launch_join<EPI_STORE>(*a, s);
  return true;
}

}  // namespace

size_t dense_part_bytes(int64_t T, int64_t H, int64_t I, bool backward) {
  const size_t up = part_bytes(T, 2 * I, H);
  if (!backward) return std::max(up, part_bytes(T, H, I));
  // The last three may run together.
  const size_t grads = std::min(
      part_bytes(T, H, 2 * I) + part_bytes(2 * I, H, T) + part_bytes(H, I, T), kMostPartBytes);
  return std::max({up, part_bytes(T, I, H), grads});
}

bool dense_fits(int64_t T, int64_t H, int64_t I) {
  // Fewer than 2^32 threads a launch, also of the kernel that joins ranges of k,
  // and rows of up to 4 MiB (a tile's offsets are 31 bits).
  auto fits = [](int64_t m, int64_t n, int64_t K, bool derivative = false) {
    const Plan q = plan_of(m, n, K, derivative);
    const double work = (double)((m + q.rows - 1) / q.rows) *
                        ((n + cols_of(q.rows) - 1) / cols_of(q.rows)) * q.splits;
    return work * (cols_of(q.rows) * 2) < 4.29e9 && work < 2.1e9 && (double)m * n / 8 < 4.29e9;
  };
  return I <= (1 << 20) && H <= (1 << 21) && fits(T, 2 * I, H) && fits(T, H, I) &&
         fits(T, I, H, true) && fits(T, H, 2 * I) && fits(2 * I, H, T) && fits(H, I, T);
}

hipError_t launch_dense_gate_up(const uint16_t* x, const uint16_t* w13, int64_t T, int H, int I,
                                float* gu, uint16_t* h, float* part, hipStream_t s) {
  DenseArgs a{};
  a.part = part;
  a.a = (const char*)x;
  a.lda = (int64_t)H * 2;
  a.b = (const char*)w13;
  a.ldb = (int64_t)H * 2;
  a.M = T;
  a.N = I;
  a.K = H;
  a.c = h;
  a.gu = gu;
  return launch_gemm<OP_ROW, OP_GATE_UP, EPI_SWIGLU>(a, "dense_gemm<gate/up>", s);
}

hipError_t launch_dense_down(const uint16_t* h, const uint16_t* w2, int64_t T, int H, int I,
                             uint16_t* y, float* part, hipStream_t s) {
  DenseArgs a{};
  a.part = part;
  a.a = (const char*)h;
  a.lda = (int64_t)I * 2;
  a.b = (const char*)w2;
  a.ldb = (int64_t)I * 2;
  a.M = T;
  a.N = H;
  a.K = I;
  a.c = y;
  return launch_gemm<OP_ROW, OP_ROW, EPI_STORE>(a, "dense_gemm<down>", s);
}

hipError_t launch_dense_backward(const uint16_t* x, const uint16_t* w13, const uint16_t* w2,
                                 const float* gu, const uint16_t* dy, int64_t T, int H, int I,
                                 uint16_t* da, uint16_t* h, uint16_t* dx, uint16_t* dw13,
                                 uint16_t* dw2, float* part, hipStream_t s) {
  const int64_t rh = (int64_t)H * 2, ri = (int64_t)I * 2;   // bytes of rows of H and I
  DenseArgs a{};
  a.part = part;
  a.a = (const char*)dy;
  a.lda = rh;
  a.b = (const char*)w2;
  a.ldb = ri;
  a.M = T;
  a.N = I;
  a.K = H;
  a.c = h;
  a.gu = const_cast<float*>(gu);
  a.da = da;
  hipError_t e = launch_gemm<OP_ROW, OP_COL, EPI_DSWIGLU>(a, "dense_gemm<dh>", s);
  if (e != hipSuccess) return e;

  DenseArgs w13a{}, w2a{}, xa{};
  w13a.part = w2a.part = xa.part = part;
  w13a.a = (const char*)da;
  w13a.lda = 2 * ri;
  w13a.b = (const char*)x;
  w13a.ldb = rh;
  w13a.M = 2 * (int64_t)I;
  w13a.N = H;
  w13a.K = T;
  w13a.c = dw13;
  w2a.a = (const char*)dy;
  w2a.lda = rh;
  w2a.b = (const char*)h;
  w2a.ldb = ri;
  w2a.M = H;
  w2a.N = I;
  w2a.K = T;
  w2a.c = dw2;
  xa.a = (const char*)da;
  xa.lda = 2 * ri;
  xa.b = (const char*)w13;
  xa.ldb = rh;
  xa.M = T;
  xa.N = H;
  xa.K = 2 * (int64_t)I;
  xa.c = dx;
  if (T && launch_grads(xa, w13a, w2a, dx == dy, s, e)) return e;

  e = launch_gemm<OP_COL, OP_COL, EPI_STORE>(w13a, "dense_gemm<dw13>", s);
  if (e == hipSuccess) e = launch_gemm<OP_COL, OP_COL, EPI_STORE>(w2a, "dense_gemm<dw2>", s);
  // Last: dx may be dy.
  if (e == hipSuccess && dx) e = launch_gemm<OP_ROW, OP_COL, EPI_STORE>(xa, "dense_gemm<dx>", s);
  return e;
}

}  // namespace moe
