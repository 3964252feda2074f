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

// Tile and k range of workgroup b.  Each XCD takes one contiguous part of the
// tiles, in groups of kGroupM tiles down by all across, column by column: the 32
// workgroups that run on an XCD together are then 8 x 4 tiles that share
// operands in its L2.
constexpr int kGroupM = 8;
__device__ __forceinline__ bool tile_of(const DenseArgs& p, int& m, int& n, int& split) {
  const int w = xcd_contiguous((int)blockIdx.x, (int)gridDim.x);
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

template <int kM, int kN, int kWM, int kWN, int kSA, int kSB, int kOpA, int kOpB, int kEpi>
__global__ void __launch_bounds__(64 * kWM * kWN, 2) dense_gemm(DenseArgs p) {
  typedef GemmTile<kM, kN, kWM, kWN, kSA, kSB, kOpA, kOpB> Tile;
  __shared__ u32x4 lds[Tile::kPieces];
  int m, n, split;
  if (!tile_of(p, m, n, split)) return;
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
  f32x16 acc[Tile::kMI][Tile::kNJ];
  Tile::run(lds, A, (int)m0, B, (int)n0, (int)((int64_t)steps * split / p.splits),
            (int)((int64_t)steps * (split + 1) / p.splits), acc);

  // The operands are read for the last time: the waves share their LDS out.
  const int w = Tile::wave();
  float* l = reinterpret_cast<float*>(lds) + w * (32 * (Tile::kNJ == 1 ? 32 : 64));
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
    // g and u of 32 rows are loaded together, each piece as soon as the one of the
    // 32 rows before is used: one by one they would each wait for memory.  Past
    // the edge the last value again.
    static_assert(kEpi != EPI_DSWIGLU || Tile::kNJ == 2, "rows of 64 columns a wave");
    const int lane = threadIdx.x & 63;
    GateUp v[4];
    auto load = [&](int i, int t) {
      v[t].load(p, min(row0 + i * 32 + t * 8 + (lane >> 3), p.M - 1),
                min(col0 + (lane & 7) * 8, p.N - 8));
    };
#pragma unroll
    for (int t = 0; t < 4; ++t) load(0, t);
#pragma unroll
    for (int i = 0; i < Tile::kMI; ++i) {
      int t = 0;
      f32x16(&block)[1][Tile::kNJ] = reinterpret_cast<f32x16(&)[1][Tile::kNJ]>(acc[i]);
      wave_rows<false>(l, block, [&](int r, int c, const float (&dh)[8]) {
        const int64_t row = row0 + i * 32 + r, col = col0 + c;
        if (row < p.M && col < p.N) epi_dswiglu(p, row, col, dh, v[t]);
        if (i + 1 < Tile::kMI) load(i + 1, t);
        ++t;
      });
    }
  }
}

// The k ranges' sums joined in their order, eight columns a thread.
template <int kEpi>
__global__ void __launch_bounds__(256) dense_join(DenseArgs p) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (i >= p.M * p.N) return;
  const int64_t row = i / p.N, col = i % p.N;
  constexpr int kParts = kEpi == EPI_SWIGLU ? 2 : 1;
  const int64_t all = p.M * p.N * kParts;
  float v[kParts][8];
#pragma unroll
  for (int h = 0; h < kParts; ++h) {
    const float* src = p.part + (row * kParts + h) * p.N + col;
    f32x4 a = {0.f, 0.f, 0.f, 0.f}, b = a;
    for (int s = 0; s < p.splits; ++s) {
      a += *reinterpret_cast<const f32x4*>(src + s * all);
      b += *reinterpret_cast<const f32x4*>(src + s * all + 4);
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

// Tile edge and k ranges of an M x n product (n rows of B, so 2 I for the gate and
// up projections) over K, by estimated time.  Measured, a step of 64 k: a tile
// of 256 takes 1.45 us with every CU at work (1.1 with few); tiles of 128 share
// a CU by twos, 1.1 us both or 0.55 one alone (bound by loading 60 GB/s a CU),
// 0.75 one alone with operands that no other tile reads, from HBM.  Ranges of k
// make more workgroups of a small product and cost a pass over their sums.
//   T = 1, H = 7168, I = 18432, gate and up projections in 1 / 3 / 4 / 7 ranges
//   about 150 / 103 / 114 / 111 us, down projection 4 / 8 / 10 ranges 71 / 55 /
//   72; both as tiles of 256 474.  T = 300: tiles of 128 in 1 / 2 / 4 ranges 448 /
//   395 / 410, of 256 639.  T = 1500, H = 2048, I = 5632: 1 / 2 ranges 138 / 186,
//   of 256 190.  T = 4096, H = 7168: of 256 2440.
// More than kMostParts workgroups' sums are never kept apart (a plan for which that
// would pay was estimated 2.5% faster at best), which bounds the workspace.
constexpr int kMostSplits = 16, kMostParts = 1024;
struct Plan {
  int edge, splits;
};
Plan plan_of(int64_t M, int64_t n, int64_t K) {
  constexpr double kCus = 256, kFill = 5.0, kJoin = 3.0;   // us
  constexpr double kHbm = 5.3e6, kSums = 5e6;                           // bytes / us
  const double steps = (double)((K + kGemmBK - 1) / kGemmBK);
  auto tiles = [&](int64_t e) { return (double)((M + e - 1) / e) * ((n + e - 1) / e); };
  // The time of `work` tiles, `slots` at once, `one` alone on a CU, `all` with
  // every slot taken, per step; `turn` what start and end of a tile add.
  auto turns = [&](double work, double slots, double per, double one, double all, double turn) {
    const double full = floor(work / slots), rest = work - full * slots;
    const double last = rest == 0 ? 0 : rest <= kCus && slots > kCus ? one
                                       : one + (all - one) * rest / slots;
    return full * (per * all + turn) + (rest > 0 ? per * last + turn : 0) + kFill;
  };
  const double floor_us = 2.0 * ((double)M + (double)n) * (double)K / kHbm;
  Plan best{256, 1};
  double least = std::max(turns(tiles(256), kCus, steps, 1.1, 1.45, 6.0), floor_us + kFill);
  // At least two steps a range: one without any would leave its sums unset.
  for (int s = 1; s <= kMostSplits && (s == 1 || steps >= 2 * s); ++s) {
    const double work = tiles(128) * s, per = ceil(steps / s);
    if (s > 1 && work > kMostParts) break;
    const double t =
        std::max(turns(work, 2 * kCus, per, M <= 256 ? 0.75 : 0.55, 1.1, 1.0), floor_us + kFill) +
        (s > 1 ? kJoin + 8.0 * s * (double)M * (double)n / kSums : 0);
    if (t < least) {
      least = t;
      best = {128, s};
    }
  }
  return best;
}
// Room for the sums of any plan of up to this size: a workspace for the largest
// batch does for the smaller ones too, which may take more ranges.
size_t part_bytes(int64_t M, int64_t n, int64_t K) {
  const int64_t splits = std::min<int64_t>(kMostSplits, (K + kGemmBK - 1) / kGemmBK / 2);
  if (splits < 2) return 0;
  return (size_t)std::min((double)splits * M * n * 4, kMostParts * 128.0 * 128.0 * 4);
}

template <int kEdge, int kSA, int kSB, int kOpA, int kOpB, int kEpi>
void launch_tiles(const DenseArgs& a, unsigned grid, const char* name, hipStream_t s) {
  constexpr int kWN = kEdge == 256 ? 4 : 2;
  MOE_TIMED_LAUNCH(s, name,
    hipLaunchKernelGGL((dense_gemm<kEdge, kEdge, 2, kWN, kSA, kSB, kOpA, kOpB, kEpi>), dim3(grid),
                       dim3(128 * kWN), 0, s, a));
}

template <int kOpA, int kOpB, int kEpi>
hipError_t launch_gemm(DenseArgs a, const char* name, hipStream_t s) {
  const int64_t n = kEpi == EPI_SWIGLU ? 2 * a.N : a.N;
  const Plan q = plan_of(a.M, n, a.K);
  a.mt = (int)((a.M + q.edge - 1) / q.edge);
  a.nt = (int)((n + q.edge - 1) / q.edge);
  a.splits = q.splits;
  const int64_t work = (int64_t)a.mt * a.nt * a.splits;
  if (work == 0) return hipSuccess;
  const unsigned grid = (unsigned)((work + kNumXcd - 1) / kNumXcd * kNumXcd);
  if (q.edge == 256) launch_tiles<256, 3, 2, kOpA, kOpB, kEpi>(a, grid, name, s);
  else launch_tiles<128, 3, 2, kOpA, kOpB, kEpi>(a, grid, name, s);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  MOE_TIMED_LAUNCH(s, "dense_join",
    hipLaunchKernelGGL(dense_join<kEpi>, dim3((unsigned)((a.M * a.N / 8 + 255) / 256)), dim3(256),
                       0, s, a));
  return hipGetLastError();
}

}  // namespace

size_t dense_part_bytes(int64_t T, int64_t H, int64_t I, bool backward) {
  size_t b = part_bytes(T, 2 * I, H);
  if (!backward) return std::max(b, part_bytes(T, H, I));
  b = std::max(b, part_bytes(T, I, H));
  b = std::max(b, part_bytes(T, H, 2 * I));
  b = std::max(b, part_bytes(2 * I, H, T));
  return std::max(b, part_bytes(H, I, T));
}

bool dense_fits(int64_t T, int64_t H, int64_t I) {
  // Fewer than 2^32 threads a launch, also of the kernel that joins ranges of k,
  // and rows of up to 4 MiB (a tile's offsets are 31 bits).
  auto fits = [](int64_t m, int64_t n, int64_t K) {
    const Plan q = plan_of(m, n, K);
    const double work = (double)((m + q.edge - 1) / q.edge) * ((n + q.edge - 1) / q.edge) * q.splits;
    return work * (q.edge * 2) < 4.29e9 && work < 2.1e9 && (double)m * n / 8 < 4.29e9;
  };
  return I <= (1 << 20) && H <= (1 << 21) && fits(T, 2 * I, H) && fits(T, H, I) &&
         fits(T, I, H) && fits(T, H, 2 * I) && fits(2 * I, H, T) && fits(H, I, T);
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

  a = DenseArgs{};
  a.part = part;
  a.a = (const char*)da;
  a.lda = 2 * ri;
  a.b = (const char*)x;
  a.ldb = rh;
  a.M = 2 * (int64_t)I;
  a.N = H;
  a.K = T;
  a.c = dw13;
  e = launch_gemm<OP_COL, OP_COL, EPI_STORE>(a, "dense_gemm<dw13>", s);
  if (e != hipSuccess) return e;

  a = DenseArgs{};
  a.part = part;
  a.a = (const char*)dy;
  a.lda = rh;
  a.b = (const char*)h;
  a.ldb = ri;
  a.M = H;
  a.N = I;
  a.K = T;
  a.c = dw2;
  e = launch_gemm<OP_COL, OP_COL, EPI_STORE>(a, "dense_gemm<dw2>", s);
  if (e != hipSuccess || !dx) return e;

  // Last: dx may be dy.
  a = DenseArgs{};
  a.part = part;
  a.a = (const char*)da;
  a.lda = 2 * ri;
  a.b = (const char*)w13;
  a.ldb = rh;
  a.M = T;
  a.N = H;
  a.K = 2 * (int64_t)I;
  a.c = dx;
  return launch_gemm<OP_ROW, OP_COL, EPI_STORE>(a, "dense_gemm<dx>", s);
}

}  // namespace moe
