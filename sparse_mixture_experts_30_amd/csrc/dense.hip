// The SwiGLU feed-forward block of a layer without routed experts, and its
// backward, on bf16 MFMA (row-major bf16 weights, fp32 accumulation):
//   [g; u] = W13 x,  h = silu(g) u,  y = W2 h;
//   dh = dy W2,  dg = dh u silu'(g),  du = dh silu(g),
//   dx = [dg du] W13,  dW2 = dy^T h,  dW13 = [dg du]^T x.
// Six matrix products, two fused epilogues (the activation behind [g; u], its
// derivative behind dh).  Every operand is read as it lies: the products
// that contract over tokens or over a weight's rows read it through the
// LDS's transposing loads.  g and u are kept in bf16 for the backward (half
// the bytes of fp32; they are read once, elementwise), h and [dg du] are
// rounded to bf16 as operands of the products that follow.
#include "dense.hpp"
#include "gemm_device.hpp"
#include "rows_device.hpp"

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
  uint16_t* gu;          // [M, 2 I]: written (EPI_SWIGLU; may be null) or read (EPI_DSWIGLU)
  uint16_t* da;          // EPI_DSWIGLU: [M, 2 I]
  int mt, nt;
};

// Tile of workgroup b.  Each XCD takes one contiguous part of the tiles, in
// groups of kGroupM tiles down by all across, column by column: the 32
// workgroups that run on an XCD together are then 8 x 4 tiles that share
// operands in its L2.
constexpr int kGroupM = 8;
__device__ __forceinline__ bool tile_of(const DenseArgs& p, int& m, int& n) {
  const int w = xcd_contiguous((int)blockIdx.x, (int)gridDim.x);
  if (w >= p.mt * p.nt) return false;
  const int per = kGroupM * p.nt, g = w / per, l = w % per;
  const int rows = min(p.mt - g * kGroupM, kGroupM);
  m = g * kGroupM + l % rows;
  n = l / rows;
  return true;
}

template <int kM, int kN, int kWM, int kWN, int kOpA, int kOpB, int kEpi>
__global__ void __launch_bounds__(64 * kWM * kWN, kWM * kWN / 4)
dense_gemm(DenseArgs p) {
  typedef GemmTile<kM, kN, kWM, kWN, kOpA, kOpB> Tile;
  __shared__ u32x4 lds[4 * Tile::kStage];
  int m, n;
  if (!tile_of(p, m, n)) return;
  constexpr int kNh = kEpi == EPI_SWIGLU ? kN / 2 : kN;   // output columns of a tile
  const int64_t m0 = (int64_t)m * kM, n0 = (int64_t)n * kNh;
  Operand A, B;
  A.ld = p.lda;
  B.ld = p.ldb;
  A.p[0] = A.p[1] = kOpA == OP_COL ? p.a : p.a + m0 * p.lda;
  A.rows = kOpA == OP_COL ? p.K : p.M - m0;
  if (kOpB == OP_COL) {
    B.p[0] = B.p[1] = p.b;
    B.rows = p.K;
  } else {
    B.p[0] = p.b + n0 * p.ldb;
    B.p[1] = B.p[0] + p.N * p.ldb;
    B.rows = p.N - n0;
  }
  f32x16 acc[Tile::kMI][Tile::kNJ];
  Tile::run(lds, A, (int)m0, B, (int)n0, p.K, acc);

  // The operands are read for the last time: the waves share their LDS out.
  const int w = Tile::wave();
  float* l = reinterpret_cast<float*>(lds) + w * (32 * (Tile::kNJ == 1 ? 32 : 64));
  const int64_t row0 = m0 + Tile::row0(w);
  const int64_t col0 = n0 + (kEpi == EPI_SWIGLU ? Tile::col0(w) / 2 : Tile::col0(w));
  if constexpr (kEpi == EPI_STORE) {
    wave_rows<false>(l, acc, [&](int r, int c, const float (&v)[8]) {
      const int64_t row = row0 + r, col = col0 + c;
      if (row < p.M && col < p.N) *reinterpret_cast<u32x4*>(p.c + row * p.N + col) = pack_bf16x8(v);
    });
  } else if constexpr (kEpi == EPI_SWIGLU) {
    wave_rows<true>(l, acc, [&](int r, int c, const float (&g)[8], const float (&u)[8]) {
      const int64_t row = row0 + r, col = col0 + c;
      if (row >= p.M || col >= p.N) return;
      if (p.gu) {
        *reinterpret_cast<u32x4*>(p.gu + row * 2 * p.N + col) = pack_bf16x8(g);
        *reinterpret_cast<u32x4*>(p.gu + row * 2 * p.N + p.N + col) = pack_bf16x8(u);
      }
      if (p.c) {
        float h[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = g[j] / (1.0f + __expf(-g[j])) * u[j];
        *reinterpret_cast<u32x4*>(p.c + row * p.N + col) = pack_bf16x8(h);
      }
    });
  } else {
    wave_rows<false>(l, acc, [&](int r, int c, const float (&dh)[8]) {
      const int64_t row = row0 + r, col = col0 + c;
      if (row >= p.M || col >= p.N) return;
      const uint16_t* gp = p.gu + row * 2 * p.N + col;
      float g[8], u[8], dg[8], du[8], h[8];
      unpack_bf16x8(*reinterpret_cast<const u32x4*>(gp), g);
      unpack_bf16x8(*reinterpret_cast<const u32x4*>(gp + p.N), u);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float s = 1.0f / (1.0f + __expf(-g[j])), gs = g[j] * s;
        dg[j] = dh[j] * u[j] * (s + gs * (1.0f - s));
        du[j] = dh[j] * gs;
        h[j] = gs * u[j];
      }
      uint16_t* dp = p.da + row * 2 * p.N + col;
      *reinterpret_cast<u32x4*>(dp) = pack_bf16x8(dg);
      *reinterpret_cast<u32x4*>(dp + p.N) = pack_bf16x8(du);
      *reinterpret_cast<u32x4*>(p.c + row * p.N + col) = pack_bf16x8(h);
    });
  }
}

template <int kOpA, int kOpB, int kEpi>
hipError_t launch_gemm(DenseArgs a, const char* name, hipStream_t s) {
  constexpr int kM = 256, kN = 256, kWM = 2, kWN = 4, kH = kEpi == EPI_SWIGLU ? kN / 2 : kN;
  a.mt = (int)((a.M + kM - 1) / kM);
  a.nt = (int)((a.N + kH - 1) / kH);
  const int64_t work = (int64_t)a.mt * a.nt;
  if (work == 0) return hipSuccess;
  const unsigned grid = (unsigned)((work + kNumXcd - 1) / kNumXcd * kNumXcd);
  MOE_TIMED_LAUNCH(s, name,
    hipLaunchKernelGGL((dense_gemm<kM, kN, kWM, kWN, kOpA, kOpB, kEpi>), dim3(grid), dim3(64 * kWM * kWN), 0, s,
                       a));
  return hipGetLastError();
}

}  // namespace

bool dense_fits(int64_t T, int64_t H, int64_t I) {
  // At most 2^23 tiles of 256 x 128 a product (a launch holds 2^32 threads), and
  // rows of up to 4 MiB (a tile's offsets are 31 bits).
  auto tiles = [](int64_t m, int64_t n) { return (double)((m + 255) / 256) * ((n + 127) / 128); };
  const double most = 8.0e6;
  return I <= (1 << 20) && H <= (1 << 21) && tiles(T, I) < most && tiles(T, H) < most &&
         tiles(2 * I, H) < most;
}

hipError_t launch_dense_gate_up(const uint16_t* x, const uint16_t* w13, int64_t T, int H, int I,
                                uint16_t* gu, uint16_t* h, hipStream_t s) {
  DenseArgs a{};
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
                             uint16_t* y, hipStream_t s) {
  DenseArgs a{};
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
                                 const uint16_t* gu, const uint16_t* dy, int64_t T, int H, int I,
                                 uint16_t* da, uint16_t* h, uint16_t* dx, uint16_t* dw13,
                                 uint16_t* dw2, hipStream_t s) {
  const int64_t rh = (int64_t)H * 2, ri = (int64_t)I * 2;   // bytes of rows of H and I
  DenseArgs a{};
  a.a = (const char*)dy;
  a.lda = rh;
  a.b = (const char*)w2;
  a.ldb = ri;
  a.M = T;
  a.N = I;
  a.K = H;
  a.c = h;
  a.gu = const_cast<uint16_t*>(gu);
  a.da = da;
  hipError_t e = launch_gemm<OP_ROW, OP_COL, EPI_DSWIGLU>(a, "dense_gemm<dh>", s);
  if (e != hipSuccess) return e;

  a = DenseArgs{};
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
