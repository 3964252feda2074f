// Expert FFNs on 4-bit weights with group scales (gfx950), for serving:
//   W[n][k] = s[n][k / g] (u[n][k] - 8),  u in 0..15, g = 128 or 32, s bf16,
// activations bf16, accumulation fp32.  Decode batches are bound by the
// weight stream, and 4 bits read a quarter of the bytes of bf16.
//
// Arithmetic.  128 + u is a bf16 number whose low mantissa bits are u, so one
// AND-OR turns two codes into two matrix operands.  Inside a group
//   sum_k x (u - 8) = sum_k x (128 + u) - 136 sum_k x;
// the second sum comes from a matrix instruction against a constant operand
// of -136 (exact in bf16) that starts the first one's accumulator.  Products
// are exact in fp32; the group's scale multiplies its fp32 sum, so the codes
// are never rounded.
//
// Layout (pack_int4): per output tile (64 h columns of gate and up together,
// or 128 output rows of the down projection) and 128-k step one block: eight
// 1 KiB fragments of 16 rows, then the scales [group][row of 16][fragment 8].
// Lane l of fragment b holds row l % 16; its dword f covers
// k = 128 step + 32 f + 8 (l / 16) + 0..7, value 2i in nibble i, value 2i + 1
// in nibble i + 4.  Fragments 0-3 of a gate/up tile are gate rows, 4-7 the up
// rows of the same columns.
//
// Each workgroup computes one tile for up to 16 * NRB rows; its four waves
// take a quarter of the k steps each and their sums are joined through LDS in
// wave order.
#include "moe_internal.hpp"

#include <algorithm>

namespace moe {

namespace {

constexpr int kThreads4 = 256;
constexpr int kStepK = 128;          // k per packed step
constexpr int kCodes16 = 512;        // 16-byte units of codes per step block
constexpr int kFrags = 8;            // 16-row fragments per tile

// 16-byte units of a step block.
constexpr __host__ __device__ int step_units(int group) { return kCodes16 + 16 * (kStepK / group); }

struct Int4Args {
  const int32_t* tiles;
  int ntn;                      // output tiles per M-tile (max over groups)
  int E, K;
  const uint16_t* a_r;
  const uint16_t* a_s;
  int64_t lda_r, lda_s;
  const int32_t* perm;          // gate/up: routed A row = perm[j] / K
  int kdim_r, kdim_s;
  const u32x4* b_r;             // packed routed weights
  int nt_r;                     // output tiles per routed expert
  const u32x4* b_s;
  int nt_s;
  uint16_t* c_r;
  uint16_t* c_s;
  int64_t ldc_r, ldc_s;
};

// Codes of dword d as bf16 operands 128 + u.
__device__ __forceinline__ bf16x8 codes_bf16(uint32_t d) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = ((d >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
  return as_bf16x8(r);
}

template <bool kGateUp, int kGroup, int NRB>
__device__ __forceinline__ void int4_tile(const Int4Args& p, float* lds, int g, int row0,
                                          int nrows, int ntile) {
  constexpr int kUnits = step_units(kGroup);
  constexpr int kScales = kStepK / kGroup;   // scale vectors per step
  const bool sh = (g == p.E);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int lr = lane & 15, lq = lane >> 4;
  const int nsteps = (sh ? p.kdim_s : p.kdim_r) / kStepK;
  const int s0 = nsteps * wave / 4, s1 = nsteps * (wave + 1) / 4;
  const uint16_t* A = sh ? p.a_s : p.a_r;
  const int64_t lda = sh ? p.lda_s : p.lda_r;
  const u32x4* bw = (sh ? p.b_s : p.b_r + (int64_t)g * p.nt_r * nsteps * kUnits) +
                    (int64_t)ntile * nsteps * kUnits;
  // This lane's activation rows (rows past the end re-read the first; their
  // results are never stored).
  const uint16_t* ap[NRB];
#pragma unroll
  for (int r = 0; r < NRB; ++r) {
    const int row = r * 16 + lr;
    const int rr = row < nrows ? row : 0;
    const int a = (!sh && kGateUp) ? p.perm[row0 + rr] / p.K : row0 + rr;
    ap[r] = A + (int64_t)a * lda + lq * 8;
  }
  const u32x4 offs_bits = {0xC308C308u, 0xC308C308u, 0xC308C308u, 0xC308C308u};   // -136
  const bf16x8 offs = as_bf16x8(offs_bits);

  f32x4 acc[NRB][kFrags];
#pragma unroll
  for (int r = 0; r < NRB; ++r)
#pragma unroll
    for (int b = 0; b < kFrags; ++b) acc[r][b] = (f32x4){0.f, 0.f, 0.f, 0.f};

  u32x4 rb[kFrags], sc[kScales], ra[NRB][4];
  auto load = [&](int step) {
    const u32x4* src = bw + (int64_t)step * kUnits;
#pragma unroll
    for (int b = 0; b < kFrags; ++b) rb[b] = __builtin_nontemporal_load(src + b * 64 + lane);
#pragma unroll
    for (int q = 0; q < kScales; ++q) sc[q] = src[kCodes16 + q * 16 + lr];
#pragma unroll
    for (int r = 0; r < NRB; ++r)
#pragma unroll
      for (int f = 0; f < 4; ++f)
        ra[r][f] = *reinterpret_cast<const u32x4*>(ap[r] + step * kStepK + f * 32);
  };
  for (int s = s0; s < s1; ++s) {
    load(s);
#pragma unroll
    for (int q = 0; q < kScales; ++q) {
      constexpr int kF = 4 / kScales;   // fragments of k per group
      float sv[kFrags];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sv[2 * i] = __uint_as_float(sc[q][i] << 16);
        sv[2 * i + 1] = __uint_as_float(sc[q][i] & 0xFFFF0000u);
      }
#pragma unroll
      for (int r = 0; r < NRB; ++r) {
        f32x4 corr = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int f = q * kF; f < (q + 1) * kF; ++f)
          corr = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(ra[r][f]), offs, corr, 0, 0, 0);
#pragma unroll
        for (int b = 0; b < kFrags; ++b) {
          f32x4 part = corr;
#pragma unroll
          for (int f = q * kF; f < (q + 1) * kF; ++f)
            part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(ra[r][f]),
                                                           codes_bf16(rb[b][f]), part, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[r][b][i] = fmaf(sv[b], part[i], acc[r][b][i]);
        }
      }
    }
  }

  // Join the four waves' sums, one row block at a time: [wave][frag][row quad
  // 4][i 4][col 16].
  uint16_t* C = sh ? p.c_s : p.c_r;
  const int64_t ldc = sh ? p.ldc_s : p.ldc_r;
#pragma unroll
  for (int r = 0; r < NRB; ++r) {
    if (r) __syncthreads();
#pragma unroll
    for (int b = 0; b < kFrags; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        lds[((wave * kFrags + b) * 16 + 4 * lq + i) * 16 + lr] = acc[r][b][i];
    __syncthreads();
    const int row = tid >> 4;
    if (r * 16 + row >= nrows) continue;   // the barrier above is passed by all threads
    uint16_t* crow = C + (int64_t)(row0 + r * 16 + row) * ldc;
    if (kGateUp) {
      const int col = (tid & 15) * 4, b = col >> 4;
      float h[4];
      f32x4 gv = {0.f, 0.f, 0.f, 0.f}, uv = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        gv += *reinterpret_cast<const f32x4*>(
            lds + ((w * kFrags + b) * 16 + row) * 16 + (col & 15));
        uv += *reinterpret_cast<const f32x4*>(
            lds + ((w * kFrags + 4 + b) * 16 + row) * 16 + (col & 15));
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) h[j] = gv[j] / (1.0f + __expf(-gv[j])) * uv[j];
      *reinterpret_cast<uint2*>(crow + ntile * 64 + col) =
          make_uint2(pack_bf16x2(h[0], h[1]), pack_bf16x2(h[2], h[3]));
    } else {
      const int col = (tid & 15) * 8, b = col >> 4;
      f32x4 v[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int w = 0; w < 4; ++w)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          v[j] += *reinterpret_cast<const f32x4*>(
              lds + ((w * kFrags + b) * 16 + row) * 16 + (col & 15) + 4 * j);
      *reinterpret_cast<u32x4*>(crow + ntile * 128 + col) =
          (u32x4){pack_bf16x2(v[0][0], v[0][1]), pack_bf16x2(v[0][2], v[0][3]),
                  pack_bf16x2(v[1][0], v[1][1]), pack_bf16x2(v[1][2], v[1][3])};
    }
  }
}

// MAXRB: 16-row blocks of the tallest tile of the list.
template <bool kGateUp, int kGroup, int MAXRB>
__global__ void __launch_bounds__(kThreads4) grouped_gemm_int4(Int4Args p) {
  __shared__ __align__(16) float lds[4 * kFrags * 256];
  const int64_t work = (int64_t)p.tiles[0] * p.ntn;
  const int64_t w = xcd_chunked(blockIdx.x, work);
  if (w < 0) return;
  int ntile;
  const int32_t* ent = decode_work(p.tiles, w, p.ntn, ntile);
  const int g = ent[0], row0 = ent[1], nrows = ent[2];
  if (ntile >= (g == p.E ? p.nt_s : p.nt_r)) return;
  switch ((nrows + 15) >> 4) {
    case 1:
      int4_tile<kGateUp, kGroup, 1>(p, lds, g, row0, nrows, ntile);
      break;
    case 2:
      if (MAXRB >= 2) int4_tile<kGateUp, kGroup, MAXRB >= 2 ? 2 : 1>(p, lds, g, row0, nrows, ntile);
      break;
    case 3:
      if (MAXRB >= 3) int4_tile<kGateUp, kGroup, MAXRB >= 3 ? 3 : 1>(p, lds, g, row0, nrows, ntile);
      break;
    case 4:
      if (MAXRB >= 4) int4_tile<kGateUp, kGroup, MAXRB >= 4 ? 4 : 1>(p, lds, g, row0, nrows, ntile);
      break;
    default:
      break;
  }
}

// One thread per 16-byte fragment piece, then per scale vector.
__global__ void __launch_bounds__(256)
pack_int4_kernel(bool gate_up, int group, const uint8_t* __restrict__ codes,
                 const uint16_t* __restrict__ scales, u32x4* __restrict__ dst, int64_t units,
                 int n, int kd, int nt) {
  const int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (u >= units) return;
  const int per = step_units(group), nsteps = kd / kStepK;
  const int o = (int)(u % per);
  const int64_t blk = u / per;
  const int step = (int)(blk % nsteps);
  const int64_t et = blk / nsteps;
  const int tile = (int)(et % nt);
  const int64_t e = et / nt;
  const int64_t rows = gate_up ? 2 * (int64_t)n : n;   // of one expert's matrix
  // Row of fragment b, lane row r in this tile.
  auto row_of = [&](int b, int r) -> int64_t {
    if (!gate_up) return (int64_t)tile * 128 + b * 16 + r;
    return (b < 4 ? 0 : n) + (int64_t)tile * 64 + (b & 3) * 16 + r;
  };
  u32x4 out = {0u, 0u, 0u, 0u};
  if (o < kCodes16) {
    const int b = o >> 6, lane = o & 63;
    const uint8_t* src = codes + ((e * rows + row_of(b, lane & 15)) * kd + step * kStepK +
                                  8 * (lane >> 4)) / 2;
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      uint32_t d = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t v = src[f * 16 + i];
        d |= (v & 15u) << (4 * i) | (v >> 4) << (16 + 4 * i);
      }
      out[f] = d;
    }
  } else {
    const int q = (o - kCodes16) >> 4, r = (o - kCodes16) & 15;
    const int64_t ng = kd / group, kg = (int64_t)step * (kStepK / group) + q;
#pragma unroll
    for (int b = 0; b < kFrags; ++b)
      out[b >> 1] |= (uint32_t)scales[(e * rows + row_of(b, r)) * ng + kg] << (16 * (b & 1));
  }
  dst[u] = out;
}

// Codes and scales of a bf16 matrix with kd columns: per group of g columns
// s = bf16(max |w| / 7), u = clamp(round(w / s), -8, 7) + 8 (ties to even;
// s = 0 gives 8).  One thread per 8 columns; g / 8 neighbouring lanes hold a
// group.
__global__ void __launch_bounds__(256)
quantize_int4_kernel(int group, const uint16_t* __restrict__ src, int64_t chunks, int kd,
                     uint8_t* __restrict__ codes, uint16_t* __restrict__ scales) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const bool ok = c < chunks;
  float v[8];
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = 0.0f;
  if (ok) {
    const u32x4 p = *reinterpret_cast<const u32x4*>(src + c * 8);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(p[j] << 16);
      v[2 * j + 1] = __uint_as_float(p[j] & 0xFFFF0000u);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[j]));
  }
  for (int off = group / 16; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
  if (!ok) return;
  const uint32_t sb = f32_to_bf16_bits(m / 7.0f);
  const float s = bf16_bits_to_f32(sb);
  uint32_t out = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float q = s > 0.0f ? fminf(fmaxf(__builtin_rintf(v[j] / s), -8.0f), 7.0f) : 0.0f;
    out |= (uint32_t)((int)q + 8) << (4 * j);
  }
  *reinterpret_cast<uint32_t*>(codes + c * 4) = out;
  if (c % (group / 8) == 0) scales[c * 8 / group] = (uint16_t)sb;
}

template <bool kGateUp, int kGroup>
hipError_t launch_gemm(const Int4Args& a, int maxrb, int64_t work, hipStream_t s) {
  const dim3 grid(xcd_grid(work));
#define MOE_INT4_LAUNCH(rb)                                                              \
  MOE_TIMED_LAUNCH(s, kGateUp ? "grouped_gemm_int4<true>" : "grouped_gemm_int4<false>",  \
    hipLaunchKernelGGL((grouped_gemm_int4<kGateUp, kGroup, rb>), grid, dim3(kThreads4), 0, s, a))
  if (maxrb == 1)
    MOE_INT4_LAUNCH(1);
  else if (maxrb == 2)
    MOE_INT4_LAUNCH(2);
  else
    MOE_INT4_LAUNCH(4);
#undef MOE_INT4_LAUNCH
  return hipGetLastError();
}

// 16-row blocks of the tallest tile: a batch of T tokens gives no expert
// more rows than that unless a caller's routing repeats one, and then the
// list cuts them.
int row_blocks(int64_t T) { return T <= 16 ? 1 : T <= 32 ? 2 : 4; }

}  // namespace

size_t int4_tiles_bytes(const FfnDims& d) {
  return (size_t)(8 + 8 * ffn_max_mtiles(d.N, d.T, d.E, 16 * row_blocks(d.T))) * sizeof(int32_t);
}

size_t packed4_bytes(bool gate_up, int64_t experts, int n, int kd, int group) {
  const int64_t nt = gate_up ? n / 64 : n / 128;
  return (size_t)(experts * nt * (kd / kStepK) * step_units(group)) * sizeof(u32x4);
}

hipError_t launch_pack_int4(bool gate_up, int group, const uint8_t* codes, const uint16_t* scales,
                            void* dst, int64_t experts, int n, int kd, hipStream_t s) {
  const int64_t units = (int64_t)(packed4_bytes(gate_up, experts, n, kd, group) / sizeof(u32x4));
  MOE_TIMED_LAUNCH(s, "pack_int4_kernel",
    hipLaunchKernelGGL(pack_int4_kernel, dim3((unsigned)((units + 255) / 256)), dim3(256), 0, s,
                       gate_up, group, codes, scales, (u32x4*)dst, units, n, kd,
                       gate_up ? n / 64 : n / 128));
  return hipGetLastError();
}

hipError_t launch_quantize_int4(int group, const uint16_t* src, int64_t rows, int kd,
                                uint8_t* codes, uint16_t* scales, hipStream_t s) {
  const int64_t chunks = rows * (kd / 8);
  MOE_TIMED_LAUNCH(s, "quantize_int4_kernel",
    hipLaunchKernelGGL(quantize_int4_kernel, dim3((unsigned)((chunks + 255) / 256)), dim3(256), 0,
                       s, group, src, chunks, kd, codes, scales));
  return hipGetLastError();
}

hipError_t launch_ffn_int4(const FfnDims& d, int group, const uint16_t* x, const int32_t* perm,
                           const int32_t* offsets, const void* w13p, const void* w2p,
                           const void* ws13p, const void* ws2p, uint16_t* h, int32_t* tiles,
                           uint16_t* y, uint16_t* ys, hipStream_t s) {
  const int maxrb = row_blocks(d.T), bm = 16 * maxrb;
  hipError_t e = ffn_build_tiles(d, offsets, bm, tiles, s, true);
  if (e != hipSuccess) return e;
  const int64_t mt = ffn_grid_mtiles(d, bm);

  Int4Args a{};
  a.tiles = tiles;
  a.nt_r = d.I / 64;
  a.nt_s = d.Is / 64;
  a.ntn = std::max(a.nt_r, a.nt_s);
  a.E = d.E;
  a.K = d.K;
  a.a_r = a.a_s = x;
  a.lda_r = a.lda_s = d.H;
  a.perm = perm;
  a.kdim_r = a.kdim_s = d.H;
  a.b_r = (const u32x4*)w13p;
  a.b_s = (const u32x4*)ws13p;
  a.c_r = h;
  a.c_s = h + d.N * d.I;
  a.ldc_r = d.I;
  a.ldc_s = d.Is;
  e = group == 32 ? launch_gemm<true, 32>(a, maxrb, mt * a.ntn, s)
                  : launch_gemm<true, 128>(a, maxrb, mt * a.ntn, s);
  if (e != hipSuccess) return e;

  a.nt_r = a.nt_s = a.ntn = d.H / 128;
  a.a_s = h + d.N * d.I;
  a.a_r = h;
  a.lda_r = a.kdim_r = d.I;
  a.lda_s = a.kdim_s = d.Is;
  a.b_r = (const u32x4*)w2p;
  a.b_s = (const u32x4*)ws2p;
  a.c_r = y;
  a.c_s = ys;
  a.ldc_r = a.ldc_s = d.H;
  return group == 32 ? launch_gemm<false, 32>(a, maxrb, mt * a.ntn, s)
                     : launch_gemm<false, 128>(a, maxrb, mt * a.ntn, s);
}

}  // namespace moe
