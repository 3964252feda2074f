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
// are never rounded.  (The code under a constant exponent and the offset taken
// out of the sum are a published way of multiplying 4-bit weights.)  h is
// rounded to bf16 like the other paths' h, as the second product's operand:
// outputs are 2.3e-3 from 64 bits instead of 1.7e-3 with the rounding of y
// alone; an h in fp32 would need three bf16 products for each of these.
//
// Layout (pack_int4): per output tile (64 h columns of gate and up together,
// or 128 output rows of the down projection) and 128-k step one block: eight
// 1 KiB fragments of 16 rows, then the scales [group][row of 16][fragment 8].
// Lane l of fragment b holds row l % 16; its dword f covers
// k = 128 step + 32 f + 8 (l / 16) + 0..7, value 2i in nibble i, value 2i + 1
// in nibble i + 4.  Fragments 0, 1 and 4, 5 of a gate/up tile are gate rows of
// its first and second 32 columns, 2, 3 and 6, 7 the up rows of the same.
//
// Two kernels.  Batches with few rows per expert (decode) read their
// activations straight from L2, 16 rows per tile, and split the k steps over
// the four waves of a workgroup.  Batches with more rows share the
// activations of 32 or 64 rows through LDS and split the output columns over
// the waves.
#include "block.hpp"

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
  const int32_t* offsets;
  int routed;                   // whether the routed experts are computed
  int per;                      // experts per lane in find_item, ceil(E / 64)
  int shared_rows;              // T, or 0 without the shared expert
  int ntn;                      // items per M-tile (max over groups)
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

// Codes of dword d as bf16 operands 128 + u.  The constants come from
// registers that the compiler cannot see through (code_constants): with
// literals it splits every AND-OR into two instructions, and unpacking is
// most of these kernels' vector work (11 instead of 7 instructions a dword).
struct CodeConstants {
  uint32_t mask, one28;
};
__device__ __forceinline__ CodeConstants code_constants() {
  CodeConstants c;
  asm("s_mov_b32 %0, 0x000f000f" : "=s"(c.mask));
  asm("v_mov_b32 %0, 0x43004300" : "=v"(c.one28));
  return c;
}
__device__ __forceinline__ bf16x8 codes_bf16(uint32_t d, const CodeConstants& c) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = ((d >> (4 * i)) & c.mask) | c.one28;
  return as_bf16x8(r);
}

// Four bf16 scales as fp32.
__device__ __forceinline__ void scales_f32(uint2 v, float* s) {
  s[0] = __uint_as_float(v.x << 16);
  s[1] = __uint_as_float(v.x & 0xFFFF0000u);
  s[2] = __uint_as_float(v.y << 16);
  s[3] = __uint_as_float(v.y & 0xFFFF0000u);
}

__device__ __forceinline__ bf16x8 minus_136() {
  return as_bf16x8((u32x4){0xC308C308u, 0xC308C308u, 0xC308C308u, 0xC308C308u});
}

__device__ __forceinline__ f32x4 mfma16(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// This workgroup's output tile and rows.  Group g < E is routed expert g with
// rows [offsets[g], offsets[g + 1]), group E the shared expert with all T
// tokens; a group of n rows is cut into mt = ceil(n / kRows) M-tiles of equal
// height (+-1 row).  Items are numbered group by group, in a group N-tile by
// N-tile, so the M-tiles that share a weight tile run together, and dealt to
// the XCDs in chunks (as xcd_chunked).  Every wave finds its item itself from
// the offsets, a few experts a lane and a scan over the lanes: a list made by
// a kernel of its own costs that kernel's 4 us in every call.
__device__ __forceinline__ uint32_t wave_inclusive_scan(uint32_t v) {
  // Data-parallel moves: within each row of 16 lanes by 1, 2, 4, 8 (lanes
  // without a source add 0), then the last lane of row 0 / 2 to row 1 / 3 and
  // of row 1 to rows 2 and 3.
  v += __builtin_amdgcn_update_dpp(0u, v, 0x111, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0u, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0u, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0u, v, 0x118, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0u, v, 0x142, 0xa, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0u, v, 0x143, 0xc, 0xf, false);
  return v;
}

struct Item {
  int g, row0, nrows, ntile;
  bool alone;   // the only M-tile of its group
};
template <int kRows>
__device__ __forceinline__ bool find_item(const Int4Args& p, Item& it) {
  const int lane = threadIdx.x & 63;
  const uint32_t b = blockIdx.x, q = b / kNumXcd;
  const uint32_t w = ((q / kXcdChunk) * kNumXcd + b % kNumXcd) * kXcdChunk + q % kXcdChunk;
  const uint32_t i0 = w / (uint32_t)p.ntn;   // M-tile the item would be if each had ntn items
  auto tiles_of = [](int32_t n) { return (uint32_t)(n + kRows - 1) / kRows; };
  // M-tiles of this lane's experts, and the end of its range of M-tiles
  uint32_t mine = 0;
  int32_t from = 0;
  if (p.routed) {
    from = p.offsets[min(lane * p.per, p.E)];
    int32_t o = from;
    for (int j = 1; j <= p.per; ++j) {
      const int32_t next = p.offsets[min(lane * p.per + j, p.E)];
      mine += tiles_of(next - o);
      o = next;
    }
  }
  const uint32_t end = wave_inclusive_scan(mine);
  const uint32_t routed = __builtin_amdgcn_readlane(end, 63);
  int32_t g, n, r0;
  uint32_t L;
  if (i0 < routed) {
    const int src = __builtin_ctzll(__ballot(end > i0));
    // that lane's experts one by one, on the scalar unit
    g = src * p.per;
    L = __builtin_amdgcn_readlane(end - mine, src);
    r0 = __builtin_amdgcn_readlane(from, src);
    for (;; ++g) {
      const int32_t next = p.offsets[g + 1];
      n = next - r0;
      if (i0 < L + tiles_of(n) || g + 1 >= p.E) break;
      L += tiles_of(n);
      r0 = next;
    }
  } else {
    g = p.E;
    n = p.shared_rows;
    r0 = 0;
    L = routed;
    if (i0 >= routed + tiles_of(n)) return false;
  }
  const uint32_t mt = tiles_of(n), local = w - L * (uint32_t)p.ntn;
  if (mt == 1) {
    it = {g, r0, n, (int)local, true};
    return true;
  }
  const uint32_t m = local % mt;
  const int32_t first = (int32_t)((uint64_t)m * n / mt),
                last = (int32_t)((uint64_t)(m + 1) * n / mt);
  it = {g, r0 + first, last - first, (int)(local / mt), false};
  return true;
}

// ---------------------------------------------------------------- few rows
// A tile of at most 16 rows and one packed output tile: the four waves take a
// quarter of the k steps each and their sums are joined through LDS in wave
// order.  One step in flight a wave, four waves a SIMD (three with groups of
// 32).  Bound by the weight stream: T = 32 (H = 7168, I = 2048, top-8 of 256,
// loads of Zipf 1.2) 340-348 us, 5.9 TB/s; two steps in flight 368 (fewer waves
// a SIMD), and before the loads past a wave's last step were dropped (358 us):
// cached instead of non-temporal weight loads 395, half the fragments a
// workgroup 400-443, k over eight waves 397, over two 356, but then T = 1 takes
// 76 instead of 50 us.
constexpr int kFewRows = 16;
constexpr int kFewWaves = 4;
constexpr int kFewThreads = 64 * kFewWaves;

template <bool kGateUp, int kGroup, bool kStream>
__device__ __forceinline__ void int4_few_tile(const Int4Args& p, float* lds, int g, int row0,
                                              int nrows, int ntile) {
  constexpr int kUnits = step_units(kGroup);
  constexpr int kScales = kStepK / kGroup;   // scale vectors per step
  constexpr int kF = 4 / kScales;            // k fragments per group
  const bool sh = (g == p.E);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int lr = lane & 15, lq = lane >> 4;
  const int nsteps = (sh ? p.kdim_s : p.kdim_r) / kStepK;
  const int s0 = nsteps * wave / kFewWaves, s1 = nsteps * (wave + 1) / kFewWaves;
  const u32x4* bw = (sh ? p.b_s : p.b_r + (int64_t)g * p.nt_r * nsteps * kUnits) +
                    (int64_t)ntile * nsteps * kUnits;

  u32x4 rb[kFrags], sc[kScales], ra[4];
  auto load_w = [&](int step) {
    const u32x4* src = bw + (int64_t)step * kUnits;
#pragma unroll
    for (int b = 0; b < kFrags; ++b)
      rb[b] = kStream ? __builtin_nontemporal_load(src + b * 64 + lane) : src[b * 64 + lane];
#pragma unroll
    for (int q = 0; q < kScales; ++q) sc[q] = src[kCodes16 + q * 16 + lr];
  };
  if (s0 < s1) load_w(s0);
  // This lane's activation row (past the end the first one; those results are
  // never stored).
  const int rr = lr < nrows ? lr : 0;
  const int arow = (!sh && kGateUp) ? p.perm[row0 + rr] / p.K : row0 + rr;
  const uint16_t* ap = (sh ? p.a_s : p.a_r) + (int64_t)arow * (sh ? p.lda_s : p.lda_r) + lq * 8;
  auto load_a = [&](int step) {
    const uint16_t* src = ap + step * kStepK;
#pragma unroll
    for (int f = 0; f < 4; ++f) ra[f] = *reinterpret_cast<const u32x4*>(src + f * 32);
  };
  if (s0 < s1) load_a(s0);

  const CodeConstants cc = code_constants();
  f32x4 acc[kFrags];
#pragma unroll
  for (int b = 0; b < kFrags; ++b) acc[b] = (f32x4){0.f, 0.f, 0.f, 0.f};
  auto compute = [&]() {
#pragma unroll
    for (int q = 0; q < kScales; ++q) {
      float sv[kFrags];
      scales_f32(make_uint2(sc[q][0], sc[q][1]), sv);
      scales_f32(make_uint2(sc[q][2], sc[q][3]), sv + 4);
      f32x4 corr = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int f = q * kF; f < (q + 1) * kF; ++f)
        corr = mfma16(as_bf16x8(ra[f]), minus_136(), corr);
#pragma unroll
      for (int b = 0; b < kFrags; ++b) {
        f32x4 part = corr;
#pragma unroll
        for (int f = q * kF; f < (q + 1) * kF; ++f)
          part = mfma16(as_bf16x8(ra[f]), codes_bf16(rb[b][f], cc), part);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[b][i] = fmaf(sv[b], part[i], acc[b][i]);
      }
    }
  };
  // Only the wave's own steps are loaded: at a few steps a wave, one read
  // ahead in vain is up to a fifth of the traffic.
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
  if (row >= nrows) return;
  uint16_t* crow = (sh ? p.c_s : p.c_r) + (int64_t)(row0 + row) * (sh ? p.ldc_s : p.ldc_r);
  auto joined = [&](int b, int col) {
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kFewWaves; ++w)
      v += *reinterpret_cast<const f32x4*>(lds + ((w * kFrags + b) * 16 + row) * 16 + col);
    return v;
  };
  if (kGateUp) {
    const int col = (tid & 15) * 4, b = (col >> 5) * 4 + (col >> 4 & 1);
    const f32x4 gv = joined(b, col & 15), uv = joined(b + 2, col & 15);
    float h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = gv[j] / (1.0f + __expf(-gv[j])) * uv[j];
    *reinterpret_cast<uint2*>(crow + ntile * 64 + col) =
        make_uint2(pack_bf16x2(h[0], h[1]), pack_bf16x2(h[2], h[3]));
  } else {
    const int col = (tid & 15) * 8, b = col >> 4;
    const f32x4 v = joined(b, col & 15), w = joined(b, (col & 15) + 4);
    *reinterpret_cast<u32x4*>(crow + ntile * 128 + col) =
        (u32x4){pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(w[0], w[1]),
                pack_bf16x2(w[2], w[3])};
  }
}

template <bool kGateUp, int kGroup>
__global__ void __launch_bounds__(kFewThreads) grouped_gemm_int4_few(Int4Args p) {
  __shared__ __align__(16) float lds[kFewWaves * kFrags * 256];
  Item it;
  if (!find_item<kFewRows>(p, it)) return;
  if (it.ntile >= (it.g == p.E ? p.nt_s : p.nt_r)) return;
  // A weight tile that only this row tile reads is not kept in cache.
  if (it.alone)
    int4_few_tile<kGateUp, kGroup, true>(p, lds, it.g, it.row0, it.nrows, it.ntile);
  else
    int4_few_tile<kGateUp, kGroup, false>(p, lds, it.g, it.row0, it.nrows, it.ntile);
}

// --------------------------------------------------------------- many rows
// A tile of at most 64 rows and two packed output tiles: each wave takes four
// fragments over the whole k range, the rows' activations pass through two
// LDS buffers in fragment order (lane-linear 16-byte reads and writes).  Tiles
// of at most 32 rows leave registers for three waves per SIMD instead of two.
// T = 512 (H = 7168, I = 2048, top-8 of 256) 1.12 ms, 5.3 TB/s of weights and
// rows; T = 1024 1.48 ms, 4.1 TB/s, the matrix cores busy 42% and the vector
// issue 49% of the time: the two and the weight stream overlap only in part.
constexpr int kMidRows = 32, kManyRows = 64;

template <bool kGateUp, int kGroup, int NRB, bool kStream>
__device__ __forceinline__ void int4_many_tile(const Int4Args& p, u32x4* lds, int g, int row0,
                                               int nrows, int npair) {
  constexpr int kUnits = step_units(kGroup);
  constexpr int kScales = kStepK / kGroup;
  constexpr int kF = 4 / kScales;
  const bool sh = (g == p.E);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int lr = lane & 15, lq = lane >> 4;
  const int nsteps = (sh ? p.kdim_s : p.kdim_r) / kStepK;
  const int nt = sh ? p.nt_s : p.nt_r;
  // An odd number of packed tiles leaves the last pair's second half to no
  // one: its waves load the first half's weights and store nothing.
  const int ntile = npair * 2 + (wave >> 1);
  const bool mine = ntile < nt;
  const u32x4* bw = (sh ? p.b_s : p.b_r + (int64_t)g * nt * nsteps * kUnits) +
                    (int64_t)(mine ? ntile : ntile - 1) * nsteps * kUnits;
  const int fh = wave & 1;   // this wave's half of the tile's fragments

  const uint16_t* ap[NRB];
#pragma unroll
  for (int r = 0; r < NRB; ++r) {
    const int rr = r * 16 + lr < nrows ? r * 16 + lr : 0;
    const int arow = (!sh && kGateUp) ? p.perm[row0 + rr] / p.K : row0 + rr;
    ap[r] = (sh ? p.a_s : p.a_r) + (int64_t)arow * (sh ? p.lda_s : p.lda_r) + wave * 32 + lq * 8;
  }
  u32x4 rb[4], st[NRB];
  uint2 sc[kScales];
  auto load_w = [&](int step) {
    const u32x4* src = bw + (int64_t)min(step, nsteps - 1) * kUnits;
#pragma unroll
    for (int b = 0; b < 4; ++b)
      rb[b] = kStream ? __builtin_nontemporal_load(src + (fh * 4 + b) * 64 + lane)
                            : src[(fh * 4 + b) * 64 + lane];
#pragma unroll
    for (int q = 0; q < kScales; ++q)
      sc[q] = reinterpret_cast<const uint2*>(src + kCodes16 + q * 16 + lr)[fh];
  };
  // Wave w stages k fragment w of every row block.
  auto load_a = [&](int step) {
#pragma unroll
    for (int r = 0; r < NRB; ++r)
      st[r] = *reinterpret_cast<const u32x4*>(ap[r] + min(step, nsteps - 1) * kStepK);
  };
  auto store_a = [&](int buf) {
#pragma unroll
    for (int r = 0; r < NRB; ++r) lds[((buf * NRB + r) * 4 + wave) * 64 + lane] = st[r];
  };

  load_a(0);
  load_w(0);
  const CodeConstants cc = code_constants();
  f32x4 acc[NRB][4];
#pragma unroll
  for (int r = 0; r < NRB; ++r)
#pragma unroll
    for (int b = 0; b < 4; ++b) acc[r][b] = (f32x4){0.f, 0.f, 0.f, 0.f};
  store_a(0);
  load_a(1);
  __syncthreads();

  // One step from LDS buffer d.
  auto compute = [&](int d) {
#pragma unroll
    for (int q = 0; q < kScales; ++q) {
      u32x4 a[NRB][kF];
#pragma unroll
      for (int r = 0; r < NRB; ++r)
#pragma unroll
        for (int f = 0; f < kF; ++f)
          a[r][f] = lds[((d * NRB + r) * 4 + q * kF + f) * 64 + lane];
      float sv[4];
      scales_f32(sc[q], sv);
      f32x4 corr[NRB];
#pragma unroll
      for (int r = 0; r < NRB; ++r) {
        corr[r] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int f = 0; f < kF; ++f)
          corr[r] = mfma16(as_bf16x8(a[r][f]), minus_136(), corr[r]);
      }
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        f32x4 part[NRB];
#pragma unroll
        for (int f = 0; f < kF; ++f) {
          const bf16x8 w = codes_bf16(rb[b][q * kF + f], cc);
#pragma unroll
          for (int r = 0; r < NRB; ++r)
            part[r] = mfma16(as_bf16x8(a[r][f]), w, f == 0 ? corr[r] : part[r]);
        }
#pragma unroll
        for (int r = 0; r < NRB; ++r)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[r][b][i] = fmaf(sv[b], part[r][i], acc[r][b][i]);
      }
    }
  };
  // One step: the next step's activations go to the buffer that was last
  // read before the previous barrier, and the loads of the step after it are
  // issued before this step's arithmetic (the scheduling barrier keeps them
  // there).  The next weights are loaded into the registers that this step
  // frees: a second set costs more in waves per SIMD than it hides (T = 1024,
  // H = 7168, I = 2048: one set 1.47 ms, two 1.50, three 1.49).
  auto one_step = [&](int d, int step) {
    store_a(d ^ 1);
    load_a(step + 2);
    __builtin_amdgcn_sched_barrier(0);
    compute(d);
    load_w(step + 1);
    __builtin_amdgcn_sched_barrier(0);
    __syncthreads();
  };
  int s = 0;
  for (; s + 2 <= nsteps; s += 2) {
    one_step(0, s);
    one_step(1, s + 1);
  }
  if (s < nsteps) one_step(0, s);   // the same for the whole workgroup

  // Results through LDS (the buffers are free after the last barrier), each
  // wave its own part: [row][its 64 output or 32 h columns] bf16.
  constexpr int kCols = kGateUp ? 32 : 64;
  uint16_t* out = reinterpret_cast<uint16_t*>(lds) + wave * (NRB * 16 * kCols);
#pragma unroll
  for (int r = 0; r < NRB; ++r)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint16_t* o = out + (r * 16 + 4 * lq + i) * kCols + lr;
      if (kGateUp) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const float gv = acc[r][b][i], uv = acc[r][2 + b][i];
          o[b * 16] = (uint16_t)f32_to_bf16_bits(gv / (1.0f + __expf(-gv)) * uv);
        }
      } else {
#pragma unroll
        for (int b = 0; b < 4; ++b) o[b * 16] = (uint16_t)f32_to_bf16_bits(acc[r][b][i]);
      }
    }
  __syncthreads();
  if (!mine) return;
  const int col0 = kGateUp ? ntile * 64 + fh * 32 : ntile * 128 + fh * 64;
  uint16_t* C = (sh ? p.c_s : p.c_r) + col0;
  const int64_t ldc = sh ? p.ldc_s : p.ldc_r;
  constexpr int kPer = kCols / 8;            // 16-byte pieces per row
  for (int i = lane; i < NRB * 16 * kPer; i += 64) {
    const int row = i / kPer, c = (i % kPer) * 8;
    if (row < nrows)
      *reinterpret_cast<u32x4*>(C + (int64_t)(row0 + row) * ldc + c) =
          *reinterpret_cast<const u32x4*>(out + row * kCols + c);
  }
}

template <bool kGateUp, int kGroup, int kRows>
__global__ void __launch_bounds__(kThreads4, kRows == kMidRows ? 3 : 2)
grouped_gemm_int4_many(Int4Args p) {
  __shared__ u32x4 lds[2 * (kRows / 16) * 4 * 64];   // 16 or 32 KiB
  Item it;
  if (!find_item<kRows>(p, it)) return;
  const int g = it.g, row0 = it.row0, nrows = it.nrows, npair = it.ntile;
  if (2 * npair >= (g == p.E ? p.nt_s : p.nt_r)) return;
  const int blocks = (nrows + 15) >> 4;
#define MOE_INT4_CASE(n)                                                          \
  if (blocks == n) {                                                              \
    if (it.alone)                                                                 \
      int4_many_tile<kGateUp, kGroup, n, true>(p, lds, g, row0, nrows, npair);    \
    else                                                                          \
      int4_many_tile<kGateUp, kGroup, n, false>(p, lds, g, row0, nrows, npair);   \
  }
  MOE_INT4_CASE(1)
  MOE_INT4_CASE(2)
  if constexpr (kRows > kMidRows) {
    MOE_INT4_CASE(3)
    MOE_INT4_CASE(4)
  }
#undef MOE_INT4_CASE
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
    return (b & 2 ? n : 0) + (int64_t)tile * 64 + (b >> 2) * 32 + (b & 1) * 16 + r;
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

// Rows of an M-tile, which name the kernel: the few-row kernel up to
// kFewAverage rows per expert on average, then tiles of 32 and of 64 rows.
// Measured at H = 7168, I = 2048, E = 256, K = 8, groups of 128, few / 32 / 64:
// T = 256 (8 rows an expert) 1.01 / - / 1.13 ms, T = 320 1.04 / 1.01 / 1.07,
// T = 512 1.25 / 1.12 / 1.17, T = 768 - / 1.29 / 1.32, T = 1024 (32 rows) 2.6 /
// 1.52 / 1.48; E = 64, groups of 32, T = 200 (25 rows) - / 0.41 / 0.46.
// A batch whose work would leave CUs idle in the tall-tile kernels takes the
// few-row kernel too, which splits k over its waves and so makes more and
// shorter workgroups; the more rows an expert has, the fewer tall workgroups
// are enough, as they re-read the weights less often.  Few against tall, by
// tall workgroups x rows per expert: 104 x 32 16 / 27 us, 224 x 32 36 / 46, 272
// x 50 94 / 110, 112 x 128 31 / 37, 388 x 22 40 / 45; 640 x 9 141 / 145; 704 x 16
// 122 / 103, 832 x 25 208 / 179, 416 x 128 193 / 175, 352 x 512 118 / 103, 152 x
// 1024 166 / 135.
// The choice is the whole layer's, whichever of its groups the launch computes:
// the few-row kernel adds k in another order, and a layer gives the same bits
// with its shared expert in a launch of its own.
constexpr int kFewAverage = 8, kMidAverage = 28;
constexpr int64_t kTallGrid = 512, kTallWork = 32768;
int tile_rows(FfnDims d) {
  d.groups = kGroupsAll;
  const int64_t tall = ffn_grid_mtiles(d, kManyRows) * (d.I / 128);
  if (d.T <= kFewRows || d.N <= (int64_t)kFewAverage * d.E ||
      (tall < kTallGrid && tall * d.N < kTallWork * d.E))
    return kFewRows;
  return d.N <= (int64_t)kMidAverage * d.E ? kMidRows : kManyRows;
}

// nt: packed tiles of the group with the most of them.
template <bool kGateUp, int kGroup>
hipError_t launch_gemm(Int4Args a, int rows, int64_t mtiles, int nt, hipStream_t s) {
  a.ntn = rows == kFewRows ? nt : (nt + 1) / 2;
  const int64_t work = mtiles * a.ntn;
  if (work > kMaxGridThreads / kThreads4 - kXcdGrid) return hipErrorInvalidValue;
  const dim3 grid(xcd_grid(work));
  if (rows == kFewRows)
    MOE_TIMED_LAUNCH(s, kGateUp ? "grouped_gemm_int4_few<true>" : "grouped_gemm_int4_few<false>",
      hipLaunchKernelGGL((grouped_gemm_int4_few<kGateUp, kGroup>), grid, dim3(kFewThreads), 0, s,
                         a));
  else
    MOE_TIMED_LAUNCH(s, kGateUp ? "grouped_gemm_int4_many<true>" : "grouped_gemm_int4_many<false>",
      hipLaunchKernelGGL((rows == kMidRows ? grouped_gemm_int4_many<kGateUp, kGroup, kMidRows>
                                           : grouped_gemm_int4_many<kGateUp, kGroup, kManyRows>),
                         grid, dim3(kThreads4), 0, s, a));
  return hipGetLastError();
}

}  // namespace

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
                           const void* ws13p, const void* ws2p, uint16_t* h, uint16_t* y,
                           uint16_t* ys, hipStream_t s) {
  const int rows = tile_rows(d);
  const int64_t mt = ffn_grid_mtiles(d, rows);

  Int4Args a{};
  a.offsets = offsets;
  a.routed = d.groups & kGroupRouted;
  a.per = (d.E + kWave - 1) / kWave;
  a.shared_rows = (d.groups & kGroupShared) && d.Is > 0 ? (int)d.T : 0;
  a.nt_r = d.I / 64;
  a.nt_s = d.Is / 64;
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
  const int nt1 = std::max(a.nt_r, a.nt_s);
  hipError_t e = group == 32 ? launch_gemm<true, 32>(a, rows, mt, nt1, s)
                             : launch_gemm<true, 128>(a, rows, mt, nt1, s);
  if (e != hipSuccess) return e;

  a.nt_r = a.nt_s = d.H / 128;
  a.a_s = h + d.N * d.I;
  a.a_r = h;
  a.lda_r = a.kdim_r = d.I;
  a.lda_s = a.kdim_s = d.Is;
  a.b_r = (const u32x4*)w2p;
  a.b_s = (const u32x4*)ws2p;
  a.c_r = y;
  a.c_s = ys;
  a.ldc_r = a.ldc_s = d.H;
  return group == 32 ? launch_gemm<false, 32>(a, rows, mt, a.nt_r, s)
                     : launch_gemm<false, 128>(a, rows, mt, a.nt_r, s);
}

}  // namespace moe
