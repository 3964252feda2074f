// One output tile of a large matrix product on bf16 MFMA (gfx950):
//   C(m, n) = sum_k A(m, k) B(k, n), fp32 accumulation,
// each operand lying along k ("row": A[m][k], B[n][k]) or across it ("col":
// A[k][m], B[k][n]), so that the products of a feed-forward block and of its
// backward need no transposed copies.
//
// Tile kM x kN of kM / kWM x 64 a wave, k in steps of 64 through two or more LDS
// stages that loads from memory fill directly.  A row operand's step is [row][64 k] in eight 16-byte
// chunks, chunk c of row r at c ^ (r & 7) ^ (r >> 3 & 3); a col operand's is [64 k][row],
// the 32-byte piece s of k row k at s ^ f(k), f = (k & 3) ^ (k & 3) << 1, and is
// transposed by the LDS's 16-bit transposing read: four k rows of 16 values a
// group of 16 lanes.  Either way the lanes that read together fall in different
// banks, and every load takes whole 128-byte lines (steps of 32, half a line of
// a row operand a load, took 14% longer where both operands are rows).
//
// A step's MFMAs come in four slices of 16 k.  Each runs while the operands of
// the next are read from LDS, across steps too.  Before a step's last slice its
// stage has been read for good and the next one has to be there: the waves
// meet, and among the last slice's MFMAs the stage's next loads are started.
// A wave alone on its SIMD would have no issue slots for this beside its MFMAs
// of a 256 x 256 tile's quarter (and its registers do not hold it): eight
// waves of 128 x 64.
//
// Loads go through buffer descriptors that end at the operand's last valid
// row (row operand) or last valid k (col operand): what lies past it arrives as
// zeros, so no size has to be a multiple of the tile and a k range that ends
// inside a step adds nothing.  Past a range's last step they are empty: those
// loads keep the waits' count and read nothing (T = 1 in three ranges read 5%
// more than its weights).
#pragma once

#include "moe_internal.hpp"

namespace moe {

typedef __attribute__((address_space(3))) void lds_void;
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int kGemmBK = 64;

enum : int { OP_ROW = 0, OP_COL = 1, OP_GATE_UP = 2 };

// An operand: the address of the tile's first row (row operand) or of the first
// k row at column 0 (col operand; the tile's first column is row0), the distance
// of rows in bytes, and the valid rows.  OP_GATE_UP is a row operand whose row
// blocks of 32 alternate between two matrices.
struct Operand {
  const char* p;
  int64_t to2;    // OP_GATE_UP: from p to the same row of the second matrix
  int64_t ld;     // bytes
  int64_t rows;   // row operand: rows from p on; col operand: valid k
};

// A value that is the same in every lane, in a scalar register.
__device__ __forceinline__ uint32_t scalar(uint32_t v) { return __builtin_amdgcn_readfirstlane(v); }

// A buffer descriptor of `bytes` from p (clamped to what it can hold).
__device__ __forceinline__ u32x4 buffer_of(const char* p, int64_t bytes) {
  const int64_t b = bytes < 0 ? 0 : bytes > 0xfffffff0LL ? 0xfffffff0LL : bytes;
  const uint64_t a = (uint64_t)(uintptr_t)p;
  return (u32x4){scalar((uint32_t)a), scalar((uint32_t)(a >> 32) & 0xffffu), scalar((uint32_t)b),
                 0x00020000u};
}

// Byte address in LDS.
__device__ __forceinline__ uint32_t lds_address(const u32x4* lds) {
  return scalar((uint32_t)(uintptr_t)(lds_void*)lds);
}

// Loads of 16 bytes a lane from memory into 1 KiB of LDS from address lds (the
// same in every lane): from an offset into a buffer, or from an address.  The
// instructions are written out because of what the compiler does with more than
// two stages: at a loop's first read of LDS it waits for every load under way.
// They have no result register; wait_and_meet waits for them.
__device__ __forceinline__ void load_to_lds(u32x4 buffer, uint32_t lds, int offset) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               ::"s"(lds), "v"(offset), "s"(buffer) : "memory");
}

__device__ __forceinline__ void load_global_to_lds(const void* p, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               ::"s"(lds), "v"(p) : "memory");
}

// Waits until at most kLeft of this wave's loads to LDS are under way and its
// LDS reads are done, then for the other waves.  (A barrier by itself would
// let the compiler move LDS accesses across it, __syncthreads waits for every
// load.)
template <int kLeft>
__device__ __forceinline__ void wait_and_meet() {
  static_assert(kLeft < 63, "the counter's range");
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kLeft) : "memory");
}

__device__ __forceinline__ int row_swizzle(int r, int c) { return c ^ (r & 7) ^ (r >> 3 & 3); }
__device__ __forceinline__ int row_chunk(int r, int c) { return r * 8 + row_swizzle(r, c); }
template <int kRows>
__device__ __forceinline__ int col_piece(int k, int s) {
  return s ^ (((k & 3) ^ ((k & 3) << 1)) & (kRows / 16 - 1));
}

// Stages one operand of kRows rows with kThreads threads.
template <int kOp, int kRows, int kThreads>
struct Stager {
  static constexpr int kLoads = kRows * 8 / kThreads;   // 16-byte pieces a thread
  static constexpr int kPer = kRows / 8;                // pieces of a k row (col operand)
  static constexpr int kPass = kThreads / 8;            // rows a load (row operand)
  const char* p;
  int64_t rows;
  int ld, wave;
  u32x4 fixed, second;   // row operand: the buffer of every step
  int at;        // this thread's offset of load 0, step 0

  __device__ __forceinline__ Stager(const Operand& o, int row0, int tid, int wave_)
      : p(o.p), rows(o.rows), ld((int)o.ld), wave(wave_) {
    // Gate / up: 32-row blocks 2 i and 2 i + 1 are rows 32 i.. of the two matrices; a
    // wave's 8 rows of a load are of one of them, the same in every load of 64
    // rows (of 32 rows: in every second load, see load).
    if (kOp != OP_COL)
      fixed = buffer_of(kOp == OP_GATE_UP && kPass == 64 ? o.p + (wave >> 2 & 1) * o.to2 : o.p,
                        o.rows * o.ld);
    if (kOp == OP_GATE_UP && kPass == 32) second = buffer_of(o.p + o.to2, o.rows * o.ld);
    if (kOp == OP_COL) {
      const int k = tid / kPer, c = tid % kPer;
      at = k * ld + (row0 + (col_piece<kRows>(k, c >> 1) * 2 + (c & 1)) * 8) * 2;
    } else {
      const int r = tid >> 3, c = row_swizzle(r, tid & 7);
      at = (kOp == OP_GATE_UP ? r & 31 : r) * ld + c * 16;
    }
  }
  // Of a k step, empty from step `end` on.
  __device__ __forceinline__ u32x4 buffer(int step, int end) const {
    const int64_t k = (int64_t)step * kGemmBK;
    u32x4 b = kOp == OP_COL ? buffer_of(p + k * ld, (rows - k) * ld) : fixed;
    b[2] = step < end ? b[2] : 0;
    return b;
  }
  // Starts load j of k step `step` into the operand's place of a stage.
  __device__ __forceinline__ void load(u32x4 buf, uint32_t lds, int step, int j) const {
    // k rows kThreads / kPer apart, a multiple of 4; or rows kPass apart
    const int off = kOp == OP_COL        ? j * (kThreads / kPer) * ld
                    : kOp == OP_GATE_UP ? j * kPass / 64 * 32 * ld + step * (kGemmBK * 2)
                                         : j * kPass * ld + step * (kGemmBK * 2);
    static_assert(kOp != OP_GATE_UP || kPass == 32 || kPass == 64, "rows a load");
    if (kOp == OP_GATE_UP && kPass == 32 && (j & 1))
      buf = (u32x4){second[0], second[1], buf[2], second[3]};   // as long as the other
    load_to_lds(buf, lds + (j * kThreads + wave * 64) * 16, at + off);
  }
};

// The MFMA operand of 32 rows from `row`, k = 16 kk + 8 (lane / 32) + 0..7.
template <int kOp, int kRows>
__device__ __forceinline__ bf16x8 fragment(const u32x4* lds, int row, int kk, int lane) {
  if (kOp == OP_COL) {
    const int g = lane >> 4, l = lane & 15;
    const int k = 16 * kk + 8 * (g >> 1) + (l >> 2);
    const int s = (row >> 4) + (g & 1);
    const char* base = reinterpret_cast<const char*>(lds) + col_piece<kRows>(k, s) * 32 + (l & 3) * 8;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(base + k * (kRows * 2)));
    const s16x4 hi =
        __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(base + (k + 4) * (kRows * 2)));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  }
  return as_bf16x8(lds[row_chunk(row + (lane & 31), 2 * kk + (lane >> 5))]);
}

// The tile's accumulators: wave (wm, wn) of kWM x kWN holds rows row0() + 32 i,
// columns col0() + 32 j.  lds: kPieces 16-byte pieces, kSA stages of A (as many as
// of B or one more), then kSB of B.
template <int kM, int kN, int kWM, int kWN, int kSA, int kSB, int kOpA, int kOpB>
struct GemmTile {
  static constexpr int kThreads = 64 * kWM * kWN;
  static constexpr int kMI = kM / kWM / 32, kNJ = kN / kWN / 32;
  static constexpr int kPieces = kSA * kM * 8 + kSB * kN * 8;
  static_assert(kNJ == 2, "64 columns a wave");

  static __device__ __forceinline__ int wave() { return (int)scalar(threadIdx.x >> 6); }
  static __device__ __forceinline__ int row0(int wave) { return wave / kWN * (kM / kWM); }
  static __device__ __forceinline__ int col0(int wave) { return wave % kWN * (kN / kWN); }

  // Sums over k steps [s0, s1).
  static __device__ __forceinline__ void run(u32x4* lds, const Operand& A, int m0,
                                             const Operand& B, int n0, int s0, int s1,
                                             f32x16 (&acc)[kMI][kNJ]) {
    const int tid = threadIdx.x, lane = tid & 63, w = wave();
    const int wrow = row0(w), wcol = col0(w);
    const uint32_t lds_at = lds_address(lds);
    const Stager<kOpA, kM, kThreads> sa(A, m0, tid, w);
    const Stager<kOpB, kN, kThreads> sb(B, n0, tid, w);
#pragma unroll
    for (int i = 0; i < kMI; ++i)
#pragma unroll
      for (int j = 0; j < kNJ; ++j)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.0f;
    if (s0 >= s1) return;

    // Loads of a step: B's (to stage sb), then A's (to stage sa).
    const uint32_t lds_b = lds_at + kSA * kM * 128;
    auto load_b = [&](const u32x4& bb, int stage, int step, int i) {
      sb.load(bb, lds_b + stage * (kN * 128), step, i);
    };
    auto load_a = [&](const u32x4& ba, int stage, int step, int i) {
      sa.load(ba, lds_at + stage * (kM * 128), step, i);
    };
    struct Slice {
      bf16x8 a[kMI], b[kNJ];
    };
    // Operand i of slice kk of a stage, in [0, kMI + kNJ): b[0], a[0], b[1], the rest.
    constexpr int kReads = kMI + kNJ, kMfma = kMI * kNJ;
    constexpr int kPer = (sa.kLoads + sb.kLoads + kMfma - 1) / kMfma;   // loads an MFMA
    auto read = [&](Slice& f, int s, int kk, int i) {   // s: the step, modulo the stages
      const u32x4 *la = lds + s % kSA * (kM * 8), *lb = lds + (kSA * kM + s % kSB * kN) * 8;
      if (i == 0 || (i >= 2 && i <= kNJ))
        f.b[i == 0 ? 0 : i - 1] =
            fragment<kOpB, kN>(lb, wcol + (i == 0 ? 0 : i - 1) * 32, kk, lane);
      else
        f.a[i == 1 ? 0 : i - kNJ] =
            fragment<kOpA, kM>(la, wrow + (i == 1 ? 0 : i - kNJ) * 32, kk, lane);
    };
    // A slice's MFMAs, and between them the reads of the next slice's operands
    // (slice kk of the step that is s modulo the stages) and, with `loads`, the
    // loads of later steps into the stages that step s - 1 was in, B's first (the
    // waits count on the order).
    auto slice = [&](const Slice& f, Slice& next, int s, int kk, bool loads, int step) {
      u32x4 ba, bb;
      if (loads) {
        ba = sa.buffer(step + kSA, s1);
        bb = sb.buffer(step + kSB, s1);
      }
#pragma unroll
      for (int q = 0; q < kMfma; ++q) {
        const int i = q / kNJ, j = q % kNJ;
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.a[i], f.b[j], acc[i][j], 0, 0, 0);
#pragma unroll
        for (int r = q; r < kReads; r += kMfma) read(next, s, kk, r);
        if (loads) {
#pragma unroll
          for (int r = q * kPer; r < (q + 1) * kPer && r < sa.kLoads + sb.kLoads; ++r)
            if (r < sb.kLoads) load_b(bb, (s + kSB - 1) % kSB, step + kSB, r);
            else load_a(ba, (s + kSA - 1) % kSA, step + kSA, r - sb.kLoads);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    // Loads that may be under way when the next step has to be there: those of
    // the steps behind it.
    constexpr int kAhead = (kSA - 2) * sa.kLoads + (kSB - 2) * sb.kLoads;
    static_assert(kSA == kSB || kSA == kSB + 1, "stages");
    Slice f0, f1;
    auto step = [&](int i, int s) {   // i: s modulo the stages
      slice(f0, f1, i, 1, false, 0);
      slice(f1, f0, i, 2, false, 0);
      slice(f0, f1, i, 3, false, 0);
      wait_and_meet<kAhead>();   // step s + 1 is there, s is read
      __builtin_amdgcn_sched_barrier(0);
      slice(f1, f0, i + 1, 0, true, s);
    };
    // In the loop's order: B's of a step, then A's of a step or of the one after.
#pragma unroll
    for (int i = 0; i < kSA; ++i) {
      const u32x4 ba = sa.buffer(s0 + i, s1), bb = sb.buffer(s0 + i - (kSA - kSB), s1);
      if (i >= kSA - kSB) {
#pragma unroll
        for (int r = 0; r < sb.kLoads; ++r) load_b(bb, i - (kSA - kSB), s0 + i - (kSA - kSB), r);
      }
#pragma unroll
      for (int r = 0; r < sa.kLoads; ++r) load_a(ba, i, s0 + i, r);
    }
    wait_and_meet<kAhead + sa.kLoads + sb.kLoads>();
#pragma unroll
    for (int i = 0; i < kReads; ++i) read(f0, 0, 0, i);
    constexpr int kTurn = kSA == kSB ? kSA : kSA * kSB;
    for (int s = s0; s < s1;) {
#pragma unroll
      for (int i = 0; i < kTurn; ++i)
        if (s < s1) step(i, s++);
    }
    wait_and_meet<0>();   // the LDS is free
  }
};

// Hands a wave's part of a tile out row by row: f(row, column, v) with v the fp32
// values of eight consecutive columns, through the wave's own 32 x 64 floats of
// LDS.  acc [kMI][2] are 32 x 32 blocks; rows and columns count from the wave's
// first.  With kPair, the two column blocks come together: f(row, column, v, w).
template <bool kPair, int kMI, class F>
__device__ __forceinline__ void wave_rows(float* l, const f32x16 (&acc)[kMI][2], F f) {
  const int lane = threadIdx.x & 63, lr = lane & 31, lh = lane >> 5;
  // physical column: the other half for every second group of four rows
  auto phys = [](int row, int col) { return row * 64 + (col ^ ((row & 4) * 8)); };
#pragma unroll
  for (int i = 0; i < kMI; ++i) {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q)
        l[phys(8 * (q >> 2) + 4 * lh + (q & 3), j * 32 + lr)] = acc[i][j][q];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    auto get = [&](int row, int col, float (&v)[8]) {
      const f32x4* p = reinterpret_cast<const f32x4*>(l + phys(row, col));
      const f32x4 x = p[0], y = p[1];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        v[t] = x[t];
        v[4 + t] = y[t];
      }
    };
    if constexpr (kPair) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int row = t * 16 + (lane >> 2), col = (lane & 3) * 8;
        float v[8], w[8];
        get(row, col, v);
        get(row, 32 + col, w);
        f(i * 32 + row, col, v, w);
      }
    } else {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int row = t * 8 + (lane >> 3), col = (lane & 7) * 8;
        float v[8];
        get(row, col, v);
        f(i * 32 + row, col, v);
      }
    }
  }
}

}  // namespace moe
