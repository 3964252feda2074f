// One output tile of a large matrix product on bf16 MFMA (gfx950):
//   C(m, n) = sum_k A(m, k) B(k, n), fp32 accumulation,
// each operand lying along k ("row": A[m][k], B[n][k]) or across it ("col":
// A[k][m], B[k][n]), so that the products of a feed-forward block and of its
// backward need no transposed copies.
//
// Tile kM x kN, k in steps of 64 through two LDS buffers that are filled by
// loads from memory straight to LDS.  A row operand's step is [row][64 k] in
// eight 16-byte chunks, chunk c of row r at c ^ (r & 7 ^ r >> 3 & 7); a col
// operand's is [64 k][row], the 32-byte piece s of k row k at s ^ f(k),
// f = (k & 3) ^ (k & 3) << 1, and is transposed by the LDS's 16-bit
// transposing read: four k rows of 16 values a group of 16 lanes.  Either way
// the lanes that read together fall in different banks.
//
// Loads go through buffer descriptors that end at the operand's last valid
// row (row operand) or last valid k (col operand): what lies past it arrives as
// zeros, so no size has to be a multiple of the tile, and a k range that ends
// inside a step adds nothing.
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
  const char* p[2];
  int64_t ld;     // bytes
  int64_t rows;   // row operand: rows from p on; col operand: valid k
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const char* p, int64_t bytes) {
  const int64_t b = bytes < 0 ? 0 : bytes > 0xfffffff0LL ? 0xfffffff0LL : bytes;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(p), 0, (int)(uint32_t)b, 0x00020000);
}

__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t r, u32x4* lds, int offset) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds, 16, offset, 0, 0, 0);
}

// The same from an address of its own a lane into the 64 pieces from lds (the
// same in every lane); kNt: not kept in cache.  The instruction is written out
// for pipelines of more than two stages: what the compiler sees of it makes it
// wait, at a loop's first read of LDS, for every load under way.  It has no
// result register; wait_and_meet waits for it.
template <bool kNt>
__device__ __forceinline__ void load_global_to_lds(const void* p, u32x4* lds) {
  const uint32_t at = (uint32_t)(uintptr_t)(lds_void*)lds;
  if (kNt)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off nt"
                 ::"s"(at), "v"(p) : "memory");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
                 ::"s"(at), "v"(p) : "memory");
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

__device__ __forceinline__ int row_chunk(int r, int c) {
  return r * 8 + (c ^ ((r ^ (r >> 3)) & 7));
}
template <int kRows>
__device__ __forceinline__ int col_piece(int k, int s) {
  return s ^ (((k & 3) ^ ((k & 3) << 1)) & (kRows / 16 - 1));
}

// Stages one operand of kRows rows with kThreads threads.
template <int kOp, int kRows, int kThreads>
struct Stager {
  static constexpr int kLoads = kRows * 8 / kThreads;   // 16-byte pieces a thread
  static constexpr int kPer = kRows / 8;                // pieces of a k row (col operand)
  const Operand& o;
  int wave;
  int at;   // this thread's offset of load 0, step 0

  __device__ __forceinline__ Stager(const Operand& op, int row0, int tid, int wave_)
      : o(op), wave(wave_) {
    if (kOp == OP_COL) {
      const int k = tid / kPer, c = tid % kPer;
      at = (int)(k * o.ld) + (row0 + (col_piece<kRows>(k, c >> 1) * 2 + (c & 1)) * 8) * 2;
    } else {
      const int r = tid >> 3, c = (tid & 7) ^ ((r ^ (r >> 3)) & 7);
      // gate / up: row blocks 2 i and 2 i + 1 of 32 are rows 32 i.. of the two
      at = (int)((kOp == OP_GATE_UP ? (r & 31) + (r >> 6) * 32 : r) * o.ld) + c * 16;
    }
  }
  // Starts the loads of k step `step` into lds [kRows * 8].
  __device__ __forceinline__ void load(u32x4* lds, int step) const {
    if (kOp == OP_COL) {
      const auto rs = buffer_of(o.p[0] + (int64_t)step * kGemmBK * o.ld,
                                (o.rows - (int64_t)step * kGemmBK) * o.ld);
#pragma unroll
      for (int j = 0; j < kLoads; ++j)   // k rows kThreads / kPer apart: a multiple of 4
        load_to_lds(rs, lds + j * kThreads + wave * 64, at + j * (kThreads / kPer) * (int)o.ld);
    } else if (kOp == OP_ROW) {
      const auto rs = buffer_of(o.p[0], o.rows * o.ld);
#pragma unroll
      for (int j = 0; j < kLoads; ++j)
        load_to_lds(rs, lds + j * kThreads + wave * 64,
                    at + j * (kThreads / 8) * (int)o.ld + step * (kGemmBK * 2));
    } else {
      const auto r0 = buffer_of(o.p[0], o.rows * o.ld), r1 = buffer_of(o.p[1], o.rows * o.ld);
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        // kThreads / 8 rows a load: 64 (the wave decides the matrix) or 32 (j does)
        const bool up = kThreads == 512 ? wave >= 4 : (j & 1);
        const int rows = kThreads == 512 ? 32 * j : 32 * (j >> 1);
        load_to_lds(up ? r1 : r0, lds + j * kThreads + wave * 64,
                    at + rows * (int)o.ld + step * (kGemmBK * 2));
      }
    }
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
// columns col0() + 32 j.  lds0, lds1: two arrays of
// (kM + kN) * 8 16-byte pieces, apart in the compiler's eyes, so that it sees
// that a load into one does not touch reads of the other.
template <int kM, int kN, int kWM, int kWN, int kOpA, int kOpB>
struct GemmTile {
  static constexpr int kThreads = 64 * kWM * kWN;
  static constexpr int kMI = kM / kWM / 32, kNJ = kN / kWN / 32;
  static constexpr int kLds = (kM + kN) * 8;

  static __device__ __forceinline__ int wave() {
    return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  }
  static __device__ __forceinline__ int row0() { return wave() / kWN * (kM / kWM); }
  static __device__ __forceinline__ int col0() { return wave() % kWN * (kN / kWN); }

  static __device__ __forceinline__ void run(u32x4* lds0, u32x4* lds1, const Operand& A, int m0,
                                             const Operand& B, int n0, int64_t K,
                                             f32x16 (&acc)[kMI][kNJ]) {
    const int tid = threadIdx.x, lane = tid & 63;
    const Stager<kOpA, kM, kThreads> sa(A, m0, tid, wave());
    const Stager<kOpB, kN, kThreads> sb(B, n0, tid, wave());
    const int nsteps = (int)((K + kGemmBK - 1) / kGemmBK);
#pragma unroll
    for (int i = 0; i < kMI; ++i)
#pragma unroll
      for (int j = 0; j < kNJ; ++j)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.0f;

    auto load = [&](u32x4* l, int step) {
      sa.load(l, step);
      sb.load(l + kM * 8, step);
    };
    auto compute = [&](const u32x4* l) {
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        bf16x8 a[kMI], b[kNJ];
#pragma unroll
        for (int i = 0; i < kMI; ++i)
          a[i] = fragment<kOpA, kM>(l, row0() + i * 32, kk, lane);
#pragma unroll
        for (int j = 0; j < kNJ; ++j)
          b[j] = fragment<kOpB, kN>(l + kM * 8, col0() + j * 32, kk, lane);
#pragma unroll
        for (int i = 0; i < kMI; ++i)
#pragma unroll
          for (int j = 0; j < kNJ; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[i], b[j], acc[i][j], 0, 0, 0);
      }
    };
    // Step s computes from one buffer while step s + 1 arrives in the other;
    // the barrier at its end waits for both.
    load(lds0, 0);
    __syncthreads();
    int s = 0;
    for (; s + 2 <= nsteps; s += 2) {
      load(lds1, s + 1);
      __builtin_amdgcn_sched_barrier(0);
      compute(lds0);
      __syncthreads();
      if (s + 2 < nsteps) load(lds0, s + 2);
      __builtin_amdgcn_sched_barrier(0);
      compute(lds1);
      __syncthreads();
    }
    if (s < nsteps) {
      compute(lds0);
      __syncthreads();
    }
  }
};

// Hands a wave's part of a tile out row by row: f(row, column, v) with v the fp32
// values of eight consecutive columns, through the wave's own 32 x 32 kNJ floats
// of LDS.  acc [kMI][kNJ] are 32 x 32 blocks; rows and columns count from the
// wave's first.  With kPair, the same columns of the two column blocks come
// together: f(row, column in a block, v, w).
template <bool kPair, int kMI, int kNJ, class F>
__device__ __forceinline__ void wave_rows(float* l, const f32x16 (&acc)[kMI][kNJ], F f) {
  static_assert(kNJ == 1 || kNJ == 2, "one or two column blocks a wave");
  constexpr int kCols = 32 * kNJ;
  const int lane = threadIdx.x & 63, lr = lane & 31, lh = lane >> 5;
  // physical column: the other half for every second group of four rows
  auto phys = [](int row, int col) {
    return row * kCols + (kNJ == 2 ? col ^ ((row & 4) * 8) : col);
  };
#pragma unroll
  for (int i = 0; i < kMI; ++i) {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int j = 0; j < kNJ; ++j)
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
      static_assert(kNJ == 2, "a pair of column blocks");
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int row = t * 16 + (lane >> 2), col = (lane & 3) * 8;
        float v[8], w[8];
        get(row, col, v);
        get(row, 32 + col, w);
        f(i * 32 + row, col, v, w);
      }
    } else {
      constexpr int kL = kCols / 8;   // lanes a row
#pragma unroll
      for (int t = 0; t < kL / 2; ++t) {
        const int row = t * (64 / kL) + lane / kL, col = (lane % kL) * 8;
        float v[8];
        get(row, col, v);
        f(i * 32 + row, col, v);
      }
    }
  }
}

}  // namespace moe
