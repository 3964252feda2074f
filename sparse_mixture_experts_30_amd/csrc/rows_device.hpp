// Sixteen bytes of a token row, bf16 or fp32 (gfx950 device code), and sums over
// lanes, shared by the kernels that work on whole rows.
#pragma once

#include "moe_internal.hpp"

namespace moe {

// A chunk is one 16-byte access: eight values in bf16, four in fp32.  Eight in
// fp32 leave every other 16 bytes of the row out of each access: the norm of
// 3000 x 4096 fp32 rows took 38.7 us instead of 33.3, the gradients of 665
// tokens of 4352 values (8 slots) 85 instead of 77.
template <typename IO>
constexpr int kWidth = 16 / (int)sizeof(IO);

__device__ __forceinline__ void unpack_bf16x8(u32x4 v, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(v[i] << 16);
    f[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ u32x4 pack_bf16x8(const float (&f)[8]) {
  return (u32x4){pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                 pack_bf16x2(f[6], f[7])};
}

// 16 bytes; kNt: non-temporal, for data that is not used again soon.
template <bool kNt, typename V>
__device__ __forceinline__ V load16(const V* p) {
  return kNt ? __builtin_nontemporal_load(p) : *p;
}
template <bool kNt, typename V>
__device__ __forceinline__ void store16(V* p, V v) {
  if (kNt)
    __builtin_nontemporal_store(v, p);
  else
    *p = v;
}

// A chunk as it lies in memory.
template <typename IO>
struct RawChunk;
template <>
struct RawChunk<uint16_t> {
  u32x4 v;
  template <bool kNt = false>
  __device__ __forceinline__ void load(const uint16_t* p) {
    v = load16<kNt>(reinterpret_cast<const u32x4*>(p));
  }
  __device__ __forceinline__ void to(float (&f)[8]) const { unpack_bf16x8(v, f); }
};
template <>
struct RawChunk<float> {
  f32x4 v;
  template <bool kNt = false>
  __device__ __forceinline__ void load(const float* p) {
    v = load16<kNt>(reinterpret_cast<const f32x4*>(p));
  }
  __device__ __forceinline__ void to(float (&f)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = v[i];
  }
};

template <typename IO>
__device__ __forceinline__ void load_chunk(const IO* p, float (&f)[kWidth<IO>]) {
  RawChunk<IO> r;
  r.load(p);
  r.to(f);
}

template <bool kNt = false>
__device__ __forceinline__ void store_chunk(uint16_t* p, const float (&f)[8]) {
  store16<kNt>(reinterpret_cast<u32x4*>(p), pack_bf16x8(f));
}
template <bool kNt = false>
__device__ __forceinline__ void store_chunk(float* p, const float (&f)[4]) {
  store16<kNt>(reinterpret_cast<f32x4*>(p), (f32x4){f[0], f[1], f[2], f[3]});
}

// N fp32 values beside a chunk of N values (norm weights and their gradient).
template <int N>
__device__ __forceinline__ void load_f32(const float* p, float (&f)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const f32x4 v = *reinterpret_cast<const f32x4*>(p + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) f[i + j] = v[j];
  }
}
template <int N>
__device__ __forceinline__ void store_f32(float* p, const float (&f)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4)
    *reinterpret_cast<f32x4*>(p + i) = (f32x4){f[i], f[i + 1], f[i + 2], f[i + 3]};
}

// v as a row of type IO holds it.
template <typename IO>
__device__ __forceinline__ float as_stored(float v);
template <>
__device__ __forceinline__ float as_stored<uint16_t>(float v) {
  return bf16_bits_to_f32(f32_to_bf16_bits(v));
}
template <>
__device__ __forceinline__ float as_stored<float>(float v) {
  return v;
}

// v of the lane n places on in the same row of 16 lanes (data-parallel move:
// no trip through LDS as a shuffle takes).
template <int n>
__device__ __forceinline__ float row_rotate(float v) {
  return __int_as_float(
      __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x120 + n, 0xf, 0xf, true));
}

// Sum of v over each row of 16 lanes; every lane gets its row's, lanes of one
// row in different orders of addition.
__device__ __forceinline__ float row_sum(float v) {
  v += row_rotate<8>(v);
  v += row_rotate<4>(v);
  v += row_rotate<2>(v);
  v += row_rotate<1>(v);
  return v;
}

__device__ __forceinline__ float lane_value(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}

// Sum of v over the wave, the same bits in every lane.
__device__ __forceinline__ float wave_sum(float v) {
  v = row_sum(v);
  return (lane_value(v, 0) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
}

// Largest v over each row of 16 lanes (NaN ignored).
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, row_rotate<8>(v));
  v = fmaxf(v, row_rotate<4>(v));
  v = fmaxf(v, row_rotate<2>(v));
  return fmaxf(v, row_rotate<1>(v));
}

}  // namespace moe
