// Eight consecutive values of a token row, bf16 or fp32 (gfx950 device code),
// shared by the kernels that work on whole rows.
#pragma once

#include "moe_internal.hpp"

namespace moe {

// A chunk is eight values: one 16-byte access in bf16, two in fp32.
constexpr int kChunk = 8;

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

// A chunk as it lies in memory.
template <typename IO>
struct RawChunk;
template <>
struct RawChunk<uint16_t> {
  u32x4 v;
  __device__ __forceinline__ void load(const uint16_t* p) {
    v = *reinterpret_cast<const u32x4*>(p);
  }
  __device__ __forceinline__ void to(float (&f)[8]) const { unpack_bf16x8(v, f); }
};
template <>
struct RawChunk<float> {
  f32x4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const f32x4*>(p);
    b = *reinterpret_cast<const f32x4*>(p + 4);
  }
  __device__ __forceinline__ void to(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = a[i];
      f[4 + i] = b[i];
    }
  }
};

template <typename IO>
__device__ __forceinline__ void load_chunk(const IO* p, float (&f)[8]) {
  RawChunk<IO> r;
  r.load(p);
  r.to(f);
}

__device__ __forceinline__ void store_chunk(uint16_t* p, const float (&f)[8]) {
  *reinterpret_cast<u32x4*>(p) = pack_bf16x8(f);
}
__device__ __forceinline__ void store_chunk(float* p, const float (&f)[8]) {
  *reinterpret_cast<f32x4*>(p) = (f32x4){f[0], f[1], f[2], f[3]};
  *reinterpret_cast<f32x4*>(p + 4) = (f32x4){f[4], f[5], f[6], f[7]};
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

// Sum of v over the NT threads of a workgroup in a fixed order (wave
// shuffles, then the waves in order); every thread gets the result.  red
// holds NT / 64 floats; every thread calls this.
template <int NT>
__device__ __forceinline__ float workgroup_sum(float v, float* red) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  if (NT == 64) return v;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int w = 0; w < NT / 64; ++w) s += red[w];
  __syncthreads();
  return s;
}

}  // namespace moe
