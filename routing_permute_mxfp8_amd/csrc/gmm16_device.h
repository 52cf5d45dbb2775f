// Device helpers of the 16-bit grouped products (gmm16.hip, gmm16_few.hip, gmm16_tile.h).
#pragma once

#include "device_common.h"
#include "fp4_device.h"

namespace moe {
namespace {

constexpr int kMaxGroups = 1024;

// The MFMAs of an element type: 16 bytes a lane of each operand.
template <typename T> struct Mfma;

template <> struct Mfma<__bf16> {
  typedef __bf16 v8 __attribute__((ext_vector_type(8)));
  static __device__ __forceinline__ v4f k32(u32x4 a, u32x4 b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
  }
  // c += a b in place; c is left alone until settled.
  static __device__ __forceinline__ void k32_into(v4f& c, u32x4 a, u32x4 b) {
    asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
  }
  static __device__ __forceinline__ uint32_t pair(float a, float b) { return bf16x2(a, b); }
  template <typename O> static __device__ __forceinline__ O out(float v) {
    if constexpr (sizeof(O) == 4) return v;
    else return (uint16_t)bf16x2(v, v);
  }
};

template <> struct Mfma<_Float16> {
  typedef _Float16 v8 __attribute__((ext_vector_type(8)));
  static __device__ __forceinline__ v4f k32(u32x4 a, u32x4 b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
  }
  // c += a b in place; c is left alone until settled.
  static __device__ __forceinline__ void k32_into(v4f& c, u32x4 a, u32x4 b) {
    asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
  }
  static __device__ __forceinline__ uint32_t pair(float a, float b) {   // to nearest even, each by itself
    typedef _Float16 h2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, h2{(_Float16)a, (_Float16)b});
  }
  template <typename O> static __device__ __forceinline__ O out(float v) {
    if constexpr (sizeof(O) == 4) return v;
    else return __builtin_bit_cast(uint16_t, (_Float16)v);
  }
};

// 16 bytes at any 16-bit element.
struct AnyChunk {
  u32x4 v;
} __attribute__((packed, aligned(2)));

// Elements 0 .. 7 at p, of which n are the row's: the others are 0.
template <bool VEC>
__device__ __forceinline__ u32x4 load_chunk(const uint16_t* p, int n) {
  u32x4 v = {};
  if constexpr (VEC) {
    if (n > 0) v = *reinterpret_cast<const u32x4*>(p);
  } else if (n >= 8) {
    v = reinterpret_cast<const AnyChunk*>(p)->v;
  } else if (n > 0) {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) v[i / 2] |= (uint32_t)p[i] << (i % 2 * 16);
  }
  return v;
}

// ends[g] = tiles of MT rows of groups 0 .. g (all 64 WAVES threads; ends has room for kMaxGroups,
// scratch for WAVES). Returns the number of tiles.
template <int MT, int WAVES>
__device__ __forceinline__ int count_tiles(const int32_t* off, int groups, int rows, int* ends, int* scratch) {
  constexpr int kEach = kMaxGroups / (64 * WAVES);
  const int t = threadIdx.x, lane = t & 63;
  int n[kEach], sum = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int g = kEach * t + i;
    int lo = 0, hi = 0;
    if (g < groups) group_rows(off, g, rows, &lo, &hi);
    sum += (hi - lo + MT - 1) / MT;
    n[i] = sum;
  }
  int incl = sum;
  for (int s = 1; s < 64; s *= 2) {
    const int v = __shfl_up(incl, s, 64);
    incl += lane >= s ? v : 0;
  }
  if (lane == 63) scratch[t >> 6] = incl;
  __syncthreads();
  int base = incl - sum, total = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    base += w < (t >> 6) ? scratch[w] : 0;
    total += scratch[w];
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) ends[kEach * t + i] = base + n[i];
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(total);
}

// The group of tile t: the first that ends behind it.
__device__ __forceinline__ int group_of_tile(const int* ends, int groups, int t) {
  int g = 0;
  for (int s = kMaxGroups / 2; s > 0; s /= 2)
    if (g + s <= groups - 1 && ends[g + s - 1] <= t) g += s;
  return g;
}

}  // namespace
}  // namespace moe
