// Device helpers of the MXFP4 product (fp4_matmul.hip): buffer loads that return zeros out
// of range, and Q_MX of 32 elements held by one lane.
#pragma once

#include "device_common.h"
#include "internal.h"

namespace moe {
namespace {

// Descriptor word 3 of raw (untyped) buffer loads.
constexpr int kBufferWord3 = 0x00020000;
// A lane offset behind every buffer used here (each is under 1 GiB, and so is what is added
// to this): the load returns zeros without memory traffic.
constexpr int kOutside = 1 << 30;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, kBufferWord3);
}

// ---- Q_MX of the 32 elements one lane holds ---------------------------------------------
// The FP4 operand layout of the block-scaled MFMA gives a lane 32 consecutive K elements of
// one row, i.e. exactly one MX group: its largest magnitude needs no other lane. The codes
// are those of moe_mx_quantize (mode 9): E8M0 = max(floor(log2 amax) - 2 + 127, 0), elements
// over 2^(E8M0 - 127) rounded to nearest even and held at +-6, by V_CVT_SCALEF32_PK_FP4_*
// (the tests compare every bf16 value).
__device__ __forceinline__ float e8m0_float(int b) { return __int_as_float(b > 0 ? b << 23 : 0x00400000); }

template <typename T> struct Group32;   // T: element type as the kernels name it

template <> struct Group32<uint16_t> {   // bf16
  static constexpr int kLoads = 4;       // 16-byte loads a lane
  static __device__ __forceinline__ int scale(const u32x4 (&u)[4]) {
    typedef unsigned short us2 __attribute__((ext_vector_type(2)));
    us2 m = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        m = __builtin_elementwise_max(m, __builtin_bit_cast(us2, u[i][j] & 0x7fff7fffu));
    const int b = ((m[0] > m[1] ? m[0] : m[1]) >> 7) - Fp8<2>::emax;
    return b < 0 ? 0 : b;
  }
  static __device__ __forceinline__ uint32_t codes(const u32x4& u, float s) {   // 8 elements
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(b2, (uint32_t)u[0]), s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(b2, (uint32_t)u[1]), s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(b2, (uint32_t)u[2]), s, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(b2, (uint32_t)u[3]), s, 3);
  }
  static __device__ __forceinline__ void run(const u32x4 (&u)[4], u32x4& q, int& b) {
    b = scale(u);
    const float s = e8m0_float(b);
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = codes(u[i], s);
  }
};

template <> struct Group32<_Float16> {
  static constexpr int kLoads = 4;
  static __device__ __forceinline__ void run(const u32x4 (&u)[4], u32x4& q, int& b) {
    typedef unsigned short us2 __attribute__((ext_vector_type(2)));
    typedef _Float16 h2 __attribute__((ext_vector_type(2)));
    us2 m = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        m = __builtin_elementwise_max(m, __builtin_bit_cast(us2, u[i][j] & 0x7fff7fffu));
    const unsigned short top = m[0] > m[1] ? m[0] : m[1];
    b = mx_scale_byte<2>((float)__builtin_bit_cast(_Float16, top));   // fp16's subnormals are normal in fp32
    const float s = e8m0_float(b);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t w = 0;
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, __builtin_bit_cast(h2, (uint32_t)u[i][0]), s, 0);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, __builtin_bit_cast(h2, (uint32_t)u[i][1]), s, 1);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, __builtin_bit_cast(h2, (uint32_t)u[i][2]), s, 2);
      q[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, __builtin_bit_cast(h2, (uint32_t)u[i][3]), s, 3);
    }
  }
};

template <> struct Group32<float> {
  static constexpr int kLoads = 8;
  static __device__ __forceinline__ void run(const u32x4 (&u)[8], u32x4& q, int& b) {
    int m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) m = max(m, (int)(u[i][j] & 0x7fffffffu));
    b = mx_scale_byte<2>(__int_as_float(m));
    const float s = e8m0_float(b);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t w = 0;
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(u[2 * i][0]), __uint_as_float(u[2 * i][1]), s, 0);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(u[2 * i][2]), __uint_as_float(u[2 * i][3]), s, 1);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(u[2 * i + 1][0]), __uint_as_float(u[2 * i + 1][1]), s, 2);
      q[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(u[2 * i + 1][2]), __uint_as_float(u[2 * i + 1][3]), s, 3);
    }
  }
};

// Rows [lo, hi) of group g, clamped into [0, rows) (offsets null: one group of all rows).
__device__ __forceinline__ void group_rows(const int32_t* off, int g, int rows, int* lo, int* hi) {
  if (!off) {
    *lo = 0;
    *hi = rows;
    return;
  }
  *lo = min(max(off[g], 0), rows);
  *hi = min(max(off[g + 1], *lo), rows);
}

// Four consecutive output channels of a row.
__device__ __forceinline__ void store4(float* p, const v4f& v) { *reinterpret_cast<v4f*>(p) = v; }
__device__ __forceinline__ void store4(uint16_t* p, const v4f& v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]));
}

}  // namespace
}  // namespace moe
