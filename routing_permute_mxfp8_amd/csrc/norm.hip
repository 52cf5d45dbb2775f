// Root-mean-square norm of the sum of a row and its residual, with MX codes of the normed row,
// and its gradient.
//
//   h = T(x + residual)                      (T: the rows' type; h is what the next layer adds to)
//   rstd = 1 / sqrt(sum_c h_c^2 / C + eps)
//   y = T(h rstd w), (codes, scales) = Q_MX(y)
// and with a = grad_y w, xh = h rstd:
//   grad_x = T(rstd (a - xh sum_c(a xh) / C) + grad_h), grad_w = sum over the rows of grad_y xh.
//
// The norm is of the sum as it is kept, rounded to T, so that the backward pass, which has only
// that, sees the same rows; and the codes are those of y rounded to T, so that they are the bytes
// that moe_mx_quantize makes of y. The squares are summed in 64 bits: no finite row overflows.
//
// A thread holds 8 neighbouring elements (16 bytes of a 16-bit type) of a row, or two such chunks,
// so every input is read and every output written once; an MX group of 32 is four lanes, whose
// largest magnitude takes two DPP steps. Rows whose chunks are no 16-byte vectors (an odd number
// of columns, a tensor that starts elsewhere) are read and written by elements.

#include <algorithm>

#include "device_common.h"
#include "internal.h"

namespace moe {
namespace {

// ---- element types ----------------------------------------------------------------------
// 8 elements of a row as floats; n of them exist (the others come as 0 and are not written).
template <typename T> struct Row8;

template <> struct Row8<uint16_t> {   // bf16
  static __device__ __forceinline__ void load(const uint16_t* p, float (&f)[8]) {
    const u32x4 u = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(u[i] << 16);
      f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ float one(const uint16_t* p) { return bf16_to_f(*p); }
  static __device__ __forceinline__ float round(float v) { return __uint_as_float(bf16x2(v, v) << 16); }
  static __device__ __forceinline__ void store(uint16_t* p, const float (&f)[8]) {
    u32x4 u;
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = bf16x2(f[2 * i], f[2 * i + 1]);
    *reinterpret_cast<u32x4*>(p) = u;
  }
  static __device__ __forceinline__ void put(uint16_t* p, float v) { *p = (uint16_t)bf16x2(v, v); }
};

template <> struct Row8<_Float16> {
  typedef _Float16 h8 __attribute__((ext_vector_type(8)));
  static __device__ __forceinline__ void load(const _Float16* p, float (&f)[8]) {
    const h8 h = *reinterpret_cast<const h8*>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = (float)h[i];
  }
  static __device__ __forceinline__ float one(const _Float16* p) { return (float)*p; }
  static __device__ __forceinline__ float round(float v) { return (float)(_Float16)v; }
  static __device__ __forceinline__ void store(_Float16* p, const float (&f)[8]) {
    h8 h;
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = (_Float16)f[i];
    *reinterpret_cast<h8*>(p) = h;
  }
  static __device__ __forceinline__ void put(_Float16* p, float v) { *p = (_Float16)v; }
};

template <> struct Row8<float> {
  static __device__ __forceinline__ void load(const float* p, float (&f)[8]) {
    const v4f a = *reinterpret_cast<const v4f*>(p), b = *reinterpret_cast<const v4f*>(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = a[i];
      f[4 + i] = b[i];
    }
  }
  static __device__ __forceinline__ float one(const float* p) { return *p; }
  static __device__ __forceinline__ float round(float v) { return v; }
  static __device__ __forceinline__ void store(float* p, const float (&f)[8]) {
    v4f a, b;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = f[i];
      b[i] = f[4 + i];
    }
    *reinterpret_cast<v4f*>(p) = a;
    *reinterpret_cast<v4f*>(p + 4) = b;
  }
  static __device__ __forceinline__ void put(float* p, float v) { *p = v; }
};

template <bool VEC, typename T>
__device__ __forceinline__ void load8(const T* p, int n, float (&f)[8]) {
  if constexpr (VEC) {
    Row8<T>::load(p, f);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = i < n ? Row8<T>::one(p + i) : 0.0f;
  }
}

template <bool VEC, typename T>
__device__ __forceinline__ void store8(T* p, int n, const float (&f)[8]) {
  if constexpr (VEC) {
    Row8<T>::store(p, f);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) Row8<T>::put(p + i, f[i]);
  }
}

// The same of the weight, which is of the rows' type or fp32.
template <bool VEC, typename T>
__device__ __forceinline__ void load_weight(const void* w, bool fp32, int c, int n, float (&f)[8]) {
  if (fp32)
    load8<VEC>((const float*)w + c, n, f);
  else
    load8<VEC>((const T*)w + c, n, f);
}

// MX codes (8 elements; F as in device_common.h) of y over its group's scale to row element c.
template <int F>
__device__ __forceinline__ int quantise8(const float (&y)[8], uint8_t* codes, int64_t at) {
  int m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_int(fabsf(y[i])));
  const int b = mx_scale_byte<F>(__int_as_float(quad_max_bits(m)));
  const float inv = mx_inv_scale(b);
  if constexpr (F == 2) {
    uint32_t q = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) q |= fp4_code(y[i] * inv) << (4 * i);
    *reinterpret_cast<uint32_t*>(codes + at / 2) = q;
  } else {
    *reinterpret_cast<uint2*>(codes + at) = make_uint2(pack4<F>(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv),
                                                       pack4<F>(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv));
  }
  return b;
}

// Sum over a row's LANES threads (a power of two; rows of fewer than 64 share a wave, wider
// ones have the block to themselves), the same in all of them. slot: 16 values of LDS.
template <int LANES, typename S>
__device__ __forceinline__ S row_sum(S v, S* slot) {
#pragma unroll
  for (int s = 1; s < (LANES < 64 ? LANES : 64); s *= 2) v += __shfl_xor(v, s, 64);
  if constexpr (LANES > 64) {
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int w = 0; w < LANES / 64; ++w) v += slot[w];
    __syncthreads();
  }
  return v;
}

// ---- the norm ---------------------------------------------------------------------------
// LANES threads a row, NV chunks a thread (chunk v of lane l: elements 8 (v LANES + l)).
template <typename T, int LANES, int NV, bool VEC, bool QUANT>
__global__ __launch_bounds__(LANES <= 64 ? 256 : LANES) void norm_kernel(NormParams p) {
  constexpr int kRows = LANES <= 64 ? 256 / LANES : 1;   // rows of a block
  __shared__ double slot[16];
  const int lane = threadIdx.x % LANES;
  const int C = p.cols;
  for (int64_t first = (int64_t)blockIdx.x * kRows; first < p.rows; first += (int64_t)gridDim.x * kRows) {
    const int64_t row = first + threadIdx.x / LANES;
    const bool live = row < p.rows;
    const T* x = (const T*)p.x + row * C;
    float h[NV][8];
    double sum = 0;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = 8 * (v * LANES + lane), n = live ? C - c : 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) h[v][i] = 0.0f;
      if (n > 0) {
        load8<VEC>(x + c, n, h[v]);
        if (p.residual) {
          float r[8];
          load8<VEC>((const T*)p.residual + row * C + c, n, r);
#pragma unroll
          for (int i = 0; i < 8; ++i) h[v][i] = Row8<T>::round(h[v][i] + r[i]);
          store8<VEC>((T*)p.h + row * C + c, n, h[v]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fma((double)h[v][i], (double)h[v][i], sum);
      }
    }
    sum = row_sum<LANES>(sum, slot);
    const float rstd = (float)(1.0 / sqrt(sum / C + (double)p.eps));
    if (live && lane == 0) p.rstd[row] = rstd;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = 8 * (v * LANES + lane), n = live ? C - c : 0;
      if (n <= 0) continue;
      float w[8], y[8];
      load_weight<VEC, T>(p.weight, p.weight_dtype == 0, c, n, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = Row8<T>::round(h[v][i] * rstd * w[i]);
      if (p.y) store8<VEC>((T*)p.y + row * C + c, n, y);
      if constexpr (QUANT) {   // (C % 32 == 0: the four lanes of a group are all here)
        const int64_t at = row * C + c;
        const int b = p.quant == 1 ? quantise8<0>(y, p.codes, at)
                      : p.quant == 2 ? quantise8<1>(y, p.codes, at) : quantise8<2>(y, p.codes, at);
        if ((lane & 3) == 0) {
          uint8_t* s = p.scales + row * p.scale_cols + (c >> 5);
          *s = (uint8_t)b;
          if (c + 32 == C && p.scale_cols > (C >> 5)) s[1] = 0;   // the pad of an odd number of groups
        }
      }
    }
  }
}

// ---- its gradient -----------------------------------------------------------------------
// Block b takes rows b kRows + i, + gridDim.x kRows, ...; the weight's gradient of these rows is
// summed in registers and goes to part[b][C].
template <typename T, int LANES, int NV, bool VEC>
__global__ __launch_bounds__(LANES <= 64 ? 256 : LANES) void norm_backward_kernel(NormGradParams p) {
  constexpr int kRows = LANES <= 64 ? 256 / LANES : 1;
  __shared__ float slot[16];
  __shared__ float parts[kRows > 1 ? kRows * 8 * LANES * NV : 1];
  const int lane = threadIdx.x % LANES, C = p.cols;
  float acc[NV][8] = {}, w[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = 8 * (v * LANES + lane);
    if (c < C) load_weight<VEC, T>(p.weight, p.weight_dtype == 0, c, C - c, w[v]);
  }
  for (int64_t first = (int64_t)blockIdx.x * kRows; first < p.rows; first += (int64_t)gridDim.x * kRows) {
    const int64_t row = first + threadIdx.x / LANES;
    const bool live = row < p.rows;
    const float rstd = live ? p.rstd[row] : 0.0f;
    float xh[NV][8], a[NV][8], dot = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = 8 * (v * LANES + lane), n = live ? C - c : 0;
      if (n <= 0) continue;
      load8<VEC>((const T*)p.h + row * C + c, n, xh[v]);
      load8<VEC>((const T*)p.grad_y + row * C + c, n, a[v]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (!VEC && i >= n) continue;
        xh[v][i] *= rstd;
        acc[v][i] = fmaf(a[v][i], xh[v][i], acc[v][i]);
        a[v][i] *= w[v][i];
        dot = fmaf(a[v][i], xh[v][i], dot);
      }
    }
    dot = row_sum<LANES>(dot, slot) / (float)C;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = 8 * (v * LANES + lane), n = live ? C - c : 0;
      if (n <= 0) continue;
      float g[8] = {};
      if (p.grad_h) load8<VEC>((const T*)p.grad_h + row * C + c, n, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] += rstd * (a[v][i] - xh[v][i] * dot);
      store8<VEC>((T*)p.grad_x + row * C + c, n, g);
    }
  }
  if constexpr (kRows > 1) {   // the block's rows side by side
    float* mine = parts + (threadIdx.x / LANES) * 8 * LANES * NV;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) mine[8 * (v * LANES + lane) + i] = acc[v][i];
    __syncthreads();
    for (int c = threadIdx.x; c < C; c += 256) {
      float s = 0.0f;
      for (int r = 0; r < kRows; ++r) s += parts[r * 8 * LANES * NV + c];
      p.part[(int64_t)blockIdx.x * C + c] = s;
    }
  } else {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = 8 * (v * LANES + lane);
      for (int i = 0; i < 8 && c + i < C; ++i) p.part[(int64_t)blockIdx.x * C + c + i] = acc[v][i];
    }
  }
}

// grad_w[c] = sum of part[b][c] over the blocks, in order: 64 columns a block, each by 16 threads
// that take every sixteenth part.
__global__ __launch_bounds__(1024) void norm_weight_kernel(const float* __restrict__ part, int parts, int cols,
                                                           float* __restrict__ grad_w) {
  __shared__ float s[16][64];
  const int c = blockIdx.x * 64 + (threadIdx.x & 63), g = threadIdx.x >> 6;
  float v = 0.0f;
  if (c < cols)
    for (int b = g; b < parts; b += 16) v += part[(int64_t)b * cols + c];
  s[g][threadIdx.x & 63] = v;
  __syncthreads();
  if (g == 0 && c < cols) {
    for (int i = 1; i < 16; ++i) v += s[i][threadIdx.x];
    grad_w[c] = v;
  }
}

bool aligned16(std::initializer_list<const void*> ps) {
  for (const void* q : ps)
    if (reinterpret_cast<uintptr_t>(q) % 16) return false;
  return true;
}

// Calls f with the number of lanes a row of `cols` elements gets and its chunks a lane: a lane a
// chunk up to 8192 columns, two chunks beyond.
template <typename F>
hipError_t with_lanes(int cols, F f) {
  const int chunks = (cols + 7) / 8;
  if (chunks <= 16) return f.template operator()<16, 1>();
  if (chunks <= 64) return f.template operator()<64, 1>();
  if (chunks <= 128) return f.template operator()<128, 1>();
  if (chunks <= 256) return f.template operator()<256, 1>();
  if (chunks <= 512) return f.template operator()<512, 1>();
  if (chunks <= 1024) return f.template operator()<1024, 1>();
  return f.template operator()<1024, 2>();
}

// Calls f with the rows' element type.
template <typename F>
hipError_t with_type(int dtype, F f) {
  switch (dtype) {
    case 0: return f.template operator()<float>();
    case 1: return f.template operator()<_Float16>();
    default: return f.template operator()<uint16_t>();
  }
}

template <typename T, bool VEC, bool QUANT>
hipError_t launch_norm_as(const NormParams& p, hipStream_t stream) {
  return with_lanes(p.cols, [&]<int LANES, int NV>() {
    constexpr int rows = LANES <= 64 ? 256 / LANES : 1, threads = LANES <= 64 ? 256 : LANES;
    // (a launch of 2^32 threads or more would be cut short: blocks go on with further rows)
    const int64_t grid = std::min<int64_t>((p.rows + rows - 1) / rows, 1 << 21);
    norm_kernel<T, LANES, NV, VEC, QUANT><<<(unsigned)grid, threads, 0, stream>>>(p);
    return hipGetLastError();
  });
}

}  // namespace

hipError_t launch_norm(const NormParams& p, hipStream_t stream) {
  const bool vec = p.cols % 8 == 0 && aligned16({p.x, p.residual, p.weight, p.y, p.h});
  return with_type(p.dtype, [&]<typename T>() {
    if (p.quant) return vec ? launch_norm_as<T, true, true>(p, stream) : launch_norm_as<T, false, true>(p, stream);
    return vec ? launch_norm_as<T, true, false>(p, stream) : launch_norm_as<T, false, false>(p, stream);
  });
}

// Blocks of the gradient's first pass (rows of parts of the weight's gradient): two a compute
// unit, and no more than there are rows.
int norm_parts(int64_t rows) { return (int)std::max<int64_t>(1, std::min<int64_t>(rows, 512)); }

hipError_t launch_norm_backward(const NormGradParams& p, hipStream_t stream) {
  const bool vec = p.cols % 8 == 0 && aligned16({p.grad_y, p.h, p.grad_h, p.weight, p.grad_x});
  hipError_t e = with_type(p.dtype, [&]<typename T>() {
    return with_lanes(p.cols, [&]<int LANES, int NV>() {
      constexpr int threads = LANES <= 64 ? 256 : LANES;
      if (vec)
        norm_backward_kernel<T, LANES, NV, true><<<p.parts, threads, 0, stream>>>(p);
      else
        norm_backward_kernel<T, LANES, NV, false><<<p.parts, threads, 0, stream>>>(p);
      return hipGetLastError();
    });
  });
  if (e != hipSuccess) return e;
  norm_weight_kernel<<<(p.cols + 63) / 64, 1024, 0, stream>>>(p.part, p.parts, p.cols, p.grad_w);
  return hipGetLastError();
}

}  // namespace moe
