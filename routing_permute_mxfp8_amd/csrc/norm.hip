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
// Both passes are bound by memory: every input is read and every output written once, 530 MB for
// 8192 x 7168 bf16 rows with a residual and MXFP8 codes, 470 MB for their gradient. A thread holds 8
// neighbouring elements (16 bytes of a 16-bit type) of a row, or two such chunks past 8192 columns;
// an MX group of 32 is four lanes, whose largest magnitude takes two DPP steps. A row has 16 lanes,
// a wave, or a block with as many waves as it has chunks for; the blocks that fit on the card at
// once go over the rows, and load the next row before they sum one. Measured at that size, each
// call's outputs in memory of their own, the gradient with the sum of its weight's partial sums:
//   a block a row, no row loaded in advance                   104 us, its gradient 117 us
//   blocks that go over the rows, rows loaded in advance, row
//   sums by DPP and lane swaps (shuffles through LDS
//   addresses: 20 more registers)                             105                   92
//   and loads and stores of rows that pass the caches by    88-93 (5.7-6.0 TB/s)    86 (5.5 TB/s)
// (the loads alone: 104 and 90; the stores alone: 100 and 89; the codes' stores too, of 8 bytes a
// lane, which the caches put together: 96). Stores pass them by where the outputs are larger than
// the cache (see with_access), so not the gradient's at this size.

#include <algorithm>

#include "device_common.h"
#include "internal.h"

namespace moe {
namespace {

// ---- element types ----------------------------------------------------------------------
// 8 elements of a row as they are in memory, in dwords (as a vector of 16-bit elements the compiler
// keeps each in a register of its own across a branch). n of them exist: the others come as 0 and
// are not written.
template <typename T> using Raw8 = uint32_t __attribute__((ext_vector_type(2 * sizeof(T))));

// They at a multiple of 16 bytes, which is what with_access looks for: an fp32 Raw8 would promise 32.
template <typename T> struct Whole8 {
  typedef uint32_t type __attribute__((ext_vector_type(2 * sizeof(T)), aligned(16)));
  static_assert(alignof(type) == 16);
};

template <typename T> __device__ __forceinline__ float value(Raw8<T> r, int i) {
  if constexpr (sizeof(T) == 4) return __uint_as_float(r[i]);
  else if constexpr (__is_same(T, _Float16)) return (float)__builtin_bit_cast(_Float16, (uint16_t)(r[i / 2] >> (i % 2 * 16)));
  else return __uint_as_float(i % 2 ? r[i / 2] & 0xffff0000u : r[i / 2] << 16);
}

// To the rows' type, each to the nearest, ties to even.
template <typename T>
__device__ __forceinline__ Raw8<T> rounded(const float (&f)[8]) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < 2 * (int)sizeof(T); ++i) {
    if constexpr (sizeof(T) == 4) {
      r[i] = __float_as_uint(f[i]);
    } else if constexpr (__is_same(T, _Float16)) {
      typedef _Float16 h2 __attribute__((ext_vector_type(2)));
      // As fp32 first, for every use of the value: the compiler may turn a product and its
      // conversion into one instruction that rounds once, here and not there, so that the codes
      // would be those of another value than the one stored.
      float a = f[2 * i], b = f[2 * i + 1];
      asm("" : "+v"(a), "+v"(b));
      r[i] = __builtin_bit_cast(uint32_t, h2{(_Float16)a, (_Float16)b});
    } else {
      r[i] = bf16x2(f[2 * i], f[2 * i + 1]);
    }
  }
  return r;
}

// How rows are read and written. WHOLE: every chunk is whole and starts at a multiple of 16 bytes;
// rows are loaded past the caches. STREAM: stored past them, too. ANY: a whole chunk is one access
// at an address that is a multiple of an element only (the memory takes it; 32768 x 1001 fp16: by
// elements 161 us, so 53), a row's last elements go one by one.
enum Access { ANY, WHOLE, STREAM };

template <typename T> struct AnyRaw8 {
  Raw8<T> v;
} __attribute__((packed, aligned(sizeof(T))));

template <Access ACC, typename T>
__device__ __forceinline__ Raw8<T> load8(const T* p, int n) {
  Raw8<T> r = {};
  if constexpr (ACC != ANY) {
    if (n > 0) r = __builtin_nontemporal_load(reinterpret_cast<const typename Whole8<T>::type*>(p));
  } else if (n >= 8) {
    r = reinterpret_cast<const AnyRaw8<T>*>(p)->v;
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) r[i] = __float_as_uint(p[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) r[i / 2] |= (uint32_t)__builtin_bit_cast(uint16_t, p[i]) << (i % 2 * 16);
  }
  return r;
}

template <Access ACC, typename T>
__device__ __forceinline__ void store8(T* p, int n, Raw8<T> r) {
  if constexpr (ACC == STREAM) {
    __builtin_nontemporal_store(r, reinterpret_cast<typename Whole8<T>::type*>(p));
  } else if constexpr (ACC == WHOLE) {
    *reinterpret_cast<typename Whole8<T>::type*>(p) = r;
  } else if (n >= 8) {
    reinterpret_cast<AnyRaw8<T>*>(p)->v = r;
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = __uint_as_float(r[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = __builtin_bit_cast(T, (uint16_t)(r[i / 2] >> (i % 2 * 16)));
  }
}

// The weight's, which is of the rows' type or fp32, as floats.
template <Access ACC, typename T>
__device__ __forceinline__ void load_weight(const void* w, bool fp32, int c, int n, float (&f)[8]) {
  const auto load = [&]<typename W>(const W* p) {
    Raw8<W> r = {};
    if constexpr (ACC == ANY) r = load8<ANY>(p, n);
    else if (n > 0) r = *reinterpret_cast<const typename Whole8<W>::type*>(p);   // (every block's: through the caches)
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = value<W>(r, i);
  };
  if (fp32) load((const float*)w + c);
  else load((const T*)w + c);
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

constexpr int rows_of(int lanes) { return lanes ? 256 / lanes : 1; }

// v + the v of the lane that step STEP exchanges with this one.
template <int STEP, typename S>
__device__ __forceinline__ S add_step(S v) {
  constexpr int kWords = sizeof(S) / 4;
  typedef uint32_t words __attribute__((ext_vector_type(2)));
  words a, b;
  if constexpr (kWords == 2) a = __builtin_bit_cast(words, v); else a[0] = __builtin_bit_cast(uint32_t, v);
#pragma unroll
  for (int i = 0; i < kWords; ++i) {
    if constexpr (STEP < 16) {   // quad_perm [1,0,3,2], [2,3,0,1], then mirrored halves of 8, rows of 16
      constexpr int ctrl = STEP == 1 ? 0xB1 : STEP == 2 ? 0x4E : STEP == 4 ? 0x141 : 0x140;
      b[i] = __builtin_amdgcn_mov_dpp((int)a[i], ctrl, 0xF, 0xF, false);
    } else {   // each lane gets both halves' values: one in each of the two results
      const auto r = STEP == 16 ? __builtin_amdgcn_permlane16_swap(a[i], a[i], false, false)
                                : __builtin_amdgcn_permlane32_swap(a[i], a[i], false, false);
      a[i] = r[0];
      b[i] = r[1];
    }
  }
  if constexpr (kWords == 2) return __builtin_bit_cast(S, a) + __builtin_bit_cast(S, b);
  else return __builtin_bit_cast(S, (uint32_t)a[0]) + __builtin_bit_cast(S, (uint32_t)b[0]);
}

// Sum of v over a row's lanes, the same in all: LANES lanes of a block of 256 threads, or (LANES = 0)
// the whole block, whatever its size. slot: one of two sets of 16 values of LDS, used in turn by
// a block's rows (a wave that is behind may still read the last row's).
template <int LANES, typename S>
__device__ __forceinline__ S row_sum(S v, S* slot) {
  v = add_step<8>(add_step<4>(add_step<2>(add_step<1>(v))));
  if constexpr (LANES != 16) v = add_step<32>(add_step<16>(v));
  if constexpr (LANES == 0) {
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) v += slot[w];   // (0 past the block's waves)
  }
  return v;
}

// ---- the norm ---------------------------------------------------------------------------
// NV chunks a thread (chunk v of lane l: elements 8 (v lanes + l)); a block takes rows
// blockIdx.x kRows + i, + gridDim.x kRows, ... and loads the next while it sums one.
template <typename T, int LANES, int NV, Access ACC, bool QUANT>
__global__ __launch_bounds__(LANES ? 256 : 1024) void norm_kernel(NormParams p) {
  constexpr int kRows = rows_of(LANES);   // rows of a block
  __shared__ double slots[2][16];
  if constexpr (LANES == 0) {
    if (threadIdx.x < 32) slots[0][threadIdx.x] = 0;
    __syncthreads();
  }
  const int lanes = LANES ? LANES : blockDim.x, lane = LANES ? threadIdx.x % (LANES + !LANES) : threadIdx.x;
  const int C = p.cols;
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t row = (int64_t)blockIdx.x * kRows + (LANES ? threadIdx.x / (LANES + !LANES) : 0);
  const int64_t mine = row - (int64_t)blockIdx.x * kRows;
  Raw8<T> x[NV], r[NV];
  const auto load = [&](int64_t at) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = 8 * (v * lanes + lane), n = at < p.rows ? C - c : 0;
      x[v] = load8<ACC>((const T*)p.x + at * C + c, n);
      if (p.residual) r[v] = load8<ACC>((const T*)p.residual + at * C + c, n);
    }
  };
  load(row);
  float w[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = 8 * (v * lanes + lane);
    load_weight<ACC, T>(p.weight, p.weight_dtype == 0, c, C - c, w[v]);
  }
  for (int turn = 0; row - mine < p.rows; row += step, turn ^= 1) {
    const bool live = row < p.rows;
    float h[NV][8];
    double sum = 0;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = 8 * (v * lanes + lane), n = live ? C - c : 0;
      if (p.residual) {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[v][i] = value<T>(x[v], i) + value<T>(r[v], i);
        x[v] = rounded<T>(h[v]);
        if (n > 0) store8<ACC>((T*)p.h + row * C + c, n, x[v]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) h[v][i] = value<T>(x[v], i);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fma((double)h[v][i], (double)h[v][i], sum);
    }
    load(row + step);
    sum = row_sum<LANES>(sum, slots[turn]);
    const float rstd = (float)(1.0 / sqrt(sum / C + (double)p.eps));
    if (live && lane == 0) p.rstd[row] = rstd;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = 8 * (v * lanes + lane), n = live ? C - c : 0;
      if (n <= 0) continue;
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = h[v][i] * rstd * w[v][i];
      const Raw8<T> out = rounded<T>(y);
      if (p.y) store8<ACC>((T*)p.y + row * C + c, n, out);
      if constexpr (QUANT) {   // (C % 32 == 0: the four lanes of a group are all here)
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = value<T>(out, i);
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
// Rows to blocks and threads as above; the weight's gradient of a block's rows is summed in
// registers and goes to part[block][C].
template <typename T, int LANES, int NV, Access ACC>
__global__ __launch_bounds__(LANES ? 256 : 1024) void norm_backward_kernel(NormGradParams p) {
  constexpr bool kAhead = NV == 1;   // (two chunks a lane, of 1024 lanes: no registers left for a second row)
  constexpr int kRows = rows_of(LANES);
  __shared__ float slots[2][16];
  if constexpr (LANES == 0) {
    if (threadIdx.x < 32) slots[0][threadIdx.x] = 0;
    __syncthreads();
  }
  __shared__ float parts[kRows > 1 ? kRows * 8 * LANES * NV : 1];
  const int lanes = LANES ? LANES : blockDim.x, lane = LANES ? threadIdx.x % (LANES + !LANES) : threadIdx.x;
  const int C = p.cols;
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t row = (int64_t)blockIdx.x * kRows + (LANES ? threadIdx.x / (LANES + !LANES) : 0);
  const int64_t mine = row - (int64_t)blockIdx.x * kRows;
  struct Set { Raw8<T> h[NV], a[NV], g[NV]; float rstd; };
  const auto load = [&](Set& s, int64_t at) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = 8 * (v * lanes + lane), n = at < p.rows ? C - c : 0;
      s.h[v] = load8<ACC>((const T*)p.h + at * C + c, n);
      s.a[v] = load8<ACC>((const T*)p.grad_y + at * C + c, n);
      s.g[v] = load8<ACC>((const T*)p.grad_h + at * C + c, p.grad_h ? n : 0);
    }
    s.rstd = at < p.rows ? p.rstd[at] : 0.0f;
  };
  float acc[NV][8] = {}, w[NV][8];
  const auto take = [&](Set& s, int turn) {
    const bool live = row < p.rows;
    const float rs = s.rstd;
    float dot = 0.0f;
    Set k = s;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xh = value<T>(k.h[v], i) * rs, gy = value<T>(k.a[v], i);
        acc[v][i] = fmaf(gy, xh, acc[v][i]);
        dot = fmaf(gy * w[v][i], xh, dot);
      }
    }
    if (kAhead) load(s, row + step);
    // Over 2^10, exactly: the sum may be C times as large as what comes of it (gradients of 5e34 in
    // 7168 columns passed fp32's largest value). What falls below its smallest number is 2^-143 of
    // the mean at most. (Row sums in 64 bits as the norm's: 93 us for 89.)
    dot = row_sum<LANES>(dot * 0x1p-10f, slots[turn]) / ((float)C * 0x1p-10f);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = 8 * (v * lanes + lane), n = live ? C - c : 0;
      if (n <= 0) continue;
      float g[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        g[i] = value<T>(k.g[v], i) + rs * (value<T>(k.a[v], i) * w[v][i] - value<T>(k.h[v], i) * rs * dot);
      store8<ACC>((T*)p.grad_x + row * C + c, n, rounded<T>(g));
    }
    row += step;
  };
  Set set;
  if (kAhead) load(set, row);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = 8 * (v * lanes + lane);
    load_weight<ACC, T>(p.weight, p.weight_dtype == 0, c, C - c, w[v]);
  }
  for (int turn = 0; row - mine < p.rows; turn ^= 1) {
    if (!kAhead) load(set, row);
    take(set, turn);
  }
  if constexpr (kRows > 1) {   // the block's rows side by side
    float* own = parts + (threadIdx.x / LANES) * 8 * LANES * NV;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) own[8 * (v * LANES + lane) + i] = acc[v][i];
    __syncthreads();
    for (int c = threadIdx.x; c < C; c += 256) {
      float s = 0.0f;
      for (int r = 0; r < kRows; ++r) s += parts[r * 8 * LANES * NV + c];
      p.part[(int64_t)blockIdx.x * C + c] = s;
    }
  } else {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = 8 * (v * lanes + lane);
#pragma unroll
      for (int i = 0; i < 8; ++i)   // (an index known here: the sums stay in registers)
        if (c + i < C) p.part[(int64_t)blockIdx.x * C + c + i] = acc[v][i];
    }
  }
}

// grad_w[c] = sum of part[b][c] over the blocks, in order: 32 columns a block, each by 32 threads
// that take every 32nd part.
__global__ __launch_bounds__(1024) void norm_weight_kernel(const float* __restrict__ part, int parts, int cols,
                                                           float* __restrict__ grad_w) {
  __shared__ float s[32][33];
  const int i = threadIdx.x & 31, g = threadIdx.x >> 5, c = blockIdx.x * 32 + i;
  float v = 0.0f;
  if (c < cols)
#pragma unroll 8
    for (int b = g; b < parts; b += 32) v += part[(int64_t)b * cols + c];
  s[g][i] = v;
  __syncthreads();
  v = s[i][g];   // part i of column g
#pragma unroll
  for (int d = 1; d < 32; d *= 2) v += __shfl_xor(v, d, 64);
  if (i == 0 && blockIdx.x * 32 + g < cols) grad_w[blockIdx.x * 32 + g] = v;
}

bool aligned16(std::initializer_list<const void*> ps) {
  for (const void* q : ps)
    if (reinterpret_cast<uintptr_t>(q) % 16) return false;
  return true;
}

// A row's lanes (0: a block of its own, of `threads`), the threads of a block and its rows.
struct Shape {
  int lanes, threads, rows;
};
Shape shape_of(int64_t cols) {
  const int chunks = (int)((cols + 7) / 8);
  if (chunks <= 16) return {16, 256, 16};
  if (chunks <= 64) return {64, 256, 4};
  const int each = chunks <= 1024 ? 1 : 2;   // chunks a lane
  return {0, (chunks + 64 * each - 1) / (64 * each) * 64, 1};
}

// Blocks that take `rows` rows: as many as `lanes` lanes a compute unit make, and no more than there
// are rows for. The norm takes 2048 (1024: 100 us at the size above, a block a row: 101), its
// gradient, whose every block writes a row of partial sums, 1024 (2048: 92 us, 4096: 103).
int64_t blocks_of(Shape s, int64_t rows, int lanes) {
  return std::max<int64_t>(1, std::min<int64_t>((rows + s.rows - 1) / s.rows, 256 * std::max(1, lanes / s.threads)));
}

// Calls f with the lanes of a row of `cols` elements and the chunks of a lane.
template <typename F>
hipError_t with_lanes(int cols, F f) {
  const Shape s = shape_of(cols);
  if (s.lanes == 16) return f.template operator()<16, 1>(s);
  if (s.lanes == 64) return f.template operator()<64, 1>(s);
  if (cols <= 8192) return f.template operator()<0, 1>(s);
  return f.template operator()<0, 2>(s);
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

// Calls f with the access to rows of `cols` elements in tensors ps, of which `bytes` are written.
// Rows that stay in the 256 MB cache are read from there by the next kernel: norm and a sum of its
// outputs (2 x 29 MB): 36 us, stored past the cache 40; the gradient and a product of it (117 MB):
// 267 and 274. Past its size nothing stays: norm (2 x 117 MB) 88 and 81, the gradient (235 MB) and
// its negation 249 and 239.
template <typename F>
hipError_t with_access(int cols, std::initializer_list<const void*> ps, int64_t bytes, F f) {
  if (cols % 8 || !aligned16(ps)) return f.template operator()<ANY>();
  if (bytes <= (int64_t)192 << 20) return f.template operator()<WHOLE>();
  return f.template operator()<STREAM>();
}

template <typename T, Access ACC, bool QUANT>
hipError_t launch_norm_as(const NormParams& p, hipStream_t stream) {
  return with_lanes(p.cols, [&]<int LANES, int NV>(Shape s) {
    norm_kernel<T, LANES, NV, ACC, QUANT><<<(unsigned)blocks_of(s, p.rows, 2048), s.threads, 0, stream>>>(p);
    return hipGetLastError();
  });
}

}  // namespace

hipError_t launch_norm(const NormParams& p, hipStream_t stream) {
  return with_type(p.dtype, [&]<typename T>() {
    const int64_t bytes = p.rows * p.cols * (int64_t)sizeof(T) * ((p.y != nullptr) + (p.residual != nullptr));
    return with_access(p.cols, {p.x, p.residual, p.weight, p.y, p.h}, bytes, [&]<Access ACC>() {
      return p.quant ? launch_norm_as<T, ACC, true>(p, stream) : launch_norm_as<T, ACC, false>(p, stream);
    });
  });
}

// Blocks of the gradient's first pass, each a row of partial sums of the weight's gradient.
int norm_parts(int64_t rows, int64_t cols) { return (int)blocks_of(shape_of(cols), rows, 1024); }

hipError_t launch_norm_backward(const NormGradParams& p, hipStream_t stream) {
  hipError_t e = with_type(p.dtype, [&]<typename T>() {
    return with_access(p.cols, {p.grad_y, p.h, p.grad_h, p.weight, p.grad_x}, p.rows * p.cols * (int64_t)sizeof(T),
                       [&]<Access ACC>() {
      return with_lanes(p.cols, [&]<int LANES, int NV>(Shape s) {
        norm_backward_kernel<T, LANES, NV, ACC><<<p.parts, s.threads, 0, stream>>>(p);
        return hipGetLastError();
      });
    });
  });
  if (e != hipSuccess) return e;
  norm_weight_kernel<<<(p.cols + 31) / 32, 1024, 0, stream>>>(p.part, p.parts, p.cols, p.grad_w);
  return hipGetLastError();
}

}  // namespace moe
