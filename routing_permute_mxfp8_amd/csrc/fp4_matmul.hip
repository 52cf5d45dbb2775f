// MXFP4 x MXFP4 product of the rows of each expert group:
//   out[r, n] = sum_k DQ(x)[r, k] DQ(w_g)[n, k]   for the rows r of group g,
// both operands E2M1 codes two a byte (element 2j in the low nibble) with an E8M0 scale per
// 32 along K. MegaMoE README, "A4W4-FP quantization scenario" (GMM1's operands), and the
// rows that quantMode 9 of MoeInitRoutingV3 / moe_token_permute makes. x may come as bf16,
// fp16 or fp32 and is then quantised here (the Q_MX of moe_mx_quantize mode 9).
//
// The block-scaled MFMA multiplies FP4 operands exactly and adds in fp32 (measured: equal to
// the fp64 sum for scale spreads up to 2^3, 1e-7 of it at 2^10 over 56 steps).

#include <algorithm>

#include "device_common.h"
#include "fp4_device.h"
#include "internal.h"

namespace moe {
namespace {

// ---- few rows a group: weights streamed into registers -----------------------------------
// Bound by the weight stream (17/32 byte an element, each used for at most 16 rows at a
// time). A block takes 16 CT channels of a group; its four waves take every fourth pair of
// K steps (a pair is one 128-byte line of a weight row) and add their sums in LDS at the
// end, so that a dense layer of a few thousand channels still fills the chip. Loads behind
// the last K step or the group's rows fall outside their buffers: zeros, no traffic.
// Measured: one bf16 row, 7168 x 4096: 8.0 us (15.6 MB, 2 TB/s: the launch and the rounds of a
// wave's loop, which loads its four K steps, waits for them and multiplies with nothing in flight);
// x 16384 24.7 us (62 MB, 2.5 TB/s; packed weights 18.1). Beyond that the LDS-tiled kernel takes
// over.
struct RowsArgs {
  const void* x;            // codes [rows, K/2], or values [rows, K]
  const uint8_t* xs;        // codes: scales [rows, K/32]
  const int32_t* off;
  int rows, K, N;
  const uint8_t* w;
  const uint8_t* ws;
};

constexpr int kRowWaves = 4;
constexpr int kPairs = 2;   // pairs of K steps in flight a wave

template <typename T> constexpr int kXBytes = sizeof(T);
struct Codes {};            // x given as codes

// The x operand (16 rows) of one K step: lane (g, r) holds row r's K block g.
template <typename X>
struct XStep {
  u32x4 u[Group32<X>::kLoads];
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t xr, __amdgpu_buffer_rsrc_t, int lane_x, int, int step, bool in) {
    const int lo = in ? lane_x : kOutside, so = step * 128 * (int)sizeof(X);
#pragma unroll
    for (int i = 0; i < Group32<X>::kLoads; ++i) u[i] = __builtin_amdgcn_raw_buffer_load_b128(xr, lo + 16 * i, so, 0);
  }
  __device__ __forceinline__ void operand(int, u32x4& q, int& b) const { Group32<X>::run(u, q, b); }
};
template <>
struct XStep<Codes> {
  u32x4 u;
  uint32_t s;
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t xr, __amdgpu_buffer_rsrc_t sr, int lane_x, int lane_s, int step,
                                       bool in) {
    u = __builtin_amdgcn_raw_buffer_load_b128(xr, in ? lane_x : kOutside, step * 64, 0);
    s = __builtin_amdgcn_raw_buffer_load_b32(sr, in ? lane_s : kOutside, step * 4, 0);
  }
  __device__ __forceinline__ void operand(int g, u32x4& q, int& b) const {
    q = u;
    b = (int)(s >> (8 * g));
  }
};

template <int CT>
struct WStep {
  u32x4 u[CT];
  uint32_t s[CT];
};

__device__ __forceinline__ v4f mfma_fp4(const u32x4& a, const u32x4& b, v4f c, int sa, int sb) {
  return mfma_mx16_ab<kFmtFp4, kFmtFp4>(join_operand(a, u32x4{}), join_operand(b, u32x4{}), c, sa, sb);
}

template <typename X, typename O, int CT, bool PACKED>
__global__ __launch_bounds__(64 * kRowWaves) void fp4_rows_kernel(RowsArgs p, O* __restrict__ out) {
  __shared__ v4f part[kRowWaves][CT][64];
  const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = blockIdx.y, tile0 = blockIdx.x * CT, n16 = p.N >> 4;
  int lo, hi;
  group_rows(p.off, group, p.rows, &lo, &hi);
  if (lo >= hi) return;
  const int ks = p.K >> 7, pairs = (ks + 1) >> 1, kq = (ks + 3) >> 2;
  const int tiles = min(CT, n16 - tile0);
  // weights: this block's channel tiles
  const int64_t code_tile = (int64_t)16 * (p.K >> 1), scale_tile = PACKED ? (int64_t)kq * 256 : (int64_t)16 * (p.K >> 5);
  const int64_t t0 = (int64_t)group * n16 + tile0;
  const __amdgpu_buffer_rsrc_t wr = buffer_of(p.w + t0 * code_tile, tiles * code_tile);
  const __amdgpu_buffer_rsrc_t sr = buffer_of(p.ws + t0 * scale_tile, tiles * scale_tile);
  const int lane_w = PACKED ? 16 * lane : r * (p.K >> 1) + 16 * g;
  const int lane_s = PACKED ? 4 * lane : r * (p.K >> 5);
  auto load_w = [&](WStep<CT>& w, int step, bool in) {
    const int lw = in ? lane_w : kOutside, ls = in ? lane_s : kOutside;
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      w.u[c] = __builtin_amdgcn_raw_buffer_load_b128(wr, lw + c * (int)code_tile, step * (PACKED ? 1024 : 64), 2);   // non-temporal
      w.s[c] = __builtin_amdgcn_raw_buffer_load_b32(sr, ls + c * (int)scale_tile, PACKED ? (step >> 2) * 256 : step * 4, 0);
    }
  };
  constexpr bool kCodes = std::is_same_v<X, Codes>;
  const int64_t row_bytes = kCodes ? (int64_t)(p.K >> 1) : (int64_t)p.K * kXBytes<std::conditional_t<kCodes, uint8_t, X>>;
  for (int row0 = lo; row0 < hi; row0 += 16) {
    const int n = min(16, hi - row0);
    const __amdgpu_buffer_rsrc_t xr = buffer_of((const uint8_t*)p.x + row0 * row_bytes, n * row_bytes);
    const __amdgpu_buffer_rsrc_t xsr = buffer_of(kCodes ? p.xs + (int64_t)row0 * (p.K >> 5) : nullptr, kCodes ? n * (p.K >> 5) : 0);
    const int lane_x = r * (int)row_bytes + (kCodes ? 16 * g : 32 * g * kXBytes<std::conditional_t<kCodes, uint8_t, X>>);
    const int lane_xs = r * (p.K >> 5);
    v4f acc[CT] = {};
    for (int p0 = wave; p0 < pairs; p0 += kRowWaves * kPairs) {
      WStep<CT> w[2 * kPairs];
      XStep<X> x[2 * kPairs];
#pragma unroll
      for (int i = 0; i < 2 * kPairs; ++i) {
        const int step = 2 * (p0 + kRowWaves * (i >> 1)) + (i & 1);
        const bool in = step < ks;
        load_w(w[i], in ? step : 0, in);
        x[i].load(xr, xsr, lane_x, lane_xs, in ? step : 0, in);
      }
#pragma unroll
      for (int i = 0; i < 2 * kPairs; ++i) {
        const int step = 2 * (p0 + kRowWaves * (i >> 1)) + (i & 1);
        u32x4 q;
        int b;
        x[i].operand(g, q, b);
#pragma unroll
        for (int c = 0; c < CT; ++c)
          acc[c] = mfma_fp4(w[i].u[c], q, acc[c], (int)(w[i].s[c] >> (PACKED ? 8 * (step & 3) : 8 * g)), b);
      }
    }
#pragma unroll
    for (int c = 0; c < CT; ++c) part[wave][c][lane] = acc[c];
    __syncthreads();
    for (int c = wave; c < tiles; c += kRowWaves) {
      v4f t = part[0][c][lane];
#pragma unroll
      for (int q = 1; q < kRowWaves; ++q) t += part[q][c][lane];
      // lane (g, r): channels 4 g .. 4 g + 3 of row r
      if (r < n) store4(out + (int64_t)(row0 + r) * p.N + (tile0 + c) * 16 + 4 * g, t);
    }
    __syncthreads();
  }
}

template <typename X, typename O, bool PACKED>
hipError_t launch_rows(const Fp4MatmulParams& p, hipStream_t stream) {
  RowsArgs a{p.x, p.x_scales, p.off, (int)p.rows, p.k, p.n, p.w, p.w_scales};
  const int n16 = p.n / 16;
  // Four channel tiles a block where that leaves enough blocks, else one: x is read, and quantised,
  // once for the four (64 groups of 4 rows, 256 x 2048, bf16: 9.8 and 17.6 us, 128 x 2048, codes:
  // 7.1 and 10.0; but one bf16 row of 7168 x 4096, on 64 blocks
  // instead of 256: 19.0 and 9.6).
  const int64_t blocks4 = (int64_t)((n16 + 3) / 4) * std::min<int64_t>(p.groups, p.rows);
  if (blocks4 >= 1024) {
    fp4_rows_kernel<X, O, 4, PACKED><<<dim3((n16 + 3) / 4, p.groups), 64 * kRowWaves, 0, stream>>>(a, (O*)p.out);
  } else {
    fp4_rows_kernel<X, O, 1, PACKED><<<dim3(n16, p.groups), 64 * kRowWaves, 0, stream>>>(a, (O*)p.out);
  }
  return hipGetLastError();
}

template <typename X, typename O>
hipError_t launch_format(const Fp4MatmulParams& p, hipStream_t stream) {
  return p.packed ? launch_rows<X, O, true>(p, stream) : launch_rows<X, O, false>(p, stream);
}
template <typename X>
hipError_t launch_out(const Fp4MatmulParams& p, hipStream_t stream) {
  return p.out_fp32 ? launch_format<X, float>(p, stream) : launch_format<X, uint16_t>(p, stream);
}

}  // namespace

// Which kernel, and its tile: 0 for the kernel above, else the rows of the LDS-staged one's.
//
// The kernel above splits K over its waves, so it is done soonest where there is little to
// read, but streams at 3 TB/s at best and reads the weights again for every 16 rows; the other
// comes to 6, after about half a microsecond for each K step of 128 and three more. (8 groups,
// 2048 x 1024, 4 rows each: 5.9 and 12 us; 16 groups, 2048 x 2048: 13.4 and 13.8; 32: 24 and
// 18; 64 groups, 7168 x 4096: 293 and 156; one row, 7168 x 8192: 12.7 and 30, x 32768: 40 and
// 35.) Values are quantised by a launch of their own there, 3 us more.
//
// Tiles a little larger than the average group, because the sizes scatter (64 groups of 7168 x
// 4096, us with tiles of 32, 64, 128 and 256 rows: 16 rows each 172, 176, 206, 228; 24: 204, 188,
// 215, 236; 48: 376, 219, 223, 245; 96: 641, 318, 214, 234; 112: 700, 379, 251, 236; 320: 1864,
// 774, 539, 504), but smaller ones where the tiles would not occupy the chip (5 groups of 155
// rows, 1408 x 2000: 14.4, 10.6, 13.6, 17.6). Where a group is at most four fifths of a tile on
// average its weights are read about once, non-temporal (tiles of 64, 40 rows each: 201 us, 212
// cached; of 128, 96 rows: 214, 245; of 256, 160 rows: 253, 281; but of 128, 160 rows: 414, 399,
// and of 256, 256 rows of 2048 x 7168: 140, 136).
//
// Limits of the rule: it was fitted on dense calls and groups of about even sizes of 7168 x 4096,
// 2048 x 7168 and 1408 x 2000, and sees `rows`, not the offsets (these are on the device): where
// rows outside the groups or a few large groups make the average a poor guide, the tile is larger
// or smaller than it should be, and tiles of 32 are non-temporal also for a group that needs many.
// The kernel above takes 16 rows after one another on a block of 16 or 64 channels, which the
// bytes do not show: many rows by few channels are slow (32768 rows, 128 to 64: 1170 us; 1024,
// 8192 to 64: 522; 4096, 1024 to 128: 342).
int fp4_tile_rows(int64_t rows, int64_t groups, int64_t n, int64_t k, bool values) {
  if (rows <= 0) return 0;
  if (rows * (k / 32) < 16) return 0;   // (it reads x's scales 16 bytes at a time, also at their end)
  constexpr int64_t kStart = 9 << 20;   // bytes the kernel above reads in 3 us
  const int64_t per = (rows + groups - 1) / groups;
  const double bytes = (double)((per + 15) / 16) * (double)(std::min(groups, rows) * n) * (double)(k / 2);
  if (bytes < (double)(kStart * (values ? 2 : 1) + k * (kStart / 6 / 128))) return 0;
  if (per <= 20) return 32;
  int mt = per <= 48 ? 64 : per <= 100 ? 128 : 256;
  const auto items = [&](int m) { return groups * ((per + m - 1) / m) * ((n + 255) / 256); };
  while (mt > 64 && items(mt) < 256) mt /= 2;
  return mt;
}

hipError_t launch_fp4_matmul(const Fp4MatmulParams& p, hipStream_t stream) {
  if (p.rows <= 0) return hipSuccess;
  if (p.mt) return launch_fp4_tiles(p, stream);
  switch (p.x_kind) {
    case 0: return launch_out<float>(p, stream);
    case 1: return launch_out<_Float16>(p, stream);
    case 2: return launch_out<uint16_t>(p, stream);
    default: return launch_out<Codes>(p, stream);
  }
}

}  // namespace moe
