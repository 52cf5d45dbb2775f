// 16-bit (bf16 or fp16) product of the rows of expert groups, and its gradients:
//   out[r] = x[r] w_g^T           w_g [n, k]      (the forward product)
//   out[r] = x[r] w_g             w_g [k, n]      (grad_x = grad_out w_g of the former)
//   out_g  = a_g^T b_g            summed over the rows of g (grad_w_g = grad_out_g^T x_g)
// Products of 16-bit values are exact in fp32; they are added in fp32 by the MFMAs and rounded to
// the output's type once.
//
// Three kernels: gmm16_few.hip for forward products of few rows, whose operands go straight to
// registers; gmm16_tile.h for the rest, whose operands are staged in LDS; and the one of this file for
// operands that do not start at a multiple of 16 bytes (views into other tensors), of any strides.
// This file chooses among them and the tile, and copies rows of odd lengths to padded ones.
//
// The kernel of this file stages operands by elements, with the contraction innermost, as
// V_MFMA_F32_16X16X32 takes them: lane l holds elements 8 (l / 16) .. + 7 of row l % 16. A block of
// four waves makes a tile of 64 x 64 outputs, 32 x 32 a wave. It is bound by the staging's 2-byte
// loads (32768 rows on 16 groups of 4096 x 7168: 54 ms, where the staged tiles take 1.6).

#include <algorithm>
#include <cmath>

#include "device_common.h"
#include "fp4_device.h"
#include "gmm16_device.h"
#include "internal.h"

namespace moe {
namespace {

constexpr int kTile = 64, kStep = 32, kPitch = kStep + 8;   // (a pitch of 80 bytes: 16-byte reads of 16 rows meet no bank twice)

// Element (i, c) of an operand: base[i * major + c * con] for i < rows, c < length, else 0.
struct Operand {
  const uint16_t* base;
  int64_t major, con;
  int rows;
};

__device__ __forceinline__ void stage(const Operand& o, int c0, int length, uint16_t* lds) {
  const int t = threadIdx.x;
#pragma unroll
  for (int j = 0; j < kTile * kStep / 256; ++j) {
    const int e = t + 256 * j;
    // neighbouring threads along the dimension that is contiguous in memory
    const int i = o.con == 1 ? e / kStep : e % kTile, c = o.con == 1 ? e % kStep : e / kTile;
    uint16_t v = 0;
    if (i < o.rows && c0 + c < length) v = o.base[i * o.major + (c0 + c) * o.con];
    lds[i * kPitch + c] = v;
  }
}

// acc[i][j]: 16 x 16 blocks of the wave's 32 channels x 32 rows.
template <typename T>
__device__ __forceinline__ void multiply(const Operand& chan, const Operand& row, int length, uint16_t* lds,
                                         v4f (&acc)[2][2]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint16_t *lc = lds, *lr = lds + kTile * kPitch;
  for (int c0 = 0; c0 < length; c0 += kStep) {
    stage(chan, c0, length, lc);
    stage(row, c0, length, lr);
    __syncthreads();
    u32x4 a[2], b[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      a[i] = *reinterpret_cast<const u32x4*>(lc + ((wave & 1) * 32 + i * 16 + (lane & 15)) * kPitch + (lane >> 4) * 8);
      b[i] = *reinterpret_cast<const u32x4*>(lr + ((wave >> 1) * 32 + i * 16 + (lane & 15)) * kPitch + (lane >> 4) * 8);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = Mfma<T>::k32(a[i], b[j], acc[i][j]);
    __syncthreads();
  }
}

// Lane l holds channels 4 (l / 16) .. + 3 of row l % 16 of a block.
template <typename T, typename O>
__device__ __forceinline__ void store(const v4f (&acc)[2][2], O* out, int64_t pitch, int channels, int rows) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int ch = (wave & 1) * 32 + i * 16 + (lane >> 4) * 4, r = (wave >> 1) * 32 + j * 16 + (lane & 15);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (ch + e < channels && r < rows) out[r * pitch + ch + e] = Mfma<T>::template out<O>(acc[i][j][e]);
    }
}

template <typename T, typename O, bool WGRAD>
__global__ __launch_bounds__(256) void gmm16_any_kernel(Gmm16Params p) {
  __shared__ __align__(16) uint16_t lds[2 * kTile * kPitch];
  __shared__ int ends[kMaxGroups], scratch[4];
  const int ncol = ((WGRAD ? p.k : p.n) + kTile - 1) / kTile, nrow = (p.n + kTile - 1) / kTile;
  const int tiles = WGRAD ? p.groups * nrow : count_tiles<kTile, 4>(p.off, p.groups, (int)p.rows, ends, scratch);
  const int64_t total = (int64_t)tiles * ncol;
  for (int64_t it = blockIdx.x; it < total; it += gridDim.x) {
    const int tile = (int)(it / ncol), c0 = (int)(it % ncol) * kTile;
    v4f acc[2][2] = {};
    int lo, hi;
    if constexpr (WGRAD) {
      const int g = tile / nrow, r0 = (tile - g * nrow) * kTile;
      group_rows(p.off, g, (int)p.rows, &lo, &hi);
      const Operand chan{(const uint16_t*)p.b + (int64_t)lo * p.k + c0, 1, p.k, p.k - c0};
      const Operand row{(const uint16_t*)p.a + (int64_t)lo * p.n + r0, 1, p.n, p.n - r0};
      multiply<T>(chan, row, hi - lo, lds, acc);
      store<T>(acc, (O*)p.out + ((int64_t)g * p.n + r0) * p.k + c0, p.k, p.k - c0, p.n - r0);
    } else {
      const int g = group_of_tile(ends, p.groups, tile);
      group_rows(p.off, g, (int)p.rows, &lo, &hi);
      const int r0 = lo + (tile - (g > 0 ? ends[g - 1] : 0)) * kTile, rows = min(kTile, hi - r0);
      const uint16_t* w = (const uint16_t*)p.b + (int64_t)g * p.n * p.k;
      const Operand chan = p.trans ? Operand{w + c0, 1, p.n, p.n - c0} : Operand{w + (int64_t)c0 * p.k, p.k, 1, p.n - c0};
      const Operand row{(const uint16_t*)p.a + (int64_t)r0 * p.k, p.k, 1, rows};
      multiply<T>(chan, row, p.k, lds, acc);
      store<T>(acc, (O*)p.out + (int64_t)r0 * p.n + c0, p.n, p.n - c0, rows);
    }
  }
}

template <typename T, typename O>
hipError_t launch_any(const Gmm16Params& p, hipStream_t stream) {
  const int64_t nrow = (p.n + kTile - 1) / kTile;
  const int64_t items = p.wgrad ? p.groups * nrow * ((p.k + kTile - 1) / kTile)
                                : ((p.rows + kTile - 1) / kTile + std::min<int64_t>(p.groups, p.rows)) * nrow;
  const unsigned grid = (unsigned)std::min<int64_t>(items, 1 << 20);
  if (p.wgrad)
    gmm16_any_kernel<T, O, true><<<grid, 256, 0, stream>>>(p);
  else
    gmm16_any_kernel<T, O, false><<<grid, 256, 0, stream>>>(p);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_as(const Gmm16Params& p, hipStream_t stream) {
  return p.out_fp32 ? launch_any<T, float>(p, stream) : launch_any<T, uint16_t>(p, stream);
}

// Rows of a matrix of 16-bit elements copied to rows of `pitch` elements, a multiple of 8, with zeros
// behind: 8 elements of the copy a thread, read in one piece (at any element: load_chunk). A block
// has `lines` rows at a time, `lines` x `per` threads at work; one row's chunks past 256 in turns.
__global__ __launch_bounds__(256) void pad16_kernel(const uint16_t* __restrict__ from, int64_t rows, int cols,
                                                    uint16_t* __restrict__ to, int pitch, int lines) {
  const int per = pitch / 8, line = lines > 1 ? threadIdx.x / per : 0, first = threadIdx.x - line * per;
  if (line >= lines) return;
  for (int64_t r = (int64_t)blockIdx.x * lines + line; r < rows; r += (int64_t)gridDim.x * lines) {
    for (int c = first; c < per; c += 256)
      *reinterpret_cast<u32x4*>(to + r * pitch + 8 * c) = load_chunk<false>(from + r * cols + 8 * c, cols - 8 * c);
  }
}

hipError_t launch_pad16(const void* from, int64_t rows, int cols, uint16_t* to, int pitch, hipStream_t stream) {
  if (rows == 0) return hipSuccess;
  const int lines = std::max(1, 256 / (pitch / 8));
  const int64_t blocks = std::min<int64_t>((rows + lines - 1) / lines, 1 << 20);
  pad16_kernel<<<(unsigned)blocks, 256, 0, stream>>>((const uint16_t*)from, rows, cols, to, pitch, lines);
  return hipGetLastError();
}

// ---- which tile -----------------------------------------------------------------------------
// The LDS-staged kernel's tiles: mt rows by nt channels, `blocks` of them at a time on a compute
// unit. step: microseconds that these take for 64 contraction elements; item: for the rest of a
// tile (its output and the next one's start). step fits products of one group, 7168 deep, of 256 or
// 512 tiles (256: 214 us, 192: 176, 160: 150, 128: 134, 64: 126, 32: 105), item the slope of shorter
// ones.
struct Shape16 {
  int mt, nt, blocks;
  float step, item;
};
constexpr Shape16 kShapes[] = {{256, 256, 1, 1.80f, 4.0f}, {192, 256, 1, 1.45f, 3.0f}, {160, 256, 1, 1.23f, 2.5f},
                               {128, 256, 1, 1.08f, 2.0f}, {64, 128, 2, 1.00f, 1.5f},  {32, 128, 3, 1.10f, 1.0f}};

// Tiles of mt rows that a group of `mean` rows fills on average. The host does not know the groups'
// sizes (they are on the device): it takes them to scatter by the square root of the mean, as those of
// rows that choose their group at random do. One group has exactly `mean` rows.
double tiles_of(double mean, int mt, bool one) {
  if (one) return std::ceil(mean / mt);
  if (mean <= 0) return 0;
  if (mean > 256.0 * mt) return mean / mt + 0.5;   // (the sum's value to 1 in 1000)
  const double sd = std::sqrt(mean);
  const double sure = std::floor(std::max(0.0, mean - 6 * sd) / mt);   // tiles that all groups fill
  double sum = sure > 0 ? sure : 1.0 - std::exp(-mean);                // (groups with rows at all)
  for (double at = mt * std::max(1.0, sure); at < mean + 6 * sd; at += mt)
    sum += 0.5 * std::erfc((at + 0.5 - mean) / (std::sqrt(2.0) * sd));
  return sum;
}

// Items of a call with tiles of shape s, and steps of one, as expected.
struct Load16 {
  double items, steps;
};
Load16 load_of(const Gmm16Params& p, const Shape16& s) {
  const double mean = (double)p.rows / p.groups;
  const double columns = std::ceil((double)(p.wgrad ? p.k : p.n) / s.nt);
  const double rows = p.wgrad ? p.groups * std::ceil((double)p.n / s.mt) : p.groups * tiles_of(mean, s.mt, p.groups == 1);
  return {rows * columns, std::max(1.0, std::ceil((p.wgrad ? mean : (double)p.k) / 64))};
}

// Blocks that share an item of the last, part-filled round of `rem` items: 1 where that saves too little.
// An expectation: where there are many groups of unknown sizes it says little about the remainder, so
// that a call may get parts and a join for nothing (5 us: 8192 rows on 32 groups, 4096 to 7168, expect
// 1792.02 items) or none where some would have helped.
double parts_of(double rem, double steps, double units) {
  const double parts = rem > 0 ? std::min(std::floor(units / rem), std::floor(steps / 4)) : 1;
  return parts >= 2 && steps - std::ceil(steps / parts) >= kGain16 ? parts : 1;
}

// Microseconds of a call with tiles of shape s, but for the memory traffic, which they share.
double estimate(const Gmm16Params& p, const Shape16& s) {
  const auto [items, steps] = load_of(p, s);
  const double units = (double)kTile16Units * s.blocks;
  const double full = std::floor(items / units), rem = items - full * units, parts = parts_of(rem, steps, units);
  double t = full * (steps * s.step + s.item);
  if (parts >= 2)
    t += std::ceil(steps / parts) * s.step + s.item + 6 + rem * parts * s.mt * s.nt * 8 / 5e6;
  else if (rem > 0)
    t += steps * s.step * (rem <= kTile16Units ? 0.5 + 0.5 / s.blocks : 1.0) + s.item;   // (fewer blocks a unit)
  return t;
}

// The tile with the least estimate. Groups of about 256 rows, e.g., take two tiles of 160 rows rather
// than one and often a second of 256 (8192 rows on 32 groups of 4096 x 7168, forward and transposed:
// 570 and 583 us, with 192 rows 608 and 626, with 256 625 and 622, with 128 728 and 731). Limits:
// where rows outside the groups or a few large groups make the mean a poor guide, the tile is larger
// or smaller than it should be; and the model is that of long contractions: a 256 x 256 item of four
// steps of the gradient by weights takes 14.6 us and not its 11.2 (the estimates of a call's tiles are
// off alike).
int tile_rows(const Gmm16Params& p) {
  int best = 0;
  double least = 0;
  for (const Shape16& s : kShapes) {
    if (p.wgrad && s.mt != 256 && s.mt != 128 && s.mt != 64) continue;
    const double t = estimate(p, s);
    if (best == 0 || t < least) {
      best = s.mt;
      least = t;
    }
  }
  return best;
}

}  // namespace

void gmm16_plan(Gmm16Params& p) {
  p.few = gmm16_is_few(p);
  if (p.few) return;
  p.mt = tile_rows(p);
  const int64_t rows_b = p.wgrad ? p.rows : (int64_t)p.groups * (p.trans ? p.k : p.n);
  const int cols_a = p.wgrad ? p.n : p.k, cols_b = p.wgrad || !p.trans ? p.k : p.n;
  p.pitch_a = (cols_a + 7) / 8 * 8;
  p.pitch_b = (cols_b + 7) / 8 * 8;
  p.copy_a = p.pitch_a != cols_a ? (size_t)p.rows * p.pitch_a : 0;
  p.copy_b = p.pitch_b != cols_b ? (size_t)rows_b * p.pitch_b : 0;
  // Parts of shared items, where some are expected: the join is a launch, needed or not (24 steps, 64
  // to 365 items: 15 us shared and 23 not, 20 not shared and 23 with a join for nothing). A group
  // that is longer than the mean may want parts in the gradient by weights (launch_tile16 knows the
  // number of items there).
  for (const Shape16& s : kShapes) {
    if (s.mt != p.mt) continue;
    const double units = (double)kTile16Units * s.blocks;
    const auto [items, steps] = load_of(p, s);
    const bool share = p.wgrad ? (p.rows + 63) / 64 - 4 >= kGain16 : parts_of(items - std::floor(items / units) * units, steps, units) >= 2;
    p.part_floats = share ? (size_t)units * s.mt * s.nt : 0;
  }
}

hipError_t launch_gmm16(const Gmm16Params& p, hipStream_t stream) {
  if (p.rows <= 0 && !p.wgrad) return hipSuccess;
  if (p.few) return launch_gmm16_few(p, stream);
  const auto on16 = [](const void* q) { return reinterpret_cast<uintptr_t>(q) % 16 == 0; };
  if (!((p.copy_a || on16(p.a)) && (p.copy_b || on16(p.b)))) {
    if (!p.wgrad && !p.trans && p.rows <= 16) return launch_gmm16_few(p, stream);   // (at any element as well)
    return p.half ? launch_as<_Float16>(p, stream) : launch_as<__bf16>(p, stream);
  }
  Gmm16Params q = p;
  hipError_t e;
  if (p.copy_a) {
    if ((e = launch_pad16(p.a, p.rows, p.wgrad ? p.n : p.k, p.a16, p.pitch_a, stream)) != hipSuccess) return e;
    q.a = p.a16;
  }
  if (p.copy_b) {
    const int64_t rows = p.wgrad ? p.rows : (int64_t)p.groups * (p.trans ? p.k : p.n);
    if ((e = launch_pad16(p.b, rows, p.wgrad || !p.trans ? p.k : p.n, p.b16, p.pitch_b, stream)) != hipSuccess) return e;
    q.b = p.b16;
  }
  q.odd = !on16(p.out) || (p.wgrad ? p.k : p.n) % (p.out_fp32 ? 4 : 8) != 0;
  if (p.wgrad) return launch_gmm16_weights(q, stream);
  return p.trans ? launch_gmm16_transposed(q, stream) : launch_gmm16_forward(q, stream);
}

}  // namespace moe
