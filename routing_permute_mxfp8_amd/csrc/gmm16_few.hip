// The 16-bit forward product of few rows (a decode step's): out[r] = x[r] w_g^T in one launch
// without a workspace.
//
// It is bound by the weights' way from memory, and small products by a launch and two trips there. A
// block makes the outputs of 8 channels for up to 32 rows of one group. Its 8 waves take the
// contraction's steps of 64 in equal runs, with several steps' loads in flight, straight from memory
// to the registers of V_MFMA_F32_16X16X32, and add their sums in LDS, always in the same order. Two
// neighbouring rows of an operand of the MFMA are the halves of a step of one channel (or of one
// row of x): a load takes 128 neighbouring bytes of each of 8 channels, and of the product's
// elements those of equal halves are added and the others left. One row, 256 channels, 7168 deep:
// 4.7 us of the card's time (16 channels a block, 64 bytes of each: 10.0; the LDS-staged tiles and
// their join: 12.7); 8 rows, 4096 channels: 10.7 us, 5.5 TB/s (16 waves a block: 11.5; tiles 21.7).
//
// Rows that are no 16-byte vectors are read in 16-byte pieces at addresses that are a multiple of
// an element only (1 row, 4001 channels, 4003 deep: 9.5 us; the tiles with a padded copy of the
// weights: 46).

#include <algorithm>

#include "device_common.h"
#include "fp4_device.h"
#include "gmm16_device.h"
#include "internal.h"

namespace moe {
namespace {

constexpr int kWaves = 8, kEach = 8, kStep = 64;   // waves, channels and rows of an operand, elements of a step
constexpr int kRows = 32;                          // rows of a block, at most

// The group that row r is in: the number of groups that end at or before it (all 64 lanes alike).
__device__ __forceinline__ int group_of_row(const int32_t* off, int groups, int r) {
  const int lane = threadIdx.x & 63;
  int n = 0;
  for (int g = 0; g < groups; g += 64) n += __popcll(__ballot(g + lane < groups && off[min(g + lane, groups - 1) + 1] <= r));
  return n;
}

// RB: blocks of 8 rows that a block of threads takes. VEC: every row is of whole 16-byte vectors.
template <typename T, typename O, int RB, bool VEC>
__global__ __launch_bounds__(64 * kWaves) void gmm16_few_kernel(Gmm16Params p) {
  constexpr int U = RB == 4 ? 4 : 8;   // steps loaded at a time
  __shared__ v4f sums[RB * kWaves * 64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = (lane & 15) >> 1, q = lane >> 4, at = 32 * (lane & 1) + 8 * q, n0 = blockIdx.x * kEach;
  // one group: block (c, 0, z) takes rows 8 RB z on; groups: block (c, r) those of the group whose
  // first row is r, if there is one
  int g = 0, lo = 0, hi = (int)p.rows;
  if (p.groups == 1) {
    if (p.off) group_rows(p.off, 0, (int)p.rows, &lo, &hi);
    lo += 8 * RB * blockIdx.z;
    hi = min(hi, lo + 8 * RB);
  } else {
    g = group_of_row(p.off, p.groups, blockIdx.y);
    if (g >= p.groups) return;
    group_rows(p.off, g, (int)p.rows, &lo, &hi);
    if (lo != (int)blockIdx.y) return;
  }
  if (lo >= hi) return;
  const uint16_t* w = (const uint16_t*)p.b + ((int64_t)g * p.n + min(n0 + r, p.n - 1)) * p.k + at;
  const uint16_t* x[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) x[b] = (const uint16_t*)p.a + (int64_t)min(lo + kEach * b + r, hi - 1) * p.k + at;
  const int steps = (p.k + kStep - 1) / kStep, end = steps * (wave + 1) / kWaves;
  v4f acc[RB] = {};
  for (int s = steps * wave / kWaves; s < end; s += U) {
    u32x4 a[U], c[U][RB];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k0 = kStep * (s + u), n = s + u < end ? p.k - k0 - at : 0;
      a[u] = load_chunk<VEC>(w + k0, n);
#pragma unroll
      for (int b = 0; b < RB; ++b) c[u][b] = load_chunk<VEC>(x[b] + k0, b == 0 || lo + kEach * b < hi ? n : 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int b = 0; b < RB; ++b) acc[b] = Mfma<T>::k32(a[u], c[u][b], acc[b]);
  }
#pragma unroll
  for (int b = 0; b < RB; ++b) sums[(b * kWaves + wave) * 64 + lane] = acc[b];
  __syncthreads();
  if (wave >= RB) return;
  v4f v = sums[wave * kWaves * 64 + lane];
#pragma unroll
  for (int i = 1; i < kWaves; ++i) v += sums[(wave * kWaves + i) * 64 + lane];
  // lane l holds elements 4 q .. + 3 of column l % 16: both halves of channels 2 q and 2 q + 1, by one
  // half of row r
  const int row = lo + kEach * wave + r;
  O* out = (O*)p.out + (int64_t)row * p.n + n0 + 2 * q;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    float sum = lane & 1 ? v[2 * c + 1] : v[2 * c];
    sum += __shfl_xor(sum, 1, 64);
    if (row < hi && !(lane & 1) && n0 + 2 * q + c < p.n) out[c] = Mfma<T>::template out<O>(sum);
  }
}

template <typename T, typename O, bool VEC>
hipError_t launch_as(const Gmm16Params& p, hipStream_t stream) {
  const unsigned strips = (p.n + kEach - 1) / kEach, rows = (unsigned)p.rows;
  const dim3 grid(strips, p.groups > 1 ? rows : 1, p.groups > 1 ? 1 : (rows + kRows - 1) / kRows);
  if (p.rows <= 8) gmm16_few_kernel<T, O, 1, VEC><<<grid, 64 * kWaves, 0, stream>>>(p);
  else if (p.rows <= 16) gmm16_few_kernel<T, O, 2, VEC><<<grid, 64 * kWaves, 0, stream>>>(p);
  else gmm16_few_kernel<T, O, 4, VEC><<<grid, 64 * kWaves, 0, stream>>>(p);
  return hipGetLastError();
}

template <typename T, typename O>
hipError_t launch(const Gmm16Params& p, hipStream_t stream) {
  const bool vec = p.k % 8 == 0 && (reinterpret_cast<uintptr_t>(p.a) | reinterpret_cast<uintptr_t>(p.b)) % 16 == 0;
  return vec ? launch_as<T, O, true>(p, stream) : launch_as<T, O, false>(p, stream);
}

}  // namespace

// The kernel of this file takes forward products whose blocks are few: a block takes 2 ns of the
// card's time (3.5 ns for more than 8 rows) even where it has little to read, and where it has much
// it reads the rows again for every 8 channels. Tiles and this kernel (us):
//   7168 deep, one group: 256 channels, 64 rows 14.7 and 10.8, 256 rows (256 blocks) 16.2 and 11.8,
//   512 (512 blocks) 24.1 and 19.4; 2048 channels, 64 rows (512) 22.9 and 19.6, 96 (768) 21.8 and
//   26.9; 8 groups of 4096, 16 rows 64 and 65, 32 rows 80 and 101;
//   8 rows, one group of 4096 channels (512 blocks), 64 deep 5.3 and 3.4; 32768 (4096), 64 deep 5.4 and
//   10.3, 288: 8.7 and 11.4, 1024: 19.9 and 13.7; 50 groups of 4400 (4400), 288 deep 11.5 and 13.3,
//   576: 15.7 and 15.9, 1024: 23.3 and 17.3;
//   16 rows on 50 groups of 512 (1024), 64 deep 5.8 and 5.7, 1024: 16.0 and 7.2; of 4400 (8800), 1024
//   deep 36 and 40, 2048: 71 and 52;
//   32 rows on 50 groups of 512 (2048), 288 deep 7.7 and 9.1, 576: 12.0 and 10.3; on 4 of 4400 (17600),
//   1024 deep 17.5 and 25.1.
// Rows of x that are no whole 16-byte vectors would have the tiles wait for a copy of the weights (32
// rows on 5 groups of 1000, 1001 deep: 27 and 12 us).
bool gmm16_is_few(const Gmm16Params& p) {
  if (p.wgrad || p.trans) return false;
  const int64_t strips = (p.n + kEach - 1) / kEach;
  const int64_t blocks = strips * (p.groups > 1 ? p.rows : (p.rows + kRows - 1) / kRows);
  if (p.k % 8 != 0 && p.rows <= kRows && std::min<int64_t>(p.rows, p.groups) * p.n * p.k <= 1 << 25) return true;
  if (p.rows <= 8) return blocks <= 1024 || p.k >= 512;
  if (p.rows <= 16) return blocks <= 1024 || p.k >= 2048;
  if (p.groups == 1) return blocks <= 512;
  return p.rows <= kRows && (blocks <= 1024 || (p.k >= 512 && blocks <= 2048));
}

hipError_t launch_gmm16_few(const Gmm16Params& p, hipStream_t stream) {
  if (p.half) return p.out_fp32 ? launch<_Float16, float>(p, stream) : launch<_Float16, uint16_t>(p, stream);
  return p.out_fp32 ? launch<__bf16, float>(p, stream) : launch<__bf16, uint16_t>(p, stream);
}

}  // namespace moe
