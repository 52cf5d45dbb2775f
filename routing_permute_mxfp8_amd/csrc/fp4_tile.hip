// MXFP4 x MXFP4 product of expert groups of many rows: both operands staged in LDS.
//
// A work item is a tile of MT rows of one group by NT output channels, computed by four
// waves (one per SIMD), each holding CB x RB accumulators of 32 channels x 32 rows
// (V_MFMA_SCALE_F32_32X32X64_F8F6F4, weights in the A slot: a lane holds 4 consecutive
// channels of one row). Blocks are persistent and XCD-aware.
//
// FP4 doubles the MFMA's rate against FP8 at the same operand rows, so the LDS reads are
// what a wave's tile shape decides: 128 x 128 a wave takes 64 of the 128 bytes a clock the
// CU's LDS delivers, 128 x 64 takes 96, 64 x 64 all of them. For many rows one wave a SIMD
// with 256 accumulator registers is therefore better than more, smaller waves. For few rows
// the weight stream is what takes the time, and two or three blocks a CU keep it going.
//
// The codes of NT weight rows and MT rows of x go straight from memory into LDS, two K steps
// of 128 at a time: 128 bytes a row, whole cache lines (64 experts of 4096 x 7168, 4 rows
// each, single steps: 199 us, pairs: 182). Two pairs are staged; the next one's loads begin as
// soon as all waves have read the one before it there, and operands are read from LDS half a
// step ahead of their MFMAs; one barrier for two steps, between the halves of the second. The
// loads go on across items, so an item's first steps are under way while the last ones of the
// item before are multiplied. The E8M0 scales of four steps (a quad) come through registers,
// 16 bytes a row.
//
// An LDS row of a pair holds eight 16-byte chunks (32 K elements each); chunk c of row r sits
// at place c ^ (r / 2 % 8), so that the sixteen lanes of a read pass (sixteen rows, one chunk)
// touch all 64 banks once (by r % 8 they met in pairs: half of the LDS's time). The
// direct-to-LDS loads write linearly; their lanes fetch the chunk that belongs at their place,
// wherever the weight format has it.
//
// Measured: 256 rows on 64 experts of 4096 x 7168 (1.0 GB of weights): 154 us, 6.4 TB/s of the
// 7.1 that a read reaches here. 32768 rows on 16 of them: 530 to 550 us, 3.5 to 3.6 PFLOP/s; these
// MFMAs alone reach 6.5 with random operands, with this kernel's LDS reads and loads dealt between
// them 5.4 to 5.9, at clocks that power holds at 1.6 to 1.9 GHz. That is nine rounds of some 2170
// items over 256 blocks, 94,000 to 112,000 cycles each: 57,000 of MFMAs (busy 42 to 45 % of all
// cycles by the counters), some 9,000 issuing an item's stores, when a compute unit's one block
// multiplies nothing. The rest is not accounted for stamp by stamp; known parts are the last round,
// half full, bursts of loads, and the first barrier of an item, which waits for every store of the
// item before (vmcnt counts stores too). 8192 rows on 32 of 7168 x 2048: 118 us; groups of about a
// tile leave half of the second tiles nearly empty, and its stores take a third.

#include <algorithm>
#include <map>
#include <mutex>

#include "device_common.h"
#include "fp4_device.h"
#include "internal.h"

namespace moe {
namespace {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void* lds_ptr;

// ---- x given as values: its codes and scales ----------------------------------------------
// One thread per group of 32 of the rows that belong to an expert group, [off[0], off[groups])
// (the others' are not read, and no tile uses their codes); row-major codes [rows, K/2] and
// scales [rows, K/32].
// Bound by the stream and, before it, the offsets' load: 8192 x 2048 bf16 (42 MB) in 10.3 us
// (8.7 for all rows without offsets; the call takes the same 132 us with either).
template <typename X>
__global__ __launch_bounds__(256) void fp4_quantise_kernel(const X* __restrict__ x, int64_t rows, int per_row,
                                                           const int32_t* __restrict__ off, int groups,
                                                           uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t first = off ? off[0] : 0, last = off ? min((int64_t)off[groups], rows) : rows;
  if (i < first * per_row || i >= last * per_row) return;
  constexpr int L = Group32<X>::kLoads;
  u32x4 u[L], c;
  const u32x4* src = reinterpret_cast<const u32x4*>(x + 32 * i);
#pragma unroll
  for (int j = 0; j < L; ++j) u[j] = src[j];
  int b;
  Group32<X>::run(u, c, b);
  reinterpret_cast<u32x4*>(codes)[i] = c;
  scales[i] = (uint8_t)b;
}

// ---- product --------------------------------------------------------------------------------
struct TileArgs {
  const uint8_t* x;         // codes [rows, K/2]
  const uint8_t* xs;        // scales [rows, K/32]
  const uint8_t* w;
  const uint8_t* ws;
  const int32_t* off;
  int groups, rows, K, N;
};

constexpr int kThreads = 256;
constexpr int kMaxGroups = 1024;
constexpr int kList = 64;   // items described at a time

// WC waves along the channels, 4 / WC along the rows; CB x RB 32 x 32 blocks a wave; BLOCKS
// blocks a CU.
template <int WC, int CB, int RB, int BLOCKS>
struct TileShape {
  static constexpr int kNT = 32 * WC * CB, kMT = 32 * (4 / WC) * RB;
  static constexpr int kA = kNT * 128, kB = kMT * 128;  // bytes of a pair of steps: weights, rows
  static constexpr int kPair = kA + kB;
  static constexpr int kSA = kNT * 16, kSB = kMT * 16;  // bytes of a quad's scales
  static constexpr int kQuad = kSA + kSB;
  // the area behind the two pairs: scales, tile ends of the groups, item list
  static constexpr int kScales = 0, kEnds = kScales + 2 * kQuad, kItems = kEnds + 4 * kMaxGroups;
  static constexpr int kLds = 2 * kPair + kItems + 16 * kList;
  static constexpr int kLA = kNT / 32, kLB = kMT / 32;   // direct-to-LDS loads a wave and pair (8 rows each)
  static_assert(kLds * BLOCKS <= 160 * 1024, "LDS of a compute unit");
  static_assert(kMT <= kThreads && kNT <= kThreads, "a thread loads a row's scales");
};

// Keeps the accumulators in accumulation registers across loop edges (left to itself the
// allocator moves most of them to vector registers and back around each quad, and spills).
template <int CB, int RB>
__device__ __forceinline__ void pin(v16f (&acc)[CB][RB]) {
#pragma unroll
  for (int i = 0; i < CB; ++i)
#pragma unroll
    for (int j = 0; j < RB; ++j) asm volatile("" : "+a"(acc[i][j]));
}

// Waits for the wave's loads and LDS accesses, then for the other waves: what was loaded or
// written is there for all, and what was read may be written again.
__device__ __forceinline__ void slot_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt((0 << 14) | (7 << 4) | (0 << 8));
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
  __builtin_amdgcn_sched_barrier(0);
}

// ends[g] = tiles of groups 0 .. g (all threads; ends has room for kMaxGroups). Returns the
// number of tiles.
template <int MT>
__device__ __forceinline__ int count_tiles(const TileArgs& p, int* ends, int* scratch) {
  const int t = threadIdx.x, lane = t & 63;
  int n[4], sum = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int g = 4 * t + i;
    int lo = 0, hi = 0;
    if (g < p.groups) group_rows(p.off, g, p.rows, &lo, &hi);
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
  for (int w = 0; w < kThreads / 64; ++w) {
    base += w < (t >> 6) ? scratch[w] : 0;
    total += scratch[w];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) ends[4 * t + i] = base + n[i];
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(total);
}

struct Item {
  int group, row0, rows, cb;
};

// Item `it` of the (tile, channel block) list: four tiles run through the channel blocks
// together, so that the items in flight on one XCD share weights as well as rows in its L2.
template <int MT>
__device__ __forceinline__ int4 describe(const TileArgs& p, const int* ends, int tiles, int ncb, int it) {
  const int block = it / (4 * ncb), in = it - block * 4 * ncb;
  const int width = min(4, tiles - 4 * block);
  const int cb = in / width, t = 4 * block + in - cb * width;
  int g = 0;   // the first group that ends behind tile t
  for (int s = kMaxGroups / 2; s > 0; s /= 2)
    if (g + s <= p.groups - 1 && ends[g + s - 1] <= t) g += s;
  int lo, hi;
  group_rows(p.off, g, p.rows, &lo, &hi);
  const int row0 = lo + (t - (g > 0 ? ends[g - 1] : 0)) * MT;
  return make_int4(g, row0, min(MT, hi - row0), cb);
}

// Lanes 16 - 31 and 48 - 63 of a change places with lanes 0 - 15 and 32 - 47 of b.
__device__ __forceinline__ void swap_rows(u32x4& a, u32x4& b) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const auto s = __builtin_amdgcn_permlane16_swap(a[c], b[c], false, false);
    a[c] = s[0];
    b[c] = s[1];
  }
}

// The body gets the two pairs of steps staged in LDS and the rest of it as three restrict
// pointers, which is what they are: apart. A pair is never read while loads into it are in
// flight (slot_barrier lies between), and so the compiler, which makes an LDS read wait for the
// direct-to-LDS loads that may write there, has nothing to wait for.
template <int WC, int CB, int RB, int BLOCKS, bool ONCE, typename O, bool PACKED>
__device__ __forceinline__ void tile_body(const TileArgs& p, O* __restrict__ out, uint8_t* __restrict__ pair0,
                                          uint8_t* __restrict__ pair1, uint8_t* __restrict__ lds) {
  using S = TileShape<WC, CB, RB, BLOCKS>;
  constexpr int MT = S::kMT, kNT = S::kNT;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wc = wave % WC, wr = wave / WC;
  const int ks = p.K >> 7, kq = (ks + 3) >> 2, half = p.K >> 1, n16 = p.N >> 4;
  const int ncb = (p.N + kNT - 1) / kNT;
  int* const ends = reinterpret_cast<int*>(lds + S::kEnds);
  int4* const list = reinterpret_cast<int4*>(lds + S::kItems);

  const int tiles = count_tiles<MT>(p, ends, reinterpret_cast<int*>(list));
  // each XCD takes a contiguous share of the items, dealt to its blocks in turn
  const int64_t total = (int64_t)tiles * ncb;
  const int xcd = blockIdx.x & 7, per = gridDim.x >> 3;
  const int64_t begin = total * xcd / 8 + (blockIdx.x >> 3), end = total * (xcd + 1) / 8;
  if (begin >= end) return;   // the whole block
  const int count = (int)((end - begin + per - 1) / per);
  auto fill = [&](int first) {   // list[i] = this block's item first + i
    __syncthreads();
    if (tid < kList && first + tid < count) list[tid] = describe<MT>(p, ends, tiles, ncb, (int)(begin + (int64_t)(first + tid) * per));
    __syncthreads();
  };
  auto item = [&](int i) {
    const int4 v = list[i % kList];
    return Item{__builtin_amdgcn_readfirstlane(v.x), __builtin_amdgcn_readfirstlane(v.y),
                __builtin_amdgcn_readfirstlane(v.z), __builtin_amdgcn_readfirstlane(v.w)};
  };

  // code loads: load i of a wave fills 8 rows, lane l place l % 8 of row l / 8
  const auto chunk_of = [&](int row) { return (lane & 7) ^ ((row >> 1) & 7); };
  int va[S::kLA], vb[S::kLB];
#pragma unroll
  for (int i = 0; i < S::kLA; ++i) {
    const int row = (wave * S::kLA + i) * 8 + (lane >> 3), c = chunk_of(row);
    va[i] = PACKED ? (row >> 4) * 16 * half + (c >> 2) * 1024 + (c & 3) * 256 + (row & 15) * 16 : row * half + c * 16;
  }
#pragma unroll
  for (int i = 0; i < S::kLB; ++i) {
    const int row = (wave * S::kLB + i) * 8 + (lane >> 3);
    vb[i] = row * half + chunk_of(row) * 16;
  }

  // The item whose codes are being loaded: buffers of exactly its rows (what lies behind
  // reads as zeros, without memory traffic).
  const uint8_t *bw, *bx;
  int wbytes, xbytes;
  auto aim_codes = [&](const Item& it) {
    const int c16 = min(kNT / 16, n16 - it.cb * (kNT / 16));
    bw = p.w + ((int64_t)it.group * n16 + it.cb * (kNT / 16)) * 16 * half;
    wbytes = c16 * 16 * half;
    bx = p.x + (int64_t)it.row0 * half;
    xbytes = it.rows * half;
  };
  // The item whose scales are being loaded; a row past its end repeats its last row.
  const uint8_t *bws, *bxs;
  uint32_t vsa, vsb;
  auto aim_scales = [&](const Item& it) {
    const int c16 = min(kNT / 16, n16 - it.cb * (kNT / 16));
    bws = p.ws + ((int64_t)it.group * n16 + it.cb * (kNT / 16)) * (PACKED ? kq * 256 : 64 * ks);
    bxs = p.xs + (int64_t)it.row0 * (4 * ks);
    const int ra = min(tid, c16 * 16 - 1), rb = min(tid, it.rows - 1);
    vsa = PACKED ? (uint32_t)((ra >> 4) * kq * 256 + (ra & 15) * 4) : (uint32_t)(ra * 4 * ks);
    vsb = (uint32_t)(rb * 4 * ks);
  };
  // Steps `step` and step + 1 (step even) into pair slot `slot`; !in: zeros. Of an odd number
  // of steps the last pair's second half is whatever follows in the item's buffer, or zeros
  // behind it; its scales are made to vanish (store_scales). The step is part of the lane's
  // offset, not of the scalar one, because only that is checked against the buffer's size.
  // ONCE: a weight is used by about one item, so weights are loaded non-temporal.
  constexpr int kCodes = S::kLA + S::kLB;   // loads of a pair
  auto issue = [&](int slot, int step, bool in, int i) {   // load i of the pair (slot: a constant)
    uint8_t* base = slot ? pair1 : pair0;
    const int s = in ? step : 0;
    if (i < S::kLA)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer_of(bw, in ? wbytes : 0),
                                               (lds_ptr)(base + (wave * S::kLA + i) * 1024), 16,
                                               va[i] + s * (PACKED ? 1024 : 64), 0, 0, ONCE ? 2 : 0);
    else
      __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer_of(bx, in ? xbytes : 0),
                                               (lds_ptr)(base + S::kA + (wave * S::kLB + i - S::kLA) * 1024), 16,
                                               vb[i - S::kLA] + s * 64, 0, 0, 0);
  };
  auto issue_pair = [&](int slot, int step, bool in) {
#pragma unroll
    for (int i = 0; i < kCodes; ++i) issue(slot, step, in, i);
  };
  // The scales of a quad: thread t holds row t's 16 bytes, dword j the four blocks of step j
  // (the packed weight scales come as dword g = block g of the four steps and are transposed).
  // The last quad's 16 bytes may reach past the row's end, and of the last rows past the
  // buffer's: those lanes read up to 12 bytes before their place and shift.
  u32x4 qa, qx;
  int early_a = 0, early_x = 0;   // bytes before the place
  const int64_t ws_bytes = (int64_t)p.groups * p.N * 4 * ks, xs_bytes = (int64_t)p.rows * 4 * ks;
  typedef u32x4 __attribute__((aligned(4))) u32x4_a4;
  auto load_scales = [&](int q) {
    if constexpr (PACKED) {
      const uint8_t* s = bws + q * 256;
#pragma unroll
      for (int g = 0; g < 4; ++g) qa[g] = *reinterpret_cast<const uint32_t*>(s + (vsa + 64 * g));
    } else {
      const int room = (int)min((int64_t)INT32_MAX, p.ws + ws_bytes - 16 - bws);   // a read may start here at the latest
      const int at = (int)vsa + 16 * q;
      early_a = max(at - room, 0);
      qa = *reinterpret_cast<const u32x4_a4*>(bws + (uint32_t)(at - early_a));
    }
    const int room = (int)min((int64_t)INT32_MAX, p.xs + xs_bytes - 16 - bxs);
    // (may be negative: the item's first row can lie within the last 16 bytes)
    const int at = (int)vsb + 16 * q;
    early_x = max(at - room, 0);
    qx = *reinterpret_cast<const u32x4_a4*>(bxs + (int64_t)(at - early_x));
  };
  // dwords shifted down by `early` bytes (0, 4, 8, 12), zeros behind
  auto shift_down = [](u32x4 v, int early) {
    const bool one = early & 4, two = early & 8;
    v = u32x4{one ? v[1] : v[0], one ? v[2] : v[1], one ? v[3] : v[2], one ? 0u : v[3]};
    return u32x4{two ? v[2] : v[0], two ? v[3] : v[1], two ? 0u : v[2], two ? 0u : v[3]};
  };
  auto store_scales = [&](int area, int q) {
    u32x4 a, x = shift_down(qx, early_x);
    if constexpr (PACKED) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        a[j] = ((qa[0] >> (8 * j)) & 0xff) | (((qa[1] >> (8 * j)) & 0xff) << 8) | (((qa[2] >> (8 * j)) & 0xff) << 16) |
               ((qa[3] >> (8 * j)) << 24);
    } else {
      a = shift_down(qa, early_a);
    }
    // a step past the last: 2^-127 on both sides, whose products vanish in fp32
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      a[j] = 4 * q + j < ks ? a[j] : 0;
      x[j] = 4 * q + j < ks ? x[j] : 0;
    }
    uint32_t* base = reinterpret_cast<uint32_t*>(lds + S::kScales + area * S::kQuad) + tid;
#pragma unroll
    for (int j = 0; j < 4; ++j) {   // [step][row]
      if (kNT == kThreads || tid < kNT) base[j * kNT] = a[j];
      if (MT == kThreads || tid < MT) base[4 * kNT + j * MT] = x[j];
    }
  };

  // operand reads of a wave: sub-step s of a step (64 elements), lane (h, r) = row r, chunk 2 s + h
  const int h = lane >> 5;
  const int read0 = (lane & 31) * 128 + ((h ^ ((lane >> 1) & 7)) * 16);
  u32x4 a[2][CB], bx_[2][RB];
  uint32_t read_s[CB + RB], sc[CB + RB];
  auto read_step = [&](int j, int s, int i) {   // operand i of sub-step s of step j (a constant)
    const uint8_t* base = (j >> 1 ? pair1 : pair0) + (read0 ^ (32 * s) ^ (64 * (j & 1)));
    if (i < CB)
      a[s][i] = *reinterpret_cast<const u32x4*>(base + (wc * CB + i) * 4096);
    else
      bx_[s][i - CB] = *reinterpret_cast<const u32x4*>(base + S::kA + (wr * RB + i - CB) * 4096);
  };
  // the lane's rows' scales of step j of the quad; shifted before their use so that block h of
  // the step is byte 0 and block 2 + h byte 2 (the MFMA selects a byte)
  auto read_scale = [&](int area, int j, int i) {
    const uint32_t* base = reinterpret_cast<const uint32_t*>(lds + S::kScales + area * S::kQuad) + (lane & 31);
    read_s[i] = base[i < CB ? j * kNT + (wc * CB + i) * 32 : 4 * kNT + j * MT + (wr * RB + i - CB) * 32];
  };
  auto take_scales = [&]() {
#pragma unroll
    for (int i = 0; i < CB + RB; ++i) sc[i] = read_s[i] >> (8 * h);
  };
  // Sub-step SUB of step J; behind MFMA m `between(m)`, in the order written (left to itself the
  // compiler moves the LDS reads to just before their use and the loads into one clump).
  v16f acc[CB][RB];
  constexpr int M = CB * RB;
  auto multiply = [&]<int SUB>(std::integral_constant<int, SUB>, auto between) {
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const int i = m % CB, j = m / CB;
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
          join_operand(a[SUB][i], u32x4{}), join_operand(bx_[SUB][j], u32x4{}), acc[i][j], kFmtFp4, kFmtFp4, 2 * SUB,
          (int)sc[i], 2 * SUB, (int)sc[CB + j]);
      between(m);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // part m of things lo .. hi - 1 dealt over the M places
  auto dealt = [](int m, int lo, int hi, auto f) {
    const int per = (hi - lo + M - 1) / M;
#pragma unroll
    for (int i = lo + m * per; i < lo + (m + 1) * per; ++i)
      if (i < hi) f(i);
  };
  constexpr std::integral_constant<int, 0> k0{};
  constexpr std::integral_constant<int, 1> k1{};
  constexpr std::integral_constant<int, 2> k2{};
  constexpr std::integral_constant<int, 3> k3{};

  fill(0);
  Item cur = item(0);
  aim_codes(cur);
  aim_scales(cur);
  load_scales(0);
  issue_pair(0, 0, true);
  issue_pair(1, 2, 2 < ks);
  store_scales(0, 0);
  slot_barrier();
  for (int i = 0; i < CB + RB; ++i) read_scale(0, 0, i);
  for (int i = 0; i < CB + RB; ++i) read_step(0, 0, i);

  int area = 0;
  // Steps 4 q .. 4 q + 3 of the current item, and the loads of quad nq: the next one, or the
  // first of item `next` (last; none when !more). Its scales are loaded at the start, its first
  // pair from step 1 on and its second from step 3 on, when all waves have read the ones before
  // them there. A pair has landed where the next one's loads begin, so there is nothing newer to
  // wait past; that is also where the scales are taken from their registers (the compiler makes
  // that wait for every direct-to-LDS load in flight).
  // Many MFMAs a step: a burst of a pair's loads meets the L2's rate and stalls the waves (about
  // 1000 cycles), so half of them go on in the next half step; of the second pair that is the
  // next quad's first (pending), but for an item's last quad.
  constexpr int kFirst = M >= 8 ? kCodes / 2 : kCodes;
  auto quad = [&](int q, bool last, bool more, const Item& next) {
    const int nq = last ? 0 : q + 1;
    const bool pending = q > 0;
    if constexpr (kFirst == kCodes) load_scales(nq);
    const auto reads = [&](int j, int m) { dealt(m, 0, CB + RB, [&](int i) { read_step(j, 1, i); }); };
    auto step = [&]<int J>(std::integral_constant<int, J>) {
      take_scales();
      if (J == 0 && kFirst < kCodes && pending)
        multiply(k0, [&](int m) {
          reads(J, m);
          dealt(m, kFirst, kCodes, [&](int i) { issue(1, 4 * q + 2, 4 * q + 2 < ks, i); });
        });
      else
        multiply(k0, [&](int m) {
          reads(J, m);
          if constexpr (J == 2)
            dealt(m, kFirst, kCodes, [&](int i) { issue(0, 4 * nq, more, i); });
        });
      if constexpr (J == 0)
        if (last) aim_codes(next);
      if constexpr (J == 0 && kFirst < kCodes) load_scales(nq);
      if constexpr (J == 1 || J == 3) slot_barrier();
      multiply(k1, [&](int m) {
        if (J == 1 && m == M / 2) store_scales(area ^ 1, nq);
        dealt(m, 0, CB + RB, [&](int i) { read_step((J + 1) & 3, 0, i); });
        dealt(m, 0, CB + RB, [&](int i) { read_scale(J == 3 ? area ^ 1 : area, (J + 1) & 3, i); });
        if constexpr (J == 1) dealt(m, 0, kFirst, [&](int i) { issue(0, 4 * nq, more, i); });
        if constexpr (J == 3) dealt(m, 0, kFirst, [&](int i) { issue(1, 4 * nq + 2, more && 4 * nq + 2 < ks, i); });
      });
      if constexpr (J == 3 && kFirst < kCodes)
        if (last)
#pragma unroll
          for (int i = kFirst; i < kCodes; ++i) issue(1, 4 * nq + 2, more && 4 * nq + 2 < ks, i);
    };
    step(k0);
    step(k1);
    step(k2);
    step(k3);
    area ^= 1;
    pin(acc);
  };
  for (int n = 0;;) {
#pragma unroll
    for (int i = 0; i < CB; ++i)
#pragma unroll
      for (int j = 0; j < RB; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
    pin(acc);
    for (int q = 0; q < kq - 1; ++q) quad(q, false, true, cur);
    // the item's last quad: the next item's first is loaded behind it
    const bool more = n + 1 < count;
    if (more && (n + 1) % kList == 0) fill(n + 1);
    const Item next = more ? item(n + 1) : cur;
    aim_scales(next);
    quad(kq - 1, true, more, next);
    // Lane (h, r) holds row r, channels 8 e + 4 h + 0..3 of a block: pieces of 8 (bf16) or 16
    // bytes, each a write request of its own to the L2 (8192 a 256 x 256 tile: 18,000 cycles).
    // Lane halves and quarters change places until a row's 64 bytes are next to one another, in
    // lanes l, l + 16, l + 32, l + 48.
#pragma unroll
    for (int j = 0; j < RB; ++j) {
#pragma unroll
      for (int i = 0; i < CB; ++i) {
        const int row = (wr * RB + j) * 32 + (lane & 15), ch = cur.cb * kNT + (wc * CB + i) * 32;
        if constexpr (sizeof(O) == 2) {
          u32x4 v[2];   // lane (h, r): channels 16 e + 8 h + 0..7
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const auto at = [&](int c) { return bf16x2(acc[i][j][8 * e + c], acc[i][j][8 * e + c + 1]); };
            const auto s0 = __builtin_amdgcn_permlane32_swap(at(0), at(4), false, false);
            const auto s1 = __builtin_amdgcn_permlane32_swap(at(2), at(6), false, false);
            v[e] = u32x4{s0[0], s1[0], s0[1], s1[1]};
          }
          swap_rows(v[0], v[1]);
          const int c = ch + 16 * ((lane >> 4) & 1) + 8 * h;
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (row + 16 * e < cur.rows && c < p.N)
              *reinterpret_cast<u32x4*>(out + (int64_t)(cur.row0 + row + 16 * e) * p.N + c) = v[e];
        } else {
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            u32x4 v[2];
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int c = 0; c < 4; ++c) v[e][c] = __float_as_uint(acc[i][j][8 * g + 4 * e + c]);
            swap_rows(v[0], v[1]);
            const int c = ch + 16 * g + 8 * ((lane >> 4) & 1) + 4 * h;
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (row + 16 * e < cur.rows && c < p.N)
                *reinterpret_cast<u32x4*>(out + (int64_t)(cur.row0 + row + 16 * e) * p.N + c) = v[e];
          }
        }
      }
    }
    if (++n >= count) break;
    cur = next;
  }
  __builtin_amdgcn_s_waitcnt((0 << 14) | (7 << 4) | (15 << 8));   // no direct-to-LDS load outlives the block
}

template <int WC, int CB, int RB, int BLOCKS, bool ONCE, typename O, bool PACKED>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(BLOCKS))) void fp4_tile_kernel(
    TileArgs p, O* __restrict__ out) {
  extern __shared__ __align__(16) uint8_t lds_area[];
  constexpr int kPair = TileShape<WC, CB, RB, BLOCKS>::kPair;
  tile_body<WC, CB, RB, BLOCKS, ONCE, O, PACKED>(p, out, lds_area, lds_area + kPair, lds_area + 2 * kPair);
}

// The device's compute units, rounded up to whole XCDs' shares; the kernel's LDS size set
// once for each device.
hipError_t tile_grid(const void* kernel, int lds, int* grid) {
  static std::mutex mu;
  static std::map<std::pair<int, const void*>, int> known;
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  auto at = known.find({dev, kernel});
  if (at == known.end()) {
    int cus = 0;
    if ((e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, lds)) != hipSuccess) return e;
    if ((e = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev)) != hipSuccess) return e;
    at = known.emplace(std::make_pair(dev, kernel), (cus + 7) / 8 * 8).first;
  }
  *grid = at->second;
  return hipSuccess;
}

template <int WC, int CB, int RB, int BLOCKS, bool ONCE, typename O, bool PACKED>
hipError_t launch_tiles(const TileArgs& a, void* out, hipStream_t stream) {
  using S = TileShape<WC, CB, RB, BLOCKS>;
  int grid = 0;
  const auto kernel = fp4_tile_kernel<WC, CB, RB, BLOCKS, ONCE, O, PACKED>;
  hipError_t e = tile_grid(reinterpret_cast<const void*>(kernel), S::kLds, &grid);
  if (e != hipSuccess) return e;
  kernel<<<grid * BLOCKS, kThreads, S::kLds, stream>>>(a, (O*)out);
  return hipGetLastError();
}

template <typename O, bool PACKED>
hipError_t launch_shape(const Fp4MatmulParams& p, const TileArgs& a, hipStream_t stream) {
  // weights of groups that mostly fit into one tile are read about once: see fp4_tile_rows
  const bool once = 5 * p.rows <= (int64_t)4 * p.mt * p.groups;
  switch (p.mt) {
    case 256: return once ? launch_tiles<2, 4, 4, 1, true, O, PACKED>(a, p.out, stream)
                          : launch_tiles<2, 4, 4, 1, false, O, PACKED>(a, p.out, stream);
    case 128: return once ? launch_tiles<2, 4, 2, 1, true, O, PACKED>(a, p.out, stream)
                          : launch_tiles<2, 4, 2, 1, false, O, PACKED>(a, p.out, stream);
    case 64: return once ? launch_tiles<4, 1, 2, 2, true, O, PACKED>(a, p.out, stream)
                         : launch_tiles<4, 1, 2, 2, false, O, PACKED>(a, p.out, stream);
    default: return launch_tiles<4, 1, 1, 3, true, O, PACKED>(a, p.out, stream);
  }
}

}  // namespace

hipError_t launch_fp4_tiles(const Fp4MatmulParams& p, hipStream_t stream) {
  TileArgs a{};
  a.x = (const uint8_t*)p.x; a.xs = p.x_scales; a.w = p.w; a.ws = p.w_scales; a.off = p.off;
  a.groups = p.groups; a.rows = (int)p.rows; a.K = p.k; a.N = p.n;
  if (p.x_codes) {
    const int per_row = p.k / 32;
    const unsigned grid = (unsigned)((p.rows * per_row + 255) / 256);
    auto quantise = [&](auto* x) {
      fp4_quantise_kernel<<<grid, 256, 0, stream>>>(x, p.rows, per_row, p.off, p.groups, p.x_codes, p.x_code_scales);
    };
    switch (p.x_kind) {
      case 0: quantise((const float*)p.x); break;
      case 1: quantise((const _Float16*)p.x); break;
      default: quantise((const uint16_t*)p.x); break;
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    a.x = p.x_codes; a.xs = p.x_code_scales;
  }
  if (p.packed)
    return p.out_fp32 ? launch_shape<float, true>(p, a, stream) : launch_shape<uint16_t, true>(p, a, stream);
  return p.out_fp32 ? launch_shape<float, false>(p, a, stream) : launch_shape<uint16_t, false>(p, a, stream);
}

}  // namespace moe
