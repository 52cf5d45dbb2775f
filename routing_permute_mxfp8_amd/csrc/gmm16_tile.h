// 16-bit grouped products with both operands staged in LDS (the kernel of the three files
// gmm16_forward.hip, gmm16_transposed.hip and gmm16_weights.hip).
//
// A work item is a tile of MT output rows by NT output channels, computed by four waves, each
// holding CB x RB accumulators of 16 channels x 16 rows (V_MFMA_F32_16X16X32: lane l holds 8
// contraction elements, 8 (l / 16) on, of row l % 16 of an operand; weights in the A slot, so that
// a lane holds 4 neighbouring channels of one row). Blocks are persistent and XCD-aware.
//
// A slot of LDS holds 64 contraction elements of both operands, two sub-steps of 32; there are two
// slots. The MFMAs of a sub-step run in groups, one for each of the wave's RB row blocks: the CB
// weight operands of the next sub-step are read beside them into a second set of registers, a row
// operand into its own when its group has been issued. Behind the first group of a slot's second
// sub-step all waves have read the slot (there is the barrier) and the loads of the step after next
// begin to fill it. Loads go on across items.
//
// An operand whose contraction is contiguous in memory ("direct") lies in LDS as rows of 64
// elements, 128 bytes; 16-byte chunk c of row r at place c ^ (r / 2 % 8), so that the sixteen lanes
// of a read pass touch all banks once. One whose channels are contiguous ("transposed") lies as
// 64 rows of the contraction, as it comes, and is transposed on its way to the registers
// (DS_READ_B64_TR_B16: of the 16 x 4 elements that four lanes a contraction row address, 4 rows of
// 16 channels, lane j gets the 4 contraction elements of channel j). 32 lanes a clock are served,
// rows 0 - 3 and 8 - 11 of 32 bytes each: 64-byte blocks of row r are exchanged by r % 4, their halves
// by r / 8 % 2, so that these lie in different banks.
//
// What bounds it: large products the card's power, at which it runs its clock down (1.66 to
// 1.81 GHz by the board, with the MFMAs at work 69 % of the cycles, forward, 32768 rows on 16 groups of
// 4096 x 7168: 1.55 to 1.66 ms, 1.25 to 1.16 PFLOP/s; the MFMAs alone, of random operands in registers, 2.06), then the items' ends: an item's
// stores and the next one's zeros take 5 us beside 1.8 a step, which a contraction of a few steps
// shows (gradient by the weights, 256 rows a group: 4 - 6 steps, 14.6 us an item). Products of few
// rows the weights' stream (256 rows on 64 groups: 3.76 GB in 0.54 ms, 7.0 TB/s). Why tiles of up to
// 256 x 256 and one block a unit: a step of it reads each operand for 256 of the other, and the L1
// is then busy half of a step's time; tiles of 128 x 256 take 1.08 us a step, 1.2 times as long for
// the same work.
//
// Measured along the way, 32768 rows as above (forward / transposed) and the weights' gradient of 16
// groups, 7168 x 2048 (ms): LDS-staged 32 x 32 MFMAs, direct-to-LDS loads 1.83 / 2.00 / 1.75; loads
// through registers, spread over a slot's time 1.73 / 1.88 / 0.89; 16 x 16 x 32 MFMAs in place 1.73 /
// 1.73 / 0.86; each load and write to LDS between MFMAs of their own 1.66 / 1.66 / 0.80; now 1.56 / 1.62 /
// 0.78.
#pragma once

#include <algorithm>
#include <atomic>

#include "gmm16_device.h"
#include "internal.h"

namespace moe {
namespace {

typedef __attribute__((address_space(3))) void* lds_ptr;

constexpr int kList = 64;   // items described at a time
constexpr int kCon = 64;    // contraction elements of a slot

enum Form { kForward, kTransposed, kWeights };

struct Tile16Args {
  const uint16_t* row;   // what makes the output's rows: [rows, con], kWeights: [rows, nr]
  const uint16_t* chan;  // and its channels: [groups, nc, con], [groups, con_t, nc], kWeights: [rows, nc]
  int pitch_row, pitch_chan;   // elements from one row of them to the next, multiples of 8
  const int32_t* off;
  int groups, rows;
  int nc, nr;            // nr: kWeights only
  int con, con_t;        // contraction, of a direct operand (with zeros up to a multiple of 8) and of a transposed one
  bool out_fp32;
  void* out;
  float* part;           // workspace of shared items: a tile for each block, or null: items are not shared
  int steps;             // of an item (not kWeights)
};

template <int WAVES, int WC, int CB, int RB>
struct Tile16 {
  static constexpr int kNT = 16 * WC * CB, kMT = 16 * (WAVES / WC) * RB;
  static constexpr int kA = kNT * 2 * kCon, kB = kMT * 2 * kCon;   // bytes of a slot: channels, rows
  static constexpr int kEnds = 0, kItems = 4 * kMaxGroups;          // behind the slots
  static constexpr int kLds = 2 * (kA + kB) + kItems + 16 * kList;
  static constexpr int kLA = kNT / (8 * WAVES), kLB = kMT / (8 * WAVES);   // loads of 1 KB a wave and slot
};

// Waits for the wave's LDS accesses (and with DMA for its direct-to-LDS loads), then for the other
// waves: what was loaded or written is there for all, and what was read may be written again.
template <bool DMA>
__device__ __forceinline__ void slot_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt(DMA ? (0 << 14) | (7 << 4) | (0 << 8) | 0 : (3 << 14) | (7 << 4) | (0 << 8) | 15);
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
  __builtin_amdgcn_sched_barrier(0);
}

// ---- which item a block works at ------------------------------------------------------------
// The items are the output's tiles by their channel blocks. Each XCD takes a contiguous share of
// them (kWeights: of each group's, whose items are as long as the group has rows; which eighth it
// takes moves on by one with each group), dealt to its blocks in turn. What is left for a last,
// part-filled round is shared: the contraction of each of these items is cut into `parts`, one for
// each block; the blocks leave fp32 tiles, which gmm16_join_kernel adds in order.
__host__ __device__ __forceinline__ int eighth(int each, int i) { return (int)((int64_t)each * i / 8); }
struct Share {
  int64_t begin;          // the XCD's first item (not kWeights)
  int full, rem, parts;   // whole rounds, items behind them, blocks an item of those
};
// each: items of a group (kWeights). steps: those of the longest item.
template <int FORM>
__host__ __device__ __forceinline__ Share share_of(const Tile16Args& p, int64_t total, int each, int steps, int xcd,
                                                   int per) {
  Share s;
  int64_t n;
  if constexpr (FORM == kWeights) {
    s.begin = 0;
    n = (int64_t)(p.groups / 8) * each;
    for (int g = 0; g < p.groups % 8; ++g) n += eighth(each, (xcd + g) % 8 + 1) - eighth(each, (xcd + g) % 8);
  } else {
    s.begin = total * xcd / 8;
    n = total * (xcd + 1) / 8 - s.begin;
  }
  s.full = (int)(n / per);
  s.rem = (int)(n - (int64_t)s.full * per);
  s.parts = s.rem ? (per / s.rem < steps / 4 ? per / s.rem : steps / 4) : 1;   // (a part has four steps at least)
  if (!p.part || s.parts < 2 || steps - (steps + s.parts - 1) / s.parts < kGain16) s.parts = 1;
  return s;
}

// Number n of the XCD's items among all.
template <int FORM>
__device__ __forceinline__ int64_t item_of(const Share& s, int each, int xcd, int64_t n) {
  if constexpr (FORM != kWeights) return s.begin + n;
  int g = (int)(n / each) * 8;   // (the XCD takes `each` items of eight groups in a row)
  int left = (int)(n % each);
  for (;; ++g) {
    const int first = eighth(each, (xcd + g) % 8), size = eighth(each, (xcd + g) % 8 + 1) - first;
    if (left < size) return (int64_t)g * each + first + left;
    left -= size;
  }
}

// The steps of the longest item: kWeights: of the largest group (all threads; scratch for WAVES).
template <int FORM, int WAVES>
__device__ __forceinline__ int longest(const Tile16Args& p, int* scratch) {
  if (FORM != kWeights || !p.part) return p.steps;
  int most = 0;
  for (int g = threadIdx.x; g < p.groups; g += 64 * WAVES) {
    int lo, hi;
    group_rows(p.off, g, p.rows, &lo, &hi);
    most = max(most, hi - lo);
  }
  for (int s = 1; s < 64; s *= 2) most = max(most, __shfl_xor(most, s, 64));
  if ((threadIdx.x & 63) == 0) scratch[threadIdx.x >> 6] = most;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < WAVES; ++w) most = max(most, scratch[w]);
  __syncthreads();
  return __builtin_amdgcn_readfirstlane((most + kCon - 1) / kCon);
}

// Item `it`: (group, first row, rows, tile and channel block). Four row tiles run through the
// channel blocks together, so that the items in flight on one XCD share both operands in its L2.
template <int FORM, int MT>
__device__ __forceinline__ int4 describe16(const Tile16Args& p, const int* ends, int tiles, int nrt, int ncb, int64_t it) {
  int64_t base = 0;
  int height = tiles;          // row tiles that are numbered together
  int g = 0;
  if constexpr (FORM == kWeights) {
    g = (int)(it / ((int64_t)nrt * ncb));
    base = (int64_t)g * nrt * ncb;
    height = nrt;
  }
  const int64_t in_all = it - base;
  const int64_t block = in_all / (4 * (int64_t)ncb);
  const int in = (int)(in_all - block * 4 * ncb);
  const int width = min(4, height - 4 * (int)block);
  const int cb = in / width, t = 4 * (int)block + in - cb * width;
  int lo, hi;
  if constexpr (FORM == kWeights) {
    group_rows(p.off, g, p.rows, &lo, &hi);
    return make_int4(g, lo, hi - lo, t * ncb + cb);
  } else {
    g = group_of_tile(ends, p.groups, t);
    group_rows(p.off, g, p.rows, &lo, &hi);
    const int row0 = lo + (t - (g > 0 ? ends[g - 1] : 0)) * MT;
    return make_int4(g, row0, min(MT, hi - row0), cb);
  }
}

// Transposed: what the chunks of a row of `width` channels are exchanged by.
__device__ constexpr int trans_swap(int width, int row) {
  return 4 * (width == 64 ? (row >> 1) & 1 : row & 3) + 2 * ((row >> 3) & 1);
}
// The first load of a wave whose lanes' chunks are exchanged as load i's are (a wave's loads begin at a
// row that is a multiple of 8): their places differ by whole rows only.
__device__ constexpr int load_like(bool direct, int width, int i) {
  if (direct) return i & 1;
  for (int k = 0; k < i; ++k)
    if (trans_swap(width, k * (512 / width)) == trans_swap(width, i * (512 / width))) return k;
  return i;
}

struct Item16 {
  int group, lo, rows;   // rows [lo, lo + rows): the tile's (kWeights: the group's, which are summed)
  int rt, cb;            // channel block; row tile of the output (kWeights)
};
template <int FORM>
__device__ __forceinline__ Item16 item16(const int4& v, int ncb) {
  Item16 r;
  r.group = __builtin_amdgcn_readfirstlane(v.x);
  r.lo = __builtin_amdgcn_readfirstlane(v.y);
  r.rows = __builtin_amdgcn_readfirstlane(v.z);
  const int w = __builtin_amdgcn_readfirstlane(v.w);
  r.rt = FORM == kWeights ? w / ncb : 0;
  r.cb = w - r.rt * ncb;
  return r;
}

// Four neighbouring values at any element of a row, `left` of which are the row's.
template <typename V>
struct AnyFour {
  V v;
} __attribute__((packed, aligned(sizeof(V) / 4)));
template <typename O, typename V>
__device__ __forceinline__ void store_any(O* to, int left, V v) {
  if (left >= 4) {
    reinterpret_cast<AnyFour<V>*>(to)->v = v;
  } else {
    O one[4];
    __builtin_memcpy(one, &v, sizeof(v));
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (i < left) to[i] = one[i];
  }
}

// ---- output -----------------------------------------------------------------------------------
// A row block's accumulators: lane (g, r) holds row r, channels 4 g + 0..3 of each 16-channel block: 64
// neighbouring bytes of a row in fp32. Of 16-bit values those of two blocks are exchanged until a
// lane has 8 neighbouring channels and a row's 64 bytes are in lanes l, l + 32, l + 16, l + 48
// (pieces of 8 bytes would be write requests of their own to the L2). ODD: the output's rows are no
// whole 16-byte vectors: a lane's 4 channels are one store at any element (store_any).
template <bool ODD, typename T, int CB>
__device__ __forceinline__ void store_rows(const Tile16Args& p, const v4f (&acc)[CB], bool valid, int64_t row, int c0) {
  const int g4 = (threadIdx.x & 63) >> 4;
  if constexpr (ODD) {
#pragma unroll
    for (int i = 0; i < CB; ++i) {
      const int c = c0 + 16 * i + 4 * g4, left = valid ? p.nc - c : 0;
      if (p.out_fp32) store_any((float*)p.out + row * p.nc + c, left, acc[i]);
      else store_any((uint16_t*)p.out + row * p.nc + c, left,
                     uint2{Mfma<T>::pair(acc[i][0], acc[i][1]), Mfma<T>::pair(acc[i][2], acc[i][3])});
    }
  } else if (p.out_fp32) {
    float* to = (float*)p.out + row * p.nc;
#pragma unroll
    for (int i = 0; i < CB; ++i) {
      const int c = c0 + 16 * i + 4 * g4;
      if (valid && c < p.nc) *reinterpret_cast<v4f*>(to + c) = acc[i];
    }
  } else {
    uint16_t* to = (uint16_t*)p.out + row * p.nc;
#pragma unroll
    for (int i = 0; i < CB; i += 2) {
      const auto at = [&](int k, int c) { return Mfma<T>::pair(acc[i + k][c], acc[i + k][c + 1]); };
      const auto s0 = __builtin_amdgcn_permlane16_swap(at(0, 0), at(1, 0), false, false);
      const auto s1 = __builtin_amdgcn_permlane16_swap(at(0, 2), at(1, 2), false, false);
      const int c = c0 + 16 * i + 16 * (g4 & 1) + 8 * (g4 >> 1);
      if (valid && c < p.nc) *reinterpret_cast<u32x4*>(to + c) = u32x4{s0[0], s1[0], s0[1], s1[1]};
    }
  }
}

// The body gets the slots (both of the channels' operand, both of the rows') and the rest of LDS as
// restrict pointers, which is what they are: apart. A slot is never read while loads into it are in
// flight, and so the compiler, which makes an LDS read wait for the direct-to-LDS loads that may
// write there, has nothing to wait for.
template <int FORM, int WAVES, int WC, int CB, int RB, bool ONCE, bool DMA, bool ODD, typename T>
__device__ __forceinline__ void tile16_body(const Tile16Args& p, uint8_t* __restrict__ a0, uint8_t* __restrict__ a1,
                                            uint8_t* __restrict__ b0, uint8_t* __restrict__ b1,
                                            uint8_t* __restrict__ lds) {
  using S = Tile16<WAVES, WC, CB, RB>;
  constexpr int MT = S::kMT, NT = S::kNT;
  constexpr bool kDirA = FORM == kForward, kDirB = FORM != kWeights;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wc = wave % WC, wr = wave / WC;
  const int ncb = (p.nc + NT - 1) / NT, nrt = (p.nr + MT - 1) / MT;
  int* const ends = reinterpret_cast<int*>(lds + S::kEnds);
  int4* const list = reinterpret_cast<int4*>(lds + S::kItems);

  int* const scratch = reinterpret_cast<int*>(list);   // (until the list is filled)
  const int tiles = FORM == kWeights ? p.groups * nrt : count_tiles<MT, WAVES>(p.off, p.groups, p.rows, ends, scratch);
  const int xcd = blockIdx.x & 7, slot_in = blockIdx.x >> 3, per = gridDim.x >> 3;
  const Share share = share_of<FORM>(p, (int64_t)tiles * ncb, nrt * ncb, longest<FORM, WAVES>(p, scratch), xcd, per);
  const bool shared = share.parts > 1 && slot_in < share.rem * share.parts;   // the block's last item is a part of one
  const int count = share.full + (share.parts > 1 ? shared : slot_in < share.rem);
  if (count == 0) return;   // the whole block
  auto fill = [&](int first) {   // list[i] = this block's item first + i
    __syncthreads();
    if (tid < kList && first + tid < count) {
      const int n = first + tid;
      const int in = n == share.full && shared ? slot_in % share.rem : slot_in;
      const int64_t it = item_of<FORM>(share, nrt * ncb, xcd, (int64_t)n * per + in);
      list[tid] = describe16<FORM, MT>(p, ends, tiles, nrt, ncb, it);
    }
    __syncthreads();
  };
  auto item = [&](int i) { return item16<FORM>(list[i % kList], ncb); };

  // ---- loads: load i of a wave and operand fills 1 KB of it, lane l the 16 bytes at 16 l -------
  // direct: 8 rows of 128 bytes; transposed: 1024 / (2 NT) rows of the contraction
  const int pitch_a = 2 * p.pitch_chan, pitch_b = 2 * p.pitch_row;
  const int tail_step = p.con % kCon ? p.con / kCon : -1;   // direct: the step that the contraction ends in
  auto direct_chunk = [&](int load) { return (lane & 7) ^ (((load * 8 + (lane >> 3)) >> 1) & 7); };
  auto lane_place = [&](bool direct, int width, int pitch, int load) {
    if (direct) return (load * 8 + (lane >> 3)) * pitch + 16 * direct_chunk(load);
    const int at = load * 64 + lane, row = at / (width / 8);
    return row * pitch + 16 * (at % (width / 8) ^ trans_swap(width, row));
  };
  int va[S::kLA], vb[S::kLB];
#pragma unroll
  for (int i = 0; i < S::kLA; ++i) va[i] = lane_place(kDirA, NT, pitch_a, wave * S::kLA + i);
#pragma unroll
  for (int i = 0; i < S::kLB; ++i) vb[i] = lane_place(kDirB, MT, pitch_b, wave * S::kLB + i);
  int ta[2], tb[2];   // what moves a lane of an even and an odd load outside in that step
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    ta[i] = kDirA && 8 * direct_chunk(wave * S::kLA + i) >= p.con % kCon ? kOutside : 0;
    tb[i] = kDirB && 8 * direct_chunk(wave * S::kLB + i) >= p.con % kCon ? kOutside : 0;
  }

  // The item being loaded: buffers of exactly what belongs to it (the rest reads as zeros,
  // without memory traffic).
  struct Step {
    const uint8_t *a, *b;   // the step's operands (direct: the item's)
    int ma, mb;             // bytes from there on that belong to the item
    int left;               // transposed: rows of the contraction from here on
    int steps, soff;        // steps from here on; direct: where the step begins in a row
  };
  Step st, nx;              // the step being loaded and the one after it
  int na, nb;               // direct: the item's bytes; transposed: bytes cut off a row's front (its first channel)
  const int stride_a = kCon * pitch_a, stride_b = kCon * pitch_b;
  auto rows_bytes = [&](int left, int pitch, int cut) { return max(min(left, kCon) * pitch - cut, 0); };   // (left may be negative)
  auto aim = [&](const Item16& it, bool part, bool there) {   // nx: the item's first step; !there: zeros
    const int con_rows = FORM == kWeights ? it.rows : p.con_t;
    const int all = ((FORM == kWeights ? it.rows : p.con) + kCon - 1) / kCon;
    int first = 0, steps = there ? all : 0;
    if (part) {
      const int each = (all + share.parts - 1) / share.parts;
      first = min(all, slot_in / share.rem * each);
      steps = min(all - first, each);
    }
    nx.steps = steps;
    nx.soff = first * 2 * kCon;
    nx.left = steps > 0 ? min(con_rows - first * kCon, steps * kCon) : 0;
    if constexpr (FORM == kWeights) {
      nx.a = reinterpret_cast<const uint8_t*>(p.chan + ((int64_t)it.lo + first * kCon) * p.pitch_chan + it.cb * NT);
      nx.b = reinterpret_cast<const uint8_t*>(p.row + ((int64_t)it.lo + first * kCon) * p.pitch_row + it.rt * MT);
      na = 2 * it.cb * NT;
      nb = 2 * it.rt * MT;
    } else {
      nx.b = reinterpret_cast<const uint8_t*>(p.row + (int64_t)it.lo * p.pitch_row);
      nb = it.rows * pitch_b;
      if constexpr (kDirA) {
        nx.a = reinterpret_cast<const uint8_t*>(p.chan + ((int64_t)it.group * p.nc + it.cb * NT) * p.pitch_chan);
        na = min(NT, p.nc - it.cb * NT) * pitch_a;
      } else {
        nx.a = reinterpret_cast<const uint8_t*>(p.chan + ((int64_t)it.group * p.con_t + first * kCon) * p.pitch_chan + it.cb * NT);
        na = 2 * it.cb * NT;
      }
    }
    nx.ma = kDirA ? (steps > 0 ? na : 0) : rows_bytes(nx.left, pitch_a, na);
    nx.mb = kDirB ? (steps > 0 ? nb : 0) : rows_bytes(nx.left, pitch_b, nb);
    return steps;
  };
  // nx from st, in parts: between the MFMAs there is room for a few scalar instructions each
  constexpr int kNextParts = 5;
  auto next_part = [&](int part) {
    if (part == 0) {
      nx.steps = st.steps - 1;
      nx.soff = st.soff + 2 * kCon;
      nx.left = st.left - kCon;
    }
    if (part == 1) nx.a = kDirA ? st.a : st.a + stride_a;
    if (part == 2) nx.b = kDirB ? st.b : st.b + stride_b;
    if (part == 3) nx.ma = kDirA ? (nx.steps > 0 ? na : 0) : rows_bytes(nx.left, pitch_a, na);
    if (part == 4) nx.mb = kDirB ? (nx.steps > 0 ? nb : 0) : rows_bytes(nx.left, pitch_b, nb);
  };
  int ua[2] = {0, 0}, ub[2] = {0, 0};
  auto take_step = [&]() {   // st = nx
    // (scalars: from vector registers, where the compiler puts some of them, each load would loop
    // over the lanes)
    auto scalar = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
    auto scalar_ptr = [&](const uint8_t* q) {
      const uint64_t u = reinterpret_cast<uint64_t>(q);
      return reinterpret_cast<const uint8_t*>((uint64_t)(uint32_t)scalar((int)(uint32_t)u) | (uint64_t)(uint32_t)scalar((int)(u >> 32)) << 32);
    };
    st.a = scalar_ptr(nx.a);
    st.b = scalar_ptr(nx.b);
    st.ma = scalar(nx.ma);
    st.mb = scalar(nx.mb);
    st.left = scalar(nx.left);
    st.steps = scalar(nx.steps);
    st.soff = scalar(nx.soff);
    const bool tail = st.soff == tail_step * 2 * kCon;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if constexpr (kDirA) ua[i] = tail ? ta[i] : 0;
      if constexpr (kDirB) ub[i] = tail ? tb[i] : 0;
    }
  };
  auto step_on = [&]() {
    for (int k = 0; k < kNextParts; ++k) next_part(k);
    take_step();
  };
  auto place = [&](int slot, int i) {   // of load i in a slot (a constant): 1 KB
    return i < S::kLA ? (slot ? a1 : a0) + (wave * S::kLA + i) * 1024 : (slot ? b1 : b0) + (wave * S::kLB + i - S::kLA) * 1024;
  };
  u32x4 held[DMA ? 1 : S::kLA + S::kLB];
  auto fetch = [&](int slot, int i) {
    const bool chan = i < S::kLA;
    const int k = chan ? i : i - S::kLA;
    const auto r = buffer_of(chan ? st.a : st.b, chan ? st.ma : st.mb);
    // (few lane places are kept, and the rows between them added: registers are short)
    const int like = chan ? load_like(kDirA, NT, k) : load_like(kDirB, MT, k);
    const int rows = (k - like) * (chan ? (kDirA ? 8 : 512 / NT) : kDirB ? 8 : 512 / MT);
    const int voff = (chan ? va[like] + ua[k & 1] : vb[like] + ub[k & 1]) + rows * (chan ? pitch_a : pitch_b), so = (chan ? kDirA : kDirB) ? st.soff : 0;
    if constexpr (DMA) {
      if (ONCE && chan) __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr)place(slot, i), 16, voff, so, 0, 2);
      else __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr)place(slot, i), 16, voff, so, 0, 0);
    } else {
      if (ONCE && chan) held[i] = __builtin_amdgcn_raw_buffer_load_b128(r, voff, so, 2);
      else held[i] = __builtin_amdgcn_raw_buffer_load_b128(r, voff, so, 0);
    }
  };
  auto put = [&](int slot, int i) {
    if constexpr (!DMA) *reinterpret_cast<u32x4*>(place(slot, i) + lane * 16) = held[i];
  };
  constexpr int kLoads = S::kLA + S::kLB;

  // ---- operand reads of a wave: sub-step s (32 elements) of a slot ---------------------------
  const int g4 = lane >> 4;
  auto read_base = [&](bool direct, int width, int blk) {   // the lane's place in block blk
    if (direct) return blk * 2048 + (lane & 15) * 128 + ((g4 ^ ((lane >> 1) & 7)) * 16);
    const int i = lane & 15, row = 8 * g4 + (i >> 2);
    return row * 2 * width + (((2 * blk + ((i & 3) >> 1)) ^ trans_swap(width, row)) * 16) + (i & 1) * 8;
  };
  int ra = read_base(kDirA, NT, wc * CB), rb = read_base(kDirB, MT, wr * RB);
  u32x4 a[2][CB], b[RB];
  auto read_trans = [&](const uint8_t* at, int pitch) {   // (rows r and r + 4 are exchanged alike)
    typedef short s4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) s4* s4_lds;
    const uint2 lo = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((s4_lds)at));
    const uint2 hi = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((s4_lds)(at + 4 * pitch)));
    return u32x4{lo.x, lo.y, hi.x, hi.y};
  };
  // (transposed: block numbers differ in the bits of 32 i, which nothing else of an address has)
  auto read_a = [&](int slot, int s, int i) {   // (constants)
    const uint8_t* base = slot ? a1 : a0;
    if constexpr (kDirA)
      a[s][i] = *reinterpret_cast<const u32x4*>(base + i * 2048 + (ra ^ (64 * s)));
    else
      a[s][i] = read_trans(base + s * 64 * NT + (ra ^ (32 * i)), 2 * NT);
  };
  auto read_b = [&](int slot, int s, int i) {
    const uint8_t* base = slot ? b1 : b0;
    if constexpr (kDirB)
      b[i] = *reinterpret_cast<const u32x4*>(base + i * 2048 + (rb ^ (64 * s)));
    else
      b[i] = read_trans(base + s * 64 * MT + (rb ^ (32 * i)), 2 * MT);
  };
  // Addresses are made anew in each turn: kept, they would take the registers of operands.
  auto renew = [&]() { asm volatile("" : "+v"(ra), "+v"(rb)); };

  // ---- MFMAs: group j of sub-step s; behind MFMA i `between(i)`, in the order written ------------
  // They are written in assembly because the compiler gives the result of a 16 x 16 MFMA other
  // registers than its accumulator had: with all 256 accumulation registers in use it moves them
  // about and spills. settle() keeps the waits that the compiler would have put between an MFMA and
  // any other access to its accumulator: 32 wait states, more than any of them needs.
  v4f acc[CB][RB];
  auto multiply = [&](int s, int j, auto between) {
#pragma unroll
    for (int i = 0; i < CB; ++i) {
      Mfma<T>::k32_into(acc[i][j], a[s][i], b[j]);
      between(i);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // Beside group j and MFMA i of sub-step s: the reads of the sub-step after it, slot `slot`, sub-step
  // `to`. The weights two a group; a group's row operand behind its last MFMA, but that of group 0
  // of a second sub-step, which lies before the barrier, with group 1.
  auto reads = [&](int slot, int to, int j, int i) {
    const int first = to == 0 ? 1 : 0;   // the first group that may read
    constexpr int kPer = (CB + RB - 2) / (RB - 1) > 2 ? (CB + RB - 2) / (RB - 1) : 2;   // weights a group
#pragma unroll
    for (int w = 0; w < kPer; ++w)
      if (i == (2 * w + 1) * CB / (2 * kPer + 2) && (j - first) * kPer + w < CB) read_a(slot, to, (j - first) * kPer + w);
    if (first && j == 1 && i == 0) read_b(slot, to, 0);
    if (i == CB - 1) read_b(slot, to, j);
  };
  // The loads beside the groups between two barriers, RB - 1 behind the one that sets slot SLOT free
  // and RB + 1 of the other slot: DMA: those of the step after next are issued in the first half.
  // Else what was fetched before is put there, a part beside each group, and in the place of each
  // part that of the step aimed at is fetched: every load has a whole slot's time, and the loads
  // are spread evenly (the CU's L1 takes half of a slot's time for them; in a burst they hold up
  // the waves). An MFMA takes the time of four other instructions: more between two of them would
  // leave the matrix core idle.
  auto loads = [&](int slot, int group, int i) {
    // (in groups of eight MFMAs away from the reads, and the two parts of a load behind different ones)
    constexpr int kPlaces = (DMA ? 1 : 2) * RB * CB, kBack = CB >= 8 ? 4 : 0, kFetch = CB >= 8 ? 1 : 0;
    static_assert((kLoads - 1) * kPlaces / kLoads + kBack + kFetch < 2 * RB * CB, "every load has its place");
#pragma unroll
    for (int l = 0; l < kLoads; ++l) {
      const int at = l * kPlaces / kLoads + kBack, here = group * CB + i;
      if (at == here) put(slot, l);
      if (at + kFetch == here) fetch(slot, l);
    }
  };
  auto end_slot = [&]<int SLOT>(std::integral_constant<int, SLOT>) {
#pragma unroll
    for (int j = 1; j < RB; ++j)
      multiply(1, j, [&](int i) {
        reads(SLOT ^ 1, 0, j, i);
        loads(SLOT, j - 1, i);
      });
  };
  auto begin_slot = [&]<int SLOT>(std::integral_constant<int, SLOT>) {   // of the other slot than SLOT
#pragma unroll
    for (int j = 0; j < RB; ++j)
      multiply(0, j, [&](int i) {
        reads(SLOT ^ 1, 1, j, i);
        loads(SLOT, RB - 1 + j, i);
        constexpr int kEach = (kNextParts + RB - 2) / (RB - 1);   // parts beside a group
        if (i == CB - 2 && j < RB - 1)
#pragma unroll
          for (int k = 0; k < kEach; ++k) next_part(j * kEach + k);
      });
    multiply(1, 0, [&](int i) { loads(SLOT, 2 * RB - 1, i); });
    slot_barrier<DMA>();
  };
  auto turn = [&](auto k) {
    renew();
    take_step();
    end_slot(k);
    begin_slot(k);
  };
  constexpr std::integral_constant<int, 0> k0{};
  constexpr std::integral_constant<int, 1> k1{};

  fill(0);
  Item16 cur = item(0);
  int steps = aim(cur, shared && share.full == 0, true);
  // DMA: steps 0 and 1 are on their way into the slots. Else step 0 is in its slot, and steps 1 and 2
  // are where the first part of a turn before the first would have left them: the parts beside its
  // RB - 1 groups of step 1 put and of step 2 fetched.
  take_step();
#pragma unroll
  for (int i = 0; i < kLoads; ++i) fetch(0, i);
#pragma unroll
  for (int i = 0; i < kLoads; ++i) put(0, i);
  step_on();
#pragma unroll
  for (int i = 0; i < kLoads; ++i) fetch(1, i);
  if constexpr (!DMA) {
    step_on();
#pragma unroll
    for (int g = 0; g < RB - 1; ++g)
#pragma unroll
      for (int i = 0; i < CB; ++i) loads(1, g, i);
  }
  slot_barrier<DMA>();
#pragma unroll
  for (int i = 0; i < CB; ++i) read_a(0, 0, i);
#pragma unroll
  for (int i = 0; i < RB; ++i) read_b(0, 0, i);
  auto settle = [&]() {
    asm volatile("s_nop 15\n\ts_nop 15" ::);
#pragma unroll
    for (int i = 0; i < CB; ++i)
#pragma unroll
      for (int j = 0; j < RB; ++j) asm volatile("" : "+a"(acc[i][j]));
    asm volatile("s_nop 15\n\ts_nop 15" ::);
  };
  auto zero = [&]() {
#pragma unroll
    for (int i = 0; i < CB; ++i)
#pragma unroll
      for (int j = 0; j < RB; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.0f;
    settle();
  };
  zero();
  begin_slot(k1);
  for (int n = 0;;) {
    // steps of the item, an even number (those behind its last are zeros)
    const int all = max(DMA ? 2 : 4, (steps + 1) / 2 * 2);
    for (int t = 0; t < all - (DMA ? 2 : 4); t += 2) {
      turn(k0);
      turn(k1);
    }
    if constexpr (!DMA) turn(k0);
    // the next item's first steps are loaded behind the item's last
    const bool more = n + 1 < count;
    if (more && (n + 1) % kList == 0) fill(n + 1);
    const Item16 next = more ? item(n + 1) : cur;
    steps = aim(next, more && shared && n + 1 == share.full, more);
    if constexpr (!DMA) turn(k1);
    turn(k0);
    take_step();
    end_slot(k1);
    settle();
    const bool part = shared && n == share.full;
    const int rows = FORM == kWeights ? min(MT, p.nr - cur.rt * MT) : cur.rows;
    const int64_t out_row = FORM == kWeights ? (int64_t)cur.group * p.nr + cur.rt * MT : cur.lo;
    const auto sums = buffer_of(p.part + ((int64_t)blockIdx.x * WAVES + wave) * (RB * CB * 256), RB * CB * 1024);
#pragma unroll
    for (int j = 0; j < RB; ++j) {
      v4f of[CB];
#pragma unroll
      for (int i = 0; i < CB; ++i) of[i] = acc[i][j];
      int row = (wr * RB + j) * 16 + (lane & 15);
      asm volatile("" : "+v"(row));   // (addresses made here: kept for all items, they would be spilled)
      if (part) {   // the sums as they are, for gmm16_join_kernel
#pragma unroll
        for (int i = 0; i < CB; ++i)
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, of[i]), sums, lane * 16, (j * CB + i) * 1024, 0);
      } else {
        store_rows<ODD, T, CB>(p, of, row < rows, out_row + row, cur.cb * NT + wc * CB * 16);
      }
    }
    if (++n >= count) break;
    cur = next;
    zero();
    begin_slot(k1);
  }
  __builtin_amdgcn_s_waitcnt((0 << 14) | (7 << 4) | (15 << 8));   // no direct-to-LDS load outlives the block
}

template <int FORM, int WAVES, int WC, int CB, int RB, int BLOCKS, bool ONCE, bool DMA, bool ODD, typename T>
__global__ __launch_bounds__(64 * WAVES) __attribute__((amdgpu_waves_per_eu(BLOCKS * WAVES / 4))) void gmm16_tile_kernel(Tile16Args p) {
  extern __shared__ __align__(16) uint8_t lds_area[];
  using S = Tile16<WAVES, WC, CB, RB>;
  uint8_t* const b = lds_area + 2 * S::kA;
  tile16_body<FORM, WAVES, WC, CB, RB, ONCE, DMA, ODD, T>(p, lds_area, lds_area + S::kA, b, b + S::kB, b + 2 * S::kB);
}

// The shared items' parts added, in the order of the contraction, and stored: blockIdx.x takes item
// blockIdx.x / 8 of XCD blockIdx.x % 8's shared ones, blockIdx.y one row block of each wave.
template <int FORM, int WAVES, int WC, int CB, int RB, bool ODD, typename T>
__global__ __launch_bounds__(64 * WAVES) void gmm16_join_kernel(Tile16Args p, int blocks) {
  using S = Tile16<WAVES, WC, CB, RB>;
  __shared__ int ends[FORM == kWeights ? 1 : kMaxGroups], scratch[WAVES];
  const int ncb = (p.nc + S::kNT - 1) / S::kNT, nrt = (p.nr + S::kMT - 1) / S::kMT;
  int tiles = p.groups * nrt;
  if constexpr (FORM != kWeights) tiles = count_tiles<S::kMT, WAVES>(p.off, p.groups, p.rows, ends, scratch);
  const int xcd = blockIdx.x & 7, r = blockIdx.x >> 3, per = blocks >> 3;
  const Share share = share_of<FORM>(p, (int64_t)tiles * ncb, nrt * ncb, longest<FORM, WAVES>(p, scratch), xcd, per);
  if (share.parts < 2 || r >= share.rem) return;
  const int64_t n = item_of<FORM>(share, nrt * ncb, xcd, (int64_t)share.full * per + r);
  const Item16 it = item16<FORM>(describe16<FORM, S::kMT>(p, ends, tiles, nrt, ncb, n), ncb);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, j = blockIdx.y;
  v4f acc[CB] = {};
  for (int part = 0; part < share.parts; ++part) {
    const int block = xcd + 8 * (part * share.rem + r);
    const v4f* from = reinterpret_cast<const v4f*>(p.part) + (((int64_t)block * WAVES + wave) * RB + j) * (CB * 64) + lane;
#pragma unroll
    for (int i = 0; i < CB; ++i) {
      const v4f v = from[i * 64];
      acc[i] += v;
    }
  }
  const int row = ((wave / WC) * RB + j) * 16 + (lane & 15);
  const int rows = FORM == kWeights ? min(S::kMT, p.nr - it.rt * S::kMT) : it.rows;
  const int64_t out_row = FORM == kWeights ? (int64_t)it.group * p.nr + it.rt * S::kMT : it.lo;
  store_rows<ODD, T, CB>(p, acc, row < rows, out_row + row, it.cb * S::kNT + (wave % WC) * CB * 16);
}

// Blocks of a launch (the device's compute units, rounded up to whole XCDs' shares, and no more than
// the workspace of shared items is laid out for); the kernel's LDS size set. `known`: what was found
// for the first devices, a kernel's own, 0 at the start.
constexpr int kDevices = 64;
inline hipError_t tile16_grid(const void* kernel, int lds, std::atomic<int> (&known)[kDevices], int* grid) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  if (dev < kDevices && (*grid = known[dev].load(std::memory_order_relaxed)) > 0) return hipSuccess;
  int cus = 0;
  if ((e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, lds)) != hipSuccess) return e;
  if ((e = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev)) != hipSuccess) return e;
  *grid = std::min((cus + 7) / 8 * 8, kTile16Units);
  if (dev < kDevices) known[dev].store(*grid, std::memory_order_relaxed);
  return hipSuccess;
}

template <int FORM, int WAVES, int WC, int CB, int RB, int BLOCKS, bool ONCE, bool DMA, bool ODD, typename T>
hipError_t launch_tile16(Tile16Args a, hipStream_t stream) {
  using S = Tile16<WAVES, WC, CB, RB>;
  static_assert(S::kLds * BLOCKS <= 160 * 1024, "LDS of a compute unit");
  static_assert(S::kMT >= 64 || FORM != kWeights, "a transposed operand is 64 wide at least");
  static_assert((FORM == kForward || S::kLA * (512 / S::kNT) % 8 == 0) && (FORM != kWeights || S::kLB * (512 / S::kMT) % 8 == 0),
                "a wave's loads of a transposed operand begin at a multiple of 8 rows");
  static std::atomic<int> known[kDevices];
  int grid = 0;
  const auto kernel = gmm16_tile_kernel<FORM, WAVES, WC, CB, RB, BLOCKS, ONCE, DMA, ODD, T>;
  hipError_t e = tile16_grid(reinterpret_cast<const void*>(kernel), S::kLds, known, &grid);
  if (e != hipSuccess) return e;
  grid *= BLOCKS;
  // Where the number of items does not depend on the groups' sizes it is known here whether any can be
  // shared; if not, the join's launch is saved (5 us).
  if (a.part && (FORM == kWeights || !a.off)) {
    const int ncb = (a.nc + S::kNT - 1) / S::kNT, nrt = (a.nr + S::kMT - 1) / S::kMT;
    const int tiles = FORM == kWeights ? a.groups * nrt : (a.rows + S::kMT - 1) / S::kMT;
    const int steps = FORM == kWeights ? (a.rows + kCon - 1) / kCon : a.steps;   // (kWeights: at most)
    bool any = false;
    for (int xcd = 0; xcd < 8; ++xcd)
      any |= share_of<FORM>(a, (int64_t)tiles * ncb, nrt * ncb, steps, xcd, grid / 8).parts > 1;
    if (!any) a.part = nullptr;
  }
  kernel<<<grid, 64 * WAVES, S::kLds, stream>>>(a);
  if ((e = hipGetLastError()) != hipSuccess || !a.part) return e;
  gmm16_join_kernel<FORM, WAVES, WC, CB, RB, ODD, T><<<dim3(grid / 2, RB), 64 * WAVES, 0, stream>>>(a, grid);
  return hipGetLastError();
}

// mt: rows of a tile, one of gmm16.hip's kShapes.
template <int FORM, bool ODD, typename T>
hipError_t launch_tile16_as(const Tile16Args& a, int mt, hipStream_t stream) {
  // Direct-to-LDS loads for the small tiles, whose few waves' MFMAs hide little (64 groups of 4096 x
  // 4096, 56 rows each: 429 us, through registers 446); but not beside transposing reads, for which
  // the compiler waits for every such load in flight.
  constexpr bool dma = FORM == kForward;
  switch (mt) {
    case 256: return launch_tile16<FORM, 4, 2, 8, 8, 1, false, false, ODD, T>(a, stream);
    case 128: return launch_tile16<FORM, 4, 2, 8, 4, 1, false, false, ODD, T>(a, stream);
    case 64: return launch_tile16<FORM, 4, 4, 2, 4, 2, FORM != kWeights, dma, ODD, T>(a, stream);
    default: break;
  }
  if constexpr (FORM != kWeights) switch (mt) {
    case 192: return launch_tile16<FORM, 4, 2, 8, 6, 1, false, false, ODD, T>(a, stream);
    case 160: return launch_tile16<FORM, 4, 2, 8, 5, 1, false, false, ODD, T>(a, stream);
    case 32: return launch_tile16<FORM, 4, 4, 2, 2, 3, true, dma, ODD, T>(a, stream);
    default: break;
  }
  return hipErrorInvalidValue;
}
template <int FORM, typename T>
hipError_t launch_tile16_odd(const Tile16Args& a, int mt, bool odd, hipStream_t stream) {
  return odd ? launch_tile16_as<FORM, true, T>(a, mt, stream) : launch_tile16_as<FORM, false, T>(a, mt, stream);
}

template <int FORM>
hipError_t launch_tile16_form(const Gmm16Params& p, hipStream_t stream) {
  Tile16Args a{};
  a.row = (const uint16_t*)p.a; a.chan = (const uint16_t*)p.b; a.pitch_row = p.pitch_a; a.pitch_chan = p.pitch_b;
  a.off = p.off; a.groups = p.groups; a.rows = (int)p.rows; a.out_fp32 = p.out_fp32; a.out = p.out;
  if (FORM == kWeights) { a.nc = p.k; a.nr = p.n; a.con = a.con_t = kCon; a.steps = 0; }
  else { a.nc = p.n; a.nr = 1; a.con = (p.k + 7) / 8 * 8; a.con_t = p.k; a.steps = (a.con + kCon - 1) / kCon; }
  a.part = p.part;
  return p.half ? launch_tile16_odd<FORM, _Float16>(a, p.mt, p.odd, stream) : launch_tile16_odd<FORM, __bf16>(a, p.mt, p.odd, stream);
}

}  // namespace
}  // namespace moe
