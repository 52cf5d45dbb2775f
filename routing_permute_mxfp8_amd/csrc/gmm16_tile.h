// 16-bit grouped products with both operands staged in LDS (the kernel of the three files
// gmm16_forward.hip, gmm16_transposed.hip and gmm16_weights.hip).
//
// A work item is a tile of MT output rows by NT output channels, computed by four waves, each
// holding CB x RB accumulators of 32 channels x 32 rows (V_MFMA_F32_32X32X16: lane l holds 8
// contraction elements, 8 (l / 32) on, of row l % 32 of an operand; weights in the A slot, so that
// a lane holds 4 neighbouring channels of one row). Blocks are persistent and XCD-aware.
//
// A slot of LDS holds 64 contraction elements of both operands; there are two. What a slot holds
// is read into registers a sub-step of 16 ahead of its MFMAs; in a slot's last sub-step all waves
// have read it (the barrier lies before), the loads of the step after next begin to fill it, and
// the next slot's first operands are read. The loads go straight to LDS and go on across items.
//
// An operand whose contraction is contiguous in memory ("direct") lies in LDS as rows of 64
// elements, 128 bytes; 16-byte chunk c of row r at place c ^ (r / 2 % 8), so that the sixteen lanes
// of a read pass touch all banks once. One whose channels are contiguous ("transposed") lies as
// 64 rows of the contraction, as it comes, and is transposed on its way to the registers
// (DS_READ_B64_TR_B16: of the 16 x 4 elements that four lanes a contraction row address, 4 rows of
// 16 channels, lane j gets the 4 contraction elements of channel j). There 64-byte blocks of row r
// are exchanged by r % 4, so that the four rows of such a read lie in different banks.
#pragma once

#include <algorithm>
#include <map>
#include <mutex>

#include "gmm16_device.h"
#include "internal.h"

namespace moe {
namespace {

typedef __attribute__((address_space(3))) void* lds_ptr;

constexpr int kThreads = 256;
constexpr int kList = 64;   // items described at a time
constexpr int kCon = 64;    // contraction elements of a slot

enum Form { kForward, kTransposed, kWeights };

struct Tile16Args {
  const uint16_t* row;   // what makes the output's rows: [rows, con], kWeights: [rows, nr]
  const uint16_t* chan;  // and its channels: [groups, nc, con], [groups, con, nc], kWeights: [rows, nc]
  const int32_t* off;
  int groups, rows;
  int nc, nr, con;       // nr: kWeights only, con: not there
  bool out_fp32;
  void* out;
};

template <int WC, int CB, int RB>
struct Tile16 {
  static constexpr int kNT = 32 * WC * CB, kMT = 32 * (4 / WC) * RB;
  static constexpr int kA = kNT * 2 * kCon, kB = kMT * 2 * kCon;   // bytes of a slot: channels, rows
  static constexpr int kSlot = kA + kB;
  static constexpr int kEnds = 0, kItems = 4 * kMaxGroups;          // behind the slots
  static constexpr int kLds = 2 * kSlot + kItems + 16 * kList;
  static constexpr int kLA = kNT / 32, kLB = kMT / 32;              // loads of 1 KB a wave and slot
};

// Keeps the accumulators in accumulation registers across loop edges.
template <int CB, int RB>
__device__ __forceinline__ void pin(v16f (&acc)[CB][RB]) {
#pragma unroll
  for (int i = 0; i < CB; ++i)
#pragma unroll
    for (int j = 0; j < RB; ++j) asm volatile("" : "+a"(acc[i][j]));
}

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

// Lanes 16 - 31 and 48 - 63 of a change places with lanes 0 - 15 and 32 - 47 of b.
__device__ __forceinline__ void swap_rows(u32x4& a, u32x4& b) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const auto s = __builtin_amdgcn_permlane16_swap(a[c], b[c], false, false);
    a[c] = s[0];
    b[c] = s[1];
  }
}

struct Item16 {
  int group, lo, rows;   // rows [lo, lo + rows): the tile's (kWeights: the group's, which are summed)
  int rt, cb;            // channel block; row tile of the output (kWeights)
};

// The body gets the two slots and the rest of LDS as three restrict pointers, which is what they
// are: apart. A slot is never read while loads into it are in flight, and so the compiler, which
// makes an LDS read wait for the direct-to-LDS loads that may write there, has nothing to wait for.
template <int FORM, int WC, int CB, int RB, bool ONCE, bool DMA, typename T>
__device__ __forceinline__ void tile16_body(const Tile16Args& p, uint8_t* __restrict__ slot0,
                                            uint8_t* __restrict__ slot1, uint8_t* __restrict__ lds) {
  using S = Tile16<WC, CB, RB>;
  constexpr int MT = S::kMT, NT = S::kNT;
  constexpr bool kDirA = FORM == kForward, kDirB = FORM != kWeights;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wc = wave % WC, wr = wave / WC;
  const int ncb = (p.nc + NT - 1) / NT, nrt = (p.nr + MT - 1) / MT;
  int* const ends = reinterpret_cast<int*>(lds + S::kEnds);
  int4* const list = reinterpret_cast<int4*>(lds + S::kItems);

  // ---- items: each XCD takes a contiguous share, dealt to its blocks in turn ----------------
  const int tiles = FORM == kWeights ? p.groups * nrt : count_tiles<MT>(p.off, p.groups, p.rows, ends, reinterpret_cast<int*>(list));
  const int64_t total = (int64_t)tiles * ncb;
  const int xcd = blockIdx.x & 7, per = gridDim.x >> 3;
  const int64_t begin = total * xcd / 8 + (blockIdx.x >> 3), end = total * (xcd + 1) / 8;
  if (begin >= end) return;   // the whole block
  const int64_t count = (end - begin + per - 1) / per;
  // Item `it`: four row tiles run through the channel blocks together, so that the items in flight
  // on one XCD share both operands in its L2.
  auto describe = [&](int64_t it) {
    int64_t base = 0;
    int height = tiles;          // row tiles that are numbered together
    int g = 0;
    if constexpr (FORM == kWeights) {
      g = (int)(it / ((int64_t)nrt * ncb));
      base = (int64_t)g * nrt * ncb;
      height = nrt;
    }
    const int64_t in_all = it - base;
    const int block = (int)(in_all / (4 * ncb)), in = (int)(in_all - (int64_t)block * 4 * ncb);
    const int width = min(4, height - 4 * block);
    const int cb = in / width, t = 4 * block + in - cb * width;
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
  };
  auto fill = [&](int64_t first) {   // list[i] = this block's item first + i
    __syncthreads();
    if (tid < kList && first + tid < count) list[tid] = describe(begin + (first + tid) * per);
    __syncthreads();
  };
  auto item = [&](int64_t i) {
    const int4 v = list[i % kList];
    Item16 r;
    r.group = __builtin_amdgcn_readfirstlane(v.x);
    r.lo = __builtin_amdgcn_readfirstlane(v.y);
    r.rows = __builtin_amdgcn_readfirstlane(v.z);
    const int w = __builtin_amdgcn_readfirstlane(v.w);
    r.rt = FORM == kWeights ? w / ncb : 0;
    r.cb = w - r.rt * ncb;
    return r;
  };
  auto steps_of = [&](const Item16& it) { return ((FORM == kWeights ? it.rows : p.con) + kCon - 1) / kCon; };

  // ---- loads: load i of a wave and operand fills 1 KB of it, lane l the 16 bytes at 16 l -------
  // direct: 8 rows of 128 bytes; transposed: 1024 / (2 NT) rows of the contraction
  int va[S::kLA], vb[S::kLB];
  int ta[2] = {0, 0}, tb[2] = {0, 0};   // direct, the step that the contraction ends in: what moves a lane outside
  const int tail_step = p.con % kCon ? p.con / kCon : -1;
  auto direct_chunk = [&](int load) {   // the chunk of a direct operand's row that belongs at the lane's place
    const int row = load * 8 + (lane >> 3);
    return (lane & 7) ^ ((row >> 1) & 7);
  };
  auto trans_place = [&](int width, int load, int* row, int* chunk) {   // width: channels of a row in LDS
    const int at = load * 64 + lane, places = width / 8;
    *row = at / places;
    const int x = width == 64 ? (*row >> 1) & 1 : *row & 3;
    *chunk = (at % places) ^ (4 * x);
  };
  if constexpr (kDirA) {
#pragma unroll
    for (int i = 0; i < S::kLA; ++i) va[i] = ((wave * S::kLA + i) * 8 + (lane >> 3)) * 2 * p.con + 16 * direct_chunk(wave * S::kLA + i);
#pragma unroll
    for (int i = 0; i < 2; ++i) ta[i] = 8 * direct_chunk(wave * S::kLA + i) >= p.con % kCon ? kOutside : 0;
  }
  if constexpr (kDirB) {
#pragma unroll
    for (int i = 0; i < S::kLB; ++i) vb[i] = ((wave * S::kLB + i) * 8 + (lane >> 3)) * 2 * p.con + 16 * direct_chunk(wave * S::kLB + i);
#pragma unroll
    for (int i = 0; i < 2; ++i) tb[i] = 8 * direct_chunk(wave * S::kLB + i) >= p.con % kCon ? kOutside : 0;
  }

  // The item being loaded: buffers of exactly what belongs to it (the rest reads as zeros,
  // without memory traffic); channels of a transposed operand behind its last are left out too.
  const uint8_t *pa, *pb;
  int na, nb, steps;      // direct: bytes; transposed: bytes cut off a row's front (its first channel)
  auto aim = [&](const Item16& it) {
    steps = steps_of(it);
    if constexpr (FORM == kWeights) {
      pa = reinterpret_cast<const uint8_t*>(p.chan + (int64_t)it.lo * p.nc + it.cb * NT);
      pb = reinterpret_cast<const uint8_t*>(p.row + (int64_t)it.lo * p.nr + it.rt * MT);
      na = 2 * it.cb * NT;
      nb = 2 * it.rt * MT;
#pragma unroll
      for (int i = 0; i < S::kLB; ++i) {
        int row, chunk;
        trans_place(MT, wave * S::kLB + i, &row, &chunk);
        vb[i] = it.rt * MT + 8 * chunk < p.nr ? row * 2 * p.nr + 16 * chunk : kOutside;
      }
    } else {
      pb = reinterpret_cast<const uint8_t*>(p.row + (int64_t)it.lo * p.con);
      nb = it.rows * 2 * p.con;
      const uint16_t* w = p.chan + (int64_t)it.group * p.nc * p.con;
      if constexpr (kDirA) {
        pa = reinterpret_cast<const uint8_t*>(w + (int64_t)it.cb * NT * p.con);
        na = min(NT, p.nc - it.cb * NT) * 2 * p.con;
      } else {
        pa = reinterpret_cast<const uint8_t*>(w + it.cb * NT);
        na = 2 * it.cb * NT;
      }
    }
    if constexpr (!kDirA) {
#pragma unroll
      for (int i = 0; i < S::kLA; ++i) {
        int row, chunk;
        trans_place(NT, wave * S::kLA + i, &row, &chunk);
        va[i] = it.cb * NT + 8 * chunk < p.nc ? row * 2 * p.nc + 16 * chunk : kOutside;
      }
    }
  };
  int con_rows = 0;   // of the item being loaded: rows of a transposed operand
  // load i of step `step`: its buffer and the lane's place in it
  struct Source {
    __amdgpu_buffer_rsrc_t r;
    int voff, soff;
  };
  auto source = [&](int step, int i) {
    const bool in = step < steps;
    const int left = min(max(con_rows - step * kCon, 0), kCon);
    if (i < S::kLA) {
      if constexpr (kDirA)
        return Source{buffer_of(pa, in ? na : 0), va[i] + (step == tail_step ? ta[i & 1] : 0), step * 2 * kCon};
      else
        return Source{buffer_of(pa + (int64_t)step * kCon * 2 * p.nc, left > 0 ? left * 2 * p.nc - na : 0), va[i], 0};
    } else {
      i -= S::kLA;
      if constexpr (kDirB)
        return Source{buffer_of(pb, in ? nb : 0), vb[i] + (step == tail_step ? tb[i & 1] : 0), step * 2 * kCon};
      else
        return Source{buffer_of(pb + (int64_t)step * kCon * 2 * p.nr, left > 0 ? left * 2 * p.nr - nb : 0), vb[i], 0};
    }
  };
  auto place = [&](int slot, int i) {   // of load i in a slot (a constant): 1 KB
    return (slot ? slot1 : slot0) + (i < S::kLA ? (wave * S::kLA + i) * 1024 : S::kA + (wave * S::kLB + i - S::kLA) * 1024);
  };
  u32x4 held[DMA ? 1 : S::kLA + S::kLB];
  auto fetch = [&](int slot, int step, int i) {
    const Source f = source(step, i);
    const bool once = ONCE && i < S::kLA;
    if constexpr (DMA) {
      if (once) __builtin_amdgcn_raw_ptr_buffer_load_lds(f.r, (lds_ptr)place(slot, i), 16, f.voff, f.soff, 0, 2);
      else __builtin_amdgcn_raw_ptr_buffer_load_lds(f.r, (lds_ptr)place(slot, i), 16, f.voff, f.soff, 0, 0);
    } else {
      if (once) held[i] = __builtin_amdgcn_raw_buffer_load_b128(f.r, f.voff, f.soff, 2);
      else held[i] = __builtin_amdgcn_raw_buffer_load_b128(f.r, f.voff, f.soff, 0);
    }
  };
  auto put = [&](int slot, int i) {
    if constexpr (!DMA) *reinterpret_cast<u32x4*>(place(slot, i) + lane * 16) = held[i];
  };
  constexpr int kLoads = S::kLA + S::kLB;

  // ---- operand reads of a wave: sub-step s (16 elements) of a slot ---------------------------
  const int h = lane >> 5;
  const int read0 = (lane & 31) * 128 + ((h ^ ((lane >> 1) & 7)) * 16);
  int ra[CB], rb[RB];   // transposed: the lane's place in each block
  auto trans_read = [&](int width, int blk) {
    const int q = lane >> 4, i = lane & 15, row = 8 * (q >> 1) + (i >> 2);
    const int x = width == 64 ? i >> 3 : i >> 2;
    return row * 2 * width + (((blk ^ x) * 4 + 2 * (q & 1) + ((i & 3) >> 1)) * 16) + (i & 1) * 8;
  };
  if constexpr (!kDirA)
#pragma unroll
    for (int i = 0; i < CB; ++i) ra[i] = trans_read(NT, wc * CB + i);
  if constexpr (!kDirB)
#pragma unroll
    for (int i = 0; i < RB; ++i) rb[i] = trans_read(MT, wr * RB + i);
  u32x4 a[2][CB], b[2][RB];
  auto read_trans = [&](const uint8_t* at, int pitch) {
    typedef short s4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) s4* s4_lds;
    const uint2 lo = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((s4_lds)at));
    const uint2 hi = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((s4_lds)(at + 4 * pitch)));
    return u32x4{lo.x, lo.y, hi.x, hi.y};
  };
  auto read = [&](int slot, int s, int i) {   // operand i of sub-step s (constants)
    const uint8_t* base = slot ? slot1 : slot0;
    if (i < CB) {
      if constexpr (kDirA)
        a[s & 1][i] = *reinterpret_cast<const u32x4*>(base + (wc * CB + i) * 4096 + (read0 ^ (32 * s)));
      else
        a[s & 1][i] = read_trans(base + s * 32 * NT + ra[i], 2 * NT);
    } else {
      i -= CB;
      if constexpr (kDirB)
        b[s & 1][i] = *reinterpret_cast<const u32x4*>(base + S::kA + (wr * RB + i) * 4096 + (read0 ^ (32 * s)));
      else
        b[s & 1][i] = read_trans(base + S::kA + s * 32 * MT + rb[i], 2 * MT);
    }
  };

  // ---- MFMAs of a sub-step; behind MFMA m `between(m)`, in the order written -------------------
  v16f acc[CB][RB];
  constexpr int M = CB * RB;
  auto multiply = [&](int s, auto between) {
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const int i = m % CB, j = m / CB;
      acc[i][j] = Mfma<T>::k16(a[s & 1][i], b[s & 1][j], acc[i][j]);
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
  // The MFMAs of a slot's last sub-step, and of the next slot's first three. Behind the barrier
  // that lies before them the slot SLOT is read: the step after next goes into it. DMA: its loads
  // are issued in the first of these sub-steps. Else what was fetched before is put there, a part
  // with each of the four sub-steps, and in the place of each part that of step `next` of the item
  // aimed at is fetched: every load has a whole slot's time, and the loads are spread evenly (the
  // CU's L1 takes half of a slot's time for them; in a burst they hold up the waves).
  auto load_part = [&]<int SLOT>(std::integral_constant<int, SLOT>, int quarter, int m, int next) {
    if constexpr (DMA) {
      if (quarter == 0) dealt(m, 0, kLoads, [&](int i) { fetch(SLOT, next, i); });
    } else {
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
        if (i * 4 * M / kLoads == quarter * M + m) {
          put(SLOT, i);
          fetch(SLOT, next, i);
        }
    }
  };
  auto end_slot = [&]<int SLOT>(std::integral_constant<int, SLOT> k, int next) {
    multiply(3, [&](int m) {
      dealt(m, 0, CB + RB, [&](int i) { read(SLOT ^ 1, 0, i); });
      load_part(k, 0, m, next);
    });
  };
  auto begin_slot = [&]<int SLOT>(std::integral_constant<int, SLOT> k, int next) {   // of the other slot than SLOT
#pragma unroll
    for (int s = 0; s < 3; ++s)
      multiply(s, [&](int m) {
        dealt(m, 0, CB + RB, [&](int i) { read(SLOT ^ 1, s + 1, i); });
        load_part(k, s + 1, m, next);
      });
    slot_barrier<DMA>();
  };
  auto turn = [&](auto k, int next) {
    end_slot(k, next);
    begin_slot(k, next);
  };
  constexpr std::integral_constant<int, 0> k0{};
  constexpr std::integral_constant<int, 1> k1{};

  fill(0);
  Item16 cur = item(0);
  aim(cur);
  con_rows = FORM == kWeights ? cur.rows : p.con;
  // DMA: steps 0 and 1 are on their way into the slots. Else step 0 is in its slot, and steps 1 and 2
  // are where the turn before the first would have left them: step 1's first quarter put and step
  // 2's fetched.
  constexpr int kQuarter = (kLoads + 3) / 4;
#pragma unroll
  for (int i = 0; i < kLoads; ++i) fetch(0, 0, i);
#pragma unroll
  for (int i = 0; i < kLoads; ++i) put(0, i);
#pragma unroll
  for (int i = 0; i < kLoads; ++i) fetch(1, 1, i);
  if constexpr (!DMA) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      if (i * 4 * M / kLoads < M) {
        put(1, i);
        fetch(1, 2, i);
      }
  }
  slot_barrier<DMA>();
#pragma unroll
  for (int i = 0; i < CB + RB; ++i) read(0, 0, i);
  auto zero = [&]() {
#pragma unroll
    for (int i = 0; i < CB; ++i)
#pragma unroll
      for (int j = 0; j < RB; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
    pin(acc);
  };
  zero();
  begin_slot(k1, 2);
  for (int64_t n = 0;;) {
    // steps of the item, an even number (those behind its last are zeros)
    const int all = max(DMA ? 2 : 4, (steps + 1) / 2 * 2);
    for (int t = 0; t < all - (DMA ? 2 : 4); t += 2) {
      turn(k0, t + (DMA ? 2 : 3));
      turn(k1, t + (DMA ? 3 : 4));
      pin(acc);
    }
    if constexpr (!DMA) turn(k0, all - 1);
    // the next item's first steps are loaded behind the item's last
    const bool more = n + 1 < count;
    if (more && (n + 1) % kList == 0) fill(n + 1);
    const Item16 next = more ? item(n + 1) : cur;
    aim(next);
    con_rows = FORM == kWeights ? next.rows : p.con;
    if (!more) steps = con_rows = 0;
    if constexpr (!DMA) turn(k1, 0);
    turn(k0, DMA ? 0 : 1);
    end_slot(k1, DMA ? 1 : 2);
    pin(acc);
    // ---- output: lane (h, r) holds row r, channels 8 e + 4 h + 0..3 of a block. Lane halves and
    // quarters change places until a row's 64 bytes are next to one another, in lanes l, l + 16,
    // l + 32, l + 48 (pieces of 8 or 16 bytes would be write requests of their own to the L2).
    const int rows = FORM == kWeights ? min(MT, p.nr - cur.rt * MT) : cur.rows;
    const int64_t first = FORM == kWeights ? (int64_t)cur.group * p.nr + cur.rt * MT : cur.lo;
#pragma unroll
    for (int j = 0; j < RB; ++j) {
#pragma unroll
      for (int i = 0; i < CB; ++i) {
        const int row = (wr * RB + j) * 32 + (lane & 15), ch = cur.cb * NT + (wc * CB + i) * 32;
        if (!p.out_fp32) {
          u32x4 v[2];   // lane (h, r): channels 16 e + 8 h + 0..7
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const auto at = [&](int c) { return Mfma<T>::pair(acc[i][j][8 * e + c], acc[i][j][8 * e + c + 1]); };
            const auto s0 = __builtin_amdgcn_permlane32_swap(at(0), at(4), false, false);
            const auto s1 = __builtin_amdgcn_permlane32_swap(at(2), at(6), false, false);
            v[e] = u32x4{s0[0], s1[0], s0[1], s1[1]};
          }
          swap_rows(v[0], v[1]);
          const int c = ch + 16 * ((lane >> 4) & 1) + 8 * h;
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (row + 16 * e < rows && c < p.nc)
              *reinterpret_cast<u32x4*>((uint16_t*)p.out + (first + row + 16 * e) * p.nc + c) = v[e];
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
              if (row + 16 * e < rows && c < p.nc)
                *reinterpret_cast<u32x4*>((float*)p.out + (first + row + 16 * e) * p.nc + c) = v[e];
          }
        }
      }
    }
    if (++n >= count) break;
    cur = next;
    zero();
    begin_slot(k1, DMA ? 1 : 2);
  }
  __builtin_amdgcn_s_waitcnt((0 << 14) | (7 << 4) | (15 << 8));   // no direct-to-LDS load outlives the block
}

template <int FORM, int WC, int CB, int RB, int BLOCKS, bool ONCE, bool DMA, typename T>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(BLOCKS))) void gmm16_tile_kernel(Tile16Args p) {
  extern __shared__ __align__(16) uint8_t lds_area[];
  constexpr int kSlot = Tile16<WC, CB, RB>::kSlot;
  tile16_body<FORM, WC, CB, RB, ONCE, DMA, T>(p, lds_area, lds_area + kSlot, lds_area + 2 * kSlot);
}

// The device's compute units, rounded up to whole XCDs' shares; the kernel's LDS size set
// once for each device.
inline hipError_t tile16_grid(const void* kernel, int lds, int* grid) {
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

template <int FORM, int WC, int CB, int RB, int BLOCKS, bool ONCE, bool DMA, typename T>
hipError_t launch_tile16(const Tile16Args& a, hipStream_t stream) {
  using S = Tile16<WC, CB, RB>;
  static_assert(S::kLds * BLOCKS <= 160 * 1024, "LDS of a compute unit");
  static_assert(S::kMT >= 64 || FORM != kWeights, "a transposed operand is 64 wide at least");
  int grid = 0;
  const auto kernel = gmm16_tile_kernel<FORM, WC, CB, RB, BLOCKS, ONCE, DMA, T>;
  hipError_t e = tile16_grid(reinterpret_cast<const void*>(kernel), S::kLds, &grid);
  if (e != hipSuccess) return e;
  kernel<<<grid * BLOCKS, kThreads, S::kLds, stream>>>(a);
  return hipGetLastError();
}

// mt: rows of a tile.
template <int FORM, typename T>
hipError_t launch_tile16_as(const Tile16Args& a, int mt, hipStream_t stream) {
  constexpr bool dma = FORM == kForward;   // (the transposing read waits for every direct-to-LDS load in flight)
  switch (mt) {
    case 256: return launch_tile16<FORM, 2, 4, 4, 1, false, false, T>(a, stream);
    case 128: return launch_tile16<FORM, 2, 4, 2, 1, false, dma, T>(a, stream);
    case 64: return launch_tile16<FORM, 4, 1, 2, 2, FORM != kWeights, dma, T>(a, stream);
    default:
      if constexpr (FORM == kWeights) return hipErrorInvalidValue;
      else return launch_tile16<FORM, 4, 1, 1, 3, true, dma, T>(a, stream);
  }
}

template <int FORM>
hipError_t launch_tile16_form(const Gmm16Params& p, hipStream_t stream) {
  Tile16Args a{};
  a.row = (const uint16_t*)p.a; a.chan = (const uint16_t*)p.b; a.off = p.off; a.groups = p.groups; a.rows = (int)p.rows;
  a.out_fp32 = p.out_fp32; a.out = p.out;
  if (FORM == kWeights) { a.nc = p.k; a.nr = p.n; a.con = kCon; }
  else { a.nc = p.n; a.nr = 1; a.con = p.k; }
  return p.half ? launch_tile16_as<FORM, _Float16>(a, p.mt, stream) : launch_tile16_as<FORM, __bf16>(a, p.mt, stream);
}

}  // namespace
}  // namespace moe
