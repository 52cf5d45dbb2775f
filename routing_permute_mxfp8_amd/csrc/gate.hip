// The router in front of the routing kernels: top-K gate, load-balance loss, and the
// gradient of both by the logits.
//
//   scores   softmax: p_e = exp(l_e - m) / sum_i exp(l_i - m); sigmoid: s_e = 1 / (1 + exp(-l_e))
//   gate     rank r_e = s_e + bias_e (the bias takes part in the choice only); with groups
//            of E / G neighbouring experts the best topk_groups groups by the sum of their
//            two best ranks stay; ids = the K best ranks in descending order, ties to the
//            lowest index; w_j = scale s_j (/ sum_i s_i over the K chosen)
//   balance  f_be = E c_be / (K T_b), P_be = (1 / T_b) sum_t p_te over the T_b counted rows
//            of sequence b (sigmoid: p = s / sum s);
//            loss = alpha / B' sum_b sum_e f_be P_be, B' = sequences with a counted row;
//            coef_be = d loss / d p_te = alpha E c_be / (K T_b^2 B')
//   gradient g_j = scale dw_j, renormalised: g_j = (scale dw_j - sum_i scale dw_i s_i / S) / S;
//            softmax: d_e = [e = id_j] g_j + dL coef_be, dl_e = p_e (d_e - sum_i d_i p_i);
//            sigmoid: q_e = dL coef_be, d_e = [e = id_j] g_j + (q_e - sum_i q_i s_i / Z) / Z
//            with Z = sum s, dl_e = s_e (1 - s_e) d_e
//
// A logit of -inf or NaN takes its expert out: score 0, ranked behind every other expert
// of the allowed groups, gradient 0. +inf counts as the largest finite float. A rank of NaN
// (a bias of NaN) is -inf; an expert of rank -inf is ranked like one taken out, by its index.
//
// One wave per row, lane l holding the V experts [l V, l V + V) (V = 1 .. 16 for up to
// 1024 experts): the row's reductions are DPP steps in one wave, without LDS or barriers.
// Up to 256 experts (the gate: and 8 choices, groups of a power of two of lanes) a row takes 16
// lanes instead, four rows a wave (see there): more of a row's values in one lane, fewer
// exchanges. Kernel times, one wave per row and 16 lanes, E = 256:
//   gate 8192 fp32 softmax 10.3, 5.7 us; 32768 bf16 sigmoid in 8 groups 55, 19;
//   loss 32768 fp32, first pass 60, 12.6 (34 MB); gradient 32768 fp32 23.3, 15.6 (70 MB, 4.5 TB/s).
// One wave per row at 8192 x 512 fp32: gate 21, with bias and groups 42, loss 17 (both passes),
// gradient 21.
// Bound: small calls by the launch, the gate by its instructions, the other two by the stream
// and the latency of few rows a wave.

#include <algorithm>
#include <cfloat>

#include "device_common.h"
#include "internal.h"

namespace moe {
namespace {

constexpr int kRowsPerBlock = 4;   // one wave each

// ---- rows -----------------------------------------------------------------------------
__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(_Float16 v) { return (float)v; }
__device__ __forceinline__ float to_float(uint16_t v) { return bf16_to_f(v); }   // bf16 bits

// A logit as the operators take it: NaN as -inf, +inf as the largest float, -0 as +0.
__device__ __forceinline__ float clean(float x) { return x != x ? -INFINITY : fminf(x, FLT_MAX) + 0.0f; }

// The lane's V logits of a row of E; experts past E are -inf. VEC: one wide load (E % V == 0
// and the address aligned for it, checked on the host).
template <typename T, int V>
__device__ __forceinline__ void load_row(const T* row, int E, int lane, bool vec, float (&x)[V]) {
  typedef T vec_t __attribute__((ext_vector_type(V)));
  const int e0 = lane * V;
  if (vec) {
    vec_t u;
    if (e0 < E) u = *reinterpret_cast<const vec_t*>(row + e0);
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = e0 < E ? clean(to_float((T)u[v])) : -INFINITY;
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = e0 + v < E ? clean(to_float(row[e0 + v])) : -INFINITY;
  }
}

// ---- reductions over the wave ---------------------------------------------------------
// DPP steps: neighbours within a row of 16 lanes, then the rows; lane 63 ends up with the
// whole wave's value, which every lane gets through a scalar register.
template <int CTRL>
__device__ __forceinline__ float dpp(float old, float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(old), __float_as_int(v), CTRL, 0xF, 0xF, false));
}
constexpr int kShr1 = 0x111, kShr2 = 0x112, kShr4 = 0x114, kShr8 = 0x118, kBcast15 = 0x142, kBcast31 = 0x143;

__device__ __forceinline__ float lane_value(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}
__device__ __forceinline__ double lane_value(double v, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)u, lane), hi = __builtin_amdgcn_readlane((uint32_t)(u >> 32), lane);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

__device__ __forceinline__ float wave_max(float v) {
  v = fmaxf(v, dpp<kShr1>(v, v));
  v = fmaxf(v, dpp<kShr2>(v, v));
  v = fmaxf(v, dpp<kShr4>(v, v));
  v = fmaxf(v, dpp<kShr8>(v, v));
  v = fmaxf(v, dpp<kBcast15>(v, v));
  v = fmaxf(v, dpp<kBcast31>(v, v));
  return lane_value(v, 63);
}
__device__ __forceinline__ double wave_max(double v) {
  for (int s = 1; s < 64; s *= 2) v = fmax(v, __shfl_xor(v, s, 64));
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp<kShr1>(0.0f, v);
  v += dpp<kShr2>(0.0f, v);
  v += dpp<kShr4>(0.0f, v);
  v += dpp<kShr8>(0.0f, v);
  v += dpp<kBcast15>(0.0f, v);   // lanes that read nothing add 0
  v += dpp<kBcast31>(0.0f, v);
  return lane_value(v, 63);
}
__device__ __forceinline__ double wave_sum(double v) {
  for (int s = 1; s < 64; s *= 2) v += __shfl_xor(v, s, 64);
  return v;
}

// ---- scores ---------------------------------------------------------------------------
__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * 1.4426950408889634f); }
__device__ __forceinline__ double exp_of(double x) { return exp(x); }

// m and 1 / sum of a row's softmax (a row of -inf only: m = 0 and every score 0).
template <typename R>
struct RowNorm {
  R m, inv;
};
template <typename R, int V>
__device__ __forceinline__ RowNorm<R> softmax_norm(const float (&x)[V]) {
  float mx = x[0];
#pragma unroll
  for (int v = 1; v < V; ++v) mx = fmaxf(mx, x[v]);
  mx = wave_max(mx);
  if (mx == -INFINITY) return RowNorm<R>{R(0), R(0)};
  R sum = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) sum += exp_of(R(x[v]) - R(mx));
  return RowNorm<R>{R(mx), R(1) / wave_sum(sum)};
}
__device__ __forceinline__ float reciprocal(float x) { return __builtin_amdgcn_rcpf(x); }   // V_RCP_F32, 1 ulp
__device__ __forceinline__ double reciprocal(double x) { return 1.0 / x; }
template <typename R, bool SOFTMAX>
__device__ __forceinline__ R score_of(float x, const RowNorm<R>& n) {
  if constexpr (SOFTMAX)
    return exp_of(R(x) - n.m) * n.inv;
  else
    return reciprocal(R(1) + exp_of(-R(x)));   // 1 / (1 + inf) = 0 for -inf
}

// ---- gate -----------------------------------------------------------------------------
struct GateArgs {
  const float* bias;      // nullable [E]
  int64_t first, rows;    // the launch's rows: [first, rows)
  int E, k;
  int groups, topk_groups, group_size;
  uint32_t group_magic;   // e / group_size = umulhi(e, group_magic) for e < 1024 (group_size > 1)
  int lanes;              // lanes of a wave per group (a power of two, 64 / lanes >= groups)
  bool renorm, vec;
  float scale;
  int32_t* ids;
  float* weights;
};

__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// A rank; NaN as -inf (the maximum of a NaN and a number is the number).
__device__ __forceinline__ float rank_of(float s, float bias) { return fmaxf(s + bias, -INFINITY); }
__device__ __forceinline__ double rank_of(double s, float bias) { return fmax(s + (double)bias, -(double)INFINITY); }

// (a, b) = the two largest of (a, b) and (c, d), a >= b, c >= d; -inf = none.
template <typename R>
__device__ __forceinline__ void merge_two(R& a, R& b, R c, R d) {
  const R lo = a < c ? a : c;
  a = a < c ? c : a;
  b = b < d ? d : b;
  b = b < lo ? lo : b;
}

// The lanes' bits of the groups that stay (group g at lanes [g lanes, (g + 1) lanes)).
// `close` is set when a group that stays and one that goes are within `tau`.
template <typename R, int V>
__device__ __forceinline__ uint64_t allowed_groups(const GateArgs& p, const R (&r)[V], R* lds, int lane, R tau, bool* close) {
  const int e0 = lane * V;
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (e0 + v < p.E) lds[e0 + v] = r[v];
  wave_lds_fence();
  const int g = lane / p.lanes, i = lane & (p.lanes - 1);
  R a = -INFINITY, b = -INFINITY;
  if (g < p.groups)
    for (int j = i; j < p.group_size; j += p.lanes) merge_two(a, b, lds[g * p.group_size + j], R(-INFINITY));
  for (int s = 1; s < p.lanes; s *= 2) {
    const R c = __shfl_xor(a, s, 64), d = __shfl_xor(b, s, 64);
    merge_two(a, b, c, d);
  }
  wave_lds_fence();   // the next row writes the area again
  const R score = a + (b == R(-INFINITY) ? R(0) : b);
  int better = 0;
  for (int h = 0; h < p.groups; ++h) {
    const R o = lane_value(score, h * p.lanes);
    better += (o > score) || (o == score && h < g);
  }
  const bool stays = g < p.groups && better < p.topk_groups;
  if (p.topk_groups < p.groups) {
    const R lowest = -wave_max(stays ? -score : R(-INFINITY));
    const R highest = wave_max(g < p.groups && !stays ? score : R(-INFINITY));
    *close = *close || (lowest - highest <= tau);   // -inf - -inf is NaN: equal ranks, not close
  }
  return __ballot(stays);
}

// The row's K best of the ranks r (dead experts -inf, experts that may not be chosen NaN):
// lane j < K ends up with id j. CHECK: sets *close when two of the K + 1 best ranks are
// within tau of each other (rounding may then have put them in the wrong order).
//
// Each lane sorts its V ranks once; then its best is at hand and each of the K rounds is a
// wave maximum, a ballot (the lowest lane holds the lowest index: experts are dealt to
// lanes in order) and a shift in the winning lane.
template <typename R, int V, bool CHECK>
__device__ __forceinline__ int pick(const GateArgs& p, R (&r)[V], int lane, R tau, R tau_rel, bool* close) {
  uint64_t order = 0;   // the local index of r[v], 4 bits each
  int at[V];
#pragma unroll
  for (int v = 0; v < V; ++v) at[v] = v;
#pragma unroll
  for (int n = V - 1; n > 0; --n)   // bubble passes: stable, so equal ranks stay in index order
#pragma unroll
    for (int v = 0; v < n; ++v) {
      const bool sw = r[v + 1] > r[v] || (r[v] != r[v] && r[v + 1] == r[v + 1]);   // NaN last
      const R t = r[v];
      const int u = at[v];
      r[v] = sw ? r[v + 1] : t;
      at[v] = sw ? at[v + 1] : u;
      r[v + 1] = sw ? t : r[v + 1];
      at[v + 1] = sw ? u : at[v + 1];
    }
#pragma unroll
  for (int v = 0; v < V; ++v) order |= (uint64_t)at[v] << (4 * v);
  int mine = 0;
  R last = INFINITY;
  const int rounds = CHECK && p.k < p.E ? p.k + 1 : p.k;
  for (int j = 0; j < rounds; ++j) {
    const R best = wave_max(r[0]);
    if constexpr (CHECK) {
      if (last - best <= tau + tau_rel * fabs(best)) *close = true;
      last = best;
    }
    const uint64_t who = __ballot(r[0] == best);
    if (who == 0) break;   // no rank is left (the host refuses K above the allowed experts)
    const int l = __builtin_ctzll(who);
    const int e = l * V + (__builtin_amdgcn_readlane((int)order, l) & 15);
    if (lane == j) mine = e;
    const bool pop = lane == l;
#pragma unroll
    for (int v = 0; v + 1 < V; ++v) r[v] = pop ? r[v + 1] : r[v];
    r[V - 1] = pop ? R(NAN) : r[V - 1];
    order = pop ? order >> 4 : order;
  }
  return mine;
}

// The ranks in type R; true where the choice is certain.
template <typename R, typename T, int V, bool SOFTMAX, bool CHECK>
__device__ __forceinline__ bool choose(const GateArgs& p, const float (&x)[V], const RowNorm<R>& norm, R* lds, int lane,
                                       int* mine) {
  // Errors of the fp32 ranks (CHECK). A softmax's sum and its reciprocal: less than 45 2^-24
  // (22 additions, the exponents' errors weighted by at most ln 1024), the same factor for all
  // scores of the row; a score's own exponential: less than 4 2^-24 of the largest. A sigmoid:
  // 2^-22. So two scores are off by less than 2^-18 of the largest together, their ranks by
  // their roundings on top; ranks closer than that, and groups' sums of two closer than four
  // times that, are decided in 64 bits.
  const R top = SOFTMAX ? norm.inv : R(1);
  const R tau = CHECK ? top * R(0x1p-18) : R(0), tau_rel = CHECK ? R(0x1p-21) : R(0);
  bool close = false;
  R r[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = lane * V + v;
    r[v] = e < p.E ? score_of<R, SOFTMAX>(x[v], norm) : R(0);
    if (p.bias) r[v] = rank_of(r[v], e < p.E ? p.bias[e] : 0.0f);
    r[v] = x[v] == -INFINITY ? R(-INFINITY) : r[v];
  }
  uint64_t stay = ~0ull;
  if (p.groups > 1) {
    R big = 0;
    if (CHECK && p.bias) {
#pragma unroll
      for (int v = 0; v < V; ++v) big = r[v] == R(-INFINITY) ? big : R(fmax(big, fabs(r[v])));
      big = wave_max(big);
    } else {
      big = top;
    }
    stay = allowed_groups<R, V>(p, r, lds, lane, 4 * (tau + tau_rel * big), &close);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = lane * V + v;
    if (!p.bias) r[v] = R(x[v]);   // the scores rise with the logits, which are exact
    if (p.groups > 1) {
      const int g = p.group_size > 1 ? (int)__umulhi((uint32_t)e, p.group_magic) : e;
      if (!(stay >> ((g * p.lanes) & 63) & 1)) r[v] = R(NAN);
    }
    if (e >= p.E) r[v] = R(NAN);
  }
  if (CHECK && p.bias)
    *mine = pick<R, V, true>(p, r, lane, tau, tau_rel, &close);
  else
    *mine = pick<R, V, false>(p, r, lane, R(0), R(0), &close);
  return !close;
}

// One row by a whole wave.
template <typename T, int V, bool SOFTMAX>
__device__ __forceinline__ void gate_row(const T* __restrict__ logits, const GateArgs& p, int64_t row, double* lds, int lane,
                                         bool vec) {
  const T* rp = logits + row * p.E;
  float x[V];
  load_row<T, V>(rp, p.E, lane, vec, x);
  RowNorm<float> norm{0.0f, 0.0f};
  if constexpr (SOFTMAX) norm = softmax_norm<float, V>(x);
  int mine;
  if (!p.bias && p.groups == 1) {
    float r[V];
#pragma unroll
    for (int v = 0; v < V; ++v) r[v] = lane * V + v < p.E ? x[v] : NAN;
    bool unused = false;
    mine = pick<float, V, false>(p, r, lane, 0.0f, 0.0f, &unused);
  } else if (!choose<float, T, V, SOFTMAX, true>(p, x, norm, reinterpret_cast<float*>(lds), lane, &mine)) {
    RowNorm<double> exact{0.0, 0.0};
    if constexpr (SOFTMAX) exact = softmax_norm<double, V>(x);
    choose<double, T, V, SOFTMAX, false>(p, x, exact, lds, lane, &mine);
  }
  float s = 0.0f;
  if (lane < p.k) {
    const float l = clean(to_float(rp[mine]));
    s = l == -INFINITY ? 0.0f : score_of<float, SOFTMAX>(l, norm);
  }
  float w = s;
  if (p.renorm) {
    const float total = wave_sum(s);
    w = total > 0.0f ? s / total : 0.0f;
  }
  if (lane < p.k) {
    p.ids[row * p.k + lane] = mine;
    p.weights[row * p.k + lane] = w * p.scale;
  }
}

template <typename T, int V, bool SOFTMAX>
__global__ __launch_bounds__(64 * kRowsPerBlock) void gate_kernel(const T* __restrict__ logits, GateArgs p) {
  extern __shared__ double lds_ranks[];   // [waves][E] with groups
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row = p.first + (int64_t)blockIdx.x * kRowsPerBlock + wave;
  if (row >= p.rows) return;
  gate_row<T, V, SOFTMAX>(logits, p, row, lds_ranks + wave * p.E, threadIdx.x & 63, p.vec);
}

// ---- gate, up to 256 experts and K up to 8: four rows a wave ------------------------------
// 16 lanes a row, lane l holding the V experts [l V, l V + V). A rank becomes one 32-bit key:
// the upper 24 bits of its fp32 value in unsigned order, then 255 - index, so a comparison
// is one instruction and equal ranks are in index order. Each lane sorts its keys, and four
// exchanges between lanes merge the lists of the eight largest: about 60 instructions a
// row, where a maximum over the wave for each of the K takes about 20 for each.
// The lower 8 bits that the keys drop and the rounding of the ranks may hide the order of two
// neighbours (not of fp16 or bf16 logits without a bias, which the 24 bits hold exactly): the
// eight and the ninth order themselves by their whole ranks, and where those are within
// their errors by ranks in 64 bits. What stays open, a tenth that near to the K-th or two
// groups that near at the border (a few rows of ten thousand), is decided row by row by
// the whole wave: deciding every near row so took 20 of 34 us at 32768 x 256 in groups, a row of
// a thousand still 9 of 25 (a wave's 8 us at the end of the launch); it is 22 now. So is, although
// its order is plain, a row of fp32 logits or with a bias that has eight live experts or fewer of
// more (8192 such rows of 256: 18 us, others 6).
constexpr int kTop = 8;

__device__ __forceinline__ uint32_t order_key(float r, int e) {
  const int b = __float_as_int(r);
  const uint32_t o = (uint32_t)b ^ ((uint32_t)(b >> 31) | 0x80000000u);
  return (o & 0xffffff00u) | (uint32_t)(255 - e);
}
__device__ __forceinline__ float key_value(uint32_t k) {   // the rank, cut to 24 bits
  const uint32_t o = k & 0xffffff00u;
  return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o & 0xffffff00u);
}

__device__ __forceinline__ void larger_first(uint32_t& a, uint32_t& b) {
  const uint32_t hi = max(a, b), lo = min(a, b);
  a = hi;
  b = lo;
}
// Descending order of a bitonic list of eight.
__device__ __forceinline__ void order_bitonic(uint32_t (&a)[kTop]) {
#pragma unroll
  for (int d = kTop / 2; d > 0; d /= 2)
#pragma unroll
    for (int i = 0; i < kTop; ++i)
      if (!(i & d)) larger_first(a[i], a[i + d]);
}
// Batcher's odd-even merge sort of eight, descending.
__device__ __forceinline__ void order_eight(uint32_t (&a)[kTop]) {
#pragma unroll
  for (int p = 1; p < kTop; p *= 2)
#pragma unroll
    for (int k = p; k > 0; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < kTop; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < kTop && (i + j) / (2 * p) == (i + j + k) / (2 * p)) larger_first(a[i + j], a[i + j + k]);
}
template <int CTRL>
__device__ __forceinline__ uint32_t dppu(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
template <int CTRL>
__device__ __forceinline__ float dppf(float v) { return __uint_as_float(dppu<CTRL>(__float_as_uint(v))); }
// Lane exchanges in a row of 16: neighbours, pairs, fours (mirrored), eights (mirrored).
constexpr int kX1 = 0xB1, kX2 = 0x4E, kX4 = 0x141, kX8 = 0x140;
template <int CTRL>
__device__ __forceinline__ void merge_lanes(uint32_t (&a)[kTop]) {
  uint32_t b[kTop];
#pragma unroll
  for (int i = 0; i < kTop; ++i) b[i] = max(a[i], dppu<CTRL>(a[kTop - 1 - i]));
#pragma unroll
  for (int i = 0; i < kTop; ++i) a[i] = b[i];
  order_bitonic(a);
}
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, dppf<kX1>(v));
  v = fmaxf(v, dppf<kX2>(v));
  v = fmaxf(v, dppf<kX4>(v));
  return fmaxf(v, dppf<kX8>(v));
}
__device__ __forceinline__ float row_sum(float v) {
  v += dppf<kX1>(v);
  v += dppf<kX2>(v);
  v += dppf<kX4>(v);
  return v + dppf<kX8>(v);
}
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  v = max(v, dppu<kX1>(v));
  v = max(v, dppu<kX2>(v));
  v = max(v, dppu<kX4>(v));
  return max(v, dppu<kX8>(v));
}

// The lane's V values of a row of E, by 16-byte loads where they fit (E % V == 0, so that a
// lane's values are all there or none, and the address aligned); past E some value of the row.
template <typename T, int V>
__device__ __forceinline__ void load_part(const T* row, int E, int sub, bool vec, T (&x)[V]) {
  constexpr int W = 16 / sizeof(T) < V ? 16 / sizeof(T) : V;
  typedef T vec_t __attribute__((ext_vector_type(W)));
  if (vec) {
    const T* at = row + (sub * V < E ? sub * V : 0);
#pragma unroll
    for (int c = 0; c < V; c += W) {
      const vec_t u = *reinterpret_cast<const vec_t*>(at + c);
#pragma unroll
      for (int v = 0; v < W; ++v) x[c + v] = u[v];
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = row[min(sub * V + v, E - 1)];
  }
}

// The logits of load_part as the operators take them; experts past E are -inf.
template <typename T, int V>
__device__ __forceinline__ void clean_part(const T (&raw)[V], int E, int sub, float (&x)[V]) {
#pragma unroll
  for (int v = 0; v < V; ++v) x[v] = clean(to_float(raw[v]));
  if (E < 16 * V) {   // uniform
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = sub * V + v < E ? x[v] : -INFINITY;
  }
}

// Where the order of a lane's experts does not matter they are dealt in 16-byte pieces (W
// values), so that a wave's loads and stores run along the rows: value v of lane `sub` is
// expert dealt<W>(sub, v). (The gradient of 32768 x 256 fp32 rows with 64 contiguous bytes a
// lane: 21 us, dealt: 16.)
template <typename T, int V> constexpr int kPiece = 16 / (int)sizeof(T) < V ? 16 / (int)sizeof(T) : V;
template <int W>
__device__ __forceinline__ int dealt(int sub, int v) { return v / W * 16 * W + sub * W + v % W; }

// VEC: every piece is whole and aligned (E % W == 0); past E some value of the row.
template <typename T, int V, int W>
__device__ __forceinline__ void load_dealt(const T* row, int E, int sub, bool vec, T (&x)[V]) {
  constexpr int N = 16 / (int)sizeof(T) < W ? 16 / (int)sizeof(T) : W;
  typedef T vec_t __attribute__((ext_vector_type(N)));
  if (vec) {
#pragma unroll
    for (int v = 0; v < V; v += N) {
      const int e = dealt<W>(sub, v);
      const vec_t u = *reinterpret_cast<const vec_t*>(row + (e < E ? e : 0));
#pragma unroll
      for (int i = 0; i < N; ++i) x[v + i] = u[i];
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = row[min(dealt<W>(sub, v), E - 1)];
  }
}
template <typename T, int V, int W>
__device__ __forceinline__ void clean_dealt(const T (&raw)[V], int E, int sub, float (&x)[V]) {
#pragma unroll
  for (int v = 0; v < V; ++v) x[v] = clean(to_float(raw[v]));
  if (E < 16 * V) {   // uniform
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = dealt<W>(sub, v) < E ? x[v] : -INFINITY;
  }
}

__device__ __forceinline__ double row_sum(double v) {
  for (int d = 1; d < 16; d *= 2) v += __shfl_xor(v, d, 64);
  return v;
}

// softmax_norm of a row held by 16 lanes.
template <typename R, int V>
__device__ __forceinline__ RowNorm<R> row_norm(const float (&x)[V]) {
  float m = x[0];
#pragma unroll
  for (int v = 1; v < V; ++v) m = fmaxf(m, x[v]);
  m = fmaxf(row_max(m), -FLT_MAX);   // (a row of -inf only: exp(-inf) = 0 throughout)
  R sum = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) sum += exp_of(R(x[v]) - R(m));
  sum = row_sum(sum);
  return RowNorm<R>{R(m), sum > R(0) ? R(1) / sum : R(0)};
}

template <typename T, int V, bool SOFTMAX, bool BIAS>
__global__ __launch_bounds__(64 * kRowsPerBlock) void gate16_kernel(const T* __restrict__ logits, GateArgs p, bool vec64, bool vec_bias) {
  extern __shared__ double lds_ranks[];   // [waves][E] with groups
  const int lane = threadIdx.x & 63, sub = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row0 = p.first + ((int64_t)blockIdx.x * kRowsPerBlock + wave) * 4;
  if (row0 >= p.rows) return;
  const int64_t row = min(row0 + (lane >> 4), p.rows - 1);
  const bool there = row0 + (lane >> 4) < p.rows;
  const T* rp = logits + row * p.E;
  float x[V];
  {
    T raw[V];
    load_part<T, V>(rp, p.E, sub, p.vec, raw);
    clean_part<T, V>(raw, p.E, sub, x);
  }
  RowNorm<float> norm{0.0f, 0.0f};
  if constexpr (SOFTMAX) norm = row_norm<float, V>(x);
  const float top = SOFTMAX ? norm.inv : 1.0f;
  // What two scores can be off together, relative to the largest, with some room. A sigmoid: t = exp(-l)
  // is off by (1.5 |l| + 2) 2^-24 of itself, which s (1 - s) <= 1/4 and s (1 - s) |l| < 0.23 make
  // less than 2^-24, 1 + t by another, the reciprocal by 2^-23: 2^-22. A softmax: its sum's
  // roundings and the exponents' errors, weighted by at most ln E, come to less than 2^-18.6.
  constexpr float kScoreError = SOFTMAX ? 0x1p-17f : 0x1p-20f;
  float r[V];
  bool redo = false;   // decided by the whole wave
  bool stays = true;
  const bool groups = p.groups > 1;   // uniform
  if (BIAS || groups) {
#pragma unroll
    for (int v = 0; v < V; ++v) r[v] = score_of<float, SOFTMAX>(x[v], norm);
    if constexpr (BIAS) {
      float bias[V];
      load_part<float, V>(p.bias, p.E, sub, vec_bias, bias);
#pragma unroll
      for (int v = 0; v < V; ++v) r[v] = rank_of(r[v], bias[v]);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) r[v] = x[v] == -INFINITY ? -INFINITY : r[v];
  }
  if (groups) {   // a group is `lanes` whole lanes (a power of two)
    float a = -INFINITY, b = -INFINITY, big = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      merge_two(a, b, r[v], -INFINITY);
      big = fmaxf(big, r[v] == -INFINITY ? 0.0f : fabsf(r[v]));
    }
    if (p.lanes > 1) merge_two(a, b, dppf<kX1>(a), dppf<kX1>(b));
    if (p.lanes > 2) merge_two(a, b, dppf<kX2>(a), dppf<kX2>(b));
    if (p.lanes > 4) merge_two(a, b, dppf<kX4>(a), dppf<kX4>(b));
    const float score = a + (b == -INFINITY ? 0.0f : b);
    // two sums of two ranks each: four scores' errors, and 8 roundings of at most `big` 2^-24
    const float tau = 2 * kScoreError * top + row_max(big) * 0x1p-20f;
    const int shift = __builtin_ctz(p.lanes), g = sub >> shift;
    int better = 0;
    auto against = [&]<int L>(std::integral_constant<int, L>) {
      const int h = L >> shift;
      if ((L & (p.lanes - 1)) == 0 && h < p.groups) {   // uniform
        const float o = dppf<0x150 + L>(score);   // lane L of each row of 16
        better += (int)(o > score) | ((int)(o == score) & (int)(h < g));
      }
    };
    [&]<int... L>(std::integer_sequence<int, L...>) { (against(std::integral_constant<int, L>{}), ...); }
    (std::make_integer_sequence<int, 16>{});
    stays = (better < p.topk_groups) & (g < p.groups);
    const float lowest = -row_max(stays ? -score : -INFINITY);
    const float highest = row_max((!stays & (g < p.groups)) ? score : -INFINITY);
    redo = lowest - highest <= tau;   // (-inf - -inf, NaN: equal groups, in index order)
  }
  uint32_t key[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    key[v] = order_key(BIAS ? r[v] : x[v], sub * V + v);   // without a bias the scores rise with the logits
    key[v] = stays ? key[v] : 0u;
  }
  if (p.E < 16 * V) {
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = sub * V + v < p.E ? key[v] : 0u;
  }
  uint32_t best[kTop];
  if constexpr (V == 16) {
    uint32_t hi[kTop];
#pragma unroll
    for (int i = 0; i < kTop; ++i) best[i] = key[i], hi[i] = key[kTop + i];
    order_eight(best);
    order_eight(hi);
#pragma unroll
    for (int i = 0; i < kTop; ++i) best[i] = max(best[i], hi[kTop - 1 - i]);
    order_bitonic(best);
  } else {
#pragma unroll
    for (int i = 0; i < kTop; ++i) best[i] = i < V ? key[i < V ? i : 0] : 0u;
    order_eight(best);
  }
  merge_lanes<kX1>(best);
  merge_lanes<kX2>(best);
  merge_lanes<kX4>(best);
  merge_lanes<kX8>(best);
  // Lane j of a row: candidate j, the eight best and the one after them.
  uint32_t mine = best[0];
#pragma unroll
  for (int i = 1; i < kTop; ++i) mine = sub == i ? best[i] : mine;
  constexpr bool kCut = BIAS || sizeof(T) == 4;   // keys may hide an order
  constexpr int kCandidates = kCut ? kTop + 1 : kTop;
  auto next_key = [&](uint32_t after) {   // the row's largest key below `after`
    uint32_t k = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) k = max(k, key[v] < after ? key[v] : 0u);
    return row_max(k);
  };
  uint32_t ninth = 0;
  if constexpr (kCut) {
    ninth = next_key(best[kTop - 1]);
    mine = sub == kTop ? ninth : mine;
  }
  const bool held = (sub < kCandidates) & (mine != 0u);
  const int id = 255 - (int)(mine & 255u);
  const float l = held ? clean(to_float(rp[held ? id : 0])) : -INFINITY;
  const float s = l == -INFINITY ? 0.0f : score_of<float, SOFTMAX>(l, norm);
  int at = sub;   // its place in the row
  if constexpr (kCut) {
    const float tau = BIAS ? kScoreError * top : 0.0f;
    // what is no candidate has to be clear of the K-th choice
    uint32_t kth = best[0];
#pragma unroll
    for (int i = 1; i < kTop; ++i) kth = p.k == i + 1 ? best[i] : kth;
    auto near = [&](uint32_t beyond) {
      const float u = key_value(kth), w = key_value(beyond);
      return (beyond != 0u) & !(u - w > tau + 0x1p-14f * fmaxf(fabsf(u), fabsf(w)));
    };
    if (__ballot(near(ninth))) redo |= near(next_key(ninth));
    // the candidates' order by their whole ranks, and where those are within their errors by
    // ranks in 64 bits
    const float b = BIAS && held ? p.bias[id] : 0.0f;
    const float rank = !held ? NAN : BIAS ? (l == -INFINITY ? -INFINITY : rank_of(s, b)) : l;
    const float reach = tau + fabsf(rank) * 0x1p-21f;
    bool close = false;
    at = 0;
    auto against = [&]<int L>(std::integral_constant<int, L>) {
      const float o = dppf<0x150 + L>(rank);
      const int oid = (int)dppu<0x150 + L>((uint32_t)id);
      at += (int)(o > rank) | ((int)(o == rank) & (int)(oid < id));
      if constexpr (BIAS) close |= (L != sub) & (fabsf(o - rank) <= reach);
    };
    auto against_all = [&]<int... L>(std::integer_sequence<int, L...>) { (against(std::integral_constant<int, L>{}), ...); };
    against_all(std::make_integer_sequence<int, kCandidates>{});
    if (BIAS && __ballot(close)) {
      RowNorm<double> exact{0.0, 0.0};
      if constexpr (SOFTMAX) exact = row_norm<double, V>(x);
      const double r64 = rank == rank && l > -INFINITY ? rank_of(score_of<double, SOFTMAX>(l, exact), b) : (double)rank;
      const uint64_t bits = __builtin_bit_cast(uint64_t, r64);
      at = 0;
      auto against64 = [&]<int L>(std::integral_constant<int, L>) {
        const uint64_t u = ((uint64_t)dppu<0x150 + L>((uint32_t)(bits >> 32)) << 32) | dppu<0x150 + L>((uint32_t)bits);
        const double o = __builtin_bit_cast(double, u);
        const int oid = (int)dppu<0x150 + L>((uint32_t)id);
        at += (int)(o > r64) | ((int)(o == r64) & (int)(oid < id));
      };
      [&]<int... L>(std::integer_sequence<int, L...>) { (against64(std::integral_constant<int, L>{}), ...); }
      (std::make_integer_sequence<int, kCandidates>{});
    }
  }
  const bool chosen = held & (at < p.k);
  float weight = chosen ? s : 0.0f;
  if (p.renorm) {
    const float total = row_sum(weight);
    weight = total > 0.0f ? weight / total : 0.0f;
  }
  uint64_t again = __ballot(redo & there);   // the same for the lanes of a row
  if (chosen & there & !redo) {
    p.ids[row * p.k + at] = id;
    p.weights[row * p.k + at] = weight * p.scale;
  }
  GateArgs q = p;   // the wave's own lanes a group
  q.lanes = 64;
  while (64 / q.lanes < q.groups) q.lanes /= 2;
  while (again) {
    const int i = __builtin_ctzll(again) >> 4;
    again &= ~(0xffffull << (16 * i));
    gate_row<T, (V + 3) / 4, SOFTMAX>(logits, q, row0 + i, lds_ranks + wave * p.E, lane, vec64);
  }
}

// ---- sequences ------------------------------------------------------------------------
// Rows [lo, hi) of sequence b, clamped into [0, rows).
__device__ __forceinline__ void seq_rows(const int32_t* off, int b, int64_t rows, int64_t* lo, int64_t* hi) {
  if (!off) {
    *lo = 0;
    *hi = rows;
    return;
  }
  *lo = min(max((int64_t)off[b], (int64_t)0), rows);
  *hi = min(max((int64_t)off[b + 1], *lo), rows);
}

// ---- balance loss ---------------------------------------------------------------------
// First pass: block (s, b) sums the scores and counts the choices of its share of sequence
// b's rows: one partial row each, in the same order on every call. A share has no upper limit
// (one sequence may hold all rows of many), so a lane adds only kSumRows rows in fp32 and then
// joins them to a sum in 64 bits in LDS: fp32 throughout was off by 2^-15 after 2048 equal rows.
// The partial row is rounded to fp32 once.
constexpr int kSumRows = 16;

template <typename T, int V, bool SOFTMAX>
__global__ __launch_bounds__(64 * kRowsPerBlock) void balance_sums_kernel(
    const T* __restrict__ logits, int64_t rows, int E, bool vec, const int32_t* __restrict__ ids, int k,
    const int32_t* __restrict__ off, const uint8_t* __restrict__ mask, float* __restrict__ sums,
    int32_t* __restrict__ counts, int32_t* __restrict__ held, unsigned* __restrict__ done) {
  // [waves] sums, then [E] counts; a lane's V sums lie V + 1 apart from the next lane's, so that
  // the lanes meet different banks (8192 x 1024, with V: 23.5 us, with V + 1: 21.3)
  extern __shared__ double lds_sums[];
  constexpr int kSums = 64 * (V + 1);
  const auto place = [](int e) { return e / V * (V + 1) + e % V; };
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int* hist = reinterpret_cast<int*>(lds_sums + kRowsPerBlock * kSums);
  const int b = blockIdx.y, splits = gridDim.x, s = blockIdx.x;
  if (threadIdx.x == 0 && s == 0 && b == 0) *done = 0;
  for (int e = threadIdx.x; e < E; e += blockDim.x) hist[e] = 0;
  __syncthreads();
  int64_t lo, hi;
  seq_rows(off, b, rows, &lo, &hi);
  const int64_t len = hi - lo, first = lo + len * s / splits, last = lo + len * (s + 1) / splits;
  float acc[V] = {};
  int seen = 0;
  bool joined = false;
  auto join = [&]() {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (lane * V + v < E) {
        double& sum = lds_sums[wave * kSums + lane * (V + 1) + v];
        sum = (joined ? sum : 0.0) + (double)acc[v];
      }
      acc[v] = 0.0f;
    }
    joined = true;
  };
  for (int64_t row = first + wave; row < last; row += kRowsPerBlock) {
    if (mask && mask[row] == 0) continue;   // uniform per wave
    if (seen > 0 && seen % kSumRows == 0) join();
    ++seen;
    float x[V];
    load_row<T, V>(logits + row * E, E, lane, vec, x);
    if (lane < k) {
      const int id = ids[row * k + lane];
      if ((unsigned)id < (unsigned)E) atomicAdd(&hist[id], 1);
    }
    if constexpr (SOFTMAX) {
      const RowNorm<float> n = softmax_norm<float, V>(x);
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] += score_of<float, true>(x[v], n);
    } else {
      float sc[V], z = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        sc[v] = score_of<float, false>(x[v], RowNorm<float>{});
        z += sc[v];
      }
      z = wave_sum(z);
      const float inv = z > 0.0f ? 1.0f / z : 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] += sc[v] * inv;
    }
  }
  join();
  __shared__ int rows_seen[kRowsPerBlock];
  if (lane == 0) rows_seen[wave] = seen;
  __syncthreads();
  const int64_t part = (int64_t)b * splits + s;
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    double t = 0.0;
#pragma unroll
    for (int w = 0; w < kRowsPerBlock; ++w) t += lds_sums[w * kSums + place(e)];
    sums[part * E + e] = (float)t;
    counts[part * E + e] = hist[e];
  }
  if (threadIdx.x == 0) {
    int t = 0;
    for (int w = 0; w < kRowsPerBlock; ++w) t += rows_seen[w];
    held[part] = t;
  }
}

// The same for up to 256 experts, four rows a wave (16 lanes each, as gate16_kernel), the
// next rows' logits loaded before these are summed.
template <typename T, int V, bool SOFTMAX>
__global__ __launch_bounds__(64 * kRowsPerBlock) void balance16_sums_kernel(
    const T* __restrict__ logits, int64_t rows, int E, bool vec, const int32_t* __restrict__ ids, int k,
    const int32_t* __restrict__ off, const uint8_t* __restrict__ mask, float* __restrict__ sums,
    int32_t* __restrict__ counts, int32_t* __restrict__ held, unsigned* __restrict__ done) {
  constexpr int W = kPiece<T, V>;
  __shared__ double lds_sums[kRowsPerBlock][16 * V];
  __shared__ int hist[16 * V];
  __shared__ int rows_seen[kRowsPerBlock];
  const int lane = threadIdx.x & 63, sub = lane & 15, part = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int b = blockIdx.y, splits = gridDim.x, s = blockIdx.x;
  if (threadIdx.x == 0 && s == 0 && b == 0) *done = 0;
  for (int e = threadIdx.x; e < 16 * V; e += blockDim.x) hist[e] = 0;
  __syncthreads();
  int64_t lo, hi;
  seq_rows(off, b, rows, &lo, &hi);
  const int64_t len = hi - lo, first = lo + len * s / splits, last = lo + len * (s + 1) / splits;
  float acc[V] = {};
  int seen = 0;
  struct Rows {   // four rows, past the end the last one
    T raw[V];
    int id[2];
    uint8_t counted;
  };
  auto load = [&](int64_t at, Rows& r) {
    const int64_t row = min(at + part, last - 1);
    load_dealt<T, V, W>(logits + row * E, E, sub, vec, r.raw);
#pragma unroll
    for (int i = 0; i < 2; ++i) r.id[i] = sub + 16 * i < k ? ids[row * k + sub + 16 * i] : -1;
    r.counted = (at + part < last) & ((mask ? mask[row] : 1) != 0);
  };
  int rounds = 0;
  auto join = [&]() {   // the wave's sums, of its four rows at a time
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float t = acc[v];
      t += __shfl_xor(t, 16, 64);
      t += __shfl_xor(t, 32, 64);
      if (part == 0) {
        double& sum = lds_sums[wave][dealt<W>(sub, v)];
        sum = (rounds > kSumRows ? sum : 0.0) + (double)t;
      }
      acc[v] = 0.0f;
    }
  };
  int64_t at = first + 4 * wave;
  Rows cur;
  if (at < last) load(at, cur);
  for (; at < last; at += 4 * kRowsPerBlock) {
    if (rounds > 0 && rounds % kSumRows == 0) join();
    ++rounds;
    Rows next;
    if (at + 4 * kRowsPerBlock < last) load(at + 4 * kRowsPerBlock, next);
    const bool counted = cur.counted;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (counted && (unsigned)cur.id[i] < (unsigned)E) atomicAdd(&hist[cur.id[i]], 1);
    seen += counted && sub == 0;
    float x[V];
    clean_dealt<T, V, W>(cur.raw, E, sub, x);
    if constexpr (SOFTMAX) {
      RowNorm<float> n = row_norm<float, V>(x);
      if (!counted) n.inv = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] += score_of<float, true>(x[v], n);
    } else {
      float sc[V], z = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        sc[v] = score_of<float, false>(x[v], RowNorm<float>{});
        z += sc[v];
      }
      z = row_sum(z);
      const float inv = counted && z > 0.0f ? 1.0f / z : 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] += sc[v] * inv;
    }
    cur = next;
  }
  join();
  const int rows_of_wave = __popcll(__ballot(seen & 1)) + 2 * __popcll(__ballot(seen & 2)) + 4 * __popcll(__ballot(seen & 4));
  int more = seen >> 3;   // (over 7 row quads a wave: long sequences)
  for (int d = 1; d < 64; d *= 2) more += __shfl_xor(more, d, 64);
  if (lane == 0) rows_seen[wave] = rows_of_wave + 8 * more;
  __syncthreads();
  const int64_t to = (int64_t)b * splits + s;
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    double t = 0.0;
#pragma unroll
    for (int w = 0; w < kRowsPerBlock; ++w) t += lds_sums[w][e];
    sums[to * E + e] = (float)t;
    counts[to * E + e] = hist[e];
  }
  if (threadIdx.x == 0) {
    int t = 0;
    for (int w = 0; w < kRowsPerBlock; ++w) t += rows_seen[w];
    held[to] = t;
  }
}

constexpr int kFinishThreads = 512;
// Experts of a block of the second pass: 16 of many partials, because one compute unit takes no
// more than about 20 GB/s of them from memory (512 partials of 256 experts: 13.4 us on 4 blocks,
// 8.7 on 16; 1024 of 512: 21.8, 10.3), else 64, where fewer blocks make the join of the loss
// cheaper (8 sequences of 128 partials: both passes 21.5 us, with 16 23.4; 63 partials of 60
// experts, one block: 7.9, 4 blocks 10.3).
constexpr int finish_experts(int splits) { return splits > 256 ? 16 : 64; }

__device__ __forceinline__ double block_sum(double v, double* lds) {
  v = wave_sum(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  double t = 0;
  for (int w = 0; w < kFinishThreads / 64; ++w) t += lds[w];
  return t;
}

// Second pass: block (c, b) joins the partials of W experts of sequence b; the last block
// to end adds the blocks' shares of the loss, in order.
template <int W>
__global__ __launch_bounds__(kFinishThreads) void balance_finish_kernel(
    int E, int k, int splits, int seqs, int lanes, const float* __restrict__ sums, const int32_t* __restrict__ counts_part,
    const int32_t* __restrict__ held, float alpha, double* __restrict__ shares, unsigned* __restrict__ done,
    float* __restrict__ loss, int32_t* __restrict__ counts, float* __restrict__ coef) {
  constexpr int kSlices = kFinishThreads / W, kAhead = W == 16 ? 8 : 4;   // (partials in flight a thread)
  __shared__ double lds_p[kSlices][W];
  __shared__ int lds_c[kSlices][W];
  __shared__ double lds_w[kFinishThreads / 64];
  __shared__ int lds_rows, lds_filled;
  const int b = blockIdx.y, lane = threadIdx.x & 63, slice = threadIdx.x / W, of = threadIdx.x % W;
  if (threadIdx.x == 0) lds_rows = lds_filled = 0;
  // this block's partials first: their loads are under way while the rows are counted
  const int e = blockIdx.x * W + of;
  double p = 0;
  int c = 0;
  if (e < E)
#pragma unroll kAhead
    for (int s = slice; s < splits; s += kSlices) {
      p += sums[((int64_t)b * splits + s) * E + e];
      c += counts_part[((int64_t)b * splits + s) * E + e];
    }
  __syncthreads();
  // sequences with a counted row, and this one's rows: `lanes` lanes a sequence
  int filled = 0;
  for (int q0 = 0; q0 < seqs; q0 += kFinishThreads / lanes) {
    const int q = q0 + threadIdx.x / lanes;
    int t = 0;
    if (q < seqs)
#pragma unroll 8
      for (int s = threadIdx.x % lanes; s < splits; s += lanes) t += held[(int64_t)q * splits + s];
    for (int d = 1; d < lanes; d *= 2) t += __shfl_xor(t, d, 64);
    const bool first = threadIdx.x % lanes == 0 && q < seqs;
    filled += __popcll(__ballot(first && t > 0));
    if (first && q == b) lds_rows = t;
  }
  if (lane == 0) atomicAdd(&lds_filled, filled);
  lds_p[slice][of] = p;
  lds_c[slice][of] = c;
  __syncthreads();
  __shared__ bool last;
  if (threadIdx.x < 64) {
    const double rows = lds_rows;
    const double f = rows > 0 ? (double)alpha * E / ((double)k * rows * rows * lds_filled) : 0.0;
    double total = 0;
    const bool mine = slice == 0 && e < E;
    if (mine) {
      for (int a = 1; a < kSlices; ++a) {
        p += lds_p[a][of];
        c += lds_c[a][of];
      }
      total = f * c * p;
    }
    const double share = wave_sum(total);
    if (lane == 0) {
      if (gridDim.x * gridDim.y == 1) {
        *loss = (float)share;
        last = false;
      } else {   // (before the other stores: the fence would wait for them)
        shares[(int64_t)b * gridDim.x + blockIdx.x] = share;
        __threadfence();
        last = atomicAdd(done, 1u) == gridDim.x * gridDim.y - 1;
      }
    }
    if (mine) {
      counts[(int64_t)b * E + e] = c;
      coef[(int64_t)b * E + e] = (float)(f * c);
    }
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  double t = 0;
  for (int64_t q = threadIdx.x; q < (int64_t)seqs * gridDim.x; q += kFinishThreads)
    t += __hip_atomic_load(&shares[q], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  t = block_sum(t, lds_w);
  if (threadIdx.x == 0) *loss = (float)t;
}

// ---- gradient -------------------------------------------------------------------------
struct GateGradArgs {
  int64_t first, rows;         // the launch's rows: [first, rows)
  int E, k;
  bool renorm, vec;
  float scale;
  const int32_t* ids;
  const float* grad_weights;   // nullable
  const float* grad_loss;      // nullable [1]; with coef
  const float* coef;           // [seqs, E]
  const int32_t* off;          // nullable
  int seqs;
  const uint8_t* mask;         // nullable
};

template <typename T>
__device__ __forceinline__ T value_as(float v) {
  if constexpr (std::is_same_v<T, uint16_t>)
    return (uint16_t)bf16x2(v, v);
  else
    return (T)v;
}

// Every term of the gradient is a gradient times a score, or times a quotient of a score by a
// sum of them: c_j = g_j s_j (renormalised: (scale dw_j - sum_i scale dw_i w_i) w_j with w_j =
// s_j / S), q_e p_e, and 1 - s for a sigmoid. A sigmoid's sums may lie near fp32's smallest, so
// that a gradient over them, the other way to write this, would overflow. A sum below 2^-126
// (its reciprocal overflows) counts as 0, like its scores.
__device__ __forceinline__ float inverse_sum(float sum) { return sum >= FLT_MIN ? 1.0f / sum : 0.0f; }
// 1 - s of a sigmoid, also of a score near 1, with t = exp(-|l|).
__device__ __forceinline__ float sigmoid_rest(float l) {
  const float t = exp_of(-fabsf(l)), r = 1.0f / (1.0f + t);
  return l > 0.0f ? t * r : r;
}

// The sequence of a row (-1: none): the last that starts at or before it, if it holds it.
__device__ __forceinline__ int row_seq(const int32_t* off, int seqs, int64_t row) {
  if (!off) return 0;
  int lo = 0, hi = seqs;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= row)
      lo = mid;
    else
      hi = mid;
  }
  return off[lo] <= row && row < off[lo + 1] ? lo : -1;
}

template <typename T, int V, bool SOFTMAX>
__global__ __launch_bounds__(64 * kRowsPerBlock) void gate_backward_kernel(const T* __restrict__ logits, GateGradArgs p,
                                                                           T* __restrict__ grad) {
  extern __shared__ float lds_grad[];   // [waves][64 V]
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row = p.first + (int64_t)blockIdx.x * kRowsPerBlock + wave;
  if (row >= p.rows) return;
  const T* rp = logits + row * p.E;
  float x[V], s[V], d[V];
  load_row<T, V>(rp, p.E, lane, p.vec, x);
  RowNorm<float> norm{0.0f, 0.0f};
  if constexpr (SOFTMAX) norm = softmax_norm<float, V>(x);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    s[v] = x[v] == -INFINITY ? 0.0f : score_of<float, SOFTMAX>(x[v], norm);
    d[v] = 0.0f;
  }
  if (p.grad_weights) {
    float* area = lds_grad + wave * 64 * V;
#pragma unroll
    for (int v = 0; v < V; ++v) area[lane * V + v] = 0.0f;
    wave_lds_fence();
    int id = -1;
    float g = 0.0f, sc = 0.0f;
    if (lane < p.k) {
      id = p.ids[row * p.k + lane];
      if ((unsigned)id >= (unsigned)p.E) id = -1;
      g = id >= 0 ? p.grad_weights[row * p.k + lane] * p.scale : 0.0f;
      const float l = id >= 0 ? clean(to_float(rp[id])) : -INFINITY;
      sc = l == -INFINITY ? 0.0f : score_of<float, SOFTMAX>(l, norm);
    }
    if (p.renorm) {
      sc *= inverse_sum(wave_sum(sc));
      g -= wave_sum(g * sc);
    }
    if (id >= 0) atomicAdd(&area[id], g * sc);   // (an id may stand in several places; one wave: a fixed order)
    wave_lds_fence();
#pragma unroll
    for (int v = 0; v < V; ++v) d[v] = area[lane * V + v];
  }
  float q[V];
#pragma unroll
  for (int v = 0; v < V; ++v) q[v] = 0.0f;
  if (p.grad_loss && !(p.mask && p.mask[row] == 0)) {
    const int b = row_seq(p.off, p.seqs, row);
    if (b >= 0) {
      const float gl = *p.grad_loss;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int e = lane * V + v;
        q[v] = e < p.E ? gl * p.coef[(int64_t)b * p.E + e] : 0.0f;
      }
    }
  }
  if constexpr (SOFTMAX) {
    float dot = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      d[v] += q[v] * s[v];
      dot += d[v];
    }
    dot = wave_sum(dot);
#pragma unroll
    for (int v = 0; v < V; ++v) d[v] -= s[v] * dot;
  } else {
    float dot = 0.0f, z = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) z += s[v];
    const float inv = inverse_sum(wave_sum(z));
#pragma unroll
    for (int v = 0; v < V; ++v) {
      s[v] *= inv;
      dot += q[v] * s[v];
    }
    dot = wave_sum(dot);
#pragma unroll
    for (int v = 0; v < V; ++v) d[v] = (d[v] + (q[v] - dot) * s[v]) * sigmoid_rest(x[v]);
  }
  T* out = grad + row * p.E;
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (lane * V + v < p.E) out[lane * V + v] = value_as<T>(d[v]);
}

// Up to 256 experts: four rows a wave (16 lanes each, as gate16_kernel).
template <typename T, int V, bool SOFTMAX>
__global__ __launch_bounds__(64 * kRowsPerBlock) void gate16_backward_kernel(const T* __restrict__ logits, GateGradArgs p,
                                                                             bool vec_coef, T* __restrict__ grad) {
  constexpr int W = kPiece<T, V>, N = W < 4 ? W : 4;
  typedef float part_t __attribute__((ext_vector_type(N)));
  __shared__ __align__(16) float lds_grad[4 * kRowsPerBlock][16 * V];
  const int lane = threadIdx.x & 63, sub = lane & 15, part = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row0 = p.first + ((int64_t)blockIdx.x * kRowsPerBlock + wave) * 4;
  if (row0 >= p.rows) return;
  const int64_t row = min(row0 + part, p.rows - 1);
  const T* rp = logits + row * p.E;
  T raw[V];
  load_dealt<T, V, W>(rp, p.E, sub, p.vec, raw);
  int id[2] = {-1, -1};
  float g[2] = {0.0f, 0.0f}, sc[2] = {0.0f, 0.0f}, l[2];
  if (p.grad_weights) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {   // choices sub and sub + 16 of the row
      const int j = sub + 16 * i;
      if (j < p.k) {
        id[i] = p.ids[row * p.k + j];
        if ((unsigned)id[i] >= (unsigned)p.E) id[i] = -1;
        g[i] = id[i] >= 0 ? p.grad_weights[row * p.k + j] * p.scale : 0.0f;
      }
      l[i] = id[i] >= 0 ? clean(to_float(rp[max(id[i], 0)])) : -INFINITY;
    }
  }
  const int seq = p.grad_loss && !(p.mask && p.mask[row] == 0) ? row_seq(p.off, p.seqs, row) : -1;
  float q[V];
#pragma unroll
  for (int v = 0; v < V; ++v) q[v] = 0.0f;
  if (seq >= 0) {
    const float gl = *p.grad_loss;
    load_dealt<float, V, W>(p.coef + (int64_t)seq * p.E, p.E, sub, vec_coef, q);
#pragma unroll
    for (int v = 0; v < V; ++v) q[v] *= gl;
  }
  float x[V], s[V], d[V];
  clean_dealt<T, V, W>(raw, p.E, sub, x);
  RowNorm<float> norm{0.0f, 0.0f};
  if constexpr (SOFTMAX) norm = row_norm<float, V>(x);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    s[v] = score_of<float, SOFTMAX>(x[v], norm);
    d[v] = 0.0f;
  }
  if (p.grad_weights) {
    float* area = lds_grad[wave * 4 + part];
#pragma unroll
    for (int v = 0; v < V; v += N) *reinterpret_cast<part_t*>(area + dealt<W>(sub, v)) = part_t{};
    wave_lds_fence();
#pragma unroll
    for (int i = 0; i < 2; ++i) sc[i] = l[i] == -INFINITY ? 0.0f : score_of<float, SOFTMAX>(l[i], norm);
    if (p.renorm) {
      const float inv = inverse_sum(row_sum(sc[0] + sc[1]));
#pragma unroll
      for (int i = 0; i < 2; ++i) sc[i] *= inv;
      const float mean = row_sum(g[0] * sc[0] + g[1] * sc[1]);
#pragma unroll
      for (int i = 0; i < 2; ++i) g[i] -= mean;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (id[i] >= 0) atomicAdd(&area[id[i]], g[i] * sc[i]);   // (an id may stand in several places)
    wave_lds_fence();
#pragma unroll
    for (int v = 0; v < V; v += N) {
      const part_t u = *reinterpret_cast<const part_t*>(area + dealt<W>(sub, v));
#pragma unroll
      for (int j = 0; j < N; ++j) d[v + j] = u[j];
    }
  }
  if constexpr (SOFTMAX) {
    float dot = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      d[v] += q[v] * s[v];
      dot += d[v];
    }
    dot = row_sum(dot);
#pragma unroll
    for (int v = 0; v < V; ++v) d[v] -= s[v] * dot;
  } else {
    float dot = 0.0f, z = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) z += s[v];
    const float inv = inverse_sum(row_sum(z));
#pragma unroll
    for (int v = 0; v < V; ++v) {
      s[v] *= inv;
      dot += q[v] * s[v];
    }
    dot = row_sum(dot);
#pragma unroll
    for (int v = 0; v < V; ++v) d[v] = (d[v] + (q[v] - dot) * s[v]) * sigmoid_rest(x[v]);
  }
  if (row0 + part >= p.rows) return;
  T* out = grad + row * p.E;
  if (p.vec) {
    typedef T vec_t __attribute__((ext_vector_type(W)));
#pragma unroll
    for (int v = 0; v < V; v += W) {
      vec_t u;
#pragma unroll
      for (int j = 0; j < W; ++j) u[j] = value_as<T>(d[v + j]);
      if (dealt<W>(sub, v) < p.E) *reinterpret_cast<vec_t*>(out + dealt<W>(sub, v)) = u;
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (dealt<W>(sub, v) < p.E) out[dealt<W>(sub, v)] = value_as<T>(d[v]);
  }
}

// V = experts a lane: the smallest power of two with 64 V >= E. The loss and the gradient come
// here above 256 experts only (with_wide), the gate also for what its 16 lanes cannot do.
template <typename F>
hipError_t with_wide(int E, F&& f) {
  if (E <= 512) return f(std::integral_constant<int, 8>{});
  return f(std::integral_constant<int, 16>{});
}
template <typename F>
hipError_t with_width(int E, F&& f) {
  if (E <= 64) return f(std::integral_constant<int, 1>{});
  if (E <= 128) return f(std::integral_constant<int, 2>{});
  if (E <= 256) return f(std::integral_constant<int, 4>{});
  return with_wide(E, f);
}
// Experts a lane of the kernels with 16 lanes a row (up to 256 experts).
constexpr int kMost16 = 256;
template <typename F>
hipError_t with_width16(int E, F&& f) {
  if (E <= 64) return f(std::integral_constant<int, 4>{});
  if (E <= 128) return f(std::integral_constant<int, 8>{});
  return f(std::integral_constant<int, 16>{});
}
template <typename F>
hipError_t with_type(int dtype, F&& f) {
  switch (dtype) {
    case 0: return f((const float*)nullptr);
    case 1: return f((const _Float16*)nullptr);
    default: return f((const uint16_t*)nullptr);
  }
}
// A launch has at most 2^32 - 1 threads along x (the runtime takes more without an error and
// leaves the rows past them undone), and a row takes up to 64: calls of more than kLaunchRows
// rows are several launches. `launch` gets the first row and the end of each.
constexpr int64_t kLaunchRows = 1 << 25;
template <typename F>
hipError_t in_launches(int64_t rows, F&& launch) {
  for (int64_t first = 0; first < rows; first += kLaunchRows) {
    launch(first, std::min(rows, first + kLaunchRows));
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}
// Blocks of `per` rows each for the rows [first, end).
unsigned blocks_of(int64_t first, int64_t end, int per) { return (unsigned)((end - first + per - 1) / per); }

template <typename T>
bool wide_rows(const void* p, int E, int V) {
  return E % V == 0 && reinterpret_cast<uintptr_t>(p) % std::min<size_t>(16, V * sizeof(T)) == 0;
}

}  // namespace

namespace {

template <typename T, int V>
void launch_gate16(const GateParams& p, GateArgs a, bool vec64, hipStream_t stream) {
  const unsigned grid = blocks_of(a.first, a.rows, 4 * kRowsPerBlock);
  const size_t lds = p.groups > 1 ? sizeof(double) * kRowsPerBlock * p.experts : 0;
  const bool vec_bias = wide_rows<float>(p.bias, p.experts, V);
  auto go = [&](auto soft, auto bias) {
    gate16_kernel<T, V, decltype(soft)::value, decltype(bias)::value>
        <<<grid, 64 * kRowsPerBlock, lds, stream>>>((const T*)p.logits, a, vec64, vec_bias);
  };
  auto with_bias = [&](auto soft) { p.bias ? go(soft, std::true_type{}) : go(soft, std::false_type{}); };
  p.sigmoid ? with_bias(std::false_type{}) : with_bias(std::true_type{});
}

}  // namespace

hipError_t launch_gate(const GateParams& p, hipStream_t stream) {
  if (p.rows <= 0) return hipSuccess;
  GateArgs a{};
  a.bias = p.bias; a.E = p.experts; a.k = p.k;
  a.groups = p.groups; a.topk_groups = p.topk_groups; a.group_size = p.experts / p.groups;
  if (a.group_size > 1) a.group_magic = (uint32_t)(((uint64_t(1) << 32) + a.group_size - 1) / a.group_size);
  a.renorm = p.renorm; a.scale = p.scale; a.ids = p.ids; a.weights = p.weights;
  // four rows a wave: up to 256 experts, K up to 8, and groups of 1, 2, 4 or 8 whole lanes of it
  const int V16 = p.experts <= 64 ? 4 : p.experts <= 128 ? 8 : 16;
  const int lanes = a.group_size / V16;
  const bool whole = p.groups == 1 || (a.group_size % V16 == 0 && (lanes & (lanes - 1)) == 0 && lanes <= 8);
  if (p.experts <= kMost16 && p.k <= kTop && whole) {
    a.lanes = std::max(lanes, 1);
    return with_type(p.dtype, [&](auto* t) {
      using T = std::remove_const_t<std::remove_pointer_t<decltype(t)>>;
      return with_width16(p.experts, [&](auto w) {
        constexpr int V = decltype(w)::value;
        a.vec = wide_rows<T>(p.logits, p.experts, V);
        return in_launches(p.rows, [&](int64_t first, int64_t end) {
          a.first = first; a.rows = end;
          launch_gate16<T, V>(p, a, wide_rows<T>(p.logits, p.experts, V / 4), stream);
        });
      });
    });
  }
  a.lanes = 64;
  while (64 / a.lanes < a.groups) a.lanes /= 2;
  const size_t lds = p.groups > 1 ? sizeof(double) * kRowsPerBlock * p.experts : 0;
  return with_type(p.dtype, [&](auto* t) {
    using T = std::remove_const_t<std::remove_pointer_t<decltype(t)>>;
    return with_width(p.experts, [&](auto w) {
      constexpr int V = decltype(w)::value;
      a.vec = wide_rows<T>(p.logits, p.experts, V);
      return in_launches(p.rows, [&](int64_t first, int64_t end) {
        a.first = first; a.rows = end;
        const unsigned grid = blocks_of(first, end, kRowsPerBlock);
        if (p.sigmoid)
          gate_kernel<T, V, false><<<grid, 64 * kRowsPerBlock, lds, stream>>>((const T*)p.logits, a);
        else
          gate_kernel<T, V, true><<<grid, 64 * kRowsPerBlock, lds, stream>>>((const T*)p.logits, a);
      });
    });
  });
}

// Shares of a sequence's rows, the same number for every sequence: enough blocks over all
// sequences for four a compute unit, of 16 rows and more of an average sequence (17 rows are two
// shares). (So a long sequence among many short ones is read by few blocks, and the second pass counts the rows
// of all sequences in every block: one of 30,000 rows among 512, 256 experts, 820 us; among 1024
// 1,630; 4096 sequences of 8 rows 383; the same rows as one sequence 21.)
int balance_splits(int64_t rows, int64_t seqs) {
  const int64_t per = std::max<int64_t>(1, rows / std::max<int64_t>(seqs, 1));
  return (int)std::max<int64_t>(1, std::min<int64_t>((1024 + seqs - 1) / seqs, (per + 15) / 16));
}

int balance_chunks(int experts, int splits) { return (experts + finish_experts(splits) - 1) / finish_experts(splits); }

hipError_t launch_balance(const BalanceParams& p, hipStream_t stream) {
  const dim3 grid((unsigned)p.splits, (unsigned)p.seqs);
  hipError_t e = with_type(p.dtype, [&](auto* t) {
    using T = std::remove_const_t<std::remove_pointer_t<decltype(t)>>;
    auto go = [&](auto kernel, bool vec, size_t lds) {
      kernel<<<grid, 64 * kRowsPerBlock, lds, stream>>>((const T*)p.logits, p.rows, p.experts, vec, p.ids, p.k, p.off, p.mask,
                                                        p.sums, p.part_counts, p.held, p.done);
      return hipGetLastError();
    };
    if (p.experts <= kMost16)
      return with_width16(p.experts, [&](auto w) {
        constexpr int V = decltype(w)::value;
        const bool vec = wide_rows<T>(p.logits, p.experts, kPiece<T, V>);
        return p.sigmoid ? go(balance16_sums_kernel<T, V, false>, vec, 0) : go(balance16_sums_kernel<T, V, true>, vec, 0);
      });
    return with_wide(p.experts, [&](auto w) {
      constexpr int V = decltype(w)::value;
      const bool vec = wide_rows<T>(p.logits, p.experts, V);
      const size_t lds = sizeof(double) * kRowsPerBlock * 64 * (V + 1) + sizeof(int) * p.experts;
      return p.sigmoid ? go(balance_sums_kernel<T, V, false>, vec, lds) : go(balance_sums_kernel<T, V, true>, vec, lds);
    });
  });
  if (e != hipSuccess) return e;
  int lanes = 1;   // a sequence's lanes where its partials are counted
  while (lanes < 64 && lanes < p.splits) lanes *= 2;
  auto finish = [&](auto kernel) {
    kernel<<<dim3((unsigned)balance_chunks(p.experts, p.splits), (unsigned)p.seqs), kFinishThreads, 0, stream>>>(
        p.experts, p.k, p.splits, p.seqs, lanes, p.sums, p.part_counts, p.held, p.alpha, p.shares, p.done, p.loss, p.counts,
        p.coef);
  };
  if (finish_experts(p.splits) == 16)
    finish(balance_finish_kernel<16>);
  else
    finish(balance_finish_kernel<64>);
  return hipGetLastError();
}

hipError_t launch_gate_backward(const GateGradParams& p, hipStream_t stream) {
  if (p.rows <= 0) return hipSuccess;
  GateGradArgs a{};
  a.E = p.experts; a.k = p.k; a.renorm = p.renorm; a.scale = p.scale; a.ids = p.ids;
  a.grad_weights = p.grad_weights; a.grad_loss = p.grad_loss; a.coef = p.coef; a.off = p.off; a.seqs = p.seqs;
  a.mask = p.mask;
  return with_type(p.dtype, [&](auto* t) {
    using T = std::remove_const_t<std::remove_pointer_t<decltype(t)>>;
    if (p.experts <= kMost16)
      return with_width16(p.experts, [&](auto w) {
        constexpr int V = decltype(w)::value;
        constexpr int W = kPiece<T, V>;
        a.vec = wide_rows<T>(p.logits, p.experts, W) && wide_rows<T>(p.grad, p.experts, W);
        const bool vec_coef = wide_rows<float>(p.coef, p.experts, W);
        auto go = [&](auto kernel) {
          return in_launches(p.rows, [&](int64_t first, int64_t end) {
            a.first = first; a.rows = end;
            kernel<<<blocks_of(first, end, 4 * kRowsPerBlock), 64 * kRowsPerBlock, 0, stream>>>((const T*)p.logits, a,
                                                                                                vec_coef, (T*)p.grad);
          });
        };
        return p.sigmoid ? go(gate16_backward_kernel<T, V, false>) : go(gate16_backward_kernel<T, V, true>);
      });
    return with_wide(p.experts, [&](auto w) {
      constexpr int V = decltype(w)::value;
      a.vec = wide_rows<T>(p.logits, p.experts, V);
      const size_t lds = sizeof(float) * kRowsPerBlock * 64 * V;
      return in_launches(p.rows, [&](int64_t first, int64_t end) {
        a.first = first; a.rows = end;
        const unsigned grid = blocks_of(first, end, kRowsPerBlock);
        if (p.sigmoid)
          gate_backward_kernel<T, V, false><<<grid, 64 * kRowsPerBlock, lds, stream>>>((const T*)p.logits, a, (T*)p.grad);
        else
          gate_backward_kernel<T, V, true><<<grid, 64 * kRowsPerBlock, lds, stream>>>((const T*)p.logits, a, (T*)p.grad);
      });
    });
  });
}

}  // namespace moe
