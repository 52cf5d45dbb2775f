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
// of the allowed groups, gradient 0. +inf counts as the largest finite float.
//
// One wave per row, lane l holding the V experts [l V, l V + V) (V = 1 .. 16 for up to
// 1024 experts): the row's reductions are DPP steps in one wave, without LDS or barriers.

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

// A logit as the operators take it: NaN as -inf, +inf as the largest float.
__device__ __forceinline__ float clean(float x) { return x != x ? -INFINITY : fminf(x, FLT_MAX); }

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
template <typename R, bool SOFTMAX>
__device__ __forceinline__ R score_of(float x, const RowNorm<R>& n) {
  if constexpr (SOFTMAX)
    return exp_of(R(x) - n.m) * n.inv;
  else
    return R(1) / (R(1) + exp_of(-R(x)));   // 1 / (1 + inf) = 0 for -inf
}

// ---- gate -----------------------------------------------------------------------------
struct GateArgs {
  const float* bias;      // nullable [E]
  int64_t rows;
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
  // Errors of the fp32 ranks (CHECK): a score is off by at most 2^-20 of the row's largest
  // (the exponent's argument, V_EXP_F32, the sum of up to 1024 terms, the reciprocal), a
  // rank by its own rounding on top; two ranks closer than twice that, and a group's sums
  // of two closer than four times that, are decided in 64 bits.
  const R top = SOFTMAX ? norm.inv : R(1);
  const R tau = CHECK ? top * R(0x1p-18) : R(0), tau_rel = CHECK ? R(0x1p-21) : R(0);
  bool close = false;
  R r[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = lane * V + v;
    r[v] = e < p.E ? score_of<R, SOFTMAX>(x[v], norm) : R(0);
    if (p.bias) r[v] += e < p.E ? R(p.bias[e]) : R(0);
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

template <typename T, int V, bool SOFTMAX>
__global__ __launch_bounds__(64 * kRowsPerBlock) void gate_kernel(const T* __restrict__ logits, GateArgs p) {
  extern __shared__ double lds_ranks[];   // [waves][E] with groups
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row = (int64_t)blockIdx.x * kRowsPerBlock + wave;
  if (row >= p.rows) return;
  double* lds = lds_ranks + wave * p.E;
  const T* rp = logits + row * p.E;
  float x[V];
  load_row<T, V>(rp, p.E, lane, p.vec, x);
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
// b's rows: one partial row each, in the same order on every call.
template <typename T, int V, bool SOFTMAX>
__global__ __launch_bounds__(64 * kRowsPerBlock) void balance_sums_kernel(
    const T* __restrict__ logits, int64_t rows, int E, bool vec, const int32_t* __restrict__ ids, int k,
    const int32_t* __restrict__ off, const uint8_t* __restrict__ mask, float* __restrict__ sums,
    int32_t* __restrict__ counts, int32_t* __restrict__ held, unsigned* __restrict__ done) {
  extern __shared__ float lds_sums[];   // [waves][E] sums, then [E] counts
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int* hist = reinterpret_cast<int*>(lds_sums + kRowsPerBlock * E);
  const int b = blockIdx.y, splits = gridDim.x, s = blockIdx.x;
  if (threadIdx.x == 0 && s == 0 && b == 0) *done = 0;
  for (int e = threadIdx.x; e < E; e += blockDim.x) hist[e] = 0;
  __syncthreads();
  int64_t lo, hi;
  seq_rows(off, b, rows, &lo, &hi);
  const int64_t len = hi - lo, first = lo + len * s / splits, last = lo + len * (s + 1) / splits;
  float acc[V] = {};
  int seen = 0;
  for (int64_t row = first + wave; row < last; row += kRowsPerBlock) {
    if (mask && mask[row] == 0) continue;   // uniform per wave
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
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (lane * V + v < E) lds_sums[wave * E + lane * V + v] = acc[v];
  __shared__ int rows_seen[kRowsPerBlock];
  if (lane == 0) rows_seen[wave] = seen;
  __syncthreads();
  const int64_t part = (int64_t)b * splits + s;
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < kRowsPerBlock; ++w) t += lds_sums[w * E + e];
    sums[part * E + e] = t;
    counts[part * E + e] = hist[e];
  }
  if (threadIdx.x == 0) {
    int t = 0;
    for (int w = 0; w < kRowsPerBlock; ++w) t += rows_seen[w];
    held[part] = t;
  }
}

constexpr int kFinishThreads = 1024;

__device__ __forceinline__ double block_sum(double v, double* lds) {
  v = wave_sum(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  double t = 0;
  for (int w = 0; w < kFinishThreads / 64; ++w) t += lds[w];
  return t;
}

// Second pass: block b joins its sequence's partials; the last block to end adds the
// sequences' losses, in order.
__global__ __launch_bounds__(kFinishThreads) void balance_finish_kernel(
    int E, int k, int splits, const float* __restrict__ sums, const int32_t* __restrict__ counts_part,
    const int32_t* __restrict__ held, float alpha, double* __restrict__ seq_loss, unsigned* __restrict__ done,
    float* __restrict__ loss, int32_t* __restrict__ counts, float* __restrict__ coef) {
  __shared__ double lds_p[kFinishThreads];
  __shared__ int lds_c[kFinishThreads];
  __shared__ double lds_w[kFinishThreads / 64];
  const int b = blockIdx.x, seqs = gridDim.x;
  // sequences with a counted row, and this one's rows
  double mine = 0, filled = 0;
  for (int q = threadIdx.x; q < seqs; q += kFinishThreads) {
    int t = 0;
    for (int s = 0; s < splits; ++s) t += held[(int64_t)q * splits + s];
    filled += t > 0;
    if (q == b) mine = t;
  }
  const double rows = block_sum(mine, lds_w);
  filled = block_sum(filled, lds_w);
  const double f = rows > 0 ? (double)alpha * E / ((double)k * rows * rows * filled) : 0.0;
  double total = 0;
  // `across` threads an expert where E is small
  const int width = min((E + 63) / 64 * 64, kFinishThreads), across = kFinishThreads / width;
  const int slice = threadIdx.x / width, col = threadIdx.x % width;
  for (int e0 = 0; e0 < E; e0 += width) {
    const int e = e0 + col;
    double p = 0;
    int c = 0;
    if (e < E && slice < across)
      for (int s = slice; s < splits; s += across) {
        p += sums[((int64_t)b * splits + s) * E + e];
        c += counts_part[((int64_t)b * splits + s) * E + e];
      }
    __syncthreads();
    lds_p[threadIdx.x] = p;
    lds_c[threadIdx.x] = c;
    __syncthreads();
    if (slice == 0 && e < E) {
      for (int a = 1; a < across; ++a) {
        p += lds_p[a * width + col];
        c += lds_c[a * width + col];
      }
      counts[(int64_t)b * E + e] = c;
      coef[(int64_t)b * E + e] = (float)(f * c);
      total += f * c * p;
    }
  }
  total = block_sum(total, lds_w);
  __shared__ bool last;
  if (threadIdx.x == 0) {
    seq_loss[b] = total;
    __threadfence();
    last = atomicAdd(done, 1u) == (unsigned)seqs - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  double t = 0;
  for (int q = threadIdx.x; q < seqs; q += kFinishThreads)
    t += __hip_atomic_load(&seq_loss[q], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  t = block_sum(t, lds_w);
  if (threadIdx.x == 0) *loss = (float)t;
}

// ---- gradient -------------------------------------------------------------------------
struct GateGradArgs {
  int64_t rows;
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

__device__ __forceinline__ void store_value(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_value(_Float16* p, float v) { *p = (_Float16)v; }
__device__ __forceinline__ void store_value(uint16_t* p, float v) { *p = (uint16_t)bf16x2(v, v); }

template <typename T, int V, bool SOFTMAX>
__global__ __launch_bounds__(64 * kRowsPerBlock) void gate_backward_kernel(const T* __restrict__ logits, GateGradArgs p,
                                                                           T* __restrict__ grad) {
  extern __shared__ float lds_grad[];   // [waves][64 V]
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row = (int64_t)blockIdx.x * kRowsPerBlock + wave;
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
      const float total = wave_sum(sc);
      const float inv = total > 0.0f ? 1.0f / total : 0.0f;
      g = (g - wave_sum(g * sc) * inv) * inv;
    }
    if (id >= 0) area[id] = g;
    wave_lds_fence();
#pragma unroll
    for (int v = 0; v < V; ++v) d[v] = area[lane * V + v];
  }
  float q[V];
#pragma unroll
  for (int v = 0; v < V; ++v) q[v] = 0.0f;
  if (p.grad_loss && !(p.mask && p.mask[row] == 0)) {
    int b = 0;
    bool counted = true;
    if (p.off) {   // the last sequence that starts at or before the row
      int hi = p.seqs;
      while (hi - b > 1) {
        const int mid = (b + hi) >> 1;
        if (p.off[mid] <= row)
          b = mid;
        else
          hi = mid;
      }
      counted = p.off[b] <= row && row < p.off[b + 1];
    }
    if (counted) {
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
      d[v] += q[v];
      dot += d[v] * s[v];
    }
    dot = wave_sum(dot);
#pragma unroll
    for (int v = 0; v < V; ++v) d[v] = s[v] * (d[v] - dot);
  } else {
    float dot = 0.0f, z = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      dot += q[v] * s[v];
      z += s[v];
    }
    z = wave_sum(z);
    const float inv = z > 0.0f ? 1.0f / z : 0.0f;
    dot = wave_sum(dot) * inv;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      // s (1 - s) = t / (1 + t)^2 with t = exp(-|l|): 1 - s would lose the digits of a score near 1
      const float t = exp_of(-fabsf(x[v])), r = 1.0f / (1.0f + t);
      d[v] = (d[v] + (q[v] - dot) * inv) * (t * r * r);
    }
  }
  T* out = grad + row * p.E;
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (lane * V + v < p.E) store_value(out + lane * V + v, d[v]);
}

// V = experts a lane: the smallest power of two with 64 V >= E.
template <typename F>
hipError_t with_width(int E, F&& f) {
  if (E <= 64) return f(std::integral_constant<int, 1>{});
  if (E <= 128) return f(std::integral_constant<int, 2>{});
  if (E <= 256) return f(std::integral_constant<int, 4>{});
  if (E <= 512) return f(std::integral_constant<int, 8>{});
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
template <typename T>
bool wide_rows(const void* p, int E, int V) {
  return E % V == 0 && reinterpret_cast<uintptr_t>(p) % std::min<size_t>(16, V * sizeof(T)) == 0;
}

}  // namespace

hipError_t launch_gate(const GateParams& p, hipStream_t stream) {
  if (p.rows <= 0) return hipSuccess;
  GateArgs a{};
  a.bias = p.bias; a.rows = p.rows; a.E = p.experts; a.k = p.k;
  a.groups = p.groups; a.topk_groups = p.topk_groups; a.group_size = p.experts / p.groups;
  if (a.group_size > 1) a.group_magic = (uint32_t)(((uint64_t(1) << 32) + a.group_size - 1) / a.group_size);
  a.lanes = 64;
  while (64 / a.lanes < a.groups) a.lanes /= 2;
  a.renorm = p.renorm; a.scale = p.scale; a.ids = p.ids; a.weights = p.weights;
  const unsigned grid = (unsigned)((p.rows + kRowsPerBlock - 1) / kRowsPerBlock);
  const size_t lds = p.groups > 1 ? sizeof(double) * kRowsPerBlock * p.experts : 0;
  return with_type(p.dtype, [&](auto* t) {
    using T = std::remove_const_t<std::remove_pointer_t<decltype(t)>>;
    return with_width(p.experts, [&](auto w) {
      constexpr int V = decltype(w)::value;
      a.vec = wide_rows<T>(p.logits, p.experts, V);
      if (p.sigmoid)
        gate_kernel<T, V, false><<<grid, 64 * kRowsPerBlock, lds, stream>>>((const T*)p.logits, a);
      else
        gate_kernel<T, V, true><<<grid, 64 * kRowsPerBlock, lds, stream>>>((const T*)p.logits, a);
      return hipGetLastError();
    });
  });
}

// Shares of a sequence's rows: enough blocks over all sequences to fill the chip twice,
// of at least 16 rows on average.
int balance_splits(int64_t rows, int64_t seqs) {
  const int64_t per = std::max<int64_t>(1, rows / std::max<int64_t>(seqs, 1));
  return (int)std::max<int64_t>(1, std::min<int64_t>((512 + seqs - 1) / seqs, (per + 15) / 16));
}

hipError_t launch_balance(const BalanceParams& p, hipStream_t stream) {
  const dim3 grid((unsigned)p.splits, (unsigned)p.seqs);
  const size_t lds = sizeof(float) * (kRowsPerBlock + 1) * p.experts;
  hipError_t e = with_type(p.dtype, [&](auto* t) {
    using T = std::remove_const_t<std::remove_pointer_t<decltype(t)>>;
    return with_width(p.experts, [&](auto w) {
      constexpr int V = decltype(w)::value;
      const bool vec = wide_rows<T>(p.logits, p.experts, V);
      if (p.sigmoid)
        balance_sums_kernel<T, V, false><<<grid, 64 * kRowsPerBlock, lds, stream>>>(
            (const T*)p.logits, p.rows, p.experts, vec, p.ids, p.k, p.off, p.mask, p.sums, p.part_counts, p.held, p.done);
      else
        balance_sums_kernel<T, V, true><<<grid, 64 * kRowsPerBlock, lds, stream>>>(
            (const T*)p.logits, p.rows, p.experts, vec, p.ids, p.k, p.off, p.mask, p.sums, p.part_counts, p.held, p.done);
      return hipGetLastError();
    });
  });
  if (e != hipSuccess) return e;
  balance_finish_kernel<<<(unsigned)p.seqs, kFinishThreads, 0, stream>>>(p.experts, p.k, p.splits, p.sums, p.part_counts,
                                                                         p.held, p.alpha, p.seq_loss, p.done, p.loss,
                                                                         p.counts, p.coef);
  return hipGetLastError();
}

hipError_t launch_gate_backward(const GateGradParams& p, hipStream_t stream) {
  if (p.rows <= 0) return hipSuccess;
  GateGradArgs a{};
  a.rows = p.rows; a.E = p.experts; a.k = p.k; a.renorm = p.renorm; a.scale = p.scale; a.ids = p.ids;
  a.grad_weights = p.grad_weights; a.grad_loss = p.grad_loss; a.coef = p.coef; a.off = p.off; a.seqs = p.seqs;
  a.mask = p.mask;
  const unsigned grid = (unsigned)((p.rows + kRowsPerBlock - 1) / kRowsPerBlock);
  return with_type(p.dtype, [&](auto* t) {
    using T = std::remove_const_t<std::remove_pointer_t<decltype(t)>>;
    return with_width(p.experts, [&](auto w) {
      constexpr int V = decltype(w)::value;
      a.vec = wide_rows<T>(p.logits, p.experts, V);
      const size_t lds = sizeof(float) * kRowsPerBlock * 64 * V;
      if (p.sigmoid)
        gate_backward_kernel<T, V, false><<<grid, 64 * kRowsPerBlock, lds, stream>>>((const T*)p.logits, a, (T*)p.grad);
      else
        gate_backward_kernel<T, V, true><<<grid, 64 * kRowsPerBlock, lds, stream>>>((const T*)p.logits, a, (T*)p.grad);
      return hipGetLastError();
    });
  });
}

}  // namespace moe
