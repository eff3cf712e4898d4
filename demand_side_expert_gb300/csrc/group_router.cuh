// Router over groups of experts: sigmoid or softmax scores, a bias that only the
// choices see, the best groups of a token, its top-K in them, and the gradient.
//   s = sigmoid(x) or softmax(x),  key = s + bias (without one: x)
//   a group's score: the sum of its group_top largest s + bias; top_groups are kept
//   I = the K largest keys in them, ties to the lower expert id
//   alpha = scale s at I (renorm: over its sum),  share = s / sum_e s
//   balance = c_b E / (n^2 K) sum_e counts_e sum_t share_te
//   d alpha -> ds,  dx = ds s (1 - s)  or  s (ds - sum s ds)
//
// Choices are whole numbers: two keys nearer than 32-bit arithmetic can tell may stand
// in the other order. Every key's error has a bound, so the kernel knows which tokens
// it cannot decide, and does those again in 64 bits. Keys of equal logits and equal
// biases are equal in any arithmetic and go by their ids.
//
// The logits are read once and little is written (T 32768 E 256 float32: 36 MB, 5.3 us of
// copy bandwidth); what bounds the kernels is the instructions of a token, about half of
// them minima and maxima (sorting, merging), and at few warps their latency. T 32768 E 256
// K 8, 4 of 8 groups, with statistics: 32 us, of which 2 to 3 are the statistics' second
// kernel and about 8 the tokens done again in 64 bits (24.8 with the doubts left as they
// are); the gradient 15.4 us, of bfloat16 15.7: half the bytes and the same instructions.
// Times in this file are of four inputs in turn with sigmoid scores and a bias in float32,
// where nothing else is said.
#pragma once

#include <algorithm>

#include "group_router.h"
#include "router.cuh"

namespace lrm {

// A lane holds NI consecutive experts, so that groups are runs of lanes. -inf past E.
template <typename T, int NI>
__device__ __forceinline__ void load_run(const T* row, int e0, int E, bool vec, float (&x)[NI]) {
  constexpr int kVec = NI * (int)sizeof(T) < 16 ? NI : 16 / (int)sizeof(T);
#pragma unroll
  for (int c = 0; c < NI; c += kVec) {
    alignas(16) T v[kVec];
    if (vec && e0 + c + kVec <= E) {
      copy_bytes<kVec * (int)sizeof(T)>(v, row + e0 + c);
#pragma unroll
      for (int i = 0; i < kVec; ++i) x[c + i] = (float)v[i];
    } else {
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        x[c + i] = e0 + c + i < E ? (float)row[e0 + c + i] : -CUDART_INF_F;
    }
  }
}

// The same of 64 bits, by integers alone: a warp's comparison of doubles takes as long as
// a division's step does here, and that is tens of cycles.
constexpr uint64_t kTopBit = 0x8000000000000000ull, kInfBits = 0x7ff0000000000000ull;
__device__ __forceinline__ uint64_t order_key(double x) {
  uint64_t u = (uint64_t)__double_as_longlong(x);
  if ((u & ~kTopBit) > kInfBits) u = kTopBit | kInfBits;
  if (u == kTopBit) u = 0;
  return u ^ ((uint64_t)((int64_t)u >> 63) | kTopBit);
}
__device__ __forceinline__ double key_double(uint64_t k) {
  return __longlong_as_double((long long)(k ^ ((k >> 63) ? kTopBit : ~0ull)));
}
constexpr uint64_t kLowestKey = ~(kTopBit | kInfBits);  // of -inf

__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Rows whose sigmoids add up to less have all of them taken over exp(m), m the largest logit: a
// score below 2^-126 is 0 in the fast form, which is then less than 1.2e-29 of the sum. (Less
// than an eighth of a unit of the keys' grid, so that the keys are the same either way.)
constexpr float kLowRow = 1e-9f;

// Keeps the larger two of (a, b) and (c, d), a >= b, c >= d.
template <typename F>
__device__ __forceinline__ void merge_two(F& a, F& b, F c, F d) {
  const F lo = a < c ? a : c;
  b = b < d ? d : b;
  b = b < lo ? lo : b;
  a = a < c ? c : a;
}

// The groups that a token keeps, of its warp: bit g of the result. v: s + bias, -inf
// where closed or past E. gap: how far the kept groups' scores stand above the others'.
template <typename F, int NI>
__device__ __forceinline__ uint32_t keep_groups(const F (&v)[NI], int lane, int size, int groups,
                                                int top_groups, int group_top, F& gap) {
  const F kLow = -(F)CUDART_INF;
  F mine = kLow;
  const int e0 = lane * NI;
  for (int g = 0; g < groups; ++g) {
    F a = kLow, b = kLow;
    const int lo = g * size - e0, hi = lo + size;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const F f = i >= lo && i < hi ? v[i] : kLow;
      merge_two(a, b, f, kLow);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const F c = __shfl_xor_sync(0xffffffffu, a, o), d = __shfl_xor_sync(0xffffffffu, b, o);
      merge_two(a, b, c, d);
    }
    const F sum = group_top == 2 && b > kLow ? a + b : a;
    if (lane == g) mine = sum;
  }
  int before = 0;
  for (int g = 0; g < groups; ++g) {
    const F other = __shfl_sync(0xffffffffu, mine, g);
    before += other > mine || (other == mine && g < lane);
  }
  const bool kept = lane < groups && before < top_groups;
  F least = kept ? mine : (F)CUDART_INF, most = kept || lane >= groups ? kLow : mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const F c = __shfl_xor_sync(0xffffffffu, least, o), d = __shfl_xor_sync(0xffffffffu, most, o);
    least = c < least ? c : least;
    most = d > most ? d : most;
  }
  gap = most == kLow ? (F)CUDART_INF : least - most;
  return __ballot_sync(0xffffffffu, kept);
}

// Takes the places of the groups that are not kept out of the keys.
template <typename U, int NI>
__device__ __forceinline__ void drop_groups(U (&key)[NI], int lane, int size, uint32_t kept) {
  int g = lane * NI / size, at = lane * NI - g * size;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    if (!(g < 32 && (kept >> g & 1))) key[i] = 0;
    if (++at == size) { at = 0; ++g; }
  }
}

__device__ __forceinline__ uint32_t warp_max(uint32_t v) {
  return __reduce_max_sync(0xffffffffu, v);
}
__device__ __forceinline__ uint64_t warp_max(uint64_t v) { return group_max<32>(v); }

// The K largest keys in order, equal ones by the lower id (0: a place that was taken,
// which the key becomes): lane k gets the k-th's expert and key.
template <typename U, int NI>
__device__ __forceinline__ void choose(U (&key)[NI], int lane, int K, int& my_idx, U& my_key) {
  for (int k = 0; k < K; ++k) {
    U best = key[0];
    int at = 0;
#pragma unroll
    for (int i = 1; i < NI; ++i)
      if (key[i] > best) { best = key[i]; at = i; }
    const U top = warp_max(best);
    const int who = __ffs(__ballot_sync(0xffffffffu, best == top)) - 1;
    const int e = __shfl_sync(0xffffffffu, lane * NI + at, who);
    if (lane == k) { my_idx = e; my_key = top; }
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if (lane == who && i == at) key[i] = 0;
  }
}

// A token's choices with keys and group scores in 64 bits: by the whole warp.
template <int NI>
__device__ __noinline__ int choose_exact(const float (&x)[NI], int lane, const RouteArgs& a) {
  const int e0 = lane * NI;
  double v[NI];
  if (a.softmax) {
    float top = -CUDART_INF_F;
#pragma unroll
    for (int i = 0; i < NI; ++i) top = fmaxf(top, x[i]);
    top = group_fmax<32>(top);
    double total = 0.0;
#pragma unroll 1
    for (int i = 0; i < NI; ++i) {
      v[i] = x[i] > -CUDART_INF_F ? exp((double)x[i] - (double)top) : 0.0;
      total += v[i];
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
#pragma unroll 1
    for (int i = 0; i < NI; ++i) v[i] /= total;
  } else {
#pragma unroll 1
    for (int i = 0; i < NI; ++i) {
      // rows of equal logits (a router before its first step) are computed once
      const bool again = i == 0 || x[i] != x[i > 0 ? i - 1 : 0];
      if (__any_sync(0xffffffffu, again)) v[i] = 1.0 / (1.0 + exp(-(double)x[i]));
      else v[i] = v[i > 0 ? i - 1 : 0];
    }
  }
  uint64_t key[NI];
#pragma unroll 1
  for (int i = 0; i < NI; ++i) {
    if (a.bias && e0 + i < a.E) v[i] += (double)a.bias[e0 + i];
    if (!(x[i] > -CUDART_INF_F)) v[i] = -CUDART_INF;  // closed, NaN, past E
    key[i] = e0 + i < a.E ? order_key(a.bias ? v[i] : (double)x[i]) : 0;
  }
  if (a.groups > 1) {
    double gap;
    drop_groups(key, lane, a.size,
                keep_groups(v, lane, a.size, a.groups, a.top_groups, a.group_top, gap));
  }
  int idx = 0;
  uint64_t last;
  choose(key, lane, a.K, idx, last);
  return idx;
}

// Keys on a grid: the range of s + bias cut into 2^23 units, kOpenUnit and above for open
// experts, 1 for closed ones (and NaN), 0 for what is no choice. A key is within 3.5 units
// of the real one: 5 2^-24 of the sigmoid's own error and 1 of two roundings to the grid;
// (22 p + 2.5) for the softmax, whose sum carries 43 2^-24 of p.
constexpr uint32_t kOpenUnit = 128;

// Where the keys' grid lies: unit = (s + bias) size + zero.
struct KeyGrid {
  float size, zero;
  __device__ __forceinline__ explicit KeyGrid(float most) {  // the largest |bias|
    size = 8388000.f / fmaf(2.f, most, 1.f);  // 2^23 less kOpenUnit and what rounds up
    zero = fmaf(most, size, (float)kOpenUnit);
  }
  // bits of the float 2^23 + unit for a score of 0
  __device__ __forceinline__ float offset(float bias) const {
    return fmaf(bias, size, zero) + 8388608.f;
  }
};

// The CTA's statistics from its warps' sums, in a fixed order; a single CTA finishes by
// itself, the sums of several are added by route_sums_kernel.
__device__ __forceinline__ void finish_stats(const RouteArgs& a, const float* sm_p,
                                             const int32_t* sm_c) {
  __shared__ float red[2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarp = blockDim.x >> 5;
  __syncthreads();
  const bool alone = gridDim.x == 1;
  float dot = 0.f, cnt = 0.f;
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
    float sum = 0.f;
#pragma unroll 8
    for (int w = 0; w < nwarp; ++w) sum += sm_p[w * a.E + e];
    const int n = sm_c[e];
    if (alone) {
      a.prob_sum[e] = sum;
      a.counts[e] = n;
      dot = fmaf((float)n, sum, dot);
      cnt += (float)n;
    } else {
      a.part[(int64_t)blockIdx.x * a.E + e] = make_float2(sum, __int_as_float(n));
    }
  }
  if (!alone) return;
  dot = warp_sum(dot);
  cnt = warp_sum(cnt);
  if (lane == 0) { red[0][warp] = dot; red[1][warp] = cnt; }
  __syncthreads();
  if (warp == 0) {
    const float d = warp_sum(lane < nwarp ? red[0][lane] : 0.f);
    // tokens that took part: every one chose K experts
    const float n = fmaxf(warp_sum(lane < nwarp ? red[1][lane] : 0.f) / (float)a.K, 1.f);
    if (lane == 0) a.loss[0] = a.balance_coef * (float)a.E * (d / (n * n * (float)a.K));
  }
}


__device__ __forceinline__ uint32_t pair_tolerance(bool softmax, float ptop) {
  return softmax ? 8u + (uint32_t)(48.f * fminf(ptop, 1.f)) : 8u;
}

// s + bias (or s) in 64 bits. Out of line, as all that few tokens need: what an SM runs
// once a launch it has to fetch first, and that took longer than running it.
struct ExactScore {
  double top, total;  // of a softmax: its row's largest logit, its sum
  bool softmax;
};
static __device__ __noinline__ double exact_score(float x, float bias, const ExactScore& s) {
  const double e = exp(s.softmax ? (double)x - s.top : -(double)x);
  return (s.softmax ? e : 1.0) / (s.softmax ? s.total : 1.0 + e) + (double)bias;
}

// The groups that a token keeps, those near the cut by their exact scores: bit g. u: units
// of the lane's experts. ~0: too many experts in doubt for a lane each.
template <typename T, int NI>
__device__ __noinline__ uint32_t settle_groups(const T* row, const uint32_t (&u)[NI], int lane,
                                               const RouteArgs& a, uint32_t tol, uint32_t zero,
                                               const ExactScore& es, uint16_t* list) {
  const int e0 = lane * NI;
  uint32_t score = 0, second = 0;  // lane g: of group g
#pragma unroll 1
  for (int g = 0; g < a.groups; ++g) {
    uint32_t k1 = 0, k2 = 0;
    const int lo = g * a.size - e0, hi = lo + a.size;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const uint32_t f = i >= lo && i < hi ? u[i] : 0u;
      k2 = max(k2, min(k1, f));
      k1 = max(k1, f);
    }
    // the warp's largest, then the largest of what is left
    const uint32_t best = __reduce_max_sync(0xffffffffu, k1);
    const int who = __ffs(__ballot_sync(0xffffffffu, k1 == best)) - 1;
    const uint32_t next = __reduce_max_sync(0xffffffffu, lane == who ? k2 : k1);
    if (lane == g && best >= kOpenUnit / 2) {
      const bool two = a.group_top == 2, has = next >= kOpenUnit / 2;
      score = best + (two ? has ? next : zero : 0u);
      second = two && has ? next : best;
    }
  }
  const bool group = lane < a.groups;
  int before = 0;
#pragma unroll 1
  for (int g = 0; g < a.groups; ++g) {
    const uint32_t other = __shfl_sync(0xffffffffu, score, g);
    before += other > score || (other == score && g < lane);
  }
  bool kept = group && before < a.top_groups;
  const uint32_t least = __reduce_min_sync(0xffffffffu, kept ? score : ~0u);
  const uint32_t next = __reduce_max_sync(0xffffffffu, group && !kept ? score : 0u);
  const uint32_t margin = 2 * tol + 2;
  if (next == 0 || least - next > margin) return __ballot_sync(0xffffffffu, kept);
  // kept for sure: those above every other's reach; the rest by their exact scores
  const bool open = group && score != 0 && score + margin >= least && score <= next + margin;
  const uint32_t in_doubt = __ballot_sync(0xffffffffu, open);
  const uint32_t sure = __ballot_sync(0xffffffffu, kept && !open);
  const uint32_t floor_of = second > tol ? second - tol : 1u;
  int n = 0, g = e0 / a.size, at = e0 - g * a.size;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const uint32_t f = __shfl_sync(0xffffffffu, floor_of, min(g, 31));
    const bool mine = u[i] >= kOpenUnit / 2 && g < 32 && (in_doubt >> (g & 31) & 1) && u[i] >= f;
    const uint32_t who = __ballot_sync(0xffffffffu, mine);
    const int place = n + __popc(who & lanemask_lt());
    if (mine && place < 32) list[place] = (uint16_t)(e0 + i);
    n += __popc(who);
    if (++at == a.size) { at = 0; ++g; }
  }
  __syncwarp();
  if (n > 32) return ~0u;
  const int e = lane < n ? list[lane] : 0;
  const uint64_t v = order_key(exact_score((float)row[e], a.bias ? a.bias[e] : 0.f, es));
  const int my_group = e / a.size;
  uint64_t k1 = 0, k2 = 0;  // lane g: of group g
#pragma unroll 1
  for (int j = 0; j < n; ++j) {
    const uint64_t f = __shfl_sync(0xffffffffu, v, j);
    if (__shfl_sync(0xffffffffu, my_group, j) == lane) merge_two(k1, k2, f, (uint64_t)0);
  }
  uint64_t mine = k1;
  if (a.group_top == 2 && k2 > kLowestKey) mine = order_key(key_double(k1) + key_double(k2));
  before = 0;
#pragma unroll 1
  for (int j = 0; j < a.groups; ++j) {
    const uint64_t other = __shfl_sync(0xffffffffu, mine, j);
    before += (in_doubt >> j & 1) && (other > mine || (other == mine && j < lane));
  }
  kept = (sure >> lane & 1) || (open && before < a.top_groups - __popc(sure));
  __syncwarp();
  return __ballot_sync(0xffffffffu, kept);
}

// A token's choices where keys of 32 bits leave some open: the few experts (and groups)
// that stand nearer to one another than their keys can tell get keys of 64 bits, a lane
// each; more than a warp of them, and all do. By the whole warp; `list`: its 64 entries.
// kept: the groups that the token keeps, where that is sure (0: it is not), `per` bits
// apart.
template <typename T, int NI, bool SOFTMAX>
__device__ __noinline__ int resolve(const T* row, int lane, const RouteArgs& a, float grid_size,
                                    float grid_zero, uint32_t kept, int per, uint16_t* list) {
  float x[NI];
  const int e0 = lane * NI;
  load_run<T, NI>(row, e0, a.E, a.vec && a.E == NI * 32, x);
  float c = 1.f, m = 0.f, s[NI];
  if constexpr (SOFTMAX) {
    float top = x[0], total = 0.f;
#pragma unroll
    for (int i = 1; i < NI; ++i) top = fmaxf(top, x[i]);
    top = group_fmax<32>(top);
    m = top > -CUDART_INF_F ? top : 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i) total += s[i] = exp_neg(x[i] - m);
    c = __frcp_rn(group_sum<32>(total));
  } else {
#pragma unroll
    for (int i = 0; i < NI; ++i) s[i] = rcp_fast(1.f + exp_neg(-x[i]));
  }
  const uint32_t tol = pair_tolerance(SOFTMAX, c);
  uint32_t u[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const float b = a.bias && e0 + i < a.E ? a.bias[e0 + i] : 0.f;
    const float o = fmaf(b, grid_size, grid_zero) + 8388608.f;
    u[i] = __float_as_uint(fmaf(s[i], c * grid_size, o)) & 0x7fffffu;
    if (!(x[i] > -CUDART_INF_F)) u[i] = e0 + i < a.E ? 1u : 0u;
  }
  ExactScore es{(double)m, 1.0, SOFTMAX};
  // the softmax's sum: the scores are over it where a bias is added to them
  if (SOFTMAX && a.bias) {
    double sum = 0.0;
#pragma unroll 1
    for (int i = 0; i < NI; ++i) {
      const float v = e0 + i < a.E ? (float)row[e0 + i] : -CUDART_INF_F;
      if (__any_sync(0xffffffffu, v > -CUDART_INF_F)) sum += exact_score(v, 0.f, es);
    }
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    es.total = sum;
  }
  if (a.groups > 1) {
    if (kept == 0) {
      kept = settle_groups<T, NI>(row, u, lane, a, tol, (uint32_t)grid_zero, es, list);
      if (kept == ~0u) return choose_exact<NI>(x, lane, a);
      per = 1;
    }
    int g = e0 / a.size, at = e0 - g * a.size;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      if (g >= a.groups || !(kept >> (g * per & 31) & 1)) u[i] = 0;
      if (++at == a.size) { at = 0; ++g; }
    }
  }
  uint32_t w[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) w[i] = u[i];
  int idx = 0;
  uint32_t key = 0;
  choose(w, lane, a.K, idx, key);
  const uint32_t last = __shfl_sync(0xffffffffu, key, a.K - 1);
  const uint32_t reach = last >= kOpenUnit / 2 ? last - min(tol, last) : kOpenUnit / 2;
  int n = 0;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const uint32_t who = __ballot_sync(0xffffffffu, u[i] >= reach);
    const int place = n + __popc(who & lanemask_lt());
    if (u[i] >= reach && place < 32) list[place] = (uint16_t)(e0 + i);
    n += __popc(who);
  }
  __syncwarp();
  if (n > 32) return choose_exact<NI>(x, lane, a);
  // (closed experts, where too few are open, stand behind in the order of their ids)
  const int e = lane < n ? list[lane] : 0;
  const float xe = (float)row[e];
  const uint64_t v = a.bias ? order_key(exact_score(xe, a.bias[e], es)) : order_key(xe);
  int place = 0;
#pragma unroll 1
  for (int j = 0; j < n; ++j) {
    const uint64_t other = __shfl_sync(0xffffffffu, v, j);
    const int oe = __shfl_sync(0xffffffffu, e, j);
    place += other > v || (other == v && oe < e);
  }
  if (lane < n) list[32 + place] = (uint16_t)e;
  __syncwarp();
  if (lane < min(n, a.K)) idx = list[32 + lane];
  __syncwarp();
  return idx;
}

template <int NI>
constexpr int group_route_threads() { return NI <= 4 ? 1024 : NI <= 8 ? 512 : 256; }

// A warp a token.
template <typename T, int NI, bool STATS>
__global__ void __launch_bounds__(group_route_threads<NI>(), 1)
group_route_kernel(const T* __restrict__ logits, const RouteArgs a) {
  pdl_begin();  // predecessor complete before any global access
  extern __shared__ float sm_p[];  // STATS: sums of the shares [warps][E], then counts [E]
  __shared__ uint16_t sm_list[group_route_threads<NI>() / 32][64];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarp = blockDim.x >> 5;
  const int E = a.E, K = a.K, e0 = lane * NI;
  int32_t* sm_c = reinterpret_cast<int32_t*>(sm_p + nwarp * E);
  float acc[NI], b[NI];
  if constexpr (STATS) {
    for (int e = threadIdx.x; e < E; e += blockDim.x) sm_c[e] = 0;
#pragma unroll
    for (int i = 0; i < NI; ++i) acc[i] = 0.f;
    __syncthreads();
  }
  float bias_most = 0.f;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    b[i] = a.bias && e0 + i < E ? a.bias[e0 + i] : 0.f;
    bias_most = fmaxf(bias_most, fabsf(b[i]));
  }
  bias_most = group_fmax<32>(bias_most);
  for (int64_t t = (int64_t)blockIdx.x * nwarp + warp; t < a.ntok; t += (int64_t)gridDim.x * nwarp) {
    const T* row = logits + t * a.stride;
    float x[NI], s[NI];
    load_run<T, NI>(row, e0, E, a.vec, x);
    const bool masked = a.mask && a.mask[t] == 0;
    float top = -CUDART_INF_F;
    bool some = false;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      top = fmaxf(top, x[i]);
      some |= x[i] != -CUDART_INF_F;
    }
    top = group_fmax<32>(top);
    const bool row_open = __any_sync(0xffffffffu, some), use = row_open && !masked;
    // s = f c: softmax f = exp(x - top), c its inverse sum; sigmoid f = exp(-m) s with
    // m = min(top, 0), so that rows of very low logits keep their shares, and c = exp(m)
    float total = 0.f, c, ptop;
    if (a.softmax) {
#pragma unroll
      for (int i = 0; i < NI; ++i) total += s[i] = row_open ? exp_neg(x[i] - top) : 0.f;
      total = group_sum<32>(total);
      c = ptop = __frcp_rn(total == 0.f ? 1.f : total);
    } else {
      const float m = top > -CUDART_INF_F ? fminf(top, 0.f) : 0.f;
      c = exp_neg(m);
      ptop = 1.f;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const float u = exp_neg(-fabsf(x[i]) - m), r = rcp_fast(1.f + u * c);
        total += s[i] = x[i] >= 0.f ? r : u * r;
      }
      total = group_sum<32>(total);
    }
    // keys in 32 bits and what they may be off by: |s| error below 5 2^-24 (sigmoid) or
    // (43 p + 1) 2^-24 (softmax, p at most the row's largest), the sum's own rounding
    float v[NI];
    uint32_t key[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const bool open = x[i] > -CUDART_INF_F;
      v[i] = open ? fmaf(s[i], c, b[i]) : -CUDART_INF_F;
      key[i] = e0 + i < E ? order_key(a.bias ? v[i] : x[i]) : 0u;
    }
    const float unit = a.softmax ? fmaf(96.f, ptop, 4.f) : 12.f;  // of two keys, 2^-24
    bool sure = true;
    if (a.groups > 1) {
      float gap, most = 0.f;
      const uint32_t kept =
          keep_groups(v, lane, a.size, a.groups, a.top_groups, a.group_top, gap);
#pragma unroll
      for (int i = 0; i < NI; ++i) most = fmaxf(most, x[i] > -CUDART_INF_F ? fabsf(v[i]) : 0.f);
      most = group_fmax<32>(most);
      sure = gap > (2.f * unit + 8.f * most) * 5.9604645e-8f;
      drop_groups(key, lane, a.size, kept);
    }
    int idx = 0;
    uint32_t kk = 0;
    choose(key, lane, K, idx, kk);
    const bool choice = lane < K;
    float xk = choice ? (float)row[idx] : -CUDART_INF_F;
    if (a.bias) {
      const float f = key_value(kk), bk = choice ? a.bias[idx] : 0.f;
      const float first = __shfl_sync(0xffffffffu, f, 0), last = __shfl_sync(0xffffffffu, f, K - 1);
      const float size = fmaxf(fabsf(first), last > -CUDART_INF_F ? fabsf(last) : 0.f);
      const float tol = (unit + 4.f * size) * 5.9604645e-8f;
      const float fn = __shfl_down_sync(0xffffffffu, f, 1), xn = __shfl_down_sync(0xffffffffu, xk, 1),
                  bn = __shfl_down_sync(0xffffffffu, bk, 1);
      bool near = lane + 1 < K && f - fn <= tol && !(xk == xn && bk == bn);
      const float xl = __shfl_sync(0xffffffffu, xk, K - 1), bl = __shfl_sync(0xffffffffu, bk, K - 1);
      const uint32_t floor_key = last > -CUDART_INF_F ? order_key(last - tol) : 0xffffffffu;
#pragma unroll
      for (int i = 0; i < NI; ++i) near |= key[i] >= floor_key && !(x[i] == xl && b[i] == bl);
      sure = sure && !__any_sync(0xffffffffu, near);
    }
    if (!sure) {
      const KeyGrid grid(bias_most);
      idx = a.softmax ? resolve<T, NI, true>(row, lane, a, grid.size, grid.zero, 0u, 1, sm_list[warp])
                      : resolve<T, NI, false>(row, lane, a, grid.size, grid.zero, 0u, 1,
                                              sm_list[warp]);
      xk = choice ? (float)row[idx] : -CUDART_INF_F;
    }
    // weights, with float32's accuracy at any logit
    float w;
    if (a.softmax) {
      const float m = a.renorm ? group_fmax<32>(xk) : top;
      w = choice && m > -CUDART_INF_F ? expf(xk - m) : 0.f;
      if (!a.renorm) w *= c;
      if (total != total) w = total;
    } else {
      const float most = group_fmax<32>(xk);
      const float m = a.renorm && most > -CUDART_INF_F ? fminf(most, 0.f) : 0.f;
      w = xk >= 0.f ? __frcp_rn(1.f + expf(-xk)) : expf(xk - m) / (1.f + expf(xk));
      if (!choice) w = 0.f;
    }
    if (a.renorm) {
      const float sum = group_sum<32>(w);
      w = sum == 0.f ? 0.f : w / sum;
    }
    if (choice) {
      a.topk_idx[t * K + lane] = idx;
      a.alpha[t * K + lane] = use ? w * a.scale : 0.f;
    }
    if constexpr (STATS) {
      if (use) {
        const float inv = total == 0.f ? 0.f : __frcp_rn(total);
#pragma unroll
        for (int i = 0; i < NI; ++i) acc[i] = fmaf(s[i], inv, acc[i]);
        if (choice) atomicAdd(&sm_c[idx], 1);
      }
    }
  }
  if constexpr (STATS) {
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if (e0 + i < E) sm_p[warp * E + e0 + i] = acc[i];
    finish_stats(a, sm_p, sm_c);
  }
}

// The common shapes: groups that are whole lanes, up to 8 choices of up to 256 experts.
// L lanes a token, NI consecutive experts a lane. A key is its unit on the grid over 8
// bits of the expert's id (the lower id is the larger key), so that sorting networks of
// 32-bit minima and maxima find the choices and equal ones go by their ids. Every lane
// sorts its keys, the two largest of a group's lanes rank the groups, the others' keys
// are dropped, and the token's lanes merge their lists of 8 pairwise. Choices that stand
// further apart than both keys' errors are sure. Bound by one token's chain: few warps an
// SM have work (T 5003 E 128, softmax, padded, with statistics: 12 us; T 1000 E 256 9.9). The
// 768 threads leave 80 registers, and 16 experts a lane with statistics spill 20 to 84 bytes.
constexpr int kTopK = 8;
constexpr int fast_route_threads(int l) { return l == 32 ? 512 : 768; }

template <typename T, int NI, int L, bool SOFTMAX, bool STATS>
__global__ void __launch_bounds__(fast_route_threads(L), 1)
group_route_fast_kernel(const T* __restrict__ logits, const RouteArgs a) {
  pdl_begin();  // predecessor complete before any global access
  extern __shared__ float sm_p[];  // STATS: sums of the shares [warps][E], then counts [E]
  __shared__ float sm_off[L < 32 ? NI * L : 1];
  __shared__ uint16_t sm_list[fast_route_threads(L) / 32][64];
  constexpr int kTokens = 32 / L, kFull = NI * L, kExact = (kFull + 31) / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarp = blockDim.x >> 5;
  const int gl = lane % L, E = a.E, K = a.K, e0 = gl * NI;
  int32_t* sm_c = reinterpret_cast<int32_t*>(sm_p + nwarp * E);
  float acc[STATS ? NI : 1], off[L == 32 ? NI : 1];
  float most = 0.f;
  if (a.bias) {
#pragma unroll
    for (int i = 0; i < kExact; ++i) {
      const int e = i * 32 + lane;
      most = fmaxf(most, e < E ? fabsf(a.bias[e]) : 0.f);
    }
    most = group_fmax<32>(most);
  }
  const KeyGrid grid(most);
  if constexpr (L == 32) {
#pragma unroll
    for (int i = 0; i < NI; ++i) off[i] = grid.offset(a.bias && e0 + i < E ? a.bias[e0 + i] : 0.f);
  } else {
    for (int e = threadIdx.x; e < kFull; e += blockDim.x)
      sm_off[e] = grid.offset(a.bias && e < E ? a.bias[e] : 0.f);
  }
  if constexpr (STATS) {
    for (int e = threadIdx.x; e < E; e += blockDim.x) sm_c[e] = 0;
#pragma unroll
    for (int i = 0; i < NI; ++i) acc[i] = 0.f;
  }
  if (STATS || L < 32) __syncthreads();
  const uint32_t zero = (uint32_t)grid.zero;
  const int per = a.size / NI;  // lanes a group
  const int64_t step = (int64_t)gridDim.x * nwarp * kTokens;
  for (int64_t first = ((int64_t)blockIdx.x * nwarp + warp) * kTokens; first < a.ntok;
       first += step) {
    // lanes of a token past the end follow token `first` and write nothing
    const bool real = first + lane / L < a.ntok;
    const int64_t t = real ? first + lane / L : first;
    const T* row = logits + t * a.stride;
    float x[NI], s[NI];
    load_run<T, NI>(row, e0, E, a.vec, x);
    const bool masked = a.mask && a.mask[t] == 0;
    float low = x[0], total = 0.f, c = 1.f, top = 0.f;
#pragma unroll
    for (int i = 1; i < NI; ++i) low = fminf(low, x[i]);
    bool row_open = true;
    float base = 0.f;
    auto score_of = [&](float v) {
      if constexpr (SOFTMAX) return exp_neg(v - base);
      float e;
      asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v * -1.4426950408889634f));
      return rcp_fast(1.f + e);
    };
    if constexpr (SOFTMAX) {
      top = x[0];
#pragma unroll
      for (int i = 1; i < NI; ++i) top = fmaxf(top, x[i]);
      top = group_fmax<L>(top);
      base = top > -CUDART_INF_F ? top : 0.f;  // nothing open: exp(-inf) each
#pragma unroll
      for (int i = 0; i < NI; ++i) total += s[i] = score_of(x[i]);
      total = group_sum<L>(total);
      row_open = total != 0.f;
      c = __frcp_rn(row_open ? total : 1.f);
    } else {
#pragma unroll
      for (int i = 0; i < NI; ++i) total += s[i] = score_of(x[i]);
      total = group_sum<L>(total);
      // low rows (and rows of none): over exp(m), m the largest logit
      const bool lost = !(total >= kLowRow);
      if (__any_sync(0xffffffffu, lost)) {
        float m = x[0], sum = 0.f;
#pragma unroll
        for (int i = 1; i < NI; ++i) m = fmaxf(m, x[i]);
        m = group_fmax<L>(m);
        m = m > -CUDART_INF_F ? fminf(m, 0.f) : 0.f;
        const float cm = exp_neg(m);
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const float u = exp_neg(-fabsf(x[i]) - m), r = rcp_fast(fmaf(u, cm, 1.f));
          const float f = x[i] >= 0.f ? r : u * r;
          sum += f;
          s[i] = lost ? f : s[i];
        }
        sum = group_sum<L>(sum);
        total = lost ? sum : total;
        c = lost ? cm : 1.f;
        row_open = total != 0.f;
      }
    }
    const bool use = row_open && !masked && real;
    if constexpr (STATS) {
      const float inv = use ? (SOFTMAX ? c : __frcp_rn(total)) : 0.f;
      if (use) {
#pragma unroll
        for (int i = 0; i < NI; ++i) acc[i] = fmaf(s[i], inv, acc[i]);
      }
    }
    uint32_t key[NI];
    const float size = c * grid.size;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const float o = L == 32 ? off[L == 32 ? i : 0] : sm_off[L == 32 ? 0 : e0 + i];
      key[i] = (__float_as_uint(fmaf(s[i], size, o)) << 8) + (uint32_t)(255 - e0) - i;
    }
    if (__any_sync(0xffffffffu, low == -CUDART_INF_F || !(total == total))) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        if (!(x[i] > -CUDART_INF_F)) key[i] = e0 + i < E ? (1u << 8) + (255 - e0) - i : 0u;
      }
    }
    // the lane's 8 largest, sorted
    constexpr int N = NI < kTopK ? NI : kTopK;
#pragma unroll
    for (int i = 0; i < NI; i += N) sort_desc<N>(key + i);
#pragma unroll
    for (int i = N; i < NI; i += N) top_of<N>(key, key + i);
    // units of two keys that may stand the other way round
    const uint32_t tol = pair_tolerance(SOFTMAX, c);
    bool sure = true;
    uint32_t kept_groups = 0;  // by their first lanes, where they are sure
    if (a.groups > 1) {
      uint32_t k1 = key[0], k2 = NI > 1 ? key[NI > 1 ? 1 : 0] : 0u;
      for (int o = 1; o < per; o <<= 1) {
        const uint32_t p = __shfl_xor_sync(0xffffffffu, k1, o), q = __shfl_xor_sync(0xffffffffu, k2, o);
        k2 = max(max(k2, q), min(k1, p));
        k1 = max(k1, p);
      }
      // a missing second expert adds a score of 0; no open expert: below all
      k1 >>= 8;
      k2 >>= 8;
      uint32_t score = 0;
      if (k1 >= kOpenUnit / 2) {
        score = k1;
        if (a.group_top == 2) score += k2 >= kOpenUnit / 2 ? k2 : zero;
      }
      const int g = gl / per, begin = lane & ~(L - 1);
      int before = 0;
      const uint32_t margin = 2 * tol + 2;
      bool close = false;
      for (int j = 0; j < a.groups; ++j) {
        const uint32_t other = __shfl_sync(0xffffffffu, score, begin + j * per);
        before += other > score || (other == score && j < g);
      }
      const bool kept = g < a.groups && before < a.top_groups;
      // the kept groups' least score and the others' largest
      const uint32_t least = ~group_max<L>(kept ? ~score : 0u);
      const uint32_t next = group_max<L>(kept || g >= a.groups ? 0u : score);
      close = next != 0 && least - next <= margin;
      sure = !close;
      kept_groups = __ballot_sync(0xffffffffu, kept) >> begin;
      if (L < 32) kept_groups &= (1u << (L & 31)) - 1;
      if (close) kept_groups = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) key[i] = kept ? key[i] : 0u;
    }
    uint32_t v[kTopK];
#pragma unroll
    for (int i = 0; i < kTopK; ++i) v[i] = i < N ? key[i] : 0u;
    merge_lanes<L, kTopK, N, 1>(v);
    uint32_t mine = 0, last = 0;  // lane k: the k-th choice; the last of all
#pragma unroll
    for (int i = 0; i < kTopK; ++i) {
      mine = gl == i ? v[i] : mine;
      last = i == K - 1 ? v[i] : last;
    }
    const bool choice = gl < K;
    int idx = min(255 - (int)(mine & 255u), E - 1);
    float xk = choice ? (float)row[idx] : -CUDART_INF_F;
    const float bk = a.bias && choice ? a.bias[idx] : 0.f;
    {
      const uint32_t next = __shfl_down_sync(0xffffffffu, mine, 1, L);
      const float xn = __shfl_down_sync(0xffffffffu, xk, 1, L),
                  bn = __shfl_down_sync(0xffffffffu, bk, 1, L);
      bool near = gl + 1 < K && (next >> 8) > 1 && (mine >> 8) - (next >> 8) <= tol &&
                  !(xk == xn && bk == bn);
      // others that may stand above the last choice: how many keys reach it
      const uint32_t reach = (last >> 8) > 1 ? ((last >> 8) - min(tol, last >> 8)) << 8 : ~0u;
      int n = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) n += key[i] >= reach;
      bool more = NI > N && key[N - 1] >= reach;  // the lane may hold others
#pragma unroll
      for (int o = 1; o < L; o <<= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
      more |= n > K && reach != ~0u;
      if (__any_sync(0xffffffffu, more)) {
        // those of the last choice's own logit and bias are below it by their ids
        const int src = (lane & ~(L - 1)) + K - 1;
        const float xl = __shfl_sync(0xffffffffu, xk, src), bl = __shfl_sync(0xffffffffu, bk, src);
        const int il = __shfl_sync(0xffffffffu, idx, src);
        load_run<T, NI>(row, e0, E, a.vec, x);
        const bool in = a.groups == 1 || key[0] != 0;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const float bi = a.bias && e0 + i < E ? a.bias[e0 + i] : 0.f;
          const float o = L == 32 ? off[L == 32 ? i : 0] : sm_off[L == 32 ? 0 : e0 + i];
          // (low rows' scores are 0 units either way)
          const float unit = fmaf(score_of(x[i]), SOFTMAX ? size : grid.size, o);
          const uint32_t k = (__float_as_uint(unit) << 8) + (255 - e0) - i;
          near |= more && in && x[i] > -CUDART_INF_F && k >= reach && k < last && e0 + i != il &&
                  !(x[i] == xl && bi == bl);
        }
      }
      sure = sure && !near;
    }
    uint32_t again = __ballot_sync(0xffffffffu, !sure && real);
    while (again) {  // a token at a time, by the whole warp
      const int at = (__ffs(again) - 1) & ~(L - 1);
      if constexpr (L == 32) again = 0;
      else again &= ~(((1u << L) - 1) << at);
      const int64_t tt = first + at / L;
      const uint32_t kept = __shfl_sync(0xffffffffu, kept_groups, at);
      const int e = resolve<T, kExact, SOFTMAX>(logits + tt * a.stride, lane, a, grid.size,
                                                grid.zero, kept, per, sm_list[warp]);
      const int got = __shfl_sync(0xffffffffu, e, gl);
      if ((lane & ~(L - 1)) == at && choice) {
        idx = got;
        xk = (float)row[idx];
      }
    }
    // weights, with float32's accuracy at any logit
    float w;
    if constexpr (SOFTMAX) {
      const float m = a.renorm ? group_fmax<L>(xk) : top;
      w = choice && m > -CUDART_INF_F ? expf(xk - m) : 0.f;
      if (!a.renorm) w *= c;
      if (total != total) w = total;
    } else {
      float m = 0.f;
      if (a.renorm) {
        const float most_x = group_fmax<L>(xk);
        m = most_x > -CUDART_INF_F ? fminf(most_x, 0.f) : 0.f;
      }
      w = xk >= 0.f ? __frcp_rn(1.f + expf(-xk)) : expf(xk - m) / (1.f + expf(xk));
      if (!choice) w = 0.f;
    }
    if (a.renorm) {
      const float sum = group_sum<L>(choice ? w : 0.f);
      w = sum == 0.f ? 0.f : w / sum;
    }
    if (choice && real) {
      a.topk_idx[t * K + gl] = idx;
      a.alpha[t * K + gl] = use ? w * a.scale : 0.f;
      if (STATS && use) atomicAdd(&sm_c[idx], 1);
    }
  }
  if constexpr (STATS) {
#pragma unroll
    for (int o = L; o < 32; o <<= 1)  // over the warp's tokens
#pragma unroll
      for (int i = 0; i < NI; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
    if (lane < L) {
#pragma unroll
      for (int i = 0; i < NI; ++i)
        if (e0 + i < E) sm_p[warp * E + e0 + i] = acc[i];
    }
    finish_stats(a, sm_p, sm_c);
  }
}

// Many tokens: L lanes hold a token's logits as above, and run through kRound of them. The
// lists are merged across tokens: of two tokens, a lane sends its neighbour the one's list
// and gets the other's, so two merges become one, and after two such steps each of four
// neighbouring lanes has a token of its own; the rest of a token (its choices' logits,
// weights, doubts) is then done for all of the round's tokens at once. What a merge leaves
// out is remembered by its largest key: the first one behind the choices.
constexpr int kRound = 4;
// 512 threads: 32768 tokens, E 256, statistics, take 32.1 us, 640 and 768 (which spill) 33.2
// and 35.7.
constexpr int kRoundThreads = 512;

// a := the 8 largest of two descending lists, descending; `out`: the largest left out.
__device__ __forceinline__ void top_with_rest(uint32_t (&a)[kTopK], const uint32_t (&b)[kTopK],
                                              uint32_t& out) {
  uint32_t rest = 0;
#pragma unroll
  for (int i = 0; i < kTopK; ++i) {
    const uint32_t p = a[i], q = b[kTopK - 1 - i];
    rest = max(rest, min(p, q));
    a[i] = max(p, q);
  }
  merge_desc<kTopK>(a);
  out = max(out, rest);
}

// Two tokens' lists, of which this lane keeps the one of its bit `o`.
__device__ __forceinline__ void merge_tokens(uint32_t (&a)[kTopK], uint32_t& rest_a,
                                             const uint32_t (&b)[kTopK], uint32_t rest_b, bool odd,
                                             int o) {
  uint32_t got[kTopK];
#pragma unroll
  for (int i = 0; i < kTopK; ++i) {
    got[i] = __shfl_xor_sync(0xffffffffu, odd ? a[i] : b[i], o);
    a[i] = odd ? b[i] : a[i];
  }
  const uint32_t r = __shfl_xor_sync(0xffffffffu, odd ? rest_a : rest_b, o);
  rest_a = max(odd ? rest_b : rest_a, r);
  top_with_rest(a, got, rest_a);
}

template <typename T, int NI, int L, bool SOFTMAX, bool STATS>
__global__ void __launch_bounds__(kRoundThreads, 1)
group_route_many_kernel(const T* __restrict__ logits, const RouteArgs a) {
  pdl_begin();  // predecessor complete before any global access
  extern __shared__ float sm_p[];  // STATS: sums of the shares [warps][E], then counts [E]
  __shared__ float sm_off[NI * L];
  __shared__ uint16_t sm_list[kRoundThreads / 32][64];
  constexpr int kGroups = 32 / L, kWarpTokens = kGroups * kRound;
  constexpr int kFull = NI * L, kExact = (kFull + 31) / 32;
  constexpr int kLanes = L / kRound, kEach = kTopK / kLanes;  // of a token; choices a lane
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarp = blockDim.x >> 5;
  const int gl = lane % L, E = a.E, K = a.K, e0 = gl * NI;
  int32_t* sm_c = reinterpret_cast<int32_t*>(sm_p + nwarp * E);
  float acc[STATS ? NI : 1];
  float most = 0.f;
  if (a.bias) {
#pragma unroll
    for (int i = 0; i < kExact; ++i) {
      const int e = i * 32 + lane;
      most = fmaxf(most, e < E ? fabsf(a.bias[e]) : 0.f);
    }
    most = group_fmax<32>(most);
  }
  const KeyGrid grid(most);
  for (int e = threadIdx.x; e < kFull; e += blockDim.x)
    sm_off[e] = grid.offset(a.bias && e < E ? a.bias[e] : 0.f);
  if constexpr (STATS) {
    for (int e = threadIdx.x; e < E; e += blockDim.x) sm_c[e] = 0;
#pragma unroll
    for (int i = 0; i < NI; ++i) acc[i] = 0.f;
  }
  __syncthreads();
  const uint32_t zero = (uint32_t)grid.zero;
  const int per = a.size / NI;  // lanes a group
  const int group = gl / per;
  const bool full = a.vec && E == kFull;
  const int64_t step = (int64_t)gridDim.x * nwarp * kWarpTokens;
  for (int64_t first = ((int64_t)blockIdx.x * nwarp + warp) * kWarpTokens; first < a.ntok;
       first += step) {
    // what the lane will know of its own token
    float my_c = 1.f, my_top = 0.f, my_total = 1.f;
    bool my_use = false, my_sure = true;
    uint32_t my_kept = 0;  // groups by their first lanes, where they are sure
    // sorted list of token q of the round
    auto one_token = [&](int q, uint32_t (&v)[kTopK], uint32_t& rest) {
      const int64_t at = first + lane / L * kRound + q;
      const bool real = at < a.ntok;
      const int64_t t = real ? at : a.ntok - 1;
      const T* row = logits + t * a.stride;
      float x[NI], s[NI];
      if (full) load_run<T, NI>(row, e0, kFull, true, x);
      else load_run<T, NI>(row, e0, E, a.vec, x);
      const bool masked = a.mask && a.mask[t] == 0;
      float low = x[0], total = 0.f, c = 1.f, top = 0.f, base = 0.f;
#pragma unroll
      for (int i = 1; i < NI; ++i) low = fminf(low, x[i]);
      bool row_open = true;
      if constexpr (SOFTMAX) {
        top = x[0];
#pragma unroll
        for (int i = 1; i < NI; ++i) top = fmaxf(top, x[i]);
        top = group_fmax<L>(top);
        base = top > -CUDART_INF_F ? top : 0.f;  // nothing open: exp(-inf) each
#pragma unroll
        for (int i = 0; i < NI; ++i) total += s[i] = exp_neg(x[i] - base);
        total = group_sum<L>(total);
        row_open = total != 0.f;
        c = __frcp_rn(row_open ? total : 1.f);
      } else {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          float e;
          asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x[i] * -1.4426950408889634f));
          total += s[i] = rcp_fast(1.f + e);
        }
        total = group_sum<L>(total);
        // low rows (and rows of none): over exp(m), m the largest logit
        const bool lost = !(total >= kLowRow);
        if (__any_sync(0xffffffffu, lost)) {
          float m = x[0], sum = 0.f;
#pragma unroll
          for (int i = 1; i < NI; ++i) m = fmaxf(m, x[i]);
          m = group_fmax<L>(m);
          m = m > -CUDART_INF_F ? fminf(m, 0.f) : 0.f;
          const float cm = exp_neg(m);
#pragma unroll
          for (int i = 0; i < NI; ++i) {
            const float u = exp_neg(-fabsf(x[i]) - m), r = rcp_fast(fmaf(u, cm, 1.f));
            const float f = x[i] >= 0.f ? r : u * r;
            sum += f;
            s[i] = lost ? f : s[i];
          }
          sum = group_sum<L>(sum);
          total = lost ? sum : total;
          c = lost ? cm : 1.f;
          row_open = total != 0.f;
        }
      }
      const bool use = row_open && !masked && real;
      if constexpr (STATS) {
        const float inv = use ? (SOFTMAX ? c : __frcp_rn(total)) : 0.f;
        if (use) {
#pragma unroll
          for (int i = 0; i < NI; ++i) acc[i] = fmaf(s[i], inv, acc[i]);
        }
      }
      uint32_t key[NI];
      const float size = c * grid.size;
#pragma unroll
      for (int i = 0; i < NI; ++i)
        key[i] = (__float_as_uint(fmaf(s[i], size, sm_off[e0 + i])) << 8) + (uint32_t)(255 - e0) - i;
      if (__any_sync(0xffffffffu, low == -CUDART_INF_F || !(total == total))) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          if (!(x[i] > -CUDART_INF_F)) key[i] = e0 + i < E ? (1u << 8) + (255 - e0) - i : 0u;
        }
      }
      // the lane's 8 largest, sorted
      constexpr int N = NI < kTopK ? NI : kTopK;
      rest = 0;
#pragma unroll
      for (int i = 0; i < NI; i += N) sort_desc<N>(key + i);
#pragma unroll
      for (int i = 0; i < kTopK; ++i) v[i] = i < N ? key[i] : 0u;
      if constexpr (NI > kTopK) {
        uint32_t other[kTopK];
#pragma unroll
        for (int i = 0; i < kTopK; ++i) other[i] = key[NI > kTopK ? kTopK + i : 0];
        top_with_rest(v, other, rest);
      }
      bool sure = true;
      uint32_t kept_groups = 0;
      if (a.groups > 1) {
        uint32_t k1 = v[0], k2 = v[1];
        for (int o = 1; o < per; o <<= 1) {
          const uint32_t p = __shfl_xor_sync(0xffffffffu, k1, o),
                         r = __shfl_xor_sync(0xffffffffu, k2, o);
          k2 = max(max(k2, r), min(k1, p));
          k1 = max(k1, p);
        }
        // a missing second expert adds a score of 0; no open expert: below all. The
        // group's id below the score, the lower one larger.
        k1 >>= 8;
        k2 >>= 8;
        uint32_t score = 0;
        if (k1 >= kOpenUnit / 2)
          score = k1 + (a.group_top == 2 ? k2 >= kOpenUnit / 2 ? k2 : zero : 0u);
        score = (score << 5) + 31u - (uint32_t)group;
        if (group >= a.groups) score = 0;
        int before = 0;
        uint32_t next = 0;  // the next one below
        const int begin = lane & ~(L - 1);
#pragma unroll 8
        for (int j = 0; j < a.groups; ++j) {
          const uint32_t other = __shfl_sync(0xffffffffu, score, begin + j * per);
          const bool above = other > score;
          before += above;
          next = max(next, above || other == score ? 0u : other);
        }
        const bool kept = group < a.groups && before < a.top_groups;
        const uint32_t margin = 2 * pair_tolerance(SOFTMAX, c) + 2;
        const bool close = before == a.top_groups - 1 && group < a.groups && next >= 32u &&
                           (score >> 5) - (next >> 5) <= margin;
        sure = (__ballot_sync(0xffffffffu, close) >> begin & ((1u << L) - 1)) == 0;
        kept_groups = __ballot_sync(0xffffffffu, kept) >> begin & ((1u << L) - 1);
        if (!sure) kept_groups = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = kept ? v[i] : 0u;
        rest = kept ? rest : 0u;
      }
      if ((gl & (kRound - 1)) == q) {
        my_c = c;
        my_top = top;
        my_total = total;
        my_use = use;
        my_sure = sure;
        my_kept = kept_groups;
      }
    };
    uint32_t v[kTopK], rest = 0;
    {
      uint32_t held[kTopK], held_rest = 0;
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        uint32_t other[kTopK], other_rest;
        one_token(2 * half, v, rest);
        one_token(2 * half + 1, other, other_rest);
        merge_tokens(v, rest, other, other_rest, gl & 1, 1);
        if (half == 0) {
#pragma unroll
          for (int i = 0; i < kTopK; ++i) held[i] = v[i];
          held_rest = rest;
        }
      }
      merge_tokens(held, held_rest, v, rest, gl & 2, 2);
#pragma unroll
      for (int i = 0; i < kTopK; ++i) v[i] = held[i];
      rest = held_rest;
    }
#pragma unroll
    for (int o = kRound; o < L; o <<= 1) {
      uint32_t got[kTopK];
#pragma unroll
      for (int i = 0; i < kTopK; ++i) got[i] = __shfl_xor_sync(0xffffffffu, v[i], o);
      rest = max(rest, __shfl_xor_sync(0xffffffffu, rest, o));
      top_with_rest(v, got, rest);
    }
    // from here on a lane is one of its token's kLanes
    const int64_t at = first + lane / L * kRound + (gl & (kRound - 1));
    const bool real = at < a.ntok;
    const int64_t t = real ? at : a.ntok - 1;
    const T* row = logits + t * a.stride;
    const int j0 = gl / kRound;  // the lane's choices: j0, j0 + kLanes, ..
    // choices that stand nearer than their keys can tell (the id's bits count as a unit)
    const uint32_t reach = (pair_tolerance(SOFTMAX, my_c) + 1) << 8;
    constexpr uint32_t kOpenKey = (kOpenUnit / 2) << 8;
    uint32_t last = v[0], behind = rest;
    bool near = false;
#pragma unroll
    for (int i = 1; i < kTopK; ++i) {
      if (i < K) {
        near |= v[i] >= kOpenKey && v[i - 1] - v[i] < reach;
        last = v[i];
      }
      if (i == K) behind = v[i];
    }
    bool sure = my_sure && !(behind >= kOpenKey && last - behind < reach);
    int idx[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      uint32_t k = v[i * kLanes];
#pragma unroll
      for (int j = 1; j < kLanes; ++j) k = j0 == j ? v[i * kLanes + j] : k;
      idx[i] = min(255 - (int)(k & 255u), E - 1);
    }
    if (__any_sync(0xffffffffu, near && sure)) {
      // equal logits and biases go by their ids, as they stand
      bool differ = false;
#pragma unroll
      for (int i = 1; i < kTopK; ++i) {
        if (near && i < K && v[i] >= kOpenKey && v[i - 1] - v[i] < reach && real) {
          const int p = 255 - (int)(v[i - 1] & 255u), q = 255 - (int)(v[i] & 255u);
          differ |= !((float)row[p] == (float)row[q] && (!a.bias || a.bias[p] == a.bias[q]));
        }
      }
      sure = sure && !differ;
    }
    uint32_t again = __ballot_sync(0xffffffffu, !sure && real && j0 == 0);
    while (again) {  // a token at a time, by the whole warp
      const int who = __ffs(again) - 1;
      again &= again - 1;
      const int64_t tt = first + who / L * kRound + who % L;
      const uint32_t kept = __shfl_sync(0xffffffffu, my_kept, who);
      const int e = resolve<T, kExact, SOFTMAX>(logits + tt * a.stride, lane, a, grid.size,
                                                grid.zero, kept, per, sm_list[warp]);
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int got = __shfl_sync(0xffffffffu, e, j0 + i * kLanes);
        if (at == tt) idx[i] = got;
      }
    }
    // weights, with float32's accuracy at any logit
    float xk[kEach], w[kEach], sum = 0.f;
#pragma unroll
    for (int i = 0; i < kEach; ++i) xk[i] = j0 + i * kLanes < K ? (float)row[idx[i]] : -CUDART_INF_F;
    auto over_token = [&](float f, auto op) {
#pragma unroll
      for (int o = kRound; o < L; o <<= 1) f = op(f, __shfl_xor_sync(0xffffffffu, f, o));
      return f;
    };
    const auto larger = [](float p, float q) { return fmaxf(p, q); };
    const auto plus = [](float p, float q) { return p + q; };
    if constexpr (SOFTMAX) {
      float m = my_top;
      if (a.renorm) {
        m = xk[0];
#pragma unroll
        for (int i = 1; i < kEach; ++i) m = fmaxf(m, xk[i]);
        m = over_token(m, larger);
      }
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        w[i] = m > -CUDART_INF_F ? expf(xk[i] - m) : 0.f;
        if (my_total != my_total) w[i] = my_total;
        sum += w[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const float e = expf(-fabsf(xk[i])), r = __frcp_rn(1.f + e);
        w[i] = xk[i] >= 0.f ? r : e * r;
        sum += w[i];
      }
    }
    float factor = a.scale;
    if (a.renorm) {
      sum = over_token(sum, plus);
      if (!SOFTMAX && __any_sync(0xffffffffu, sum < 1e-6f)) {
        // one of the scores may be below 32 bits' normal numbers and a weight all the same: over
        // exp(m), m the largest logit
        float m = xk[0], low_sum = 0.f;
#pragma unroll
        for (int i = 1; i < kEach; ++i) m = fmaxf(m, xk[i]);
        m = over_token(m, larger);
        const bool lost = sum < 1e-6f;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          const float f = m > -CUDART_INF_F ? expf(xk[i] - m) / (1.f + expf(xk[i])) : 0.f;
          low_sum += f;
          w[i] = lost ? f : w[i];
        }
        low_sum = over_token(low_sum, plus);
        sum = lost ? low_sum : sum;
      }
      factor = sum == 0.f ? 0.f : __frcp_rn(sum) * a.scale;
    } else if (SOFTMAX) {
      factor *= my_c;
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int k = j0 + i * kLanes;
      if (k < K && real) {
        a.topk_idx[t * K + k] = idx[i];
        a.alpha[t * K + k] = my_use ? w[i] * factor : 0.f;
        if (STATS && my_use) atomicAdd(&sm_c[idx[i]], 1);
      }
    }
  }
  if constexpr (STATS) {
#pragma unroll
    for (int o = L; o < 32; o <<= 1)  // over the warp's tokens
#pragma unroll
      for (int i = 0; i < NI; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
    if (lane < L) {
#pragma unroll
      for (int i = 0; i < NI; ++i)
        if (e0 + i < E) sm_p[warp * E + e0 + i] = acc[i];
    }
    finish_stats(a, sm_p, sm_c);
  }
}

// Gradient: the G lanes of a token write what every expert has (the balance loss), then
// lane k adds what choice k has on top and writes that element again. kPer: choices a lane.
// The row's exponentials are the hardware's (off by up to 7e-8 for each unit of a logit),
// the choices' own are expf's.
constexpr int kGroupBwdThreads = 256;
// Four CTAs an SM are said outright for rows of 16 experts a lane (T 32768 E 256: 15.4 us, 21.3
// with the two that the compiler's registers leave room for, though 64 registers spill 16 to
// 44 bytes). A token's choices are distinct: two lanes with one expert would write one element.
template <typename T, int NI, int G, int kPer, bool SOFTMAX>
__global__ void __launch_bounds__(kGroupBwdThreads, NI == 16 && kPer == 1 ? 4 : 0)
group_route_bwd_kernel(const T* __restrict__ logits, const RouteBwdArgs a, T* dlogits) {
  pdl_begin();  // predecessor complete before any global access
  using S = RowShape<T, NI, G>;
  constexpr int kTokens = 32 / G, nwarp = kGroupBwdThreads / 32;
  const int lane = threadIdx.x & 31, gl = lane % G, E = a.E, K = a.K;
  const int64_t step = (int64_t)gridDim.x * nwarp * kTokens;
  int64_t first = ((int64_t)blockIdx.x * nwarp + (threadIdx.x >> 5)) * kTokens;
  // the lane's own choices of token t: read a round ahead, because their logits are
  // read by them
  int next[kPer];
  auto read_choices = [&](int64_t t) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int k = j * G + gl;
      next[j] = t < a.ntok && k < K ? a.topk_idx[t * K + k] : 0;
    }
  };
  read_choices(first + lane / G);
  float cost[NI];
  int pairs = 0;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int e = S::expert(i, gl), n = e < E ? a.counts[e] : 0;
    cost[i] = (float)n;
    pairs += n;
  }
#pragma unroll
  for (int o = 1; o < G; o <<= 1) pairs += __shfl_xor_sync(0xffffffffu, pairs, o);
  // tokens that took part: every one chose K experts
  const float inv_n = 1.f / fmaxf((float)pairs / (float)K, 1.f);
  const float kb = (a.dloss ? a.dloss[0] : 1.f) * a.balance_coef * (float)E * inv_n *
                   (inv_n / (float)K);
#pragma unroll
  for (int i = 0; i < NI; ++i) cost[i] *= kb;
  const bool full = a.vec && E == NI * G;
  for (; first < a.ntok; first += step) {
    const bool real = first + lane / G < a.ntok;
    const int64_t t = real ? first + lane / G : first;
    const T* row = logits + t * a.stride;
    float x[NI];
    if (full) load_row<T, NI, G>(row, gl, NI * G, true, x);
    else load_row<T, NI, G>(row, gl, E, a.vec, x);
    const bool masked = a.mask && a.mask[t] == 0;
    int idx[kPer];
    float da[kPer], xc[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int k = j * G + gl;
      idx[j] = -1;
      da[j] = 0.f;
      xc[j] = -CUDART_INF_F;
      if (k < K && real) {
        const int q = next[j];
        if (q >= 0 && q < E) {
          idx[j] = q;
          xc[j] = (float)row[q];
          if (a.dalpha) da[j] = a.dalpha[t * K + k] * a.scale;
        } else {
          flag_error(a.err, LRM_DEVERR_EXPERT_ID);
        }
      }
    }
    read_choices(first + step + lane / G);
    // x becomes the score over exp(m), d what its own derivative makes of it: s (1 - s) over
    // exp(m), or the softmax's s
    float d[NI], total = 0.f, cdot = 0.f, m = 0.f, inv = 0.f;
    bool row_open = true;
    if constexpr (SOFTMAX) {
      float top = x[0];
#pragma unroll
      for (int i = 1; i < NI; ++i) top = fmaxf(top, x[i]);
      top = group_fmax<G>(top);
      m = top > -CUDART_INF_F ? top : 0.f;  // nothing open: exp(-inf) each
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        total += d[i] = exp_neg(x[i] - m);
        cdot = fmaf(d[i], cost[i], cdot);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        float e;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x[i] * -1.4426950408889634f));
        e = fminf(e, 1e38f);  // NaN too: seen by the sum below
        const float s = rcp_fast(1.f + e);
        total += x[i] != x[i] ? x[i] : s;
        cdot = fmaf(s, cost[i], cdot);
        d[i] = s * (e * s);
      }
    }
    total = group_sum<G>(total);
    cdot = group_sum<G>(cdot);
    const bool lost = !(total >= kLowRow);
    if (__any_sync(0xffffffffu, lost)) {
      // rows of very low logits, of nothing open, with NaN: over exp(m), m the largest logit
      float top = x[0], sum = 0.f, dot = 0.f;
#pragma unroll
      for (int i = 1; i < NI; ++i) top = fmaxf(top, x[i]);
      top = group_fmax<G>(top);
      if (!SOFTMAX && lost) m = top > -CUDART_INF_F ? fminf(top, 0.f) : 0.f;
      const float cm = exp_neg(m);
      if constexpr (!SOFTMAX) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const float u = exp_neg(-fabsf(x[i]) - m), z = u * cm, r = rcp_fast(1.f + z);
          const float f = x[i] >= 0.f ? r : u * r;
          sum += f;
          dot = fmaf(f, cost[i], dot);
          if (lost) d[i] = f * (x[i] >= 0.f ? z * r : r);
        }
        sum = group_sum<G>(sum);
        dot = group_sum<G>(dot);
        if (lost) { total = sum; cdot = dot; }
      }
      row_open = total != 0.f;
    }
    const bool use = row_open && !masked;
    inv = row_open ? __frcp_rn(total) : 0.f;
    const float cmean = cdot * inv;
    // the choices' scores over exp(mc): their ratios are right however low they are
    float most = -CUDART_INF_F;
#pragma unroll
    for (int j = 0; j < kPer; ++j) most = fmaxf(most, xc[j]);
    most = group_fmax<G>(most);
    float mc = m;  // at most m, so that exp(mc - m) does not overflow
    if (most > -CUDART_INF_F) mc = SOFTMAX ? most : fminf(most, 0.f);
    float sc[kPer], lc[kPer], chosen = 0.f, adot = 0.f;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const float xj = xc[j];
      if constexpr (SOFTMAX) {
        sc[j] = idx[j] >= 0 && xj > -CUDART_INF_F ? expf(xj - mc) : 0.f;
        if (xj != xj) sc[j] = xj;
        lc[j] = 1.f;
      } else {
        const float z = expf(-fabsf(xj)), r = __frcp_rn(1.f + z);
        sc[j] = xj >= 0.f ? r : mc < 0.f ? expf(xj - mc) * r : z * r;
        lc[j] = xj >= 0.f ? z * r : r;
        if (idx[j] < 0) sc[j] = 0.f;
      }
      chosen += sc[j];
      adot = fmaf(sc[j], da[j], adot);
    }
    chosen = group_sum<G>(chosen);
    adot = group_sum<G>(adot);
    const float to_row = mc < m ? expf(mc - m) : 1.f;  // sc to_row inv: the choice's share
    // s = sc back
    const float back = SOFTMAX ? to_row * inv : mc < 0.f ? expf(mc) : 1.f;
    const float inv_c = chosen == 0.f ? 0.f : __frcp_rn(chosen);
    const float mean = a.renorm ? adot * inv_c : SOFTMAX ? adot * back : 0.f;
    const float common = -cmean - (SOFTMAX && !a.renorm ? mean : 0.f);
    T* out = dlogits + t * E;
#pragma unroll
    for (int q = 0; q < NI / S::kVec; ++q) {
      const int e = S::expert(q * S::kVec, gl);
      alignas(16) T v[S::kVec];
#pragma unroll
      for (int i = 0; i < S::kVec; ++i) {
        const int s = q * S::kVec + i;
        v[i] = (T)(use ? d[s] * (inv * (cost[s] + common)) : 0.f);
      }
      if (real) {
        if (full || (a.out_vec && e + S::kVec <= E)) {
          copy_bytes<S::kVec * (int)sizeof(T)>(out + e, v);
        } else {
#pragma unroll
          for (int i = 0; i < S::kVec; ++i)
            if (e + i < E) out[e + i] = v[i];
        }
      }
    }
    __syncwarp();  // the choices' elements are written after the row's
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (idx[j] >= 0 && use && real) {
        const float share = sc[j] * to_row * inv;
        const float base = share * (kb * (float)a.counts[idx[j]] + common);
        const float own = a.renorm ? sc[j] * inv_c * (da[j] - mean) : sc[j] * back * da[j];
        out[idx[j]] = (T)((base + own) * lc[j]);
      }
    }
  }
}

// `warps` of them have work, `most` of a CTA's threads; the statistics want `capacity`
// floats a warp.
template <typename T>
static lrm_status launch_route_kernel(void (*kern)(const T*, RouteArgs), const void* logits,
                                      const RouteArgs& a, int64_t warps, int max_warps,
                                      int capacity, cudaStream_t cs) {
  const bool stats = a.counts != nullptr;
  int nwarp;
  int64_t grid;
  if (stats) {
    // one CTA an SM at most (each leaves a row for the last sums), its warps in even
    // rounds; tokens that fit one CTA stay in one, without that second launch. Eight warps
    // at least: T 1000 E 256 takes 10.1 us, 11.3 with 16 and 10.1 with 4 (T 8192 17.2, 19.8,
    // 17.5)
    const int64_t ctas = std::min(num_sms(), kRouterMaxCtas);
    const int64_t rounds = (warps + ctas * max_warps - 1) / (ctas * max_warps);
    const int64_t need = (warps + rounds - 1) / rounds;
    nwarp = (int)(need <= max_warps
                      ? need
                      : std::max<int64_t>(std::min(8, max_warps), (need + ctas - 1) / ctas));
    grid = (need + nwarp - 1) / nwarp;
  } else {
    nwarp = (int)std::min<int64_t>(4, warps);  // a warp for each scheduler of an SM
    grid = std::min<int64_t>((warps + nwarp - 1) / nwarp, 1 << 30);
  }
  const size_t smem = stats ? ((size_t)nwarp + 1) * a.E * 4 : 0;
  // the limit is the kernel's, for all host threads: only ever set to the most any call needs
  const int most_smem = (max_warps + 1) * capacity * 4;
  if (smem > 40 * 1024 &&
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most_smem) !=
          cudaSuccess) {
    (void)cudaGetLastError();
    return LRM_ERR_CUDA;
  }
  if (launch_k(kern, dim3((unsigned)grid), dim3(nwarp * 32), smem, cs, (const T*)logits, a) !=
      cudaSuccess) {
    (void)cudaGetLastError();
    return LRM_ERR_CUDA;
  }
  if (stats && grid > 1)
    launch_k(route_sums_kernel, dim3(kSumCtas), dim3(kSumThreads), 0, cs, (const float2*)a.part,
             (const float*)nullptr, (int)grid, a.E, a.K, a.balance_coef, 0.f, a.counts,
             a.prob_sum, a.loss);
  return launch_status();
}

template <typename T, int NI>
static int run_vec(int64_t stride) {
  constexpr int kVec = NI * (int)sizeof(T) < 16 ? NI : 16 / (int)sizeof(T);
  return stride % kVec == 0;
}

template <typename T, int NI>
static lrm_status launch_group_route(const void* logits, RouteArgs a, cudaStream_t cs) {
  a.vec = run_vec<T, NI>(a.stride);
  return launch_route_kernel<T>(
      a.counts ? group_route_kernel<T, NI, true> : group_route_kernel<T, NI, false>, logits, a,
      std::max(1, a.ntok), group_route_threads<NI>() / 32, NI * 32, cs);
}

template <typename T, int NI, int L>
static lrm_status launch_many_route(const void* logits, RouteArgs a, cudaStream_t cs) {
  a.vec = run_vec<T, NI>(a.stride);
  constexpr int kTokens = 32 / L * kRound;
  const bool stats = a.counts != nullptr;
  auto kern = a.softmax ? (stats ? group_route_many_kernel<T, NI, L, true, true>
                                 : group_route_many_kernel<T, NI, L, true, false>)
                        : (stats ? group_route_many_kernel<T, NI, L, false, true>
                                 : group_route_many_kernel<T, NI, L, false, false>);
  return launch_route_kernel<T>(kern, logits, a,
                                std::max<int64_t>(1, ((int64_t)a.ntok + kTokens - 1) / kTokens),
                                kRoundThreads / 32, NI * L, cs);
}

template <typename T, int NI, int L>
static lrm_status launch_fast_route(const void* logits, RouteArgs a, cudaStream_t cs) {
  a.vec = run_vec<T, NI>(a.stride);
  constexpr int kTokens = 32 / L;
  const bool stats = a.counts != nullptr;
  auto kern = a.softmax ? (stats ? group_route_fast_kernel<T, NI, L, true, true>
                                 : group_route_fast_kernel<T, NI, L, true, false>)
                        : (stats ? group_route_fast_kernel<T, NI, L, false, true>
                                 : group_route_fast_kernel<T, NI, L, false, false>);
  return launch_route_kernel<T>(kern, logits, a,
                                std::max<int64_t>(1, ((int64_t)a.ntok + kTokens - 1) / kTokens),
                                fast_route_threads(L) / 32, NI * L, cs);
}

// Whether groups are whole lanes of NI experts, a power of two of them.
static bool whole_lanes(const RouteArgs& a, int ni) {
  if (a.groups == 1) return true;
  const int per = a.size / ni;
  return a.size % ni == 0 && (per & (per - 1)) == 0;
}

template <typename T>
lrm_status pick_group_route(const void* logits, const RouteArgs& a, cudaStream_t cs) {
  if (a.E <= 256 && a.K <= kTopK) {
    const int cap = a.E <= 32 ? 32 : a.E <= 64 ? 64 : a.E <= 128 ? 128 : 256;
    // From 20 tokens an SM on they share warps (T 3040, with statistics, us shared | a warp a
    // token: E 32 7.9 | 10.8, E 64 10.9 | 13.2, E 128 10.4 | 12.3, E 256 12.8 | 13.3, softmax of
    // bfloat16 E 128 21.0 | 19.6, E 256 26.5 | 27.6; T 1520 E 32 7.7 | 8.4, E 128 10.4 | 10.2,
    // softmax of bfloat16 17.9 | 15.6, E 256 10.9 | 10.6).
    const bool many = (int64_t)a.ntok > (int64_t)num_sms() * 20;
    const int shared_ni = cap == 32 ? 4 : cap == 64 ? 8 : 16;
    if (many && whole_lanes(a, shared_ni)) {
      // From 800 lanes of tokens an SM on the lists are merged across tokens (us merged | not:
      // E 256, 16 lanes a token, T 5003 14.2 | 13.6, T 7600 15.4 | 17.5, T 16384 19.7 | 24.1,
      // T 32768 32.5 | 38.1; E 128, 8 lanes, T 8192 14.9 | 12.7, T 15200 16.7 | 17.4, T 32768
      // 19.9 | 23.0). Lists of few experts a lane gain nothing (E 64 T 32768 19.1 | 18.7).
      const bool most = (int64_t)a.ntok * (cap / 16) >= (int64_t)num_sms() * 800;
      if (cap == 32) return launch_fast_route<T, 4, 8>(logits, a, cs);
      if (cap == 64) return launch_fast_route<T, 8, 8>(logits, a, cs);
      if (cap == 128) return most ? launch_many_route<T, 16, 8>(logits, a, cs)
                                  : launch_fast_route<T, 16, 8>(logits, a, cs);
      return most ? launch_many_route<T, 16, 16>(logits, a, cs)
                  : launch_fast_route<T, 16, 16>(logits, a, cs);
    }
    if (whole_lanes(a, cap / 32)) {
      if (cap == 32) return launch_fast_route<T, 1, 32>(logits, a, cs);
      if (cap == 64) return launch_fast_route<T, 2, 32>(logits, a, cs);
      if (cap == 128) return launch_fast_route<T, 4, 32>(logits, a, cs);
      return launch_fast_route<T, 8, 32>(logits, a, cs);
    }
  }
  if (a.E <= 32) return launch_group_route<T, 1>(logits, a, cs);
  if (a.E <= 64) return launch_group_route<T, 2>(logits, a, cs);
  if (a.E <= 128) return launch_group_route<T, 4>(logits, a, cs);
  if (a.E <= 256) return launch_group_route<T, 8>(logits, a, cs);
  if (a.E <= 512) return launch_group_route<T, 16>(logits, a, cs);
  return launch_group_route<T, 32>(logits, a, cs);
}

template <typename T, int NI, int G, int kPer>
static lrm_status launch_group_bwd(const void* logits, RouteBwdArgs a, void* dlogits,
                                   cudaStream_t cs) {
  constexpr int kTokens = 32 / G * (kGroupBwdThreads / 32);  // tokens a CTA and round
  const int64_t blocks =
      std::min<int64_t>(((int64_t)a.ntok + kTokens - 1) / kTokens, (int64_t)num_sms() * 8);
  a.vec = a.stride % RowShape<T, NI, G>::kVec == 0;
  a.out_vec = a.E % RowShape<T, NI, G>::kVec == 0;
  auto kern = a.softmax ? group_route_bwd_kernel<T, NI, G, kPer, true>
                        : group_route_bwd_kernel<T, NI, G, kPer, false>;
  launch_k(kern, dim3((unsigned)blocks), dim3(kGroupBwdThreads), 0, cs, (const T*)logits, a,
           (T*)dlogits);
  return launch_status();
}

template <typename T, int NI, int G>
lrm_status pick_group_choices(const void* logits, const RouteBwdArgs& a, void* dlogits,
                                     cudaStream_t cs) {
  if (a.K <= G) return launch_group_bwd<T, NI, G, 1>(logits, a, dlogits, cs);
  return launch_group_bwd<T, NI, G, kRouterMaxK / G>(logits, a, dlogits, cs);
}

template <typename T>
lrm_status pick_group_bwd(const void* logits, const RouteBwdArgs& a, void* dlogits,
                                 cudaStream_t cs) {
  if (a.E <= 32) return pick_group_choices<T, 4, 8>(logits, a, dlogits, cs);
  if (a.E <= 64) return pick_group_choices<T, 8, 8>(logits, a, dlogits, cs);
  if (a.E <= 128) return pick_group_choices<T, 16, 8>(logits, a, dlogits, cs);
  if (a.E <= 256) return pick_group_choices<T, 16, 16>(logits, a, dlogits, cs);
  if (a.E <= 512) return pick_group_choices<T, 16, 32>(logits, a, dlogits, cs);
  return pick_group_choices<T, 32, 32>(logits, a, dlogits, cs);
}

}  // namespace lrm
