// Router of the MoE layer: top-K experts of every token with their routing
// weights, per-expert counts, the balance loss and the z-loss, and the
// gradient of all of them with respect to the logits.
//
// For the tokens t that take part (mask, and at least one logit above -inf):
//   p_t = softmax(x_t),  lse_t = log sum_e exp(x_te)
//   I_t = the K largest logits, ties to the lower expert id
//   alpha_tk = p at I_t (renorm: divided by its sum over I_t)
//   counts_e = #{(t, k): I_tk = e},  P_e = sum_t p_te,  n = #tokens
//   balance = c_b E / (n^2 K) sum_e counts_e P_e,   z = c_z / n sum_t lse_t^2
// counts are constants to the gradient (they are piecewise constant).
//
// G lanes of a warp hold a token's row in registers, NI experts a lane, so a
// row is read once and no shared memory is touched before the statistics. The
// bytes are few (T 32768 E 128 bfloat16: 10.5 MB, 1.5 us); what bounds the
// kernels is the minima, maxima and selections of a token (at that size 60% of the
// integer pipe's cycles with statistics and 66% without, 47% and 51% for float32) and,
// for few tokens, latency. So many tokens share a warp (G = 8 or 16) and few get a
// whole one. Measured at T 32768 E 128 K 8: choices and weights 7.2 us (bfloat16) and
// 9.6 us (float32), with the statistics 11.9 and 15.3 us, the gradient 6.7 and 7.7 us.
#include <algorithm>

#include "router.cuh"

namespace lrm {

// A choice's key: the logit's order first, then the lower expert id, so that
// keys are unique (a lane's places past E hold -inf and rank behind the row's). A
// bfloat16 leaves the low half of its 32 bits free for the id; a float32 needs 64 bits.
template <typename T>
struct ChoiceKey;
template <>
struct ChoiceKey<__nv_bfloat16> {
  using Key = uint32_t;
  __device__ __forceinline__ static Key make(float x, int e) {
    return (order_key(x) & 0xffff0000u) | (0xffffu - (uint32_t)e);
  }
  __device__ __forceinline__ static int expert(Key k) { return 0xffff - (int)(k & 0xffffu); }
  __device__ __forceinline__ static float value(Key k) {
    return key_value((k >> 31) ? k & 0xffff0000u : k | 0xffffu);
  }
};
template <>
struct ChoiceKey<float> {
  using Key = uint64_t;
  __device__ __forceinline__ static Key make(float x, int e) {
    return (uint64_t)order_key(x) << 32 | (0xffffffffu - (uint32_t)e);
  }
  __device__ __forceinline__ static int expert(Key k) { return (int)(0xffffffffu - (uint32_t)k); }
  __device__ __forceinline__ static float value(Key k) { return key_value((uint32_t)(k >> 32)); }
};

// Whether token t takes part: its row maximum is above -inf, or it holds a
// NaN (which then reaches the outputs), and it is not masked out.
template <int NI, int G>
__device__ __forceinline__ bool takes_part(const float (&x)[NI], float top, bool masked) {
  bool some = top > -CUDART_INF_F;
  if (__any_sync(0xffffffffu, !some)) {
    bool nan = false;
#pragma unroll
    for (int i = 0; i < NI; ++i) nan |= x[i] != x[i];
    const uint32_t who = __ballot_sync(0xffffffffu, nan);
    const int lane = threadIdx.x & 31;
    if constexpr (G == 32) some |= who != 0;
    else some |= (who >> (lane & ~(G - 1)) & ((1u << G) - 1)) != 0;
  }
  return some && !masked;
}

// The lane's keys as sorted lists of (up to) 4, largest first: a choice is
// the largest front over the token's lanes, and is taken from its list. A
// longer list would cost more to sort than the shorter lists cost to look at.
template <typename Key, int NI>
struct KeyLists {
  static constexpr int kLen = NI < 4 ? NI : 4;
  Key key[NI];
  __device__ __forceinline__ void exchange(int a, int b) {
    const Key hi = max(key[a], key[b]), lo = min(key[a], key[b]);
    key[a] = hi;
    key[b] = lo;
  }
  __device__ __forceinline__ void sort() {
#pragma unroll
    for (int l = 0; l < NI; l += kLen) {
      if constexpr (kLen == 2) exchange(l, l + 1);
      if constexpr (kLen == 4) {
        exchange(l, l + 1);
        exchange(l + 2, l + 3);
        exchange(l, l + 2);
        exchange(l + 1, l + 3);
        exchange(l + 1, l + 2);
      }
    }
  }
  __device__ __forceinline__ Key front() const {
    Key m = key[0];
#pragma unroll
    for (int l = kLen; l < NI; l += kLen) m = max(m, key[l]);
    return m;
  }
  __device__ __forceinline__ void take(Key k) {
#pragma unroll
    for (int l = 0; l < NI; l += kLen) {
      const bool here = key[l] == k;
#pragma unroll
      for (int i = 0; i + 1 < kLen; ++i) key[l + i] = here ? key[l + i + 1] : key[l + i];
      key[l + kLen - 1] = here ? (Key)0 : key[l + kLen - 1];
    }
  }
};

// Choices by merging, for tokens that share a warp: every lane sorts its keys
// and keeps the KC >= K largest, then the token's lanes merge their lists
// pairwise until all hold the token's. Minima and maxima on registers only, so
// the keys are 32 bits: a logit's order with the expert id in the low bits (16
// for bfloat16, where those are free; log2(NI G) for float32).
template <typename T, int NI, int G, int KC>
__device__ __forceinline__ uint32_t choose_merged(const float (&x)[NI], int gl) {
  using S = RowShape<T, NI, G>;
  constexpr uint32_t kId = sizeof(T) == 2 ? 0xffffu : NI * G - 1;
  static_assert((NI * G & (NI * G - 1)) == 0, "ids fill whole bits");
  uint32_t key[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    // places past E hold -inf and ids past the row's: they rank last
    key[i] = (order_key(x[i]) & ~kId) | (kId - (uint32_t)S::expert(i, gl));
  }
  constexpr int L = NI < KC ? NI : KC;
  uint32_t v[KC];
#pragma unroll
  for (int i = 0; i < NI; i += L) sort_desc<L>(key + i);
#pragma unroll
  for (int i = L; i < NI; i += L) top_of<L>(key, key + i);
#pragma unroll
  for (int i = 0; i < KC; ++i) v[i] = i < L ? key[i] : 0u;
  merge_lanes<G, KC, L, 1>(v);
  uint32_t mine = 0;  // lane k keeps the k-th choice
#pragma unroll
  for (int i = 0; i < KC; ++i) mine = gl == i ? v[i] : mine;
  return mine;
}

// What is wrong with choices by float32 keys, whose low bits are the id's: bit
// 0, they do not descend; bit 1, the row has something above the least of them
// that is not among them. (Equal logits have equal keys but for the id, which
// orders them.)
template <int NI, int G>
__device__ __forceinline__ int choices_wrong(const float (&x)[NI], int gl, int K, float my_x) {
  const float least = -group_fmax<G>(gl < K ? -my_x : -CUDART_INF_F);
  const float next = __shfl_down_sync(0xffffffffu, my_x, 1, G);
  int above = gl < K && my_x > least ? -1 : 0;
#pragma unroll
  for (int i = 0; i < NI; ++i) above += x[i] > least;
#pragma unroll
  for (int o = 1; o < G; o <<= 1) above += __shfl_xor_sync(0xffffffffu, above, o);
  return (above != 0 ? 2 : 0) | (gl + 1 < K && my_x < next ? 1 : 0);
}

// The second fault: the choices whose key (without the id) is above the last
// one's are right as a set; the other places go, one by one on the whole
// logits, to the row's experts with that very key.
template <typename T, int NI, int G>
__device__ __noinline__ void choose_again(const float (&x)[NI], int gl, int E, int K,
                                          uint32_t mine, int& my_idx, float& my_x) {
  using S = RowShape<T, NI, G>;
  constexpr uint32_t kId = NI * G - 1;
  const uint32_t last = __shfl_sync(0xffffffffu, mine, K - 1, G) & ~kId;
  const uint32_t sure = __ballot_sync(0xffffffffu, gl < K && (mine & ~kId) > last);
  const int lane = threadIdx.x & 31;
  const int n = __popc(sure >> (lane & ~(G - 1)) & ((1u << G) - 1));
  const int rounds = __reduce_max_sync(0xffffffffu, K - n);
  uint32_t taken = 0;
  for (int k = 0; k < rounds; ++k) {
    uint32_t best = 0;
    int at = 0;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const uint32_t key = order_key(x[i]);
      if (S::expert(i, gl) < E && (key & ~kId) == last && !(taken >> i & 1) && key > best) {
        best = key;
        at = i;
      }
    }
    const uint32_t hi = group_max<G>(best);
    // the lowest expert of the lanes that hold it
    const uint32_t e = (uint32_t)S::expert(at, gl);
    const uint32_t low = ~group_max<G>(best == hi ? ~e : 0u);
    if (gl == n + k && gl < K) { my_idx = (int)low; my_x = key_value(hi); }
    if (best == hi && e == low) taken |= 1u << at;
  }
}

// The first fault: a choice's place is its rank among the token's K.
template <int G>
__device__ __forceinline__ int rank_of(int K, int my_idx, float my_x) {
  int place = 0;
  for (int j = 0; j < K; ++j) {
    const float v = __shfl_sync(0xffffffffu, my_x, j, G);
    const int e = __shfl_sync(0xffffffffu, my_idx, j, G);
    place += v > my_x || (v == my_x && e < my_idx);
  }
  return place;
}

// Threads of a routing CTA: what NI experts a lane leave registers for.
template <typename T>
constexpr int router_threads(int ni, int g) {
  return ni <= 8 ? 1024 : ni == 16 ? (g < 32 || sizeof(T) == 2 ? 1024 : 512) : 256;
}

// KC: the length of the merged lists where several tokens share a warp (G < 32).
// One CTA an SM is said outright: left to choose, the compiler takes 32 registers
// for two and spills (T 32768 E 32 K 4: 9.2 us instead of 6.8).
template <typename T, int NI, int G, int KC, bool STATS>
__global__ void __launch_bounds__(router_threads<T>(NI, G), 1)
route_kernel(const T* __restrict__ logits, const uint8_t* __restrict__ mask, int ntok, int E,
             int K, int64_t stride, int vec, int renorm, float balance_coef, float z_coef,
             int32_t* __restrict__ topk_idx, float* __restrict__ alpha,
             int32_t* __restrict__ counts, float* __restrict__ prob_sum,
             float* __restrict__ loss, float2* __restrict__ part, float* __restrict__ part_z) {
  pdl_begin();  // predecessor complete before any global access
  extern __shared__ float sm_p[];  // STATS: sums of p [warps][E], then counts [E]
  using C = ChoiceKey<T>;
  using S = RowShape<T, NI, G>;
  constexpr int kTokens = 32 / G;  // tokens a warp
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarp = blockDim.x >> 5;
  const int gl = lane % G;
  int32_t* sm_c = reinterpret_cast<int32_t*>(sm_p + nwarp * E);
  float acc[NI];
  float zacc = 0.f;
  if constexpr (STATS) {
    for (int e = threadIdx.x; e < E; e += blockDim.x) sm_c[e] = 0;
#pragma unroll
    for (int i = 0; i < NI; ++i) acc[i] = 0.f;
    __syncthreads();
  }
  const int64_t step = (int64_t)gridDim.x * nwarp * kTokens;
  for (int64_t first = ((int64_t)blockIdx.x * nwarp + warp) * kTokens; first < ntok;
       first += step) {
    // lanes of a token past the end follow token `first` and write nothing
    const bool real = first + lane / G < ntok;
    const int64_t t = real ? first + lane / G : first;
    float x[NI];
    load_row<T, NI, G>(logits + t * stride, gl, E, vec, x);
    const bool masked = mask && mask[t] == 0;
    // lane k of the token gets its k-th choice: the expert and its logit
    int my_idx = 0, place = gl;
    float my_x = 0.f, top = 0.f;
    if constexpr (G == 32) {
      KeyLists<typename C::Key, NI> list;
#pragma unroll
      for (int i = 0; i < NI; ++i) list.key[i] = C::make(x[i], S::expert(i, gl));
      list.sort();
      typename C::Key my_key = 0;
      for (int k = 0; k < K; ++k) {
        const typename C::Key best = group_max<G>(list.front());
        if (k == 0) top = C::value(best);
        if (gl == k) my_key = best;
        list.take(best);
      }
      my_idx = C::expert(my_key);
      my_x = C::value(my_key);
    } else {
      const uint32_t mine = choose_merged<T, NI, G, KC>(x, gl);
      if constexpr (sizeof(T) == 2) {
        my_idx = ChoiceKey<T>::expert(mine);
        my_x = ChoiceKey<T>::value(mine);
      } else {
        my_idx = (int)(NI * G - 1 - (mine & (NI * G - 1)));
        my_x = gl < K ? fmaxf((float)logits[t * stride + my_idx], -CUDART_INF_F) : 0.f;
        const int wrong = choices_wrong<NI, G>(x, gl, K, my_x);
        if (__any_sync(0xffffffffu, wrong)) {
          if (__any_sync(0xffffffffu, wrong & 2))
            choose_again<T, NI, G>(x, gl, E, K, mine, my_idx, my_x);
          place = rank_of<G>(K, my_idx, my_x);
        }
      }
      top = group_fmax<G>(gl < K ? my_x : -CUDART_INF_F);
    }
    const bool use = takes_part<NI, G>(x, top, masked) && real;
    // p, its sum over the row, and the weights of the K choices
    float total = 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      x[i] = exp_neg(x[i] - top);  // 0 past E, where x is -inf
      total += x[i];
    }
    total = group_sum<G>(total);
    const float inv_total = __frcp_rn(total);
    const bool choice = gl < K;
    float a = choice ? expf(my_x - top) : 0.f;
    // every lane of the warp takes part in the sum, whatever its token holds
    const float inv_a = renorm ? __frcp_rn(group_sum<G>(a)) : inv_total;
    // a NaN in the row makes every weight NaN, also where the choices' own sum has none
    a = total != total ? total : a * inv_a;
    if (choice && real) {
      topk_idx[t * K + place] = my_idx;
      alpha[t * K + place] = use ? a : 0.f;
    }
    if constexpr (STATS) {
      if (use) {
#pragma unroll
        for (int i = 0; i < NI; ++i) acc[i] = fmaf(x[i], inv_total, acc[i]);
        const float lse = top + logf(total);
        zacc = fmaf(lse, lse, zacc);
        if (choice) atomicAdd(&sm_c[my_idx], 1);
      }
    }
  }
  if constexpr (STATS) {
    // the CTA's sums, in a fixed order; a single CTA finishes by itself, the
    // sums of several are added by route_sums_kernel
    __shared__ float red[3][32];
#pragma unroll
    for (int o = G; o < 32; o <<= 1) {  // over the warp's tokens
      zacc += __shfl_xor_sync(0xffffffffu, zacc, o);
#pragma unroll
      for (int i = 0; i < NI; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
    }
    if (lane < G) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int e = S::expert(i, gl);
        if (e < E) sm_p[warp * E + e] = acc[i];
      }
    }
    if (lane == 0) red[2][warp] = zacc;
    __syncthreads();
    float z = 0.f;  // warp 0: the CTA's sum of lse^2
    if (warp == 0) z = warp_sum(lane < nwarp ? red[2][lane] : 0.f);
    const bool alone = gridDim.x == 1;
    float dot = 0.f;
    int64_t pairs = 0;
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
      float s = 0.f;
#pragma unroll 8
      for (int w = 0; w < nwarp; ++w) s += sm_p[w * E + e];
      const int c = sm_c[e];
      if (alone) {
        prob_sum[e] = s;
        counts[e] = c;
        dot = fmaf((float)c, s, dot);
        pairs += c;
      } else {
        part[(int64_t)blockIdx.x * E + e] = make_float2(s, __int_as_float(c));
      }
    }
    if (!alone) {
      if (threadIdx.x == 0) part_z[blockIdx.x] = z;
      return;
    }
    // tokens that took part: every one chose K experts
    dot = warp_sum(dot);
    const float cnt = warp_sum((float)pairs);
    if (lane == 0) { red[0][warp] = dot; red[1][warp] = cnt; }
    __syncthreads();
    if (warp == 0) {
      const float d = warp_sum(lane < nwarp ? red[0][lane] : 0.f);
      const float n = fmaxf(warp_sum(lane < nwarp ? red[1][lane] : 0.f) / (float)K, 1.f);
      if (lane == 0) {
        loss[0] = balance_coef * (float)E * (d / (n * n * (float)K));
        loss[1] = z_coef * (z / n);
      }
    }
  }
}

// The G lanes of a token write the gradient that every expert has; then lane k
// adds what choice k has on top and writes that element again.
// kPer: choices a lane. Three CTAs an SM are said outright where expf makes the
// compiler take registers for two (T 32768 E 128 K 12 float32: 12.1 us instead of 10.4).
constexpr int kRouteBwdThreads = 256;
template <typename T, int NI, int G, int kPer>
__global__ void __launch_bounds__(kRouteBwdThreads, sizeof(T) == 4 && NI == 16 ? 3 : 0)
route_bwd_kernel(const T* __restrict__ logits, const uint8_t* __restrict__ mask,
                 const int32_t* __restrict__ topk_idx, const int32_t* __restrict__ counts,
                 const float* __restrict__ dalpha, const float* __restrict__ dloss, int ntok,
                 int E, int K, int64_t stride, int vec, int out_vec, int renorm,
                 float balance_coef, float z_coef, T* dlogits, int32_t* err) {
  pdl_begin();  // predecessor complete before any global access
  using S = RowShape<T, NI, G>;
  constexpr int kTokens = 32 / G;
  const int lane = threadIdx.x & 31, gl = lane % G;
  const int nwarp = kRouteBwdThreads / 32;
  const int64_t step = (int64_t)gridDim.x * nwarp * kTokens;
  int64_t first = ((int64_t)blockIdx.x * nwarp + (threadIdx.x >> 5)) * kTokens;
  // the lane's own choices of token t: read a round ahead, because their logits
  // are read by them
  int next[kPer];
  auto read_choices = [&](int64_t t) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int k = j * G + gl;
      next[j] = t < ntok && k < K ? topk_idx[t * K + k] : 0;
    }
  };
  read_choices(first + lane / G);
  // the token's lanes hold every expert's count once
  float cost[NI];
  int pairs = 0;
#pragma unroll
  for (int c = 0; c < NI / S::kVec; ++c) {
    const int e = S::expert(c * S::kVec, gl);
    alignas(16) int32_t v[S::kVec];
    if (e + S::kVec <= E) {
      constexpr int kWord = S::kVec * 4 < 16 ? S::kVec * 4 : 16;
#pragma unroll
      for (int i = 0; i < S::kVec * 4 / kWord; ++i)
        copy_bytes<kWord>(v + i * (kWord / 4), counts + e + i * (kWord / 4));
    } else {
#pragma unroll
      for (int i = 0; i < S::kVec; ++i) v[i] = e + i < E ? counts[e + i] : 0;
    }
#pragma unroll
    for (int i = 0; i < S::kVec; ++i) {
      cost[c * S::kVec + i] = (float)v[i];
      pairs += v[i];
    }
  }
#pragma unroll
  for (int o = 1; o < G; o <<= 1) pairs += __shfl_xor_sync(0xffffffffu, pairs, o);
  // tokens that took part: every one chose K experts
  const float n = fmaxf((float)pairs / (float)K, 1.f);
  const float inv_n = 1.f / n;
  const float d0 = dloss ? dloss[0] : 1.f, d1 = dloss ? dloss[1] : 1.f;
  // d balance / d p_te = kb counts_e, and 2 c_z / n of the z-loss
  const float kb = d0 * balance_coef * (float)E * inv_n * (inv_n / (float)K);
  const float kz = d1 * 2.f * z_coef * inv_n;
#pragma unroll
  for (int i = 0; i < NI; ++i) cost[i] *= kb;
  for (; first < ntok; first += step) {
    const bool real = first + lane / G < ntok;
    const int64_t t = real ? first + lane / G : first;
    const T* row = logits + t * stride;
    float x[NI];
    load_row<T, NI, G>(row, gl, E, vec, x);
    const bool masked = mask && mask[t] == 0;
    // the lane's own choices: expert, dalpha, logit
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
          if (dalpha) da[j] = dalpha[t * K + k];
        } else {
          flag_error(err, LRM_DEVERR_EXPERT_ID);
        }
      }
    }
    read_choices(first + step + lane / G);
    float top = -CUDART_INF_F;
#pragma unroll
    for (int i = 0; i < NI; ++i) top = fmaxf(top, x[i]);
    top = group_fmax<G>(top);
    const bool use = takes_part<NI, G>(x, top, masked);
    float total = 0.f, cdot = 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      x[i] = exp_grad<T>(x[i] - top);  // 0 past E, where x is -inf
      total += x[i];
      cdot = fmaf(x[i], cost[i], cdot);
    }
    total = group_sum<G>(total);
    const float inv_total = inverse_grad<T>(total);
    const float cmean = group_sum<G>(cdot) * inv_total;
    float chosen = 0.f, adot = 0.f;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      xc[j] = idx[j] >= 0 ? exp_grad<T>(xc[j] - top) : 0.f;
      chosen += xc[j];
      adot = fmaf(xc[j], da[j], adot);
    }
    // mean of dalpha under alpha (renorm), or under p
    adot = group_sum<G>(adot);
    const float inv_a = renorm ? inverse_grad<T>(group_sum<G>(chosen)) : inv_total;
    const float mean = adot * inv_a;
    // what p_e is multiplied by, but for its own balance cost
    const float common = kz * (top + log_grad<T>(total)) - cmean - (renorm ? 0.f : mean);
    T* out = dlogits + t * E;
#pragma unroll
    for (int c = 0; c < NI / S::kVec; ++c) {
      const int e = S::expert(c * S::kVec, gl);
      alignas(16) T v[S::kVec];
#pragma unroll
      for (int i = 0; i < S::kVec; ++i) {
        const int s = c * S::kVec + i;
        v[i] = (T)(use ? x[s] * inv_total * (cost[s] + common) : 0.f);
      }
      if (real) {
        if (out_vec && e + S::kVec <= E) {
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
        const float p = xc[j] * inv_total;
        const float base = p * (kb * (float)counts[idx[j]] + common);
        const float own = xc[j] * inv_a * (renorm ? da[j] - mean : da[j]);
        out[idx[j]] = (T)(base + own);
      }
    }
  }
}

static lrm_status check_router(const lrm_router* r) {
  if (!r) return LRM_ERR_INVALID_ARG;
  if (r->T < 0 || r->E <= 0 || r->K <= 0 || r->K > r->E) return LRM_ERR_INVALID_ARG;
  if (r->dtype != LRM_F32 && r->dtype != LRM_BF16) return LRM_ERR_INVALID_ARG;
  if (r->stride < r->E) return LRM_ERR_INVALID_ARG;
  if (r->E > kRouterMaxE || r->K > kRouterMaxK) return LRM_ERR_UNSUPPORTED;
  if ((int64_t)r->T * r->K >= (int64_t)1 << 31) return LRM_ERR_UNSUPPORTED;
  return LRM_OK;
}

static size_t router_bytes(const lrm_router* r) {
  // header, then sums of p, counts and lse^2 of every CTA
  const size_t b = kWsHeaderBytes + (size_t)kRouterMaxCtas * (8 * (size_t)r->E + 4);
  return (b + 255) / 256 * 256;
}

static lrm_status check_router_ws(const lrm_router* r, const void* ws, size_t ws_bytes) {
  if (!ws) return LRM_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return LRM_ERR_UNSUPPORTED;
  if (ws_bytes < router_bytes(r)) return LRM_ERR_WORKSPACE;
  return LRM_OK;
}

// Rows begin on a multiple of a lane's chunk (the base is 16-byte aligned).
template <typename T, int NI, int G>
static bool chunks_aligned(int64_t stride) {
  return stride % RowShape<T, NI, G>::kVec == 0;
}

template <typename T, int NI, int G, int KC>
static lrm_status launch_route(const lrm_router* r, const void* logits, const uint8_t* mask,
                               int32_t* topk_idx, float* alpha, int32_t* counts,
                               float* prob_sum, float* loss, void* ws, cudaStream_t cs) {
  const bool stats = counts != nullptr;
  constexpr int kMaxWarps = router_threads<T>(NI, G) / 32, kTokens = 32 / G;
  const int64_t warps = std::max<int64_t>(1, ((int64_t)r->T + kTokens - 1) / kTokens);
  int nwarp;
  int64_t grid;
  if (stats) {
    // one CTA an SM at most (each leaves a row for the last sums), its warps in
    // even rounds; tokens that fit one CTA stay in one, without that second launch
    const int64_t ctas = std::min(num_sms(), kRouterMaxCtas);
    const int64_t rounds = (warps + ctas * kMaxWarps - 1) / (ctas * kMaxWarps);
    const int64_t need = (warps + rounds - 1) / rounds;
    nwarp = (int)(need <= kMaxWarps
                      ? need
                      : std::max<int64_t>(std::min(16, kMaxWarps), (need + ctas - 1) / ctas));
    grid = (need + nwarp - 1) / nwarp;
  } else {
    nwarp = (int)std::min<int64_t>(4, warps);  // a warp for each scheduler of an SM
    grid = std::min<int64_t>((warps + nwarp - 1) / nwarp, 1 << 30);
  }
  float2* part = reinterpret_cast<float2*>((char*)ws + kWsHeaderBytes);
  float* part_z = reinterpret_cast<float*>(part + (size_t)kRouterMaxCtas * r->E);
  auto kern = stats ? route_kernel<T, NI, G, KC, true> : route_kernel<T, NI, G, KC, false>;
  const size_t smem = stats ? ((size_t)nwarp + 1) * r->E * 4 : 0;
  // The limit is the kernel's, for all host threads, so it is only ever set to the
  // most that any call needs: a smaller call in another thread cannot lower it
  // before this one's launch.
  constexpr int kMostSmem = (kMaxWarps + 1) * NI * G * 4;
  if (smem > 40 * 1024 &&
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem) !=
          cudaSuccess) {
    (void)cudaGetLastError();
    return LRM_ERR_CUDA;
  }
  if (launch_k(kern, dim3((unsigned)grid), dim3(nwarp * 32), smem, cs, (const T*)logits, mask,
               r->T, r->E, r->K, r->stride, (int)chunks_aligned<T, NI, G>(r->stride), r->renorm,
               r->balance_coef, r->z_coef, topk_idx, alpha, counts, prob_sum, loss, part, part_z) != cudaSuccess) {
    (void)cudaGetLastError();
    return LRM_ERR_CUDA;
  }
  if (stats && grid > 1)
    launch_k(route_sums_kernel, dim3(kSumCtas), dim3(kSumThreads), 0, cs, (const float2*)part,
             (const float*)part_z, (int)grid, r->E, r->K, r->balance_coef, r->z_coef, counts,
             prob_sum, loss);
  return launch_status();
}

template <typename T, int NI, int G, int kPer>
static lrm_status launch_route_bwd(const lrm_router* r, const void* logits, const uint8_t* mask,
                                   const int32_t* topk_idx, const int32_t* counts,
                                   const float* dalpha, const float* dloss, void* dlogits,
                                   int32_t* err, cudaStream_t cs) {
  constexpr int kTokens = 32 / G * (kRouteBwdThreads / 32);  // tokens a CTA and round
  const int64_t blocks =
      std::min<int64_t>(((int64_t)r->T + kTokens - 1) / kTokens, (int64_t)num_sms() * 8);
  launch_k(route_bwd_kernel<T, NI, G, kPer>, dim3((unsigned)blocks), dim3(kRouteBwdThreads), 0, cs,
           (const T*)logits, mask, topk_idx, counts, dalpha, dloss, r->T, r->E, r->K, r->stride,
           (int)chunks_aligned<T, NI, G>(r->stride), (int)chunks_aligned<T, NI, G>(r->E),
           r->renorm, r->balance_coef, r->z_coef, (T*)dlogits, err);
  return launch_status();
}

using RouteFn = lrm_status (*)(const lrm_router*, const void*, const uint8_t*, int32_t*, float*,
                               int32_t*, float*, float*, void*, cudaStream_t);

template <typename T, int KC>
static RouteFn pick_shared(int E) {
  if (E <= 32) return launch_route<T, 4, 8, KC>;
  if (E <= 64) return launch_route<T, 8, 8, KC>;
  if (E <= 128) return launch_route<T, 16, 8, KC>;
  return launch_route<T, 16, 16, KC>;
}

template <typename T>
static RouteFn pick_route(const lrm_router* r) {
  // From 20 tokens an SM on several share a warp. Measured without statistics,
  // E 128 K 8 (a warp each | shared, us): T 2500 bfloat16 2.1 | 2.3, float32 2.6 |
  // 3.0; T 4864 3.4 | 2.4, 3.8 | 3.3; T 32768 13.8 | 7.3, 16.6 | 9.5.
  const bool many = (int64_t)r->T > (int64_t)num_sms() * 20;
  if (many && r->E <= 256 && r->K <= 8)
    return r->K <= 2   ? pick_shared<T, 2>(r->E)
           : r->K <= 4 ? pick_shared<T, 4>(r->E)
                       : pick_shared<T, 8>(r->E);
  if (r->E <= 32) return launch_route<T, 1, 32, 0>;
  if (r->E <= 64) return launch_route<T, 2, 32, 0>;
  if (r->E <= 128) return launch_route<T, 4, 32, 0>;
  if (r->E <= 256) return launch_route<T, 8, 32, 0>;
  if (r->E <= 512) return launch_route<T, 16, 32, 0>;
  return launch_route<T, 32, 32, 0>;
}

using RouteBwdFn = lrm_status (*)(const lrm_router*, const void*, const uint8_t*, const int32_t*,
                                  const int32_t*, const float*, const float*, void*, int32_t*,
                                  cudaStream_t);

template <typename T, int NI, int G>
static RouteBwdFn pick_choices(int K) {
  if (K <= G) return launch_route_bwd<T, NI, G, 1>;
  return launch_route_bwd<T, NI, G, kRouterMaxK / G>;
}
template <typename T>
static RouteBwdFn pick_route_bwd(const lrm_router* r) {
  if (r->E <= 32) return pick_choices<T, 4, 8>(r->K);
  if (r->E <= 64) return pick_choices<T, 8, 8>(r->K);
  if (r->E <= 128) return pick_choices<T, 16, 8>(r->K);
  if (r->E <= 256) return pick_choices<T, 16, 16>(r->K);
  if (r->E <= 512) return pick_choices<T, 16, 32>(r->K);
  return pick_choices<T, 32, 32>(r->K);
}

}  // namespace lrm

using namespace lrm;

extern "C" size_t lrm_router_workspace_bytes(const lrm_router* r) {
  return check_router(r) == LRM_OK ? router_bytes(r) : 0;
}

extern "C" lrm_status lrm_route(const lrm_router* r, const void* logits, const uint8_t* mask,
                                int32_t* topk_idx, float* alpha, int32_t* counts,
                                float* prob_sum, float* loss, void* ws, size_t ws_bytes,
                                void* stream) {
  LRM_NVTX("lrm_route");
  lrm_status st = check_router(r);
  if (st != LRM_OK) return st;
  if ((st = check_router_ws(r, ws, ws_bytes)) != LRM_OK) return st;
  const int given = !!counts + !!prob_sum + !!loss;
  if (given != 0 && given != 3) return LRM_ERR_INVALID_ARG;
  if (r->T > 0 && (!logits || !topk_idx || !alpha)) return LRM_ERR_INVALID_ARG;
  if ((st = check_aligned({logits, topk_idx, alpha, counts, prob_sum, loss})) != LRM_OK)
    return st;
  if (r->T == 0 && !counts) return LRM_OK;
  cudaStream_t cs = (cudaStream_t)stream;
  auto go = r->dtype == LRM_BF16 ? pick_route<__nv_bfloat16>(r) : pick_route<float>(r);
  return go(r, logits, mask, topk_idx, alpha, counts, prob_sum, loss, ws, cs);
}

extern "C" lrm_status lrm_route_bwd(const lrm_router* r, const void* logits, const uint8_t* mask,
                                    const int32_t* topk_idx, const int32_t* counts,
                                    const float* dalpha, const float* dloss, void* dlogits,
                                    void* ws, size_t ws_bytes, void* stream) {
  LRM_NVTX("lrm_route_bwd");
  lrm_status st = check_router(r);
  if (st != LRM_OK) return st;
  if ((st = check_router_ws(r, ws, ws_bytes)) != LRM_OK) return st;
  if (r->T == 0) return LRM_OK;
  if (!logits || !topk_idx || !counts || !dlogits) return LRM_ERR_INVALID_ARG;
  if ((st = check_aligned({logits, topk_idx, counts, dalpha, dloss, dlogits})) != LRM_OK)
    return st;
  cudaStream_t cs = (cudaStream_t)stream;
  auto go = r->dtype == LRM_BF16 ? pick_route_bwd<__nv_bfloat16>(r) : pick_route_bwd<float>(r);
  return go(r, logits, mask, topk_idx, counts, dalpha, dloss, dlogits, error_word(ws), cs);
}
