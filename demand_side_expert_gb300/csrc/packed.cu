// The saved state [a | b] of the experts in 8 bits, and its use in the backward pass.
//   pack:    s = max(amax, 2^-100) / 448 over each `cols` columns of a and of b,
//            q = e4m3(v / s), phi_sq = sum (SiLU(a) b)^2 of the unquantised values
//   score:   R_u = alpha_u^2 ||g_t||^2 phi_sq_u
//   compact: dy = alpha g, (a, b) = q s, phi = SiLU(a) b for the retained rows, in
//            their expert-major order
#include <algorithm>
#include <type_traits>

#include "rows.cuh"

namespace lrm {

constexpr float kLog2e = 1.4426950408889634f;

// a sigmoid(a) = a / (1 + 2^(-a log2 e)) on the hardware's power of two and reciprocal:
// the product's rounding puts it off by up to 9e-8 |a| of itself for a below 0, where
// SiLU falls as |a| e^a, and by 3e-7 elsewhere. From -87.3 down, where |SiLU| is below
// 1.1e-36, the reciprocal is below 2^-126 and the result 0. -inf gives NaN, as the formula does.
__device__ __forceinline__ float silu(float a) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-a * kLog2e));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return a * r;
}

__device__ __forceinline__ Pair silu2(Pair a) {
  const float2 x = floats(mul2(a, pair(-kLog2e, -kLog2e)));
  float2 e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(x.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(x.y));
  const float2 d = floats(add2(pair(e.x, e.y), pair(1.f, 1.f)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(d.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(d.y));
  return mul2(a, pair(r.x, r.y));
}

// What a group's values are divided by: 448 v / amax, corrected by its own remainder
// so that quotients which lie between two codes (bfloat16 values often do) round as
// the exact ones. Both sides of the remainder are scaled by 2^-9, so that neither
// overflows.
struct Divisor {
  Pair k, a, r;  // 448 / amax, -amax / 512, 512 / amax
  __device__ __forceinline__ explicit Divisor(float amax) {
    const float inv = __frcp_rn(amax);
    k = pair(inv * kF8Max, inv * kF8Max);
    a = pair(amax * -0.001953125f, amax * -0.001953125f);
    r = pair(inv * 512.f, inv * 512.f);
  }
  __device__ __forceinline__ uint32_t codes(Pair v, Pair seven_eighths) const {
    const Pair t = mul2(v, k);
    const float2 q = floats(fma2(fma2(t, a, mul2(v, seven_eighths)), r, t));
    return __nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3);
  }
};

// The largest magnitudes (NaN aside) of a group's values: 2^shift lanes have its units of a
// and of b. Of bfloat16 both at once, in the halves of a word.
template <typename T>
__device__ __forceinline__ void group_amax(const Unit8<T>& a, const Unit8<T>& b, int shift,
                                           float& ma, float& mb) {
  if constexpr (sizeof(T) == 2) {
    const __nv_bfloat162* pa = reinterpret_cast<const __nv_bfloat162*>(&a.v[0]);
    const __nv_bfloat162* pb = reinterpret_cast<const __nv_bfloat162*>(&b.v[0]);
    auto top = [](const __nv_bfloat162* p) {
      return __hmax2(__hmax2(__habs2(p[0]), __habs2(p[1])), __hmax2(__habs2(p[2]), __habs2(p[3])));
    };
    const __nv_bfloat162 ta = top(pa), tb = top(pb);
    __nv_bfloat162 m = __hmax2(__lows2bfloat162(ta, tb), __highs2bfloat162(ta, tb));
#pragma unroll
    for (int o = 0; o < 4; ++o)
      if (o < shift) m = __hmax2(m, __shfl_xor_sync(0xffffffffu, m, 1 << o));
    const float2 f = __bfloat1622float2(m);
    ma = fmaxf(f.x, kAmaxMin);
    mb = fmaxf(f.y, kAmaxMin);
  } else {
    float fa[kUnit], fb[kUnit];
    a.get(fa);
    b.get(fb);
    ma = mb = kAmaxMin;
#pragma unroll
    for (int j = 0; j < kUnit; ++j) {
      ma = fmaxf(ma, fabsf(fa[j]));
      mb = fmaxf(mb, fabsf(fb[j]));
    }
#pragma unroll
    for (int o = 0; o < 4; ++o) {
      if (o < shift) {
        ma = fmaxf(ma, __shfl_xor_sync(0xffffffffu, ma, 1 << o));
        mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, 1 << o));
      }
    }
  }
}

template <typename T>
__device__ __forceinline__ void pairs_of(const Unit8<T>& u, Pair (&p)[4]) {
  float f[kUnit];
  u.get(f);
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = pair(f[2 * i], f[2 * i + 1]);
}

__device__ __forceinline__ uint2 codes8(const Pair (&p)[4], float amax) {
  const Divisor d(amax);
  const Pair c = pair(0.875f, 0.875f);
  return make_uint2(d.codes(p[0], c) | d.codes(p[1], c) << 16,
                    d.codes(p[2], c) | d.codes(p[3], c) << 16);
}

// LANES lanes a row; lane l holds the 8 columns l, l + LANES, .. of both halves, so that a
// scale's group is neighbouring lanes. NI of them are loaded before any is used. HBM-bound:
// 262,144 pairs of H 768 in bfloat16, 1.22 GB, take 194 us, 0.93 of the copy bandwidth.
constexpr int kPackThreads = 128;

template <typename T, int NI, int LANES>
__global__ void __launch_bounds__(kPackThreads)
pack_kernel(const T* __restrict__ ab, int64_t rows, int H, int shift, uint8_t* __restrict__ q,
            float* __restrict__ scale, float* __restrict__ phi_sq) {
  pdl_begin();  // predecessor complete before any global access
  const int lane = threadIdx.x % LANES;
  const int64_t at = (int64_t)blockIdx.x * (kPackThreads / LANES) + threadIdx.x / LANES;
  if (LANES == 32 && at >= rows) return;
  const bool real = at < rows;  // lanes of a row past the end stay with their warp
  const int64_t r = real ? at : rows - 1;
  const int units = H / kUnit, groups = ((units - 1) >> shift) + 1;
  const T* row = ab + r * 2 * H;
  uint8_t* out = q + r * 2 * H;
  float* sc = scale + r * 2 * groups;
  Pair sq2 = pair(0.f, 0.f);
  for (int u0 = lane; u0 - lane < units; u0 += LANES * NI) {
    Unit8<T> va[NI], vb[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int u = u0 + LANES * i;
      va[i].load(row + u * kUnit, u < units);
      vb[i].load(row + H + u * kUnit, u < units);
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int u = u0 + LANES * i;
      if (u - lane >= units) break;
      float ma, mb;
      group_amax(va[i], vb[i], shift, ma, mb);
      Pair a[4], b[4];
      pairs_of(va[i], a);
      pairs_of(vb[i], b);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const Pair p = mul2(silu2(a[j]), b[j]);
        sq2 = fma2(p, p, sq2);
      }
      if (u < units && real) {
        *reinterpret_cast<uint2*>(out + u * kUnit) = codes8(a, ma);
        *reinterpret_cast<uint2*>(out + H + u * kUnit) = codes8(b, mb);
        if ((u & ((1 << shift) - 1)) == 0) {
          sc[u >> shift] = ma * kF8MaxInv;
          sc[groups + (u >> shift)] = mb * kF8MaxInv;
        }
      }
    }
  }
  const float2 part = floats(sq2);
  float sq = part.x + part.y;
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
  if (lane == 0 && real) phi_sq[r] = sq;
}

// LANES lanes a token: lane k holds slot k's position, ||g_t||^2 is their sum. HBM-bound for wide
// rows (T 16384 D 4096: 21.5 us, 0.92 of the copy bandwidth); a token of a narrow row costs a
// lane the same instructions, so fewer lanes have it (T 29084 bfloat16, us with 8 | 16 | 32: D 80
// 4.6 | 6.7 | 11.3, D 512 7.2 | 8.2 | 12.3, D 1024 13.3 | 13.3 | 14.9; T 300 D 512 3.6 | 2.8 | 2.6).
constexpr int kScoreWarps = 4;

template <typename T, int LANES>
__global__ void __launch_bounds__(32 * kScoreWarps)
score_packed_kernel(const T* __restrict__ g, const float* __restrict__ phi_sq,
                    const float* __restrict__ alpha, const int32_t* __restrict__ inv,
                    float* __restrict__ score, int ntok, int D, int K, int32_t* err) {
  pdl_begin();  // predecessor complete before any global access
  constexpr int V = Vec16<T>::kElems, kAhead = 8;
  const int lane = threadIdx.x & (LANES - 1);
  const int64_t t = (int64_t)blockIdx.x * (32 * kScoreWarps / LANES) + threadIdx.x / LANES;
  if (LANES == 32 && t >= ntok) return;
  const bool real = LANES == 32 || t < ntok;
  const int64_t N = (int64_t)ntok * K;
  const int chunks = D / V;
  const T* row = g + t * D;
  float s = 0.f;
  for (int c0 = lane; c0 - lane < chunks; c0 += LANES * kAhead) {
    uint4 v[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      v[i] = load_if(row + (c0 + LANES * i) * V, real && c0 + LANES * i < chunks);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      float f[V];
      Vec16<T>::unpack(v[i], f);
#pragma unroll
      for (int j = 0; j < V; ++j) s = fmaf(f[j], f[j], s);
    }
  }
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (!real) return;
  for (int k = lane; k < K; k += LANES) {
    const int pos = inv[t * K + k];
    if (pos >= 0 && pos < N) {
      const float a = alpha[t * K + k];
      score[pos] = (a * a) * s * phi_sq[pos];
    } else {
      flag_error(err, LRM_DEVERR_INDEX);
    }
  }
}

// 8 values of e4m3 codes (a byte each) times their scale.
__device__ __forceinline__ void decode8(uint2 c, float scale, float (&f)[kUnit]) {
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
        (__nv_fp8x2_storage_t)(w[i / 2] >> (i % 2 * 16) & 0xffffu), __NV_E4M3);
    const float2 v = __half22float2(__half2(h));
    f[2 * i] = v.x * scale;
    f[2 * i + 1] = v.y * scale;
  }
}

// LANES lanes a retained row; the row count M = sel_off[E] is read on the device. The rows stand by
// expert, and each expert's by token, so the rows of one token are far apart. Where L2 does not
// hold the cotangents (SPREAD, a warp a row) the warps therefore go through all experts'
// segments side by side: in each of `rounds` rounds every segment's next part is dealt out,
// and the rows of a token, at about the same place of their segments, are met while its
// cotangent is still in L2 (T 16384 D 4096 H 1408, half of the pairs, 1.28 GB: 241 us; in the
// rows' own order, at the best number of CTAs, 296). Bound by HBM: of the cotangents, what L2
// did not keep is read again.
constexpr int kUnpackThreads = 256;

// The row of warp `w` in the round whose parts lie between the fractions f0 and f1 (of
// 2^32; the last round's f1 is 0) of the segments; -1: none. Each part is rounded to whole
// rows, so a round holds up to E more than its share.
__device__ __forceinline__ int64_t row_of_round(const int32_t* sel_off, int E, int64_t M,
                                                uint32_t f0, uint32_t f1, int64_t w, int lane) {
  const int per = (E + 31) / 32;  // experts a lane, consecutive
  auto part = [&](int e, uint32_t& begin) -> uint32_t {
    if (e >= E) return 0;
    const int64_t lo = min(max((int64_t)sel_off[e], (int64_t)0), M);
    const uint32_t m = (uint32_t)(min(max((int64_t)sel_off[e + 1], lo), M) - lo);
    const uint32_t at = __umulhi(m, f0), end = f1 ? __umulhi(m, f1) : m;
    begin = (uint32_t)lo + at;
    return end - at;
  };
  uint32_t begin = 0, sum = 0;
  for (int q = 0; q < per; ++q) sum += part(lane * per + q, begin);
  uint32_t upto = sum;  // with the lanes before
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += v;
  }
  const uint32_t has = __ballot_sync(0xffffffffu, upto > w);
  if (has == 0) return -1;
  const int who = __ffs(has) - 1;
  uint32_t left = (uint32_t)w - (upto - sum), row = 0;
  for (int q = 0; q < per; ++q) {  // (only lane `who` finds its place)
    const uint32_t n = part(lane * per + q, begin);
    if (left < n) {
      row = begin + left;
      break;
    }
    left -= n;
  }
  return (int64_t)__shfl_sync(0xffffffffu, row, who);
}

template <typename T>
__device__ __forceinline__ void stream8(T* p, const float (&f)[kUnit]) {
  constexpr int V = Vec16<T>::kElems;
#pragma unroll
  for (int i = 0; i < (int)(sizeof(T) / 2); ++i)
    __stcs(reinterpret_cast<uint4*>(p) + i, Vec16<T>::pack(f + i * V));
}

// Four CTAs an SM (T 16384 D 4096 H 1408, half of the pairs: 241 us; three 248, five, six and
// eight 270, 268, 307), and 4 of a lane's 16-byte pieces of a cotangent ahead (8: as long, 12:
// 266; a short block, T 1021 D 2048: 1.1 and 2.4 us longer), for which its 64 registers spill 24 to
// 80 bytes. Their results are not read here: stores
// that leave L2 first keep the cotangents in it (plain ones 249 us).
constexpr int kUnpackCtas = 4, kAheadG = 4;

// SPREAD: there may be more rows than warps (else they are all met at once), and many more
// warps than experts. A round's rows are then no more than the warps. Wants a warp a row.
template <typename T, int LANES, bool SPREAD>
__global__ void __launch_bounds__(kUnpackThreads, kUnpackCtas)
compact_packed_kernel(const uint8_t* __restrict__ q, const float* __restrict__ scale, int shift,
                      const int32_t* __restrict__ perm, const uint8_t* __restrict__ keep,
                      const int32_t* __restrict__ sel_off, const int32_t* __restrict__ sel_pos,
                      const float* __restrict__ alpha, const void* __restrict__ x,
                      const float* __restrict__ x_scale, int x_cols, const T* __restrict__ g,
                      T* __restrict__ dy_c, T* __restrict__ x_c, T* __restrict__ ab_c,
                      T* __restrict__ phi_c, int32_t* __restrict__ tok_c,
                      int32_t* __restrict__ row_of_pos, int ntok, int D, int H, int K, int E,
                      int32_t* err) {
  pdl_begin();  // predecessor complete before any global access
  static_assert(!SPREAD || LANES == 32, "the warp looks for its row");
  constexpr int V = Vec16<T>::kElems;
  const int64_t N = (int64_t)ntok * K;
  const int64_t gtid = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t nthr = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = gtid; i < N; i += nthr)
    if (!keep[i]) row_of_pos[i] = -1;

  const int lane = threadIdx.x & (LANES - 1);
  int64_t M = sel_off[E];
  if (M < 0 || M > N) {  // not of a selection: no row past the buffers is addressed
    if (gtid == 0) flag_error(err, LRM_DEVERR_INDEX);
    M = M < 0 ? 0 : N;
  }
  const int dv = D / V, units = H / kUnit, groups = ((units - 1) >> shift) + 1;
  {  // the zero rows behind dy_c that the FC2 weight-gradient product reads
    const int64_t zrows = M < N ? min((int64_t)64, N - M) : 0;
    uint4* z = reinterpret_cast<uint4*>(dy_c + M * D);
    for (int64_t i = gtid; i < zrows * dv; i += nthr) z[i] = make_uint4(0, 0, 0, 0);
  }
  const int x_groups = x_cols ? (D + x_cols - 1) / x_cols : 1;
  // a fraction is off by up to 8 of 2^32, which is 4 rows of the most that there can be
  const int64_t teams = nthr / LANES, team = gtid / LANES;
  const int64_t deal = SPREAD ? teams - E - 8 : teams;
  const int64_t rounds = (M + deal - 1) / deal;
  const uint64_t share = rounds ? ((uint64_t)1 << 48) / (uint64_t)rounds : 0;  // 48 bits
  auto fraction = [&](int64_t r) { return (uint32_t)((uint64_t)r * share >> 16); };
  auto row = [&](int64_t round) -> int64_t {
    if (round >= rounds) return -1;
    const int64_t j =
        SPREAD ? row_of_round(sel_off, E, M, fraction(round),
                              round + 1 == rounds ? 0u : fraction(round + 1), team, lane)
               : round * teams + team;
    return j < M ? j : -1;
  };
  // in the rows' own order the next one's place and pair are looked up before this one's data
  int64_t j_next = -1;
  int i_next = -1, p_next = -1;
  auto look = [&](int64_t round) {
    j_next = row(round);
    i_next = j_next >= 0 ? sel_pos[j_next] : -1;
    p_next = i_next >= 0 && i_next < N ? perm[i_next] : -1;
  };
  if (!SPREAD) look(0);
  for (int64_t round = 0; round < rounds; ++round) {
    if (SPREAD) look(round);
    const int64_t j = j_next;
    const int i = i_next, p = p_next;
    if (!SPREAD) look(round + 1);
    if (j < 0) continue;
    if (p < 0 || p >= N) {
      if (lane == 0) flag_error(err, LRM_DEVERR_INDEX);
      continue;
    }
    const int64_t t = p / K;
    const float al = alpha[p];
    const uint8_t* qr = q + (int64_t)i * 2 * H;
    const float* sr = scale + (int64_t)i * 2 * groups;
    const uint4* gs = reinterpret_cast<const uint4*>(g + t * D);
    uint4* dyd = reinterpret_cast<uint4*>(dy_c + j * D);
    for (int c0 = lane; c0 < dv; c0 += LANES * kAheadG) {
      uint4 v[kAheadG];
#pragma unroll
      for (int u = 0; u < kAheadG; ++u)
        if (c0 + LANES * u < dv) v[u] = gs[c0 + LANES * u];
#pragma unroll
      for (int u = 0; u < kAheadG; ++u) {
        if (c0 + LANES * u < dv) {
          float f[V];
          Vec16<T>::unpack(v[u], f);
#pragma unroll
          for (int e = 0; e < V; ++e) f[e] *= al;
          __stcs(dyd + c0 + LANES * u, Vec16<T>::pack(f));
        }
      }
    }
    if (x_c) {
      if (x_scale) {
        const uint8_t* xr = (const uint8_t*)x + t * D;
        const float* xs = x_scale + t * x_groups;
        for (int u = lane; u < D / kUnit; u += LANES) {
          float f[kUnit];
          decode8(*reinterpret_cast<const uint2*>(xr + u * kUnit),
                  xs[x_cols ? u * kUnit / x_cols : 0], f);
          stream8(x_c + j * D + u * kUnit, f);
        }
      } else {
        const uint4* xr = reinterpret_cast<const uint4*>((const T*)x + t * D);
        uint4* xd = reinterpret_cast<uint4*>(x_c + j * D);
        for (int c = lane; c < dv; c += LANES) __stcs(xd + c, xr[c]);
      }
    }
    T* abd = ab_c + j * 2 * H;
    T* pd = phi_c + j * H;
#pragma unroll 1
    for (int u = lane; u < units; u += LANES) {
      const uint2 ca = __ldcs(reinterpret_cast<const uint2*>(qr + u * kUnit));
      const uint2 cb = __ldcs(reinterpret_cast<const uint2*>(qr + H + u * kUnit));
      float a[kUnit], b[kUnit], ph[kUnit];
      decode8(ca, sr[u >> shift], a);
      decode8(cb, sr[groups + (u >> shift)], b);
#pragma unroll
      for (int e = 0; e < kUnit; ++e) ph[e] = silu(a[e]) * b[e];
      stream8(abd + u * kUnit, a);
      stream8(abd + H + u * kUnit, b);
      stream8(pd + u * kUnit, ph);
    }
    if (lane == 0) {
      tok_c[j] = (int32_t)t;
      row_of_pos[i] = (int32_t)j;
    }
  }
}

static lrm_status check_packed(const lrm_packed* p) {
  if (!p) return LRM_ERR_INVALID_ARG;
  if (p->rows < 0 || p->H <= 0) return LRM_ERR_INVALID_ARG;
  if (p->dtype != LRM_F32 && p->dtype != LRM_BF16) return LRM_ERR_INVALID_ARG;
  if (p->H % 8 != 0 || p->rows >= (int64_t)1 << 31) return LRM_ERR_UNSUPPORTED;
  if (p->cols != 32 && p->cols != 64 && p->cols != 128) return LRM_ERR_UNSUPPORTED;
  if (p->rows > 0 && (!p->q || !p->scale || !p->phi_sq)) return LRM_ERR_INVALID_ARG;
  for (const void* b : {(const void*)p->q, (const void*)p->scale, (const void*)p->phi_sq})
    if (!aligned16(b)) return LRM_ERR_UNSUPPORTED;
  return LRM_OK;
}

static int group_shift(int cols) { return cols == 32 ? 2 : cols == 64 ? 3 : 4; }

// The state is the layer's: as many pairs, the same width and type.
static lrm_status check_layer(const lrm_shape* s, const lrm_packed* p, const void* ws,
                              size_t ws_bytes) {
  lrm_status st = check_shape(s);
  if (st != LRM_OK) return st;
  if ((st = check_packed(p)) != LRM_OK) return st;
  if (p->rows != (int64_t)s->T * s->K || p->H != s->H || p->dtype != s->dtype)
    return LRM_ERR_INVALID_ARG;
  return check_ws(s, ws, ws_bytes);
}

template <typename T>
static lrm_status launch_pack(const lrm_packed* p, const void* ab, cudaStream_t cs) {
  const int units = p->H / kUnit;
  const int lanes = units <= 4 ? 4 : units <= 8 ? 8 : units <= 16 ? 16 : 32;
  // a lane's units in even rounds of up to four
  const int mine = (units + 31) / 32, rounds = (mine + 3) / 4, ni = (mine + rounds - 1) / rounds;
  auto kern = lanes == 4    ? pack_kernel<T, 1, 4>
              : lanes == 8  ? pack_kernel<T, 1, 8>
              : lanes == 16 ? pack_kernel<T, 1, 16>
              : ni == 1     ? pack_kernel<T, 1, 32>
              : ni == 2     ? pack_kernel<T, 2, 32>
              : ni == 3     ? pack_kernel<T, 3, 32>
                            : pack_kernel<T, 4, 32>;
  const int per_cta = kPackThreads / lanes;
  // a group that is wider than the row is the row
  int shift = group_shift(p->cols);
  while (shift > 0 && (1 << shift) > lanes) --shift;
  launch_k(kern, dim3((unsigned)((p->rows + per_cta - 1) / per_cta)), dim3(kPackThreads), 0, cs,
           (const T*)ab, p->rows, p->H, shift, p->q, p->scale, p->phi_sq);
  return launch_status();
}

}  // namespace lrm

using namespace lrm;

extern "C" lrm_status lrm_pack_state(const lrm_packed* p, const void* ab, void* stream) {
  LRM_NVTX("lrm_pack_state");
  lrm_status st = check_packed(p);
  if (st != LRM_OK) return st;
  if (p->rows == 0) return LRM_OK;
  if (!ab) return LRM_ERR_INVALID_ARG;
  if (!aligned16(ab)) return LRM_ERR_UNSUPPORTED;
  return p->dtype == LRM_BF16 ? launch_pack<__nv_bfloat16>(p, ab, (cudaStream_t)stream)
                              : launch_pack<float>(p, ab, (cudaStream_t)stream);
}

extern "C" lrm_status lrm_score_packed(const lrm_shape* s, const lrm_packed* p, const void* g,
                                       const float* alpha, const int32_t* inv, float* score,
                                       void* ws, size_t ws_bytes, void* stream) {
  LRM_NVTX("lrm_score_packed");
  lrm_status st = check_layer(s, p, ws, ws_bytes);
  if (st != LRM_OK) return st;
  if (s->T == 0) return LRM_OK;
  if (!g || !alpha || !inv || !score) return LRM_ERR_INVALID_ARG;
  if (!aligned16(g)) return LRM_ERR_UNSUPPORTED;
  cudaStream_t cs = (cudaStream_t)stream;
  auto go = [&](auto kern, auto* type, int lanes) {
    using T = std::remove_pointer_t<decltype(type)>;
    const int per_cta = 32 * kScoreWarps / lanes;
    launch_k(kern, dim3((unsigned)(((int64_t)s->T + per_cta - 1) / per_cta)),
             dim3(32 * kScoreWarps), 0, cs, (const T*)g, (const float*)p->phi_sq, alpha, inv, score,
             s->T, s->D, s->K, error_word(ws));
  };
  auto pick = [&](auto* type) {
    using T = std::remove_pointer_t<decltype(type)>;
    // by the width alone: a token's score does not depend on how many others there are
    const int chunks = s->D / Vec16<T>::kElems;
    if (chunks <= 32) go(score_packed_kernel<T, 8>, type, 8);
    else if (chunks <= 128) go(score_packed_kernel<T, 16>, type, 16);
    else go(score_packed_kernel<T, 32>, type, 32);
  };
  if (s->dtype == LRM_BF16) pick((__nv_bfloat16*)nullptr);
  else pick((float*)nullptr);
  return launch_status();
}

extern "C" lrm_status lrm_compact_packed(
    const lrm_shape* s, const lrm_packed* pk, const int32_t* perm, const uint8_t* keep,
    const int32_t* sel_off, const int32_t* sel_pos, const float* alpha, const void* x,
    const float* x_scale, int32_t x_cols, const void* g, void* dy_c, void* x_c, void* ab_c,
    void* phi_c, int32_t* tok_c, int32_t* row_of_pos, void* ws, size_t ws_bytes, void* stream) {
  LRM_NVTX("lrm_compact_packed");
  lrm_status st = check_layer(s, pk, ws, ws_bytes);
  if (st != LRM_OK) return st;
  if (x_c && x_scale && x_cols != 0 && x_cols != 32 && x_cols != 64 && x_cols != 128 &&
      x_cols != 256)
    return LRM_ERR_UNSUPPORTED;
  if (pk->rows == 0) return LRM_OK;
  for (const void* p : {(const void*)perm, (const void*)keep, (const void*)sel_off,
                        (const void*)sel_pos, (const void*)alpha, g, (const void*)dy_c,
                        (const void*)ab_c, (const void*)phi_c, (const void*)tok_c,
                        (const void*)row_of_pos})
    if (!p) return LRM_ERR_INVALID_ARG;
  if (x_c && !x) return LRM_ERR_INVALID_ARG;
  for (const void* p : {x, g, (const void*)dy_c, (const void*)x_c, (const void*)ab_c,
                        (const void*)phi_c})
    if (!aligned16(p)) return LRM_ERR_UNSUPPORTED;
  const dim3 grid(num_sms() * kUnpackCtas);
  cudaStream_t cs = (cudaStream_t)stream;
  const int shift = group_shift(pk->cols);
  const int64_t warps = (int64_t)grid.x * (kUnpackThreads / 32);
  // Cotangents that L2 holds are read from it in any order, and narrow rows pass faster in their
  // own, each one's place known before its turn (bfloat16, half of 8 a token, us spread | in
  // order: T 16384 D 512 H 256 53 | 40, D 1024 H 512 82 | 79, D 2048 H 768 131 | 146; T 8192
  // D 2048 H 704 66 | 67; T 32768 D 1024 H 512 160 | 169, 4 a token H 256 72 | 63). The line at
  // 4096 bytes a row leaves the one that loses by 6% on the wrong side of it.
  const int64_t row_bytes = (int64_t)s->D * (s->dtype == LRM_BF16 ? 2 : 4);
  const bool spread = pk->rows > warps && warps > 2 * (int64_t)s->E + 16 && row_bytes >= 4096 &&
                      row_bytes * s->T >= 32 << 20;
  // Few lanes for a narrow row (T 29084 D 80 H 48 float32, us with 8 | 16 | 32 lanes: 30 | 35 |
  // 54; T 7260 D 320 H 128 bfloat16 15 | 16 | 23; T 16384 D 512 H 256 42 | 40 | 41), as long as
  // the rows are more than the teams (T 969 of 4, D 168 H 208: 5.3 | 4.6 | 4.1).
  int lanes = row_bytes <= 512 && s->H <= 64 ? 8 : row_bytes <= 1024 && s->H <= 256 ? 16 : 32;
  while (lanes < 32 && pk->rows <= warps * 16 / lanes) lanes *= 2;
  auto go = [&](auto kern, auto* type) {
    using T = std::remove_pointer_t<decltype(type)>;
    launch_k(kern, grid, dim3(kUnpackThreads), 0, cs, (const uint8_t*)pk->q,
             (const float*)pk->scale, shift, perm, keep, sel_off, sel_pos, alpha, x, x_scale,
             x_cols, (const T*)g, (T*)dy_c, (T*)x_c, (T*)ab_c, (T*)phi_c, tok_c, row_of_pos,
             s->T, s->D, s->H, s->K, s->E, error_word(ws));
  };
  auto pick = [&](auto* type) {
    using T = std::remove_pointer_t<decltype(type)>;
    if (spread) go(compact_packed_kernel<T, 32, true>, type);
    else if (lanes == 8) go(compact_packed_kernel<T, 8, false>, type);
    else if (lanes == 16) go(compact_packed_kernel<T, 16, false>, type);
    else go(compact_packed_kernel<T, 32, false>, type);
  };
  if (s->dtype == LRM_BF16) pick((__nv_bfloat16*)nullptr);
  else pick((float*)nullptr);
  return launch_status();
}
