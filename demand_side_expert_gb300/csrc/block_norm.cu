// The norms around a block with what stands between them, and the gradients.
//   u = block rstd_b w_post,  h = c res + gate u,  y = h rstd w (or e4m3 rows of it)
//   dhs = rstd (w dy - xhat mean(w dy xhat)) + dh,  dres = c dhs,  dw = sum_t dy xhat
//   du = gate dhs,  dblock = rstd_b (w_post du - ohat mean(w_post du ohat))
//   xhat = h rstd,  ohat = block rstd_b
// The backward pass needs two means of a row, the second of what the first gives. With
// k = w_post (times the gate of a column) and P = sum k ohat dhs, which is the gradient
// of a token's gate too, dhs is linear in m = mean(w dy xhat):
//   P = sum k ohat (rstd w dy + dh) - m sum k ohat rstd xhat,
// so one round over the row's threads gives all three sums.
// w_post's and a column gate's gradients are one sum of columns, c_d = sum_t dhs ohat:
// dw_post = gate c and dgate = w_post c (a token's gate is inside the sum).
#include <algorithm>

#include "rows.cuh"

namespace lrm {

constexpr int kBlockMaxD = 8192;
constexpr int kBlockMaxCtas = 160;  // partial column sums in the workspace

// Forward: TPR threads a row (lanes of a warp, or a CTA), UPT units of 8 columns a
// thread; the row stays in registers from its loads to its stores.
template <int TPR>
constexpr int block_threads() { return TPR < 64 ? 128 : TPR; }

template <typename T, typename O, int TPR, int UPT>
__global__ void __launch_bounds__(block_threads<TPR>())
block_norm_kernel(const O* __restrict__ block, const T* res, const T* __restrict__ w,
                  const T* __restrict__ w_post, const T* __restrict__ gate, T* h,
                  T* __restrict__ y, uint8_t* __restrict__ q, float* __restrict__ q_scale,
                  float* __restrict__ rstd, float* __restrict__ block_rstd, int rows, int D,
                  int64_t block_stride, int64_t res_stride, int gate_kind, int q_shift, float eps,
                  float res_scale) {
  pdl_begin();  // predecessor complete before any global access
  __shared__ float red[3][32];
  const int tl = threadIdx.x % TPR;
  const int units = D / kUnit;
  const int64_t r = (int64_t)blockIdx.x * (block_threads<TPR>() / TPR) + threadIdx.x / TPR;
  if (TPR >= 32 && r >= rows) return;
  // several rows a warp: its lanes stay together, those past the end only reduce
  const bool real = TPR >= 32 || r < rows;
  const O* po = block + r * block_stride + tl * kUnit;
  const T* pr = res + r * res_stride + tl * kUnit;
  const int64_t at = r * D + tl * kUnit;  // of the thread's first unit in an output
  Unit8<O> vo[UPT];
  Unit8<T> vr[UPT];
#pragma unroll
  for (int i = 0; i < UPT; ++i) vo[i].load(po + i * TPR * kUnit, real && tl + i * TPR < units);
#pragma unroll
  for (int i = 0; i < UPT; ++i) vr[i].load(pr + i * TPR * kUnit, real && tl + i * TPR < units);
  float g = 1.f;
  if (gate_kind == LRM_GATE_TOKEN && real) g = (float)gate[r];
  float rb = 1.f;
  if (w_post) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
      float f[kUnit];
      vo[i].get(f);
#pragma unroll
      for (int j = 0; j < kUnit; ++j) s = fmaf(f[j], f[j], s);
    }
    s = row_reduce<TPR, false>(s, red, 0);
    rb = rsqrtf(fmaf(s, 1.f / (float)D, eps));
    if (block_rstd && tl == 0 && real) block_rstd[r] = rb;
  }
  float f[UPT][kUnit];
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < UPT; ++i) {
    const int col = (tl + i * TPR) * kUnit;
    float v[kUnit];
    vo[i].get(f[i]);
    vr[i].get(v);
    if (tl + i * TPR < units) {
      float m[kUnit];
      if (w_post) {
        Unit8<T> vw;
        vw.load_cached(w_post + col);
        vw.get(m);
#pragma unroll
        for (int j = 0; j < kUnit; ++j) f[i][j] = f[i][j] * rb * m[j];
      }
      if (gate_kind == LRM_GATE_COLUMN) {
        Unit8<T> vw;
        vw.load_cached(gate + col);
        vw.get(m);
#pragma unroll
        for (int j = 0; j < kUnit; ++j) f[i][j] *= m[j];
      }
    }
#pragma unroll
    for (int j = 0; j < kUnit; ++j) {
      f[i][j] = fmaf(res_scale, v[j], g * f[i][j]);
      s = fmaf(f[i][j], f[i][j], s);
    }
  }
  s = row_reduce<TPR, false>(s, red, 1);
  const float rs = rsqrtf(fmaf(s, 1.f / (float)D, eps));
  if (rstd && tl == 0 && real) rstd[r] = rs;
  float rowmax = 0.f;
#pragma unroll
  for (int i = 0; i < UPT; ++i) {
    const int u = tl + i * TPR;
    const bool in = real && u < units;
    if (in) {
      store8(h + at + i * TPR * kUnit, f[i]);
      Unit8<T> vw;
      vw.load_cached(w + u * kUnit);
      float m[kUnit];
      vw.get(m);
#pragma unroll
      for (int j = 0; j < kUnit; ++j) f[i][j] = f[i][j] * rs * m[j];
      if (y) store8(y + at + i * TPR * kUnit, f[i]);
    }
    if (q) {
      float m = 0.f;  // units past the row are 0
#pragma unroll
      for (int j = 0; j < kUnit; ++j) m = fmaxf(m, fabsf(f[i][j]));
      if (q_shift >= 0) {
        // a group is 2^q_shift consecutive lanes, or the whole of a shorter row
#pragma unroll
        for (int b = 0; b < 5; ++b)
          if ((1 << b) < TPR && b < q_shift) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1 << b));
        m = fmaxf(m, kAmaxMin);
        if (in) {
          store_e4m3(q + at + i * TPR * kUnit, f[i], __frcp_rn(m) * kF8Max);
          if ((u & ((1 << q_shift) - 1)) == 0)
            q_scale[r * ((units - 1 >> q_shift) + 1) + (u >> q_shift)] = m * kF8MaxInv;
        }
      } else {
        rowmax = fmaxf(rowmax, m);
      }
    }
  }
  if (q && q_shift < 0) {
    const float m = fmaxf(row_reduce<TPR, true>(rowmax, red, 2), kAmaxMin);
    const float k = __frcp_rn(m) * kF8Max;
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
      const int u = tl + i * TPR;
      if (real && u < units) store_e4m3(q + at + i * TPR * kUnit, f[i], k);
    }
    if (tl == 0 && real) q_scale[r] = m * kF8MaxInv;
  }
}

// Backward: `tpr` threads a row (4, 8 or 16 lanes, or whole warps), UPT units a thread,
// as many row groups a CTA as its threads and the shared memory hold, one CTA an SM. A
// row's inputs are copied to their thread's own places in shared memory `stages` - 1 rows
// ahead, so an SM's loads do not stop while a row's sums are formed; the column sums stay
// in registers over all of a thread's rows. HBM-bound: T 16384 D 4096, float32 block and
// gradients, moves 1.34 GB in 206 us, 0.96 of the copy bandwidth.
constexpr int kBlockThreads = 512;
constexpr int kBlockRing = 224 * 1024;  // bytes of a CTA's copies in flight, at most
constexpr int kBlockStages = 6;
constexpr int kColumnsSmem = 216 * 1024;  // the last kernel's, which it does not use

__device__ __forceinline__ void block_wait(int stages) {
  switch (stages) {
    case 1: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 3: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    case 4: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    case 5: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
  }
}

// Three sums over a row's threads. Every thread of the CTA calls it as often as the
// others, whether its row exists or not.
struct RowSums {
  int tpr, group, tl;
  float4 (*red)[kBlockThreads / 32];  // [2][warps of the CTA]
  int flip = 0;
  __device__ __forceinline__ void sum(float (&v)[3]) {
    for (int o = min(tpr, 32) / 2; o > 0; o >>= 1)
#pragma unroll
      for (int k = 0; k < 3; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    if (tpr > 32) {
      const int warps = tpr >> 5;
      float4* mine = red[flip] + group * warps;
      if ((threadIdx.x & 31) == 0) mine[tl >> 5] = make_float4(v[0], v[1], v[2], 0.f);
      asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(tpr) : "memory");
      const int k = threadIdx.x & 15;  // a warp of the row's, of at most 16
      const float4 q = k < warps ? mine[k] : make_float4(0.f, 0.f, 0.f, 0.f);
      v[0] = q.x;
      v[1] = q.y;
      v[2] = q.z;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1)
#pragma unroll
        for (int j = 0; j < 3; ++j) v[j] += __shfl_xor_sync(0xffffffffu, v[j], o);
      flip ^= 1;  // the other buffer next: one barrier a sum is enough
    }
  }
};

template <typename T, typename O, typename G>
struct BlockBwd {
  const G *dy, *dh;
  const T* h;
  const O* block;
  const T *w, *w_post, *gate;
  const float *rstd, *block_rstd;
  G* dres;
  T* dblock;
  float *dw, *dw_post, *dgate;
  float* part;  // [CTAs][2][D]
  int rows, D, gate_kind, tpr, stages;
  float res_scale;
};

// The gradients that a column's two sums stand for.
template <typename T, typename O, typename G>
__device__ __forceinline__ void write_columns(const BlockBwd<T, O, G>& a, int c, float sw,
                                              float sc) {
  a.dw[c] = sw;
  const bool column = a.gate_kind == LRM_GATE_COLUMN;
  if (a.w_post) a.dw_post[c] = column ? (float)a.gate[c] * sc : sc;
  if (column) a.dgate[c] = a.w_post ? (float)a.w_post[c] * sc : sc;
}

// What a lane loads and stores at once in the backward pass: Q consecutive columns, the 16
// bytes of 4 float32 ones (or 8 where every row is bfloat16), so that a warp's access is 512
// bytes in a row. With 8 columns of float32, two pieces of 16 bytes a lane, T 16384 D 4096
// took 284 us instead of 206.
template <typename O, typename G>
constexpr int lane_columns() { return sizeof(O) == 2 && sizeof(G) == 2 ? 8 : 4; }

template <int BYTES>
struct Bytes;
template <>
struct Bytes<8> { using type = uint2; };
template <>
struct Bytes<16> { using type = uint4; };

template <typename T, int Q>
struct alignas(Q * sizeof(T)) Columns {
  uint32_t w[Q * sizeof(T) / 4];
  __device__ __forceinline__ void get(Pair (&f)[Q / 2]) const {
    const auto v = *reinterpret_cast<const typename Bytes<Q * sizeof(T)>::type*>(w);
    const uint32_t* u = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < Q / 2; ++i) {
      if constexpr (sizeof(T) == 4)
        f[i] = pair(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]));
      else
        f[i] = pair(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
    }
  }
  __device__ __forceinline__ void set(const Pair (&f)[Q / 2]) {
    typename Bytes<Q * sizeof(T)>::type v;
    uint32_t* u = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < Q / 2; ++i) {
      const float2 p = floats(f[i]);
      if constexpr (sizeof(T) == 4) {
        u[2 * i] = __float_as_uint(p.x);
        u[2 * i + 1] = __float_as_uint(p.y);
      } else {
        __nv_bfloat162 h = __float22bfloat162_rn(p);
        u[i] = *reinterpret_cast<uint32_t*>(&h);
      }
    }
    *reinterpret_cast<typename Bytes<Q * sizeof(T)>::type*>(w) = v;
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(w) / 4); ++i) w[i] = 0;
  }
};
template <int Q, typename T>
__device__ __forceinline__ void load_columns(const T* p, Pair (&f)[Q / 2]) {
  reinterpret_cast<const Columns<T, Q>*>(p)->get(f);
}
template <int Q, typename T>
__device__ __forceinline__ void store_columns(T* p, const Pair (&f)[Q / 2]) {
  if constexpr (Q * sizeof(T) <= 16) {
    reinterpret_cast<Columns<T, Q>*>(p)->set(f);
  } else {
    reinterpret_cast<Columns<T, Q / 2>*>(p)[0].set(*reinterpret_cast<const Pair(*)[Q / 4]>(&f[0]));
    reinterpret_cast<Columns<T, Q / 2>*>(p)[1].set(*reinterpret_cast<const Pair(*)[Q / 4]>(&f[Q / 4]));
  }
}
// Columns from global to shared memory.
template <int Q, typename T>
__device__ __forceinline__ void copy_columns(uint32_t dst, const T* src) {
  if constexpr (Q * sizeof(T) == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}

// With q = rstd^2 m the row is a line in h: dhs = (w rstd dy + dh) - q h.
template <typename T, typename O, typename G, int UPT>
__global__ void __launch_bounds__(kBlockThreads)
block_norm_bwd_kernel(const BlockBwd<T, O, G> a) {
  constexpr int Q = lane_columns<O, G>(), kPairs = Q / 2;
  extern __shared__ uint4 ring[];  // [stages][UPT][h, block, dy, dh][threads]
  __shared__ float4 red[2][kBlockThreads / 32];
  const int threads = blockDim.x, tpr = a.tpr, groups = threads / tpr, D = a.D, rows = a.rows;
  RowSums row{tpr, (int)threadIdx.x / tpr, (int)threadIdx.x % tpr, red};
  const int tl = row.tl;
  const int chunks = D / Q;
  // bytes of a chunk's inputs, and of a stage; where a thread's own places begin
  const uint32_t each = threads * Q * (uint32_t)(sizeof(T) + sizeof(O) + sizeof(G) * (a.dh ? 2 : 1));
  const uint32_t stage = UPT * each;
  const uint32_t at_h = threadIdx.x * Q * sizeof(T);
  const uint32_t at_o = threads * Q * sizeof(T) + threadIdx.x * Q * sizeof(O);
  const uint32_t at_d = threads * Q * (sizeof(T) + sizeof(O)) + threadIdx.x * Q * sizeof(G);
  const uint32_t at_e = at_d + threads * Q * sizeof(G);
  const float inv_d = 1.f / (float)D;
  const bool post = a.w_post != nullptr, token = a.gate_kind == LRM_GATE_TOKEN;
  pdl_begin();  // predecessor complete before any global access
  const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(ring);
  char* const ring_c = reinterpret_cast<char*>(ring);
  // A row's columns into the thread's own places of a stage. Places without columns, or
  // without a row, are set to 0, so that they are read like any other.
  auto copy_row = [&](int64_t r, int slot) {
    uint32_t dst = slot * stage;
    const int64_t at = r * D + tl * Q;
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
      const int64_t p = at + i * tpr * Q;
      if (r < rows && tl + i * tpr < chunks) {
        copy_columns<Q>(ring_at + dst + at_h, a.h + p);
        copy_columns<Q>(ring_at + dst + at_o, a.block + p);
        copy_columns<Q>(ring_at + dst + at_d, a.dy + p);
        if (a.dh) copy_columns<Q>(ring_at + dst + at_e, a.dh + p);
      } else {
        reinterpret_cast<Columns<T, Q>*>(ring_c + dst + at_h)->zero();
        reinterpret_cast<Columns<O, Q>*>(ring_c + dst + at_o)->zero();
        reinterpret_cast<Columns<G, Q>*>(ring_c + dst + at_d)->zero();
        if (a.dh) reinterpret_cast<Columns<G, Q>*>(ring_c + dst + at_e)->zero();
      }
      dst += each;
    }
    copies_commit();
  };
  int64_t base = (int64_t)blockIdx.x * groups;
  const int64_t dr = (int64_t)gridDim.x * groups;
  for (int i = 0; i < a.stages - 1; ++i) copy_row(base + row.group + i * dr, i);
  // the thread's columns: w, and k = w_post times a column's gate
  Pair fw[UPT][kPairs], kc[UPT][kPairs], sum_w[UPT][kPairs], sum_c[UPT][kPairs];
#pragma unroll
  for (int i = 0; i < UPT; ++i) {
    const int c = (tl + i * tpr) * Q;
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      kc[i][j] = pair(1.f, 1.f);
      fw[i][j] = sum_w[i][j] = sum_c[i][j] = pair(0.f, 0.f);
    }
    if (c < D) {
      load_columns<Q>(a.w + c, fw[i]);
      if (post) load_columns<Q>(a.w_post + c, kc[i]);
      if (a.gate_kind == LRM_GATE_COLUMN) {
        Pair m[kPairs];
        load_columns<Q>(a.gate + c, m);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) kc[i][j] = mul2(kc[i][j], m[j]);
      }
    }
  }
  // a row's scalars, read a row ahead
  float next_rs, next_rb, next_g;
  auto scalars = [&](int64_t r) {
    const bool in = r < rows;
    next_rs = in ? __ldg(a.rstd + r) : 0.f;
    next_rb = in && post ? __ldg(a.block_rstd + r) : 1.f;
    next_g = in && token ? (float)a.gate[r] : 1.f;
  };
  scalars(base + row.group);
  int slot = 0;
  for (; base < rows; base += dr) {
    const int64_t r = base + row.group;
    copy_row(r + (a.stages - 1) * dr, slot == 0 ? a.stages - 1 : slot - 1);
    const float rs = next_rs, rb = next_rb, g = next_g;
    scalars(r + dr);
    block_wait(a.stages);
    const char* v = ring_c + slot * stage;
    auto take = [&](int i, Pair (&h)[kPairs], Pair (&o)[kPairs], Pair (&d)[kPairs],
                    Pair (&e)[kPairs]) {
      const char* p = v + i * each;
      reinterpret_cast<const Columns<T, Q>*>(p + at_h)->get(h);
      reinterpret_cast<const Columns<O, Q>*>(p + at_o)->get(o);
      reinterpret_cast<const Columns<G, Q>*>(p + at_d)->get(d);
      for (int j = 0; j < kPairs; ++j) e[j] = pair(0.f, 0.f);
      if (a.dh) reinterpret_cast<const Columns<G, Q>*>(p + at_e)->get(e);
    };
    // 8 columns a thread: their values stay in registers for the second look
    constexpr bool kKeep = UPT * Q <= 8;
    constexpr int kHeld = kKeep ? UPT : 1;
    Pair h[kHeld][kPairs], o[kHeld][kPairs], d[kHeld][kPairs], e[kHeld][kPairs];
    const Pair rs2 = pair(rs, rs);
    Pair s0 = pair(0.f, 0.f), s1 = s0, s2 = s0;
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
      const int n = kKeep ? i : 0;
      take(i, h[n], o[n], d[n], e[n]);
#pragma unroll
      for (int j = 0; j < kPairs; ++j) {
        const Pair t = mul2(rs2, d[n][j]), wt = mul2(fw[i][j], t), ko = mul2(kc[i][j], o[n][j]);
        sum_w[i][j] = fma2(t, h[n][j], sum_w[i][j]);
        s0 = fma2(wt, h[n][j], s0);
        s2 = fma2(ko, h[n][j], s2);
        e[n][j] = fma2(fw[i][j], t, e[n][j]);
        s1 = fma2(ko, e[n][j], s1);
      }
    }
    float s[3] = {floats(s0).x + floats(s0).y, floats(s1).x + floats(s1).y,
                  floats(s2).x + floats(s2).y};
    row.sum(s);
    const float q = rs * rs * (s[0] * inv_d), P = rb * fmaf(-q, s[2], s[1]);
    if (token && tl == 0 && r < rows) a.dgate[r] = P;
    const float m2 = post ? -rb * rb * (g * P * inv_d) : 0.f;
    const Pair nq2 = pair(-q, -q), m22 = pair(m2, m2), gb2 = pair(g * rb, g * rb),
               c2 = pair(a.res_scale, a.res_scale);
    if (r < rows) {
#pragma unroll
      for (int i = 0; i < UPT; ++i) {
        const int n = kKeep ? i : 0, c = (tl + i * tpr) * Q;
        if (c < D) {
          if (!kKeep) {
            take(i, h[n], o[n], d[n], e[n]);
#pragma unroll
            for (int j = 0; j < kPairs; ++j)
              e[n][j] = fma2(fw[i][j], mul2(rs2, d[n][j]), e[n][j]);
          }
#pragma unroll
          for (int j = 0; j < kPairs; ++j) {
            const Pair dhs = fma2(nq2, h[n][j], e[n][j]), v2 = mul2(gb2, dhs);
            sum_c[i][j] = fma2(v2, o[n][j], sum_c[i][j]);
            d[n][j] = mul2(c2, dhs);
            e[n][j] = fma2(kc[i][j], v2, mul2(m22, o[n][j]));
          }
          store_columns<Q>(a.dres + r * D + c, d[n]);
          store_columns<Q>(a.dblock + r * D + c, e[n]);
        }
      }
    }
    slot = slot + 1 == a.stages ? 0 : slot + 1;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  // the CTA's sums over its row groups, in a fixed order: the groups of a warp by
  // exchanges, the rest through shared memory
  for (int o = tpr; o < 32; o <<= 1)
#pragma unroll
    for (int i = 0; i < UPT; ++i)
#pragma unroll
      for (int j = 0; j < kPairs; ++j) {
        sum_w[i][j] = add2(sum_w[i][j], __shfl_xor_sync(0xffffffffu, sum_w[i][j], o));
        sum_c[i][j] = add2(sum_c[i][j], __shfl_xor_sync(0xffffffffu, sum_c[i][j], o));
      }
  const int wide = max(tpr, 32), sums = threads / wide;
  const bool writes = (int)threadIdx.x % wide < tpr;
  float* out = a.part + (int64_t)blockIdx.x * 2 * D;
  __syncthreads();  // the ring is free
  float* sm = reinterpret_cast<float*>(ring);  // [sums][2][D]
#pragma unroll
  for (int i = 0; i < UPT; ++i)
    if (writes && tl + i * tpr < chunks) {
      float* p = sm + ((int)threadIdx.x / wide * 2) * D + (tl + i * tpr) * Q;
      store_columns<Q>(p, sum_w[i]);
      store_columns<Q>(p + D, sum_c[i]);
    }
  __syncthreads();
  for (int c = threadIdx.x; c < D; c += threads) {
    float t0 = 0.f, t1 = 0.f;
    for (int k = 0; k < sums; ++k) {
      t0 += sm[2 * k * D + c];
      t1 += sm[(2 * k + 1) * D + c];
    }
    if (gridDim.x == 1) {
      write_columns(a, c, t0, t1);
    } else {
      out[c] = t0;
      out[D + c] = t1;
    }
  }
}

// The column sums of the CTAs, added in a fixed order: 32 columns a CTA, 16 threads a
// column, every load before any use.
constexpr int kBlockColThreads = 512;
template <typename T, typename O, typename G>
__global__ void __launch_bounds__(kBlockColThreads)
block_columns_kernel(const BlockBwd<T, O, G> a, int nrows) {
  pdl_begin();  // predecessor complete before any global access
  constexpr int kWarps = kBlockColThreads / 32, kEach = (kBlockMaxCtas + kWarps - 1) / kWarps;
  __shared__ float2 sm[kWarps][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane, D = a.D;
  float2 v[kEach];
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int r = warp + k * kWarps;
    const bool in = c < D && r < nrows;
    const float* p = a.part + (int64_t)r * 2 * D + c;
    v[k] = in ? make_float2(p[0], p[D]) : make_float2(0.f, 0.f);
  }
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    s.x += v[k].x;
    s.y += v[k].y;
  }
  sm[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < D) {
    float2 t = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      t.x += sm[k][lane].x;
      t.y += sm[k][lane].y;
    }
    write_columns(a, c, t.x, t.y);
  }
}

__global__ void zero_columns_kernel(float* dw, float* dw_post, float* dgate, int D) {
  pdl_begin();  // predecessor complete before any global access
  for (int c = threadIdx.x; c < D; c += blockDim.x) {
    dw[c] = 0.f;
    if (dw_post) dw_post[c] = 0.f;
    if (dgate) dgate[c] = 0.f;
  }
}

static lrm_status check_block(const lrm_block* b) {
  if (!b) return LRM_ERR_INVALID_ARG;
  if (b->T < 0 || b->D <= 0 || b->q_cols < 0) return LRM_ERR_INVALID_ARG;
  for (int32_t dt : {b->dtype, b->block_dtype, b->grad_dtype})
    if (dt != LRM_F32 && dt != LRM_BF16) return LRM_ERR_INVALID_ARG;
  if (b->gate < LRM_GATE_NONE || b->gate > LRM_GATE_TOKEN) return LRM_ERR_INVALID_ARG;
  if (!(b->eps >= 0.f)) return LRM_ERR_INVALID_ARG;
  if (b->block_stride < b->D || b->res_stride < b->D) return LRM_ERR_INVALID_ARG;
  if (b->block_dtype != LRM_F32 && b->block_dtype != b->dtype) return LRM_ERR_UNSUPPORTED;
  if (b->D % kUnit != 0 || b->D > kBlockMaxD) return LRM_ERR_UNSUPPORTED;
  if (b->block_stride % kUnit != 0 || b->res_stride % kUnit != 0) return LRM_ERR_UNSUPPORTED;
  if (b->q_cols != 0 && b->q_cols != 32 && b->q_cols != 64 && b->q_cols != 128 &&
      b->q_cols != 256)
    return LRM_ERR_UNSUPPORTED;
  return LRM_OK;
}

static size_t block_bytes(const lrm_block* b) {
  const size_t n = kWsHeaderBytes + (size_t)kBlockMaxCtas * 2 * b->D * 4;
  return (n + 255) / 256 * 256;
}

struct BlockFwd {
  const void *block, *res, *w, *w_post, *gate;
  void *h, *y;
  uint8_t* q;
  float *q_scale, *rstd, *block_rstd;
};

template <typename T, typename O, int TPR, int UPT>
static lrm_status launch_block(const lrm_block* b, const BlockFwd& a, cudaStream_t cs) {
  constexpr int kRows = block_threads<TPR>() / TPR;
  int q_shift = -1;  // log2 of a group's units, -1: the row is the group
  for (int u = b->q_cols / kUnit; u > 0; u >>= 1) ++q_shift;
  launch_k(block_norm_kernel<T, O, TPR, UPT>,
           dim3((unsigned)((b->T + (int64_t)kRows - 1) / kRows)), dim3(block_threads<TPR>()), 0,
           cs, (const O*)a.block, (const T*)a.res, (const T*)a.w, (const T*)a.w_post,
           (const T*)a.gate, (T*)a.h, (T*)a.y, a.q, a.q_scale, a.rstd, a.block_rstd, b->T, b->D,
           b->block_stride, b->res_stride, b->gate, q_shift, b->eps, b->residual_scale);
  return launch_status();
}

template <typename T, typename O>
static lrm_status pick_block(const lrm_block* b, const BlockFwd& a, cudaStream_t cs) {
  const int D = b->D;
  // Few elements an SM: as many threads a row as it has units (512 at most), for the latency of
  // one row (bfloat16 rows, float32 block, us so | several units a thread: D 1024 T 608 2.9 | 4.5,
  // T 2432 7.2 | 9.0, past the edge T 4864 11.2 | 15.7, T 19456 33.0 | 36.7, T 58368 91 | 93;
  // D 2048 T 304 3.0 | 3.5, T 1216 7.7 | 6.9, T 29184 95 | 90; D 4096 T 152 3.4 | 3.8, T 608
  // 8.5 | 7.2, T 14592 105 | 92; D 8192 T 304 7.6 | 9.9, T 7296 99 | 98).
  // Rows of 8192 columns that are all float32 would gain by it at any T (T 7296 174 | 198, 0.81
  // and 0.71 of the copy bandwidth; D 6144 182 | 173).
  // Narrow rows have a unit a thread up to 256 columns; of the copy bandwidth, 0.17 to 0.34 GB in
  // all, and with two units a thread: D 32 0.91 | 0.80, D 64 0.96 | 0.97, D 128 0.96 | 0.94,
  // D 256 0.95 | 0.95. D 512 has two units, 0.94; one on 64 threads 0.72.
  const bool few = (int64_t)b->T * D <= (int64_t)num_sms() * 16384;
  if (D <= 32) return launch_block<T, O, 4, 1>(b, a, cs);
  if (D <= 64) return launch_block<T, O, 8, 1>(b, a, cs);
  if (D <= 128) return launch_block<T, O, 16, 1>(b, a, cs);
  if (D <= 256) return launch_block<T, O, 32, 1>(b, a, cs);
  if (D <= 512) return launch_block<T, O, 32, 2>(b, a, cs);
  if (D <= 1024)
    return few ? launch_block<T, O, 128, 1>(b, a, cs) : launch_block<T, O, 32, 4>(b, a, cs);
  if (D <= 2048)
    return few ? launch_block<T, O, 256, 1>(b, a, cs) : launch_block<T, O, 128, 2>(b, a, cs);
  if (D <= 4096)
    return few ? launch_block<T, O, 512, 1>(b, a, cs) : launch_block<T, O, 256, 2>(b, a, cs);
  return few ? launch_block<T, O, 512, 2>(b, a, cs) : launch_block<T, O, 256, 4>(b, a, cs);
}

// The limit of dynamic shared memory is the kernel's, for all host threads, so it is
// only ever set to the most that any call needs.
template <typename K>
static bool allow_smem(K kern, size_t smem, int most) {
  if (smem <= 40 * 1024) return true;
  if (smem <= (size_t)most &&
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most) ==
          cudaSuccess)
    return true;
  (void)cudaGetLastError();
  return false;
}

template <typename T, typename O, typename G, int UPT>
static lrm_status launch_block_bwd(BlockBwd<T, O, G> a, cudaStream_t cs) {
  const int64_t rows = a.rows;
  constexpr int Q = lane_columns<O, G>();
  const int need = (a.D / Q + UPT - 1) / UPT;
  a.tpr = need <= 4 ? 4 : need <= 8 ? 8 : need <= 16 ? 16 : (need + 31) / 32 * 32;
  const int bytes =  // of a thread's inputs
      UPT * Q * (int)(sizeof(T) + sizeof(O) + sizeof(G) * (a.dh ? 2 : 1));
  // rows a CTA works on at once: what its threads hold and what leaves room for two
  // stages, but no more than it takes to give every CTA some
  const int row_bytes = a.tpr * bytes;
  const int64_t most = std::max<int64_t>(
      1, std::min<int64_t>(kBlockThreads / a.tpr, kBlockRing / (2 * row_bytes)));
  const int64_t ctas = rows <= most ? 1 : std::min(num_sms(), kBlockMaxCtas);
  const int64_t share = std::min<int64_t>(most, (rows + ctas - 1) / ctas);
  int threads = std::max(1, (int)((share * a.tpr + 31) / 32)) * 32;
  if (a.tpr > 32) threads = (int)share * a.tpr;
  const int groups = threads / a.tpr;
  const int64_t grid = std::min<int64_t>(ctas, (rows + groups - 1) / groups);
  const int64_t turns = (rows + grid * groups - 1) / (grid * groups);
  const int stage = threads * bytes;
  a.stages = (int)std::max<int64_t>(
      1, std::min<int64_t>(std::min<int64_t>(kBlockStages, turns), kBlockRing / stage));
  const size_t smem = std::max((size_t)a.stages * stage,
                               (size_t)(threads / std::max(a.tpr, 32)) * 2 * a.D * 4);
  auto kern = block_norm_bwd_kernel<T, O, G, UPT>;
  // both before the first launch: a refusal leaves the gradients as they were
  auto columns = block_columns_kernel<T, O, G>;
  const size_t columns_smem = std::min(smem, (size_t)kColumnsSmem);
  if (!allow_smem(kern, smem, kBlockRing) ||
      (grid > 1 && !allow_smem(columns, columns_smem, kColumnsSmem)))
    return LRM_ERR_CUDA;
  if (launch_k(kern, dim3((unsigned)grid), dim3(threads), smem, cs, a) != cudaSuccess) {
    (void)cudaGetLastError();
    return LRM_ERR_CUDA;
  }
  if (grid > 1)  // it asks for as much shared memory: an SM need not split its L1 anew
    launch_k(columns, dim3((a.D + 31) / 32), dim3(kBlockColThreads), columns_smem, cs, a,
             (int)grid);
  return launch_status();
}

struct BlockGrad {
  const void *dy, *dh, *h, *block, *w, *w_post, *gate;
  const float *rstd, *block_rstd;
  void *dres, *dblock;
  float *dw, *dw_post, *dgate, *part;
};

template <typename T, typename O, typename G>
static lrm_status pick_block_bwd(const lrm_block* b, const BlockGrad& g, cudaStream_t cs) {
  BlockBwd<T, O, G> a{(const G*)g.dy, (const G*)g.dh, (const T*)g.h, (const O*)g.block,
                      (const T*)g.w, (const T*)g.w_post, (const T*)g.gate, g.rstd, g.block_rstd,
                      (G*)g.dres, (T*)g.dblock, g.dw, g.dw_post, g.dgate, g.part, b->T, b->D,
                      b->gate, 0, 0, b->residual_scale};
  // Two chunks a thread wherever 512 threads hold the row so (T 32768, float32 gradients, two
  // | four: D 512 56 us | 58, D 1024 103 | 112, D 4096 T 16384 207 | 224; with one, D 2048 takes
  // 398 instead of 222).
  // A bfloat16 layer's float32 block with bfloat16 gradients has the fewest bytes a chunk, and
  // four there put more rows into a turn (us two | four: T 32768 D 768 67 | 68, D 1024 87 | 76,
  // D 1536 134 | 115, T 16384 D 2048 89 | 77, D 3200 154 | 159, T 8192 D 4096 91 | 80; widths
  // like 3200 are not told apart).
  // Where everything is float32 four chunks of a row of D 8192 with dh fill the ring, so one row
  // is in flight: T 8192 252 us, 0.94 of the copy bandwidth (D 7168 0.93).
  constexpr bool kLight = sizeof(T) == 2 && sizeof(O) == 4 && sizeof(G) == 2;
  constexpr int two = kLight ? 1023 : kBlockThreads * 2 * lane_columns<O, G>();
  if constexpr (two < kBlockMaxD)
    if (b->D > two) return launch_block_bwd<T, O, G, 4>(a, cs);
  return launch_block_bwd<T, O, G, 2>(a, cs);
}

template <typename... P>
static bool block_aligned(P... p) {
  return (aligned16(p) && ...);
}

}  // namespace lrm

using namespace lrm;

extern "C" size_t lrm_block_workspace_bytes(const lrm_block* b) {
  return check_block(b) == LRM_OK ? block_bytes(b) : 0;
}

extern "C" lrm_status lrm_block_norm(const lrm_block* b, const void* block, const void* res,
                                     const void* w, const void* w_post, const void* gate, void* h,
                                     void* y, void* q, float* q_scale, float* rstd,
                                     float* block_rstd, void* stream) {
  LRM_NVTX("lrm_block_norm");
  lrm_status st = check_block(b);
  if (st != LRM_OK) return st;
  if (b->T == 0) return LRM_OK;
  if (!!q != !!q_scale || (!y && !q)) return LRM_ERR_INVALID_ARG;
  if (!block || !res || !w || !h || !!gate != (b->gate != LRM_GATE_NONE))
    return LRM_ERR_INVALID_ARG;
  if (!block_aligned(block, res, w, w_post, h, y, q, q_scale, rstd, block_rstd) ||
      (b->gate == LRM_GATE_COLUMN && !aligned16(gate)))
    return LRM_ERR_UNSUPPORTED;
  if (h == res && b->res_stride != b->D) return LRM_ERR_INVALID_ARG;
  const BlockFwd a{block, res, w, w_post, gate, h, y, (uint8_t*)q, q_scale, rstd, block_rstd};
  cudaStream_t cs = (cudaStream_t)stream;
  using B = __nv_bfloat16;
  if (b->dtype == LRM_F32) return pick_block<float, float>(b, a, cs);
  return b->block_dtype == LRM_F32 ? pick_block<B, float>(b, a, cs) : pick_block<B, B>(b, a, cs);
}

extern "C" lrm_status lrm_block_norm_bwd(const lrm_block* b, const void* dy, const void* dh,
                                         const void* h, const void* block, const void* w,
                                         const void* w_post, const void* gate, const float* rstd,
                                         const float* block_rstd, void* dres, void* dblock,
                                         float* dw, float* dw_post, float* dgate, void* ws,
                                         size_t ws_bytes, void* stream) {
  LRM_NVTX("lrm_block_norm_bwd");
  lrm_status st = check_block(b);
  if (st != LRM_OK) return st;
  if (!ws || ws_bytes < block_bytes(b)) return LRM_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return LRM_ERR_UNSUPPORTED;
  const bool gated = b->gate != LRM_GATE_NONE;
  if (!dw || (w_post && !dw_post) || (gated && b->T > 0 && !dgate)) return LRM_ERR_INVALID_ARG;
  if (b->gate == LRM_GATE_COLUMN && !dgate) return LRM_ERR_INVALID_ARG;
  if (b->T > 0 && (!dy || !h || !block || !w || !rstd || !dres || !dblock || !!gate != gated ||
                   (w_post && !block_rstd)))
    return LRM_ERR_INVALID_ARG;
  if (!block_aligned(dy, dh, h, block, w, w_post, rstd, block_rstd, dres, dblock, dw, dw_post) ||
      (b->gate == LRM_GATE_COLUMN && !block_aligned(gate, dgate)))
    return LRM_ERR_UNSUPPORTED;
  cudaStream_t cs = (cudaStream_t)stream;
  if (b->T == 0) {
    launch_k(zero_columns_kernel, dim3(1), dim3(1024), 0, cs, dw, w_post ? dw_post : nullptr,
             b->gate == LRM_GATE_COLUMN ? dgate : nullptr, b->D);
    return launch_status();
  }
  const BlockGrad g{dy, dh, h, block, w, w_post, gate, rstd, block_rstd, dres, dblock, dw, dw_post,
                    dgate, reinterpret_cast<float*>((char*)ws + kWsHeaderBytes)};
  using B = __nv_bfloat16;
  const bool g16 = b->grad_dtype == LRM_BF16;
  if (b->dtype == LRM_F32)
    return g16 ? pick_block_bwd<float, float, B>(b, g, cs)
               : pick_block_bwd<float, float, float>(b, g, cs);
  if (b->block_dtype == LRM_F32)
    return g16 ? pick_block_bwd<B, float, B>(b, g, cs) : pick_block_bwd<B, float, float>(b, g, cs);
  return g16 ? pick_block_bwd<B, B, B>(b, g, cs) : pick_block_bwd<B, B, float>(b, g, cs);
}
