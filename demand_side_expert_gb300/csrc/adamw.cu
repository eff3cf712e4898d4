// One AdamW step over many tensors in a few launches, moments in 32 bits or in 8.
//   g' = s g,  m = b1 m + (1 - b1) g',  v = b2 v + (1 - b2) g'^2
//   p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// 8-bit moments: blocks of 256 consecutive values of a tensor share one float
// scale, max(amax, 2^-100) / 448; m is held as e4m3(m / scale) and v by its
// root, e4m3(sqrt(v) / scale): the root halves the exponent range that the
// code has to span, and a positive root never rounds to zero (it is raised to
// the smallest positive code), so that no step divides by eps alone. The step
// itself uses the unrounded new moments.
//
// HBM-bound (604 million values with FP32 master copies: 32-bit moments 18.1 GB in
// 2.56 ms, 8-bit ones 10.9 GB in 1.56 ms, 1.04 and 1.03 of the copy bandwidth):
// every value is read and written once, 8 consecutive values a thread, so that a
// warp covers one 8-bit block and its maxima are warp reductions. Each operation is rounded on its own (no contraction): moments
// and parameters do not depend on how the compiler fuses them.
#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>

#include "common.cuh"

namespace lrm {

// 128 threads: 1571 us for 604 million values with 8-bit moments, where 256 and
// 512 take 1657 and 1761 (32-bit moments: 2568, 2562 and 2550).
constexpr int kAdamThreads = 128;
constexpr int kAdamUnit = 8;
constexpr int kAdamBlock = 256;  // values under one scale
constexpr int kAdamChunk = kAdamThreads * kAdamUnit;
// Tensors a launch, described in its parameters: few, or as many as fit.
constexpr int kAdamFew = 16, kAdamMany = 256;
constexpr float kAdamF8Max = 448.f, kAdamF8Step = 0.001953125f;  // largest, smallest e4m3
constexpr float kAdamF8MaxInv = 1.f / kAdamF8Max;
constexpr float kAdamAmaxMin = 7.888609052210118e-31f;           // 2^-100

struct AdamSeg {
  void* param;
  const void* grad;
  float* master;
  void *m, *v;
  float *m_scale, *v_scale;
  int64_t n;
  float keep;  // 1 - lr wd
};
struct AdamStep {
  int nseg;
  float b1, c1, b2, c2, inv_sqrt_bc2, eps, step;
  const float* grad_scale;
};
template <int SEGS>
struct AdamArgs : AdamStep {
  uint32_t first[SEGS];  // first chunk of the launch that is the tensor's
  AdamSeg seg[SEGS];
};
static_assert(sizeof(AdamArgs<kAdamMany>) <= 32764, "kernel parameters");

template <typename T>
__device__ __forceinline__ void adam_load(const T* p, int count, float (&f)[8]) {
  if (count == 8) {
    constexpr int V = Vec16<T>::kElems;
#pragma unroll
    for (int i = 0; i < 8 / V; ++i)
      Vec16<T>::unpack(__ldcs(reinterpret_cast<const uint4*>(p) + i), f + i * V);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = i < count ? (float)p[i] : 0.f;
  }
}
template <typename T>
__device__ __forceinline__ void adam_store(T* p, int count, const float (&f)[8]) {
  if (count == 8) {
    constexpr int V = Vec16<T>::kElems;
#pragma unroll
    for (int i = 0; i < 8 / V; ++i)
      __stcs(reinterpret_cast<uint4*>(p) + i, Vec16<T>::pack(f + i * V));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < count) p[i] = (T)f[i];
  }
}

__device__ __forceinline__ void e4m3_load(const uint8_t* p, int count, float scale,
                                          float (&f)[8]) {
  uint2 c = make_uint2(0, 0);
  if (count == 8) {
    c = __ldcs(reinterpret_cast<const uint2*>(p));
  } else {
    uint8_t* b = reinterpret_cast<uint8_t*>(&c);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < count) b[i] = p[i];
  }
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_fp8x2_storage_t two = (__nv_fp8x2_storage_t)(w[i >> 1] >> (16 * (i & 1)));
    const float2 t = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(two, __NV_E4M3)));
    f[2 * i] = __fmul_rn(t.x, scale);
    f[2 * i + 1] = __fmul_rn(t.y, scale);
  }
}

// Quantises the warp's 256 values: the codes of the lane's 8, and the scale.
template <bool ROOT>
__device__ __forceinline__ void e4m3_store(uint8_t* p, float* scale, int count,
                                           const float (&f)[8], int lane) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(f[i]));
  // non-negative floats order like their bits
  m = fmaxf(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m))), kAdamAmaxMin);
  const float k = __fmul_rn(__frcp_rn(m), kAdamF8Max);
  float s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    s[i] = __fmul_rn(f[i], k);
    if (ROOT && f[i] > 0.f) s[i] = fmaxf(s[i], kAdamF8Step);
  }
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = __nv_cvt_float2_to_fp8x2(make_float2(s[2 * i], s[2 * i + 1]), __NV_SATFINITE,
                                    __NV_E4M3);
  const uint2 c = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
  if (count == 8) {
    __stcs(reinterpret_cast<uint2*>(p), c);
  } else {
    const uint8_t* b = reinterpret_cast<const uint8_t*>(&c);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < count) p[i] = b[i];
  }
  if (lane == 0 && count > 0) *scale = __fmul_rn(m, kAdamF8MaxInv);
}

template <typename P, typename G, bool MASTER, bool F8, int SEGS>
__global__ void __launch_bounds__(kAdamThreads)
adamw_kernel(const __grid_constant__ AdamArgs<SEGS> a) {
  pdl_begin();  // predecessor complete before any global access
  // the tensor of this chunk: the last one whose first chunk is not after it
  int lo = 0, hi = a.nseg - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.first[mid] <= blockIdx.x) lo = mid;
    else hi = mid - 1;
  }
  const AdamSeg& sg = a.seg[lo];
  const int64_t at = (int64_t)(blockIdx.x - a.first[lo]) * kAdamChunk + threadIdx.x * kAdamUnit;
  const int lane = threadIdx.x & 31;
  const int64_t left = sg.n - at;
  const int count = left >= 8 ? 8 : left > 0 ? (int)left : 0;
  if (at - lane * kAdamUnit >= sg.n) return;  // the whole warp is past the end
  float p[8], g[8], m[8], v[8];
  adam_load<G>((const G*)sg.grad + at, count, g);
  if constexpr (MASTER) adam_load<float>(sg.master + at, count, p);
  else adam_load<P>((const P*)sg.param + at, count, p);
  if constexpr (F8) {
    const int64_t blk = at / kAdamBlock;
    const float ms = __ldcs(sg.m_scale + blk), vs = __ldcs(sg.v_scale + blk);
    e4m3_load((const uint8_t*)sg.m + at, count, ms, m);
    e4m3_load((const uint8_t*)sg.v + at, count, vs, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(v[i], v[i]);
  } else {
    adam_load<float>((const float*)sg.m + at, count, m);
    adam_load<float>((const float*)sg.v + at, count, v);
  }
  if (a.grad_scale) {
    const float s = __ldg(a.grad_scale);
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = __fmul_rn(g[i], s);
  }
  float root[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    m[i] = __fadd_rn(__fmul_rn(m[i], a.b1), __fmul_rn(g[i], a.c1));
    v[i] = __fadd_rn(__fmul_rn(v[i], a.b2), __fmul_rn(__fmul_rn(g[i], g[i]), a.c2));
    root[i] = __fsqrt_rn(v[i]);
    const float den = __fadd_rn(__fmul_rn(root[i], a.inv_sqrt_bc2), a.eps);
    p[i] = __fsub_rn(__fmul_rn(p[i], sg.keep), __fmul_rn(__fdiv_rn(m[i], den), a.step));
  }
  if constexpr (MASTER) adam_store<float>(sg.master + at, count, p);
  adam_store<P>((P*)sg.param + at, count, p);
  if constexpr (F8) {
    const int64_t blk = at / kAdamBlock;
    e4m3_store<false>((uint8_t*)sg.m + at, sg.m_scale + blk, count, m, lane);
    e4m3_store<true>((uint8_t*)sg.v + at, sg.v_scale + blk, count, root, lane);
  } else {
    adam_store<float>((float*)sg.m + at, count, m);
    adam_store<float>((float*)sg.v + at, count, v);
  }
}

static lrm_status check_tensor(const lrm_adamw_tensor& t) {
  if (t.n < 0) return LRM_ERR_INVALID_ARG;
  if ((t.param_dtype != LRM_F32 && t.param_dtype != LRM_BF16) ||
      (t.grad_dtype != LRM_F32 && t.grad_dtype != LRM_BF16) ||
      (t.state != LRM_STATE_F32 && t.state != LRM_STATE_F8))
    return LRM_ERR_INVALID_ARG;
  if (t.n == 0) return LRM_OK;
  if (!t.param || !t.grad || !t.m || !t.v) return LRM_ERR_INVALID_ARG;
  if (t.state == LRM_STATE_F8 && (!t.m_scale || !t.v_scale)) return LRM_ERR_INVALID_ARG;
  if (t.master && t.param_dtype == LRM_F32) return LRM_ERR_INVALID_ARG;
  if (!aligned16(t.param) || !aligned16(t.grad) || !aligned16(t.master) || !aligned16(t.m) ||
      !aligned16(t.v))
    return LRM_ERR_UNSUPPORTED;
  if (((reinterpret_cast<uintptr_t>(t.m_scale) | reinterpret_cast<uintptr_t>(t.v_scale)) & 3u) != 0)
    return LRM_ERR_UNSUPPORTED;
  // chunk numbers are 32-bit
  if (t.n > (int64_t)kAdamChunk * 0x7fffffff) return LRM_ERR_UNSUPPORTED;
  return LRM_OK;
}

// The kernel of a tensor's combination of types.
static int adam_kind(const lrm_adamw_tensor& t) {
  const int p = t.param_dtype == LRM_F32 ? 0 : t.master ? 2 : 1;
  return p * 4 + (t.grad_dtype == LRM_BF16) * 2 + (t.state == LRM_STATE_F8);
}
template <int SEGS>
using AdamKernel = void (*)(const AdamArgs<SEGS>);
template <typename P, bool MASTER, int SEGS>
static AdamKernel<SEGS> adam_types(int kind) {
  switch (kind & 3) {
    case 0: return adamw_kernel<P, float, MASTER, false, SEGS>;
    case 1: return adamw_kernel<P, float, MASTER, true, SEGS>;
    case 2: return adamw_kernel<P, __nv_bfloat16, MASTER, false, SEGS>;
    default: return adamw_kernel<P, __nv_bfloat16, MASTER, true, SEGS>;
  }
}

// Launches the tensors of one kind, SEGS at a time.
template <int SEGS>
static lrm_status adam_launch(const AdamStep& step, double lr, int kind,
                              const lrm_adamw_tensor* tensors, int count, cudaStream_t cs) {
  const AdamKernel<SEGS> kern = kind < 4   ? adam_types<float, false, SEGS>(kind)
                                : kind < 8 ? adam_types<__nv_bfloat16, false, SEGS>(kind)
                                           : adam_types<__nv_bfloat16, true, SEGS>(kind);
  AdamArgs<SEGS> a;
  static_cast<AdamStep&>(a) = step;
  int64_t chunks = 0;
  a.nseg = 0;
  for (int i = 0; i <= count; ++i) {
    const bool end = i == count;
    if (!end && (tensors[i].n == 0 || adam_kind(tensors[i]) != kind)) continue;
    const int64_t more = end ? 0 : (tensors[i].n + kAdamChunk - 1) / kAdamChunk;
    if (a.nseg > 0 && (end || a.nseg == SEGS || chunks + more > 0x7fffffff)) {
      if (launch_k(kern, dim3((unsigned)chunks), dim3(kAdamThreads), 0, cs, a) != cudaSuccess) {
        (void)cudaGetLastError();
        return LRM_ERR_CUDA;
      }
      a.nseg = 0;
      chunks = 0;
    }
    if (end) break;
    const lrm_adamw_tensor& t = tensors[i];
    a.first[a.nseg] = (uint32_t)chunks;
    a.seg[a.nseg++] = {t.param, t.grad, t.master, t.m, t.v, t.m_scale, t.v_scale, t.n,
                       (float)(1.0 - lr * t.weight_decay)};
    chunks += more;
  }
  return LRM_OK;
}

}  // namespace lrm

using namespace lrm;

extern "C" lrm_status lrm_adamw_step(const lrm_adamw* h, const lrm_adamw_tensor* tensors,
                                     int32_t count, void* stream) {
  LRM_NVTX("lrm_adamw_step");
  if (!h || count < 0 || (count > 0 && !tensors)) return LRM_ERR_INVALID_ARG;
  if (!(h->beta1 >= 0 && h->beta1 < 1) || !(h->beta2 >= 0 && h->beta2 < 1) ||
      !(h->eps >= 0) || h->step < 1)
    return LRM_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(h->grad_scale) & 3u) != 0) return LRM_ERR_UNSUPPORTED;
  for (int i = 0; i < count; ++i) {
    const lrm_status st = check_tensor(tensors[i]);
    if (st != LRM_OK) return st;
  }
  int of_kind[12] = {};
  for (int i = 0; i < count; ++i)
    if (tensors[i].n > 0) ++of_kind[adam_kind(tensors[i])];
  const double bc1 = 1.0 - std::pow(h->beta1, (double)h->step);
  const double bc2 = 1.0 - std::pow(h->beta2, (double)h->step);
  const AdamStep step{0,
                      (float)h->beta1,
                      (float)(1.0 - h->beta1),
                      (float)h->beta2,
                      (float)(1.0 - h->beta2),
                      (float)(1.0 / std::sqrt(bc2)),
                      (float)h->eps,
                      (float)(h->lr / bc1),
                      h->grad_scale};
  for (int kind = 0; kind < 12; ++kind) {
    if (of_kind[kind] == 0) continue;
    const lrm_status st =
        of_kind[kind] <= kAdamFew
            ? adam_launch<kAdamFew>(step, h->lr, kind, tensors, count, (cudaStream_t)stream)
            : adam_launch<kAdamMany>(step, h->lr, kind, tensors, count, (cudaStream_t)stream);
    if (st != LRM_OK) return st;
  }
  return launch_status();
}
