// What the kernels that work on rows share: 8 elements at a time as loaded and as
// floats, e4m3 codes, reductions over a row's threads, asynchronous copies.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace lrm {

constexpr float kF8Max = 448.f;    // largest e4m3 value
constexpr float kF8MaxInv = 1.f / kF8Max;
constexpr float kAmaxMin = 7.888609052210118e-31f;  // 2^-100

// A unit is 8 consecutive elements: what one thread loads at a time.
constexpr int kUnit = 8;

// 16 bytes, or zeros: a predicated load, which no branch keeps apart from the
// loads before and after it.
__device__ __forceinline__ uint4 load_if(const void* p, bool ok) {
  uint4 v;
  asm volatile(
      "{\n\t.reg .pred ok;\n\tsetp.ne.b32 ok, %5, 0;\n\t"
      "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
      "@ok ld.global.cs.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(p), "r"((int)ok)
      : "memory");
  return v;
}

template <typename T>
struct Unit8 {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) v[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void load(const T* p, bool ok) {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i)
      v[i] = load_if(reinterpret_cast<const uint4*>(p) + i, ok);
  }
  __device__ __forceinline__ void load_cached(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void get(float (&f)[kUnit]) const {
    constexpr int V = Vec16<T>::kElems;
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) Vec16<T>::unpack(v[i], f + i * V);
  }
};

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&f)[kUnit]) {
  constexpr int V = Vec16<T>::kElems;
#pragma unroll
  for (int i = 0; i < (int)(sizeof(T) / 2); ++i)
    reinterpret_cast<uint4*>(p)[i] = Vec16<T>::pack(f + i * V);
}

__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}

__device__ __forceinline__ void store_e4m3(uint8_t* p, const float (&f)[kUnit], float k) {
  uint2 c;
  c.x = pack_e4m3(f[0] * k, f[1] * k, f[2] * k, f[3] * k);
  c.y = pack_e4m3(f[4] * k, f[5] * k, f[6] * k, f[7] * k);
  *reinterpret_cast<uint2*>(p) = c;
}

// Two floats in one operation.
using Pair = unsigned long long;
__device__ __forceinline__ Pair pair(float lo, float hi) {
  Pair p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(lo), "f"(hi));
  return p;
}
__device__ __forceinline__ float2 floats(Pair p) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(p));
  return f;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair p;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(p) : "l"(a), "l"(b));
  return p;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
  Pair p;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(p) : "l"(a), "l"(b));
  return p;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair p;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(p) : "l"(a), "l"(b), "l"(c));
  return p;
}
// Sum (or maximum) over the TPR threads of a row in the forward kernel; `slot`
// is a shared buffer of its own for each of the two.
template <int TPR, bool MAX>
__device__ __forceinline__ float row_reduce(float v, float (*red)[32], int slot) {
#pragma unroll
  for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? fmaxf(v, u) : v + u;
  }
  if constexpr (TPR > 32) {
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) red[slot][warp] = v;
    __syncthreads();
    v = red[slot][0];
#pragma unroll
    for (int w = 1; w < TPR / 32; ++w) v = MAX ? fmaxf(v, red[slot][w]) : v + red[slot][w];
  }
  return v;
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}

}  // namespace lrm
