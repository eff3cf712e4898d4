// Root-mean-square norm of a row with the residual's addition in front and an
// 8-bit output behind, and its gradients.
//   h = x + res,  rstd = 1 / sqrt(mean(h^2) + eps),  y = h rstd w
//   8 bits: scale = max(amax, 2^-100) / 448 over each q_cols columns,
//           q = e4m3(y / scale)
//   dx = rstd (w dy - xhat mean(w dy xhat)) + dh,  dw = sum_t dy xhat,
//   xhat = h rstd
// The sum h is rounded to the layer type only where it is stored: the norm is
// taken of the 32-bit sum. All of it is HBM-bound; a row is read once into
// registers by one group of threads and everything is computed from there.
#include <cuda_fp8.h>

#include <algorithm>

#include "common.cuh"

namespace lrm {

constexpr int kNormMaxD = 16384;
constexpr int kNormMaxCtas = 640;  // partial dw rows in the workspace
constexpr float kF8Max = 448.f;    // largest e4m3 value
constexpr float kF8MaxInv = 1.f / kF8Max;
constexpr float kAmaxMin = 7.888609052210118e-31f;  // 2^-100

// A unit is 8 consecutive elements: what one thread loads at a time.
constexpr int kUnit = 8;

template <typename T>
struct Unit8 {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) v[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i)
      v[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
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

// Sum (or maximum) over the TPR threads of a row; `slot` alternates between
// two shared buffers so that one barrier a reduction suffices.
template <int TPR, bool MAX>
__device__ __forceinline__ float row_reduce(float v, float (*red)[32], int slot) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
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

// TPR threads a row, UPT units a thread: TPR * UPT * 8 >= D.
template <typename T, int TPR, int UPT>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR)
add_rmsnorm_kernel(const T* x, const T* res, const T* __restrict__ w, T* h, T* y, uint8_t* q,
                   float* q_scale, float* rstd, int rows, int D, int64_t x_stride,
                   int64_t res_stride, int group_units, float eps) {
  pdl_begin();  // predecessor complete before any global access
  constexpr int kThreads = TPR < 128 ? 128 : TPR;
  constexpr int RPC = kThreads / TPR;
  __shared__ float red[2][32];
  const int lane = threadIdx.x % TPR;
  const int units = D / kUnit;
  const int groups = group_units ? (units + group_units - 1) / group_units : 1;
  for (int64_t r = (int64_t)blockIdx.x * RPC + threadIdx.x / TPR; r < rows;
       r += (int64_t)gridDim.x * RPC) {
    Unit8<T> vx[UPT], vr[UPT];
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
      const int u = lane + i * TPR;
      vx[i].zero();
      vr[i].zero();
      if (u < units) {
        vx[i].load(x + r * x_stride + u * kUnit);
        if (res) vr[i].load(res + r * res_stride + u * kUnit);
      }
    }
    float f[UPT][kUnit];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
      vx[i].get(f[i]);
      if (res) {
        float g[kUnit];
        vr[i].get(g);
#pragma unroll
        for (int j = 0; j < kUnit; ++j) f[i][j] += g[j];
      }
#pragma unroll
      for (int j = 0; j < kUnit; ++j) s = fmaf(f[i][j], f[i][j], s);
    }
    s = row_reduce<TPR, false>(s, red, 0);
    const float rs = 1.f / sqrtf(s / (float)D + eps);
    if (rstd && lane == 0) rstd[r] = rs;
    float rowmax = 0.f;
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
      const int u = lane + i * TPR;
      if (u < units) {
        if (h) store8(h + r * D + u * kUnit, f[i]);
        Unit8<T> vw;
        vw.load_cached(w + u * kUnit);
        float g[kUnit];
        vw.get(g);
#pragma unroll
        for (int j = 0; j < kUnit; ++j) f[i][j] = f[i][j] * rs * g[j];
        if (y) store8(y + r * D + u * kUnit, f[i]);
      }
      if (q) {
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < kUnit; ++j) m = fmaxf(m, fabsf(f[i][j]));
        if (group_units) {
          for (int o = 1; o < group_units; o <<= 1)
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
          m = fmaxf(m, kAmaxMin);
          if (u < units) {
            const float k = __frcp_rn(m) * kF8Max;
            uint2 c;
            c.x = pack_e4m3(f[i][0] * k, f[i][1] * k, f[i][2] * k, f[i][3] * k);
            c.y = pack_e4m3(f[i][4] * k, f[i][5] * k, f[i][6] * k, f[i][7] * k);
            *reinterpret_cast<uint2*>(q + r * D + u * kUnit) = c;
            if (u % group_units == 0) q_scale[r * groups + u / group_units] = m * kF8MaxInv;
          }
        } else {
          rowmax = fmaxf(rowmax, m);
        }
      }
    }
    if (q && !group_units) {
      const float m = fmaxf(row_reduce<TPR, true>(rowmax, red, 1), kAmaxMin);
      const float k = __frcp_rn(m) * kF8Max;
#pragma unroll
      for (int i = 0; i < UPT; ++i) {
        const int u = lane + i * TPR;
        if (u < units) {
          uint2 c;
          c.x = pack_e4m3(f[i][0] * k, f[i][1] * k, f[i][2] * k, f[i][3] * k);
          c.y = pack_e4m3(f[i][4] * k, f[i][5] * k, f[i][6] * k, f[i][7] * k);
          *reinterpret_cast<uint2*>(q + r * D + u * kUnit) = c;
        }
      }
      if (lane == 0) q_scale[r] = m * kF8MaxInv;
    }
    if (TPR > 32) __syncthreads();  // the buffers are free for the next row
  }
}

template <typename T, typename G, int TPR, int UPT>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR)
rmsnorm_bwd_kernel(const G* dy, const G* dh, const T* __restrict__ h,
                   const T* __restrict__ w, const float* __restrict__ rstd, G* dx,
                   float* __restrict__ dw_part, int rows, int D) {
  pdl_begin();  // predecessor complete before any global access
  constexpr int kThreads = TPR < 128 ? 128 : TPR;
  constexpr int RPC = kThreads / TPR;
  __shared__ float red[2][32];
  const int lane = threadIdx.x % TPR;
  const int units = D / kUnit;
  Unit8<T> vw[UPT];
  float acc[UPT][kUnit];
#pragma unroll
  for (int i = 0; i < UPT; ++i) {
    vw[i].zero();
    if (lane + i * TPR < units) vw[i].load_cached(w + (lane + i * TPR) * kUnit);
#pragma unroll
    for (int j = 0; j < kUnit; ++j) acc[i][j] = 0.f;
  }
  int slot = 0;
  for (int64_t r = (int64_t)blockIdx.x * RPC + threadIdx.x / TPR; r < rows;
       r += (int64_t)gridDim.x * RPC) {
    Unit8<G> vdy[UPT], vdh[UPT];
    Unit8<T> vh[UPT];
    const float rs = rstd[r];
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
      const int u = lane + i * TPR;
      vdy[i].zero();
      vh[i].zero();
      vdh[i].zero();
      if (u < units) {
        vdy[i].load(dy + r * D + u * kUnit);
        vh[i].load(h + r * D + u * kUnit);
        if (dh) vdh[i].load(dh + r * D + u * kUnit);
      }
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
      float fd[kUnit], fh[kUnit], fw[kUnit];
      vdy[i].get(fd);
      vh[i].get(fh);
      vw[i].get(fw);
#pragma unroll
      for (int j = 0; j < kUnit; ++j) {
        const float xhat = fh[j] * rs;
        s = fmaf(fd[j] * fw[j], xhat, s);
        acc[i][j] = fmaf(fd[j], xhat, acc[i][j]);
      }
    }
    s = row_reduce<TPR, false>(s, red, slot) / (float)D;
    slot ^= 1;
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
      const int u = lane + i * TPR;
      if (u < units) {
        float fd[kUnit], fh[kUnit], fw[kUnit], fr[kUnit];
        vdy[i].get(fd);
        vh[i].get(fh);
        vw[i].get(fw);
        vdh[i].get(fr);
#pragma unroll
        for (int j = 0; j < kUnit; ++j)
          fr[j] = fmaf(rs, fd[j] * fw[j] - fh[j] * rs * s, fr[j]);
        store8(dx + r * D + u * kUnit, fr);
      }
    }
  }
  // the CTA's sum over its rows, rows of a CTA in a fixed order
  if constexpr (RPC > 1) {
    __shared__ float sum[RPC][TPR * UPT * kUnit];
#pragma unroll
    for (int i = 0; i < UPT; ++i)
#pragma unroll
      for (int j = 0; j < kUnit; ++j)
        sum[threadIdx.x / TPR][(lane + i * TPR) * kUnit + j] = acc[i][j];
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += kThreads) {
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < RPC; ++k) s += sum[k][c];
      dw_part[(int64_t)blockIdx.x * D + c] = s;
    }
  } else {
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
      const int u = lane + i * TPR;
      if (u < units) store8(dw_part + (int64_t)blockIdx.x * D + u * kUnit, acc[i]);
    }
  }
}

// dw[c] = sum over the CTAs' partial rows, in a fixed order: 32 columns a CTA,
// 8 threads a column.
constexpr int kColThreads = 256;
__global__ void __launch_bounds__(kColThreads)
dw_sum_kernel(const float* __restrict__ part, int nrows, int D, float* __restrict__ dw) {
  pdl_begin();  // predecessor complete before any global access
  __shared__ float sm[kColThreads / 32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < D)
    for (int r = warp; r < nrows; r += kColThreads / 32) s += part[(int64_t)r * D + c];
  sm[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < D) {
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < kColThreads / 32; ++k) t += sm[k][lane];
    dw[c] = t;
  }
}

__global__ void zero_dw_kernel(float* dw, int D) {
  pdl_begin();  // predecessor complete before any global access
  for (int c = threadIdx.x; c < D; c += blockDim.x) dw[c] = 0.f;
}

static lrm_status check_norm(const lrm_norm* n) {
  if (!n) return LRM_ERR_INVALID_ARG;
  if (n->T < 0 || n->D <= 0 || n->q_cols < 0) return LRM_ERR_INVALID_ARG;
  if (n->dtype != LRM_F32 && n->dtype != LRM_BF16) return LRM_ERR_INVALID_ARG;
  if (n->grad_dtype != LRM_F32 && n->grad_dtype != LRM_BF16) return LRM_ERR_INVALID_ARG;
  if (!(n->eps >= 0.f)) return LRM_ERR_INVALID_ARG;
  if (n->x_stride < n->D || n->res_stride < n->D) return LRM_ERR_INVALID_ARG;
  if (n->D % kUnit != 0 || n->D > kNormMaxD) return LRM_ERR_UNSUPPORTED;
  if (n->x_stride % kUnit != 0 || n->res_stride % kUnit != 0) return LRM_ERR_UNSUPPORTED;
  if (n->q_cols != 0 && n->q_cols != 32 && n->q_cols != 64 && n->q_cols != 128 &&
      n->q_cols != 256)
    return LRM_ERR_UNSUPPORTED;
  return LRM_OK;
}

static size_t norm_bytes(const lrm_norm* n) {
  const size_t b = kWsHeaderBytes + (size_t)kNormMaxCtas * n->D * 4;
  return (b + 255) / 256 * 256;
}

struct NormFwd {
  const void *x, *res, *w;
  void *h, *y;
  uint8_t* q;
  float *q_scale, *rstd;
};
struct NormBwd {
  const void *dy, *dh, *h, *w;
  const float* rstd;
  void* dx;
  float *dw, *part;
};

template <typename T, int TPR, int UPT>
static lrm_status launch_norm(const lrm_norm* n, const NormFwd& a, cudaStream_t cs) {
  constexpr int kThreads = TPR < 128 ? 128 : TPR;
  constexpr int RPC = kThreads / TPR;
  const int64_t blocks = std::min<int64_t>(((int64_t)n->T + RPC - 1) / RPC, 1 << 20);
  launch_k(add_rmsnorm_kernel<T, TPR, UPT>, dim3((unsigned)blocks), dim3(kThreads), 0, cs,
           (const T*)a.x, (const T*)a.res, (const T*)a.w, (T*)a.h, (T*)a.y, a.q, a.q_scale,
           a.rstd, n->T, n->D, n->x_stride, n->res_stride, n->q_cols / kUnit, n->eps);
  return launch_status();
}

template <typename T, typename G, int TPR, int UPT>
static lrm_status launch_norm_bwd(const lrm_norm* n, const NormBwd& a, cudaStream_t cs) {
  constexpr int kThreads = TPR < 128 ? 128 : TPR;
  constexpr int RPC = kThreads / TPR;
  const int64_t ctas = std::min<int64_t>((int64_t)num_sms() * 4, kNormMaxCtas);
  const int64_t blocks = std::min<int64_t>(((int64_t)n->T + RPC - 1) / RPC, ctas);
  float* part = blocks == 1 ? a.dw : a.part;
  launch_k(rmsnorm_bwd_kernel<T, G, TPR, UPT>, dim3((unsigned)blocks), dim3(kThreads), 0, cs,
           (const G*)a.dy, (const G*)a.dh, (const T*)a.h, (const T*)a.w, a.rstd, (G*)a.dx, part,
           n->T, n->D);
  if (blocks > 1)
    launch_k(dw_sum_kernel, dim3((n->D + 31) / 32), dim3(kColThreads), 0, cs, (const float*)part,
             (int)blocks, n->D, a.dw);
  return launch_status();
}

// Threads a row and units a thread: a warp holds rows of up to 1024 columns, a
// CTA of 128 threads up to 4096, one of 512 up to 16384.
#define LRM_NORM_PICK(call, ...)                          \
  (n->D <= 256     ? call<__VA_ARGS__, 32, 1>             \
   : n->D <= 512   ? call<__VA_ARGS__, 32, 2>             \
   : n->D <= 1024  ? call<__VA_ARGS__, 32, 4>             \
   : n->D <= 2048  ? call<__VA_ARGS__, 128, 2>            \
   : n->D <= 4096  ? call<__VA_ARGS__, 128, 4>            \
   : n->D <= 8192  ? call<__VA_ARGS__, 512, 2>            \
                   : call<__VA_ARGS__, 512, 4>)

template <typename... P>
static bool all_aligned(P... p) {
  return (aligned16(p) && ...);
}

}  // namespace lrm

using namespace lrm;

extern "C" size_t lrm_norm_workspace_bytes(const lrm_norm* n) {
  return check_norm(n) == LRM_OK ? norm_bytes(n) : 0;
}

extern "C" lrm_status lrm_add_rmsnorm(const lrm_norm* n, const void* x, const void* res,
                                      const void* w, void* h, void* y, void* q, float* q_scale,
                                      float* rstd, void* stream) {
  LRM_NVTX("lrm_add_rmsnorm");
  lrm_status st = check_norm(n);
  if (st != LRM_OK) return st;
  if (n->T == 0) return LRM_OK;
  if (!!q != !!q_scale || (!y && !q)) return LRM_ERR_INVALID_ARG;
  if (!x || !w) return LRM_ERR_INVALID_ARG;
  if (!all_aligned(x, res, w, h, y, q, q_scale, rstd)) return LRM_ERR_UNSUPPORTED;
  const NormFwd a{x, res, w, h, y, (uint8_t*)q, q_scale, rstd};
  auto go = n->dtype == LRM_BF16 ? LRM_NORM_PICK(launch_norm, __nv_bfloat16)
                                 : LRM_NORM_PICK(launch_norm, float);
  return go(n, a, (cudaStream_t)stream);
}

extern "C" lrm_status lrm_add_rmsnorm_bwd(const lrm_norm* n, const void* dy, const void* dh,
                                          const void* h, const void* w, const float* rstd,
                                          void* dx, float* dw, void* ws, size_t ws_bytes,
                                          void* stream) {
  LRM_NVTX("lrm_add_rmsnorm_bwd");
  lrm_status st = check_norm(n);
  if (st != LRM_OK) return st;
  if (!ws || ws_bytes < norm_bytes(n)) return LRM_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return LRM_ERR_UNSUPPORTED;
  if (!dw) return LRM_ERR_INVALID_ARG;
  if (n->T > 0 && (!dy || !h || !w || !rstd || !dx)) return LRM_ERR_INVALID_ARG;
  if (!all_aligned(dy, dh, h, w, rstd, dx, dw)) return LRM_ERR_UNSUPPORTED;
  cudaStream_t cs = (cudaStream_t)stream;
  if (n->T == 0) {
    launch_k(zero_dw_kernel, dim3(1), dim3(1024), 0, cs, dw, n->D);
    return launch_status();
  }
  float* part = reinterpret_cast<float*>((char*)ws + kWsHeaderBytes);
  const NormBwd a{dy, dh, h, w, rstd, dx, dw, part};
  using B = __nv_bfloat16;
  auto go = n->dtype == LRM_BF16 ? (n->grad_dtype == LRM_BF16 ? LRM_NORM_PICK(launch_norm_bwd, B, B)
                                                              : LRM_NORM_PICK(launch_norm_bwd, B, float))
                                 : (n->grad_dtype == LRM_BF16 ? LRM_NORM_PICK(launch_norm_bwd, float, B)
                                                              : LRM_NORM_PICK(launch_norm_bwd, float, float));
  return go(n, a, cs);
}
