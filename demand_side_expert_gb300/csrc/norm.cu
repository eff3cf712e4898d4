// Root-mean-square norm of a row with the residual's addition in front and an
// 8-bit output behind, and its gradients.
//   h = x + res,  rstd = 1 / sqrt(mean(h^2) + eps),  y = h rstd w
//   8 bits: scale = max(amax, 2^-100) / 448 over each q_cols columns,
//           q = e4m3(y / scale)
//   dx = rstd (w dy - xhat mean(w dy xhat)) + dh,  dw = sum_t dy xhat,
//   xhat = h rstd
// The sum h is rounded to the layer type only where it is stored: the norm is
// taken of the 32-bit sum. Few operations a byte: HBM-bound from some MB on
// (T 32768 D 2048 bfloat16, residual and 8-bit rows: 472 MB in 71 us, 0.97 of the
// copy bandwidth; T 16384 D 4096 backward, float32 gradients: 940 MB in 138 us,
// 1.00), and bound by latency and launches below.
#include <algorithm>

#include "rows.cuh"

namespace lrm {

constexpr int kNormMaxD = 16384;
constexpr int kNormMaxCtas = 160;  // partial dw rows in the workspace

// Forward: TPR threads a row (lanes of a warp, or a CTA), UPT units a thread,
// TPR * UPT * 8 >= D, one row (of a warp: 32 / TPR rows) a thread and CTA. The
// row stays in registers from its loads to its stores. Many small CTAs keep an
// SM loading while some of them sum: a persistent form with the rows copied
// ahead into shared memory, as the backward pass has it, measured 101-113 us
// against 71 us (T 32768 D 2048, residual, 8-bit rows). Every load of a row comes
// before any use and the group of a unit is found by shifts: with branches
// between the loads it took 91 us, with divisions 76.
template <int TPR>
constexpr int norm_threads() { return TPR < 64 ? 128 : TPR; }

template <typename T, int TPR, int UPT>
__global__ void __launch_bounds__(norm_threads<TPR>())
add_rmsnorm_kernel(const T* x, const T* res, const T* __restrict__ w, T* h, T* y, uint8_t* q,
                   float* q_scale, float* rstd, int rows, int D, int64_t x_stride,
                   int64_t res_stride, int q_shift, float eps) {
  pdl_begin();  // predecessor complete before any global access
  __shared__ float red[2][32];
  const int tl = threadIdx.x % TPR;
  const int units = D / kUnit;
  const int64_t r = (int64_t)blockIdx.x * (norm_threads<TPR>() / TPR) + threadIdx.x / TPR;
  if (TPR >= 32 && r >= rows) return;
  // several rows a warp: its lanes stay together, those past the end only reduce
  const bool real = TPR >= 32 || r < rows;
  const T* px = x + r * x_stride + tl * kUnit;
  const T* pr = res ? res + r * res_stride + tl * kUnit : nullptr;
  const T* pw = w + tl * kUnit;
  const int64_t at = r * D + tl * kUnit;  // of the thread's first unit in an output
  Unit8<T> vx[UPT], vr[UPT];
#pragma unroll
  for (int i = 0; i < UPT; ++i) vx[i].load(px + i * TPR * kUnit, real && tl + i * TPR < units);
  if (res) {
#pragma unroll
    for (int i = 0; i < UPT; ++i) vr[i].load(pr + i * TPR * kUnit, real && tl + i * TPR < units);
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
  const float rs = rsqrtf(fmaf(s, 1.f / (float)D, eps));
  if (rstd && tl == 0 && real) rstd[r] = rs;
  float rowmax = 0.f;
#pragma unroll
  for (int i = 0; i < UPT; ++i) {
    const int u = tl + i * TPR;
    const bool in = real && u < units;
    if (in) {
      if (h) store8(h + at + i * TPR * kUnit, f[i]);
      Unit8<T> vw;
      vw.load_cached(pw + i * TPR * kUnit);
      float g[kUnit];
      vw.get(g);
#pragma unroll
      for (int j = 0; j < kUnit; ++j) f[i][j] = f[i][j] * rs * g[j];
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
    const float m = fmaxf(row_reduce<TPR, true>(rowmax, red, 1), kAmaxMin);
    const float k = __frcp_rn(m) * kF8Max;
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
      const int u = tl + i * TPR;
      if (real && u < units) store_e4m3(q + at + i * TPR * kUnit, f[i], k);
    }
    if (tl == 0 && real) q_scale[r] = m * kF8MaxInv;
  }
}

// Backward: `tpr` threads a row (4, 8 or 16 lanes, or whole warps), UPT units a
// thread, as many row groups a CTA as its threads hold, one CTA an SM. A row's
// inputs are copied to their thread's own places in shared memory `stages` - 1
// rows ahead, so an SM's loads do not stop while a row's sum is formed, and dw
// stays in registers over all of a thread's rows; a thread waits for its own
// copies only, and the row's threads meet once, for the sum. The copies go
// through L1 (.ca): a thread's 8 float32 values are two 16-byte pieces, and
// past L1 each would fetch their 32-byte sector anew (T 16384 D 4096, float32
// gradients: 204 us instead of 140, which is 0.99 of the copy bandwidth).
constexpr int kNormThreads = 512;
constexpr int kNormRing = 200 * 1024;  // bytes of a CTA's copies in flight, at most

// One group of copies a row: all but the newest `stages` - 1 have landed.
constexpr int kNormStages = 6;
__device__ __forceinline__ void copies_wait(int stages) {
  switch (stages) {
    case 1: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 3: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    case 4: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    case 5: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
  }
}

// Sum over a row's threads. Every thread of the CTA calls it as often as the
// others, whether its row exists or not. `red`: two buffers, zeroed at first.
struct RowGroup {
  int tpr, group, tl;
  float4 (*red)[kNormThreads / 64][kNormThreads / 128];
  int flip = 0;
  __device__ __forceinline__ float sum(float v) {
    for (int o = min(tpr, 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (tpr > 32) {
      float* mine = reinterpret_cast<float*>(red[flip][group]);
      if ((threadIdx.x & 31) == 0) mine[tl >> 5] = v;
      asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(tpr) : "memory");
      v = 0.f;  // places past the row's warps hold 0
#pragma unroll
      for (int k = 0; k < kNormThreads / 128; ++k) {
        const float4 q = red[flip][group][k];
        v += (q.x + q.y) + (q.z + q.w);
      }
      flip ^= 1;  // the other buffer next: one barrier a sum is enough
    }
    return v;
  }
};

template <typename T, typename G, int UPT>
__global__ void __launch_bounds__(kNormThreads)
rmsnorm_bwd_kernel(const G* dy, const G* dh, const T* __restrict__ h, const T* __restrict__ w,
                   const float* __restrict__ rstd, G* dx, float* __restrict__ dw_part, int rows,
                   int D, int tpr, int stages) {
  constexpr int TP = sizeof(T) / 2, GP = sizeof(G) / 2;  // 16-byte pieces of a unit
  extern __shared__ uint4 ring[];  // [stages][pieces][threads]
  __shared__ float4 red[2][kNormThreads / 64][kNormThreads / 128];
  const int threads = blockDim.x, groups = threads / tpr;
  RowGroup row{tpr, (int)threadIdx.x / tpr, (int)threadIdx.x % tpr, red};
  for (int i = threadIdx.x; i < (int)(sizeof(red) / sizeof(float)); i += threads)
    reinterpret_cast<float*>(red)[i] = 0.f;
  __syncthreads();
  const int tl = row.tl;
  const int per_unit = TP + GP * (dh ? 2 : 1), pieces = UPT * per_unit;
  const int units = D / kUnit;
  const float inv_d = 1.f / (float)D;
  pdl_begin();  // predecessor complete before any global access
  const uint32_t mine = (uint32_t)__cvta_generic_to_shared(ring + threadIdx.x);
  auto copy_row = [&](int64_t r, int slot) {
    if (r < rows) {
      uint32_t dst = mine + (uint32_t)(slot * pieces * threads) * 16;
#pragma unroll
      for (int i = 0; i < UPT; ++i) {
        const int u = tl + i * tpr;
        const int64_t at = r * D + u * kUnit;
        if (u < units) {
#pragma unroll
          for (int k = 0; k < TP; ++k)
            copy16(dst + k * threads * 16, reinterpret_cast<const uint4*>(h + at) + k);
#pragma unroll
          for (int k = 0; k < GP; ++k)
            copy16(dst + (TP + k) * threads * 16, reinterpret_cast<const uint4*>(dy + at) + k);
          if (dh) {
#pragma unroll
            for (int k = 0; k < GP; ++k)
              copy16(dst + (TP + GP + k) * threads * 16,
                     reinterpret_cast<const uint4*>(dh + at) + k);
          }
        }
        dst += per_unit * threads * 16;
      }
    }
    copies_commit();
  };
  int64_t base = (int64_t)blockIdx.x * groups;
  const int64_t dr = (int64_t)gridDim.x * groups;
  for (int i = 0; i < stages - 1; ++i) copy_row(base + row.group + i * dr, i);
  Unit8<T> vw[UPT];
  float acc[UPT][kUnit];
#pragma unroll
  for (int i = 0; i < UPT; ++i) {
    vw[i].zero();
    if (tl + i * tpr < units) vw[i].load_cached(w + (tl + i * tpr) * kUnit);
#pragma unroll
    for (int j = 0; j < kUnit; ++j) acc[i][j] = 0.f;
  }
  float next_rs = base + row.group < rows ? __ldg(rstd + base + row.group) : 0.f;
  int slot = 0;
  for (; base < rows; base += dr) {
    const int64_t r = base + row.group;
    copy_row(r + (stages - 1) * dr, slot == 0 ? stages - 1 : slot - 1);
    const float rs = next_rs;
    next_rs = r + dr < rows ? __ldg(rstd + r + dr) : 0.f;
    copies_wait(stages);
    const uint4* v = ring + slot * pieces * threads + threadIdx.x;
    float fd[UPT][kUnit], xhat[UPT][kUnit];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
      const uint4* p = v + i * per_unit * threads;
      const bool in = tl + i * tpr < units && r < rows;
      Unit8<T> vh;
      Unit8<G> vd;
#pragma unroll
      for (int k = 0; k < TP; ++k) vh.v[k] = in ? p[k * threads] : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int k = 0; k < GP; ++k) vd.v[k] = in ? p[(TP + k) * threads] : make_uint4(0, 0, 0, 0);
      float fw[kUnit];
      vh.get(xhat[i]);
      vd.get(fd[i]);
      vw[i].get(fw);
#pragma unroll
      for (int j = 0; j < kUnit; ++j) {
        xhat[i][j] *= rs;
        acc[i][j] = fmaf(fd[i][j], xhat[i][j], acc[i][j]);
        fd[i][j] *= fw[j];
        s = fmaf(fd[i][j], xhat[i][j], s);
      }
    }
    s = row.sum(s) * inv_d;
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
      const int u = tl + i * tpr;
      if (u < units && r < rows) {
        float fr[kUnit];
        Unit8<G> vr;
        vr.zero();
        if (dh) {
#pragma unroll
          for (int k = 0; k < GP; ++k) vr.v[k] = v[(i * per_unit + TP + GP + k) * threads];
        }
        vr.get(fr);
#pragma unroll
        for (int j = 0; j < kUnit; ++j) fr[j] = fmaf(rs, fd[i][j] - xhat[i][j] * s, fr[j]);
        store8(dx + r * D + u * kUnit, fr);
      }
    }
    slot = slot + 1 == stages ? 0 : slot + 1;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  // the CTA's sum over its row groups, in a fixed order: the groups of a warp
  // by exchanges, the rest through shared memory
  for (int o = tpr; o < 32; o <<= 1)
#pragma unroll
    for (int i = 0; i < UPT; ++i)
#pragma unroll
      for (int j = 0; j < kUnit; ++j) acc[i][j] += __shfl_xor_sync(0xffffffffu, acc[i][j], o);
  float* out = dw_part + (int64_t)blockIdx.x * D;
  const int wide = max(tpr, 32), sums = threads / wide;
  const bool writes = (int)threadIdx.x % wide < tpr;
  if (sums == 1) {
#pragma unroll
    for (int i = 0; i < UPT; ++i)
      if (writes && tl + i * tpr < units) store8(out + (tl + i * tpr) * kUnit, acc[i]);
    return;
  }
  __syncthreads();  // the ring is free
  float* sum = reinterpret_cast<float*>(ring);  // [sums][D]
#pragma unroll
  for (int i = 0; i < UPT; ++i)
    if (writes && tl + i * tpr < units)
      store8(sum + (int)threadIdx.x / wide * D + (tl + i * tpr) * kUnit, acc[i]);
  __syncthreads();
  for (int c = threadIdx.x; c < D; c += threads) {
    float t = 0.f;
    for (int k = 0; k < sums; ++k) t += sum[k * D + c];
    out[c] = t;
  }
}

// dw[c] = sum over the CTAs' partial rows, in a fixed order: 32 columns a CTA,
// 16 threads a column.
constexpr int kColThreads = 512;
__global__ void __launch_bounds__(kColThreads)
dw_sum_kernel(const float* __restrict__ part, int nrows, int D, float* __restrict__ dw) {
  pdl_begin();  // predecessor complete before any global access
  __shared__ float sm[kColThreads / 32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  // every load before any use: a loop over the rows that exist would wait for
  // each in turn (8 us instead of 2)
  constexpr int kWarps = kColThreads / 32;
  float v[(kNormMaxCtas + kWarps - 1) / kWarps];
#pragma unroll
  for (int k = 0; k < (int)(sizeof(v) / sizeof(float)); ++k) {
    const int r = warp + k * kWarps;
    v[k] = c < D && r < nrows ? part[(int64_t)r * D + c] : 0.f;
  }
  float s = 0.f;
#pragma unroll
  for (int k = 0; k < (int)(sizeof(v) / sizeof(float)); ++k) s += v[k];
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

// How the backward pass deals out its rows.
struct RowPlan {
  int tpr, threads, stages;
  int64_t ctas;
  size_t smem;
};

// `pieces`: 16-byte pieces of a unit's inputs.
static RowPlan plan_rows(int64_t rows, int D, int upt, int pieces) {
  RowPlan p;
  const int need = (D / kUnit + upt - 1) / upt;
  p.tpr = need <= 4 ? 4 : need <= 8 ? 8 : need <= 16 ? 16 : (need + 31) / 32 * 32;
  // rows a CTA works on at once: what its threads hold, but no more than it
  // takes to give every CTA some. Rows that fit one CTA at once stay in one: a
  // second costs the launch that adds the CTAs' sums of dw (T 4 D 2048: 4.4 us
  // on the host and 3.4 on the GPU instead of 3.1 and 4.3; two rounds of rows in
  // one CTA would be 5.8 on the GPU).
  const int64_t most = kNormThreads / p.tpr;
  const int64_t ctas = rows <= most ? 1 : std::min(num_sms(), kNormMaxCtas);
  const int64_t share = std::min<int64_t>(most, (rows + ctas - 1) / ctas);
  p.threads = std::max(1, (int)((share * p.tpr + 31) / 32)) * 32;
  if (p.tpr > 32) p.threads = std::max<int>(1, (int)share) * p.tpr;
  const int groups = p.threads / p.tpr;
  p.ctas = std::min<int64_t>(ctas, (rows + groups - 1) / groups);
  const int stage = p.threads * 16 * upt * pieces;
  // no more stages than a group has rows
  const int64_t turns = (rows + p.ctas * groups - 1) / (p.ctas * groups);
  p.stages = (int)std::max<int64_t>(
      1, std::min<int64_t>(std::min<int64_t>(kNormStages, turns), kNormRing / stage));
  p.smem = (size_t)p.stages * stage;
  return p;
}

// Lets a kernel have `smem` bytes of dynamic shared memory. The limit is the
// kernel's, for all host threads, so it is only ever set to the most that any call
// needs: a smaller call in another thread cannot lower it before this one's launch.
template <typename K>
static bool allow_smem(K kern, size_t smem) {
  if (smem <= 40 * 1024) return true;
  if (smem <= kNormRing &&
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormRing) ==
          cudaSuccess)
    return true;
  (void)cudaGetLastError();
  return false;
}

template <typename T, int TPR, int UPT>
static lrm_status launch_norm(const lrm_norm* n, const NormFwd& a, cudaStream_t cs) {
  constexpr int kRows = norm_threads<TPR>() / TPR;
  int q_shift = -1;  // log2 of a group's units, -1: the row is the group
  for (int u = n->q_cols / kUnit; u > 0; u >>= 1) ++q_shift;
  launch_k(add_rmsnorm_kernel<T, TPR, UPT>, dim3((unsigned)((n->T + (int64_t)kRows - 1) / kRows)),
           dim3(norm_threads<TPR>()), 0, cs, (const T*)a.x, (const T*)a.res, (const T*)a.w,
           (T*)a.h, (T*)a.y, a.q, a.q_scale, a.rstd, n->T, n->D, n->x_stride, n->res_stride,
           q_shift, n->eps);
  return launch_status();
}

template <typename T, typename G, int UPT>
static lrm_status launch_norm_bwd(const lrm_norm* n, const NormBwd& a, cudaStream_t cs) {
  RowPlan p =
      plan_rows(n->T, n->D, UPT, (int)sizeof(T) / 2 + (int)sizeof(G) / 2 * (a.dh ? 2 : 1));
  const int sums = p.threads / std::max(p.tpr, 32);
  if (sums > 1) p.smem = std::max(p.smem, (size_t)sums * n->D * 4);
  auto kern = rmsnorm_bwd_kernel<T, G, UPT>;
  // both before the first launch: a refusal leaves dx and dw as they were
  if (!allow_smem(kern, p.smem) || (p.ctas > 1 && !allow_smem(dw_sum_kernel, p.smem)))
    return LRM_ERR_CUDA;
  if (launch_k(kern, dim3((unsigned)p.ctas), dim3(p.threads), p.smem, cs, (const G*)a.dy,
               (const G*)a.dh, (const T*)a.h, (const T*)a.w, a.rstd, (G*)a.dx,
               p.ctas == 1 ? a.dw : a.part, n->T, n->D, p.tpr, p.stages) != cudaSuccess) {
    (void)cudaGetLastError();
    return LRM_ERR_CUDA;
  }
  if (p.ctas > 1) {
    // It asks for the same shared memory, which it does not use: an SM that had
    // to change its split of L1 would start it later (9.7 us instead of 8.6 for
    // both kernels at T 1021 D 2048).
    launch_k(dw_sum_kernel, dim3((n->D + 31) / 32), dim3(kColThreads), p.smem, cs,
             (const float*)a.part, (int)p.ctas, n->D, a.dw);
  }
  return launch_status();
}

// Threads a row and units a thread. Up to 16384 values an SM the latency of a
// row is all there is: one unit a thread, where a CTA holds the row so. Beyond,
// two units (several rows an SM keep it loading while one is summed); four where
// that makes a row a warp's (a CTA for each row of 1024 columns takes longer to
// start than to run) or keeps it to 256 threads. Measured (bf16, residual, 8-bit
// rows, 1 | 2 | 4 units, us): T 4 D 4096 2.8 | 3.0 | 3.9, T 1021 D 2048 4.6 | 5.2 |
// 5.1, T 2432 D 4096 14.6 | 12.2 | 12.9, T 32768 D 2048 90.7 | 70.8 | 72.1,
// T 16384 D 4096 96.5 | 71.6 | 71.6, T 2432 D 8192 (2 | 4) 26.7 | 23.0. A bfloat16
// row without a residual is half the bytes and wants four units: T 16384 D 4096,
// y alone, 45.5 us with two and 41.2 with four.
template <typename T>
static lrm_status pick_norm(const lrm_norm* n, const NormFwd& a, cudaStream_t cs) {
  const int D = n->D;
  const bool few = (int64_t)n->T * D <= (int64_t)num_sms() * 16384;
  if (D <= 32) return launch_norm<T, 4, 1>(n, a, cs);
  if (D <= 64) return launch_norm<T, 8, 1>(n, a, cs);
  if (D <= 128) return launch_norm<T, 16, 1>(n, a, cs);
  if (D <= 256) return launch_norm<T, 32, 1>(n, a, cs);
  if (D <= 512) return launch_norm<T, 32, 2>(n, a, cs);
  if (D <= 1024) return few ? launch_norm<T, 128, 1>(n, a, cs) : launch_norm<T, 32, 4>(n, a, cs);
  const bool light = sizeof(T) == 2 && !a.res;
  if (D <= 2048)
    return few     ? launch_norm<T, 256, 1>(n, a, cs)
           : light ? launch_norm<T, 64, 4>(n, a, cs)
                   : launch_norm<T, 128, 2>(n, a, cs);
  if (D <= 4096)
    return few     ? launch_norm<T, 512, 1>(n, a, cs)
           : light ? launch_norm<T, 128, 4>(n, a, cs)
                   : launch_norm<T, 256, 2>(n, a, cs);
  if (D <= 8192) return few ? launch_norm<T, 512, 2>(n, a, cs) : launch_norm<T, 256, 4>(n, a, cs);
  return launch_norm<T, 512, 4>(n, a, cs);
}
// Two units a thread up to 8192 columns. One, in two CTAs an SM, measured the
// same at T 32768 D 2048 (float32 gradients, 140 us) and 7% more at T 16384
// D 4096 with bfloat16 gradients (93 us against 86).
template <typename T, typename G>
static lrm_status pick_norm_bwd(const lrm_norm* n, const NormBwd& a, cudaStream_t cs) {
  if (n->D <= kNormThreads * kUnit * 2) return launch_norm_bwd<T, G, 2>(n, a, cs);
  return launch_norm_bwd<T, G, 4>(n, a, cs);
}

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
  // an output over an input has to have its rows
  for (const void* out : {(const void*)h, (const void*)y})
    if (out && ((out == x && n->x_stride != n->D) || (out == res && n->res_stride != n->D)))
      return LRM_ERR_INVALID_ARG;
  const NormFwd a{x, res, w, h, y, (uint8_t*)q, q_scale, rstd};
  return n->dtype == LRM_BF16 ? pick_norm<__nv_bfloat16>(n, a, (cudaStream_t)stream)
                              : pick_norm<float>(n, a, (cudaStream_t)stream);
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
  if (n->dtype == LRM_BF16)
    return n->grad_dtype == LRM_BF16 ? pick_norm_bwd<B, B>(n, a, cs)
                                     : pick_norm_bwd<B, float>(n, a, cs);
  return n->grad_dtype == LRM_BF16 ? pick_norm_bwd<float, B>(n, a, cs)
                                   : pick_norm_bwd<float, float>(n, a, cs);
}
