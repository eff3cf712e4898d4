// Gradient of the routing weights. The layer's output is
// out_t = sum_k alpha_tk y_(t,k), so
//   dalpha[t,k] = <g_t, y[inv[t*K+k]]>,
// the dot product of the token's cotangent with the output row of each expert
// it was routed to (y in dispatch order, as the forward pass leaves it).
//
// HBM-bound: every y row is read once (K rows a token against one row of g).
// What counts is the bytes an SM keeps in flight: loads into registers got to
// 0.70-0.90 of the copy bandwidth (257-198 us at T 16384 D 4096 K 8, bf16, by
// how many were unrolled), a ring of asynchronous copies in shared memory gets
// to 1.00 (178 us, 6.8 TB/s).
#include <algorithm>

#include "common.cuh"

namespace lrm {

constexpr int kGateThreads = 128;
constexpr int kGateRows = 8;   // y rows summed per pass over g_t
// Steps in flight. 2, 3, 4 and 6 measured 191, 178, 192 and 239 us at T 16384
// D 4096 K 8 (fewer CTAs fit an SM where the rings are deeper).
constexpr int kGateSteps = 3;

// Adds kGateRows values over the warp: lane r (mod 8) ends with row r's sum.
// Three steps trade half of the values against half of the lanes, so that 9
// exchanges do the work of 40.
__device__ __forceinline__ float fold_rows(const float (&v)[kGateRows]) {
  static_assert(kGateRows == 8, "three halvings");
  const int lane = threadIdx.x & 31;
  float a[4], b[2];
  const bool h4 = lane & 4, h2 = lane & 2, h1 = lane & 1;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float keep = h4 ? v[i + 4] : v[i], give = h4 ? v[i] : v[i + 4];
    a[i] = keep + __shfl_xor_sync(0xffffffffu, give, 4);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float keep = h2 ? a[i + 2] : a[i], give = h2 ? a[i] : a[i + 2];
    b[i] = keep + __shfl_xor_sync(0xffffffffu, give, 2);
  }
  const float keep = h1 ? b[1] : b[0], give = h1 ? b[0] : b[1];
  float s = keep + __shfl_xor_sync(0xffffffffu, give, 1);
  s += __shfl_xor_sync(0xffffffffu, s, 8);
  s += __shfl_xor_sync(0xffffffffu, s, 16);
  return s;
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool valid) {
  // an invalid source is not read: 16 zero bytes are written
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}

// TPT threads a token (a warp, or the CTA), S steps of its rows in flight.
// A step is one 16-byte piece of g_t and of up to 8 y rows for every thread;
// it is copied to the thread's own places in shared memory, S - 1 steps ahead
// of the one being summed, across the ends of tokens. Nobody else reads them,
// so a thread waits for its own copies and there is no barrier.
template <typename T, int TPT, int S>
__global__ void __launch_bounds__(kGateThreads)
gate_grad_kernel(const T* __restrict__ g, const T* __restrict__ y,
                 const int32_t* __restrict__ inv, float* __restrict__ dalpha, int ntok, int D,
                 int K, int32_t* err) {
  pdl_begin();  // predecessor complete before any global access
  constexpr int V = Vec16<T>::kElems;
  constexpr int W = kGateThreads / 32;
  constexpr int kTokens = kGateThreads / TPT;
  extern __shared__ uint4 ring[];  // [S][kGateRows + 1][threads]
  __shared__ float part[2][W][kGateRows];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tl = threadIdx.x % TPT;
  const int64_t N = (int64_t)ntok * K;
  const int nv = D / V;
  const int steps = (nv + TPT - 1) / TPT;
  const int64_t t0 = (int64_t)blockIdx.x * kTokens + threadIdx.x / TPT;
  const int64_t dt = (int64_t)gridDim.x * kTokens;
  const uint32_t mine = (uint32_t)__cvta_generic_to_shared(ring + threadIdx.x);

  // copies: token, first row of the pass, step; lane r has row r's position
  int64_t ct = t0;
  int ck = 0, cs = 0;
  auto positions = [&](int64_t t, int k0) {
    int q = -1;
    if (t < ntok && lane < kGateRows && k0 + lane < K) {
      q = inv[t * K + k0 + lane];
      if (q < 0 || q >= N) {
        flag_error(err, LRM_DEVERR_INDEX);
        q = -1;
      }
    }
    return q;
  };
  int pos = positions(ct, 0);
  // of the pass after that one, read a pass ahead
  int64_t nt = K > kGateRows ? ct : ct + dt;
  int nk = K > kGateRows ? kGateRows : 0;
  int next_pos = positions(nt, nk);
  auto copy_step = [&](int slot) {
    if (ct < ntok) {
      const int c = tl + cs * TPT;
      const bool in = c < nv;
      const uint32_t dst = mine + (uint32_t)slot * (kGateRows + 1) * kGateThreads * 16;
      const int at = in ? c : 0;
      copy16(dst, reinterpret_cast<const uint4*>(g + ct * D) + at, in);
#pragma unroll
      for (int r = 0; r < kGateRows; ++r) {
        const int q = __shfl_sync(0xffffffffu, pos, r);
        if (ck + r < K)
          copy16(dst + (r + 1) * kGateThreads * 16,
                 reinterpret_cast<const uint4*>(y + (int64_t)max(q, 0) * D) + at, in && q >= 0);
      }
      if (++cs == steps) {
        cs = 0;
        ct = nt;
        ck = nk;
        pos = next_pos;
        nk += kGateRows;
        if (nk >= K) {
          nk = 0;
          nt += dt;
        }
        next_pos = positions(nt, nk);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) copy_step(i);
  int slot = 0, buf = 0;
  for (int64_t t = t0; t < ntok; t += dt) {
    for (int k0 = 0; k0 < K; k0 += kGateRows) {
      float acc[kGateRows];
#pragma unroll
      for (int r = 0; r < kGateRows; ++r) acc[r] = 0.f;
      for (int i = 0; i < steps; ++i) {
        copy_step(slot == 0 ? S - 1 : slot - 1);  // the place of the step summed last
        asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
        const uint4* v = ring + slot * (kGateRows + 1) * kGateThreads + threadIdx.x;
        float fg[V];
        Vec16<T>::unpack(v[0], fg);
#pragma unroll
        for (int r = 0; r < kGateRows; ++r) {
          if (k0 + r < K) {
            float fy[V];
            Vec16<T>::unpack(v[(r + 1) * kGateThreads], fy);
#pragma unroll
            for (int j = 0; j < V; ++j) acc[r] = fmaf(fg[j], fy[j], acc[r]);
          }
        }
        slot = slot + 1 == S ? 0 : slot + 1;
      }
      float s = fold_rows(acc);
      if constexpr (TPT == 32) {
        if (lane < kGateRows && k0 + lane < K) dalpha[t * K + k0 + lane] = s;
      } else {
        if (lane < kGateRows) part[buf][warp][lane] = s;
        __syncthreads();
        if (threadIdx.x < kGateRows && k0 + (int)threadIdx.x < K) {
          s = 0.f;
#pragma unroll
          for (int w = 0; w < W; ++w) s += part[buf][w][threadIdx.x];
          dalpha[t * K + k0 + threadIdx.x] = s;
        }
        buf ^= 1;  // the other buffer next: one barrier a pass is enough
      }
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

template <typename T, int TPT>
static lrm_status launch_gate(const lrm_shape* s, const void* g, const void* y,
                              const int32_t* inv, float* dalpha, int32_t* err,
                              cudaStream_t cs) {
  constexpr size_t kSmem = (size_t)kGateSteps * (kGateRows + 1) * kGateThreads * 16;
  constexpr int64_t kPerSm = 4;  // CTAs that fit an SM's shared memory
  static_assert(kPerSm * (kSmem + 2048) <= 227 * 1024, "the rings of an SM's CTAs");
  const int64_t need = ((int64_t)s->T * TPT + kGateThreads - 1) / kGateThreads;
  // More CTAs than fit at once, so that an SM which starts late or reads slowly
  // gets fewer tokens. Behind lrm_route_bwd (T 16384 D 4096, both, us): 210, 187,
  // 181 and 177 for 1, 4, 8 and 16 times as many as fit; a warp a token
  // (D 256): 27.4, 24.0 and 24.5 for 1, 3 and 4.
  constexpr int64_t kTimes = TPT == 32 ? 3 : 16;
  const int blocks = (int)std::min<int64_t>(need, num_sms() * kPerSm * kTimes);
  auto kern = gate_grad_kernel<T, TPT, kGateSteps>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem) !=
      cudaSuccess) {
    (void)cudaGetLastError();
    return LRM_ERR_CUDA;
  }
  launch_k(kern, dim3(blocks), dim3(kGateThreads), kSmem, cs, (const T*)g, (const T*)y, inv,
           dalpha, s->T, s->D, s->K, err);
  return launch_status();
}

// A CTA a token from rows of 4 KB on, a warp a token below. Measured (bf16, K 8
// unless said, warp | CTA, us): T 16384 D 4096 195 | 178, T 200 D 4096 13.9 | 5.5,
// T 3000 D 2048 25.7 | 21.6, T 8192 D 704 K 4 15.8 | 24.1, T 16384 D 256 18.0 | 51.
template <typename T>
static lrm_status pick_gate(const lrm_shape* s, const void* g, const void* y, const int32_t* inv,
                            float* dalpha, int32_t* err, cudaStream_t cs) {
  if ((int64_t)s->D * (int64_t)sizeof(T) >= 4096)
    return launch_gate<T, kGateThreads>(s, g, y, inv, dalpha, err, cs);
  return launch_gate<T, 32>(s, g, y, inv, dalpha, err, cs);
}

}  // namespace lrm

using namespace lrm;

extern "C" lrm_status lrm_gate_grad(const lrm_shape* s, const void* g, const void* y,
                                    const int32_t* inv, float* dalpha, void* ws,
                                    size_t ws_bytes, void* stream) {
  LRM_NVTX("lrm_gate_grad");
  lrm_status st = check_shape(s);
  if (st != LRM_OK) return st;
  if ((st = check_ws(s, ws, ws_bytes)) != LRM_OK) return st;
  if ((st = check_ptrs(s, {}, {g, y, inv, dalpha})) != LRM_OK) return st;
  if (s->T == 0) return LRM_OK;
  cudaStream_t cs = (cudaStream_t)stream;
  return s->dtype == LRM_BF16
             ? pick_gate<__nv_bfloat16>(s, g, y, inv, dalpha, error_word(ws), cs)
             : pick_gate<float>(s, g, y, inv, dalpha, error_word(ws), cs);
}
