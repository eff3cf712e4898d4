// Gradient of the routing weights. The layer's output is
// out_t = sum_k alpha_tk y_(t,k), so
//   dalpha[t,k] = <g_t, y[inv[t*K+k]]>,
// the dot product of the token's cotangent with the output row of each expert
// it was routed to (y in dispatch order, as the forward pass leaves it).
//
// HBM-bound: every y row is read once (K rows a token against one row of g).
#include <algorithm>

#include "common.cuh"

namespace lrm {

constexpr int kGateThreads = 128;
constexpr int kGateRows = 8;  // y rows summed per pass over g_t

template <typename T>
__global__ void __launch_bounds__(kGateThreads)
gate_grad_kernel(const T* __restrict__ g, const T* __restrict__ y,
                 const int32_t* __restrict__ inv, float* __restrict__ dalpha, int ntok, int D,
                 int K, int32_t* err) {
  pdl_begin();  // predecessor complete before any global access
  constexpr int V = Vec16<T>::kElems;
  constexpr int W = kGateThreads / 32;
  __shared__ float part[W][kGateRows];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t N = (int64_t)ntok * K;
  const int nv = D / V;
  for (int64_t t = blockIdx.x; t < ntok; t += gridDim.x) {
    const uint4* grow = reinterpret_cast<const uint4*>(g + t * D);
    for (int k0 = 0; k0 < K; k0 += kGateRows) {
      const uint4* row[kGateRows];
      bool ok[kGateRows];
      float acc[kGateRows];
#pragma unroll
      for (int r = 0; r < kGateRows; ++r) {
        int q = 0;
        ok[r] = k0 + r < K;
        if (ok[r]) {
          q = inv[t * K + k0 + r];
          if (q < 0 || q >= N) {
            flag_error(err, LRM_DEVERR_INDEX);
            ok[r] = false;
            q = 0;
          }
        }
        row[r] = reinterpret_cast<const uint4*>(y + (int64_t)q * D);
        acc[r] = 0.f;
      }
      for (int c = threadIdx.x; c < nv; c += kGateThreads) {
        uint4 vy[kGateRows];
        const uint4 vg = grow[c];
#pragma unroll
        for (int r = 0; r < kGateRows; ++r)
          vy[r] = ok[r] ? ld_stream(row[r] + c) : make_uint4(0, 0, 0, 0);
        float fg[V];
        Vec16<T>::unpack(vg, fg);
#pragma unroll
        for (int r = 0; r < kGateRows; ++r) {
          float fy[V];
          Vec16<T>::unpack(vy[r], fy);
#pragma unroll
          for (int i = 0; i < V; ++i) acc[r] = fmaf(fg[i], fy[i], acc[r]);
        }
      }
#pragma unroll
      for (int r = 0; r < kGateRows; ++r) {
        const float s = warp_sum(acc[r]);
        if (lane == 0) part[warp][r] = s;
      }
      __syncthreads();
      if (threadIdx.x < kGateRows && k0 + (int)threadIdx.x < K) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) s += part[w][threadIdx.x];
        dalpha[t * K + k0 + threadIdx.x] = s;
      }
      __syncthreads();
    }
  }
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
  const int blocks = (int)std::min<int64_t>(s->T, (int64_t)num_sms() * 64);
  cudaStream_t cs = (cudaStream_t)stream;
  if (s->dtype == LRM_BF16)
    launch_k(gate_grad_kernel<__nv_bfloat16>, dim3(blocks), dim3(kGateThreads), 0, cs,
             (const __nv_bfloat16*)g, (const __nv_bfloat16*)y, inv, dalpha, s->T, s->D, s->K,
             error_word(ws));
  else
    launch_k(gate_grad_kernel<float>, dim3(blocks), dim3(kGateThreads), 0, cs, (const float*)g,
             (const float*)y, inv, dalpha, s->T, s->D, s->K, error_word(ws));
  return launch_status();
}
