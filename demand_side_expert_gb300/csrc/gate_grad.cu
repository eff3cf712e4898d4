// Gradient of the routing weights. The layer's output is
// out_t = sum_k alpha_tk y_(t,k), so
//   dalpha[t,k] = <g_t, y[inv[t*K+k]]>,
// the dot product of the token's cotangent with the output row of each expert
// it was routed to (y in dispatch order, as the forward pass leaves it).
//
// HBM-bound: every y row is read once (K rows a token against one row of g).
// What counts is the bytes an SM keeps in flight and the instructions for them:
// loads into registers got to 0.70-0.90 of the copy bandwidth (257-198 us at
// T 16384 D 4096 K 8, bf16, by how many were unrolled), a ring of asynchronous
// copies in shared memory gets to 1.05 (169 us, 7.1 TB/s); with its step made for
// 8 rows whatever K, K 2 took 99 us where it takes 62. Bad entries of inv cost only
// where there are any.
#include <algorithm>

#include "common.cuh"

namespace lrm {

constexpr int kGateThreads = 128;
constexpr int kGateRows = 8;  // y rows summed in one pass over g_t, at most
// Steps of copies in flight. With 8 rows 2, 3, 4 and 6 measured 191, 178, 192 and
// 239 us at T 16384 D 4096 (fewer CTAs fit an SM where the rings are deeper).
constexpr int kGateSteps = 3;
// Pieces of every row in a step of R rows: a step has 8 to 10 pieces in all.
constexpr int gate_pieces(int R) { return R == 8 ? 1 : R == 4 ? 2 : R == 2 ? 3 : 4; }

// Adds R values over the warp: lane r (mod R) ends with row r's sum. Every
// halving trades half of the values against half of the lanes, so that 9
// exchanges do the work of 40 for R = 8.
template <int R>
__device__ __forceinline__ float fold_rows(float (&v)[R]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = R / 2; o > 0; o >>= 1) {
    const bool high = lane & o;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float keep = high ? v[i + o] : v[i], give = high ? v[i] : v[i + o];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  float s = v[0];
#pragma unroll
  for (int o = R; o < 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool valid) {
  // an invalid source is not read: 16 zero bytes are written
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}

// TPT threads a token (a warp, or the CTA), R rows of y a pass. A step is a few
// 16-byte pieces of g_t and of the rows for every thread; it is copied to the
// thread's own places in shared memory, kGateSteps - 1 steps ahead of the one
// being summed, across the ends of tokens. Nobody else reads them, so a thread
// waits for its own copies and there is no barrier. Four CTAs an SM, what their
// rings leave room for, are said outright: left to choose, the compiler squeezes the
// registers and spills (T 16384 D 4096 K 8: 175 us instead of 169).
template <typename T, int TPT, int R>
__global__ void __launch_bounds__(kGateThreads, 4)
gate_grad_kernel(const T* __restrict__ g, const T* __restrict__ y,
                 const int32_t* __restrict__ inv, float* __restrict__ dalpha, int ntok, int D,
                 int K, int32_t* err) {
  pdl_begin();  // predecessor complete before any global access
  constexpr int V = Vec16<T>::kElems;
  constexpr int W = kGateThreads / 32;
  constexpr int kTokens = kGateThreads / TPT;
  constexpr int U = gate_pieces(R), S = kGateSteps;
  extern __shared__ uint4 ring[];  // [S][U][R + 1][threads]
  __shared__ float part[2][W][R];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tl = threadIdx.x % TPT;
  const int64_t N = (int64_t)ntok * K;
  const int nv = D / V;
  const int steps = (nv + TPT * U - 1) / (TPT * U);
  const int64_t t0 = (int64_t)blockIdx.x * kTokens + threadIdx.x / TPT;
  const int64_t dt = (int64_t)gridDim.x * kTokens;
  const uint32_t mine = (uint32_t)__cvta_generic_to_shared(ring + threadIdx.x);

  // copies: token, step, the rows' positions
  int64_t ct = t0;
  int cs = 0;
  int row[R];
  // lane r: position of row r of a pass; a bad entry reads nothing
  bool bad = false;
  auto positions = [&](int64_t t, int k0) {
    int q = -1;
    if (t < ntok && lane < R && k0 + lane < K) {
      q = inv[t * K + k0 + lane];
      if (q < 0 || q >= N) {
        flag_error(err, LRM_DEVERR_INDEX);
        bad = true;
        q = -1;
      }
    }
    return q;
  };
  auto spread = [&](int pos) {
#pragma unroll
    for (int r = 0; r < R; ++r) row[r] = __shfl_sync(0xffffffffu, pos, r);
  };
  // positions of the pass after that one, read a pass ahead
  int64_t nt = K > R ? ct : ct + dt;
  int nk = K > R ? R : 0;
  const int first_pos = positions(ct, 0);
  int next_pos = positions(nt, nk);
  spread(first_pos);
  auto copy_step = [&](int slot) {
    if (ct < ntok) {
      uint32_t dst = mine + (uint32_t)slot * U * (R + 1) * kGateThreads * 16;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = tl + (cs * U + u) * TPT;
        const bool in = c < nv;
        const int at = in ? c : 0;
        copy16(dst, reinterpret_cast<const uint4*>(g + ct * D) + at, in);
#pragma unroll
        for (int r = 0; r < R; ++r)
          copy16(dst + (r + 1) * kGateThreads * 16,
                 reinterpret_cast<const uint4*>(y + (int64_t)max(row[r], 0) * D) + at,
                 in && row[r] >= 0);
        dst += (R + 1) * kGateThreads * 16;
      }
      if (++cs == steps) {
        cs = 0;
        ct = nt;
        spread(next_pos);
        nk += R;
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
    for (int k0 = 0; k0 < K; k0 += R) {
      float acc[R];
#pragma unroll
      for (int r = 0; r < R; ++r) acc[r] = 0.f;
      for (int i = 0; i < steps; ++i) {
        copy_step(slot == 0 ? S - 1 : slot - 1);  // the place of the step summed last
        asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
        const uint4* v = ring + slot * U * (R + 1) * kGateThreads + threadIdx.x;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float fg[V];
          Vec16<T>::unpack(v[u * (R + 1) * kGateThreads], fg);
#pragma unroll
          for (int r = 0; r < R; ++r) {
            float fy[V];
            Vec16<T>::unpack(v[(u * (R + 1) + r + 1) * kGateThreads], fy);
#pragma unroll
            for (int j = 0; j < V; ++j) acc[r] = fmaf(fg[j], fy[j], acc[r]);
          }
        }
        slot = slot + 1 == S ? 0 : slot + 1;
      }
      float s = fold_rows<R>(acc);
      if constexpr (TPT == 32) {
        if (lane < R && k0 + lane < K) dalpha[t * K + k0 + lane] = s;
      } else {
        if (lane < R) part[buf][warp][lane] = s;
        __syncthreads();
        if (threadIdx.x < R && k0 + (int)threadIdx.x < K) {
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
  // A bad entry yields 0: the zeros copied in its row's place made NaN of an infinite
  // g. The lane that wrote it writes it again, here, where almost no call comes.
  if (bad && (TPT == 32 || warp == 0)) {
    for (int64_t t = t0; t < ntok; t += dt)
      for (int k = lane; k < K; k += R) {
        const int q = inv[t * K + k];
        if (q < 0 || q >= N) dalpha[t * K + k] = 0.f;
      }
  }
}

// Bytes of a CTA's ring, and CTAs that fit an SM's shared memory with theirs.
constexpr size_t gate_smem(int R) {
  return (size_t)kGateSteps * gate_pieces(R) * (R + 1) * kGateThreads * 16;
}
constexpr int64_t gate_per_sm(int R) { return 227 * 1024 / (gate_smem(R) + 2048); }

template <typename T, int TPT, int R>
static lrm_status launch_gate(const lrm_shape* s, const void* g, const void* y,
                              const int32_t* inv, float* dalpha, int32_t* err,
                              cudaStream_t cs) {
  constexpr size_t kSmem = gate_smem(R);
  const int64_t need = ((int64_t)s->T * TPT + kGateThreads - 1) / kGateThreads;
  // More CTAs than fit at once, so that an SM which starts late or reads slowly
  // gets fewer tokens. Behind lrm_route_bwd (T 16384 D 4096, both, us): 210, 187,
  // 181 and 177 for 1, 4, 8 and 16 times as many as fit; a warp a token
  // (D 256): 27.4, 24.0 and 24.5 for 1, 3 and 4.
  constexpr int64_t kTimes = TPT == 32 ? 3 : 16;
  const int blocks = (int)std::min<int64_t>(need, num_sms() * gate_per_sm(R) * kTimes);
  auto kern = gate_grad_kernel<T, TPT, R>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem) !=
      cudaSuccess) {
    (void)cudaGetLastError();
    return LRM_ERR_CUDA;
  }
  launch_k(kern, dim3(blocks), dim3(kGateThreads), kSmem, cs, (const T*)g, (const T*)y, inv,
           dalpha, s->T, s->D, s->K, err);
  return launch_status();
}

// A CTA a token where every token's CTA is resident at once and a token has 8 KB or
// more (a warp a token would leave SMs with a few warps each), and for any number of
// tokens of 35 KB or more where four CTAs fit an SM (not so with R = 4); a warp a token
// else. Measured (warp | CTA, us), bf16:
//   K 8        T 305        600        900        1500       6000       16384
//   D  512     3.2 |  3.2   3.9 | 4.0  4.4 | 5.6  5.5 | 7.5  12.2|20.8  27.6| 47.2
//   D 1000     4.4 |  4.0   5.4 | 5.2  6.3 | 6.7  8.8 | 8.8  21.6|25.9  51.1| 56.6
//   D 2040     6.5 |  5.4   7.5 | 7.3  9.1 | 9.1  13.6|12.4  38.3|37.8  97.6| 94.7
//   D 4096     9.0 |  7.1  11.2 |10.4 13.9 |14.4  22.0|21.2  68.9|67.0 178.7|169.5
//   K 4 D 4096 6.3 |  5.2   7.5 | 7.7  9.1 | 9.7  13.0|13.2  39.2|42.3 100.1|100.9
//   K 2 D 4096 4.7 |  4.4   5.8 | 5.8  7.1 | 7.5   9.8| 9.9  26.3|29.7  62.2| 68.1
//   K 1 D  512 2.6 |  2.8   2.8 | 3.0  2.8 | 4.2   3.2| 5.8   7.0|16.9  10.8| 34.5
// and float32: K 8 D 1000 (36 KB) 12.4 | 11.9 at T 1500, 92.3 | 90.2 at 16384; K 2
// D 4096 (48 KB) 15.3 | 14.7, 115.2 | 115.6; bf16 K 16 D 1000 (34 KB) 13.4 | 12.8,
// 93.5 | 95.8.
template <typename T, int R>
static lrm_status pick_threads(const lrm_shape* s, const void* g, const void* y,
                               const int32_t* inv, float* dalpha, int32_t* err,
                               cudaStream_t cs) {
  const int64_t token = ((int64_t)s->K + 1) * s->D * (int64_t)sizeof(T);
  if ((token >= 8 * 1024 && s->T <= num_sms() * gate_per_sm(R)) ||
      (token >= 35 * 1024 && gate_per_sm(R) >= 4))
    return launch_gate<T, kGateThreads, R>(s, g, y, inv, dalpha, err, cs);
  return launch_gate<T, 32, R>(s, g, y, inv, dalpha, err, cs);
}

template <typename T>
static lrm_status pick_gate(const lrm_shape* s, const void* g, const void* y, const int32_t* inv,
                            float* dalpha, int32_t* err, cudaStream_t cs) {
  if (s->K == 1) return pick_threads<T, 1>(s, g, y, inv, dalpha, err, cs);
  if (s->K == 2) return pick_threads<T, 2>(s, g, y, inv, dalpha, err, cs);
  if (s->K <= 4) return pick_threads<T, 4>(s, g, y, inv, dalpha, err, cs);
  return pick_threads<T, kGateRows>(s, g, y, inv, dalpha, err, cs);
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
