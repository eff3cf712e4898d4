/*
 * lrm.h -- C ABI of the recalibrated MoE expert backward on one GB300 GPU.
 *
 * The path follows "LRMoE: Demand-Side Load Re-Calibration for Efficient MoE
 * Training on Memory-Constrained Nodes" (arXiv 2610.37720) on a single GPU:
 *   forward dispatch permutation -> LRM score of every routed pair ->
 *   per-expert top-q selection -> physical compaction -> SwiGLU expert
 *   backward as variable-size grouped GEMMs over the retained rows only.
 * Multi-GPU routing, replicas, all-to-all and the CPU offload queue of the
 * paper are not part of this library.
 *
 * Notation: T tokens, D model dim, H expert FFN dim, E experts, K routed
 * experts per token, N = T*K routed pairs; pair index p = t*K + k.
 * "Dispatch order" lists the pairs grouped by expert (expert-major), inside a
 * group by ascending p.
 *
 * Conventions shared by every entry point:
 *  - Pointers are DEVICE pointers owned by the caller unless stated; the
 *    library never allocates or frees memory and keeps no global state
 *    (calls on different streams are independent).
 *  - All calls are asynchronous on `stream` (a cudaStream_t passed as void*;
 *    NULL = legacy default stream) and never synchronise the host, except
 *    lrm_get_device_error.
 *  - Row-major contiguous layouts. Floating-point activations and weights
 *    (x, g, ab, phi, W_*, dy_c, x_c, ab_c, phi_c, dab_c) have the element type
 *    of lrm_shape.dtype (LRM_BF16: bfloat16, LRM_F32: float); routing weights,
 *    scores and all gradients in float32; indices int32.
 *  - Every pointer must be 16-byte aligned and D, H multiples of 8, else
 *    LRM_ERR_UNSUPPORTED. The BF16 grouped backward also needs D and H to be
 *    multiples of 64.
 *  - Argument errors are returned before anything is launched. A failed
 *    launch returns LRM_ERR_CUDA. Bad DATA found on the device (an expert id
 *    outside [0, E), a quota outside [0, n_e], an index out of range, a
 *    pipeline wait that timed out) never traps: the kernel clamps or skips,
 *    ORs an LRM_DEVERR_* bit into the device error word kept in the first 4
 *    bytes of the caller's workspace, and the call returns LRM_OK; read the
 *    word with lrm_get_device_error.
 *  - ws / ws_bytes: caller-owned device workspace of at least
 *    lrm_workspace_bytes(shape) bytes, 256-byte aligned. Its first 256 bytes
 *    are a header: the device error word and the tile-queue counters of the
 *    weight-gradient products, which every such launch leaves at zero for
 *    the next one. Zero the header once with lrm_clear_device_error before
 *    first use, and let one workspace serve one stream at a time (two
 *    weight-gradient launches in flight together would share the queue).
 */
#ifndef LRM_H_
#define LRM_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum lrm_status {
  LRM_OK = 0,
  LRM_ERR_INVALID_ARG = 1, /* null pointer, negative or inconsistent size */
  LRM_ERR_UNSUPPORTED = 2, /* alignment / dimension not supported */
  LRM_ERR_WORKSPACE = 3,   /* workspace missing or too small */
  LRM_ERR_CUDA = 4         /* a CUDA launch or runtime call failed */
} lrm_status;

typedef enum lrm_dtype { LRM_F32 = 0, LRM_BF16 = 1 } lrm_dtype;

/* Layer shape. dtype is an lrm_dtype. N = T*K must be < 2^31. */
typedef struct lrm_shape {
  int32_t T, D, H, E, K;
  int32_t dtype;
} lrm_shape;

/* Bits of the device error word. */
#define LRM_DEVERR_EXPERT_ID 1 /* topk_idx outside [0,E): clamped          */
#define LRM_DEVERR_QUOTA 2     /* quota outside [0,n_e]: clamped           */
#define LRM_DEVERR_INDEX 4     /* inv / perm / sel_pos out of range: row skipped */
#define LRM_DEVERR_TIMEOUT 8   /* a GEMM pipeline wait gave up: outputs invalid */
#define LRM_DEVERR_QUEUE 16    /* a weight-gradient tile queue did not hand out
                                  every tile once (header not zeroed before first
                                  use, or shared by concurrent launches): outputs
                                  invalid; the queue is rewound for the next call */

/* Bytes of workspace every call of this shape needs (host only, pure). */
size_t lrm_workspace_bytes(const lrm_shape* shape);

/* Zero the workspace header (the device error word in its first 4 bytes and
 * the tile-queue counters). Async on stream. */
lrm_status lrm_clear_device_error(void* ws, size_t ws_bytes, void* stream);

/* Synchronise `stream`, then copy the device error word into *code_out. */
lrm_status lrm_get_device_error(const void* ws, size_t ws_bytes,
                                int32_t* code_out, void* stream);

/* Human-readable name of a status code (static string). */
const char* lrm_status_string(lrm_status status);

/*
 * Forward dispatch permutation: a stable counting sort of the pairs by
 * expert id. "Least-Loaded Expert Parallelism" (LLEP) Sec. 2.1 re-index
 * (tokens [a,b,c,d] routed to experts [2,6,2,1] become [d,a,c,b]) and LLEP
 * Alg. 4 sort of the flattened indices; LRMoE Alg. 1 forward admission
 * counts N_e = |P_e|.
 *   topk_idx [T,K] int32 : expert of pair p = t*K+k (read).
 *   perm     [N]   int32 : perm[pos] = p, dispatch position -> pair (written).
 *   inv      [N]   int32 : inv[p] = pos (written).
 *   counts   [E]   int32 : n_e (written).
 *   off      [E+1] int32 : exclusive prefix of counts, off[E] = N (written).
 * Ids outside [0,E) are clamped into range and flag LRM_DEVERR_EXPERT_ID.
 */
lrm_status lrm_dispatch_permute(const lrm_shape* shape, const int32_t* topk_idx,
                                int32_t* perm, int32_t* inv, int32_t* counts,
                                int32_t* off, void* ws, size_t ws_bytes,
                                void* stream);

/*
 * Row re-index into dispatch order, dst[pos] = src[perm[pos]] for
 * pos < n_rows (LLEP Sec. 2.1: B' is B with its rows taken in dispatch
 * order). row_bytes must be a positive multiple of 16; src and dst must not
 * overlap. Rows whose perm entry is outside [0, n_rows) are left untouched.
 */
lrm_status lrm_permute_rows(const int32_t* perm, int32_t n_rows, const void* src,
                            void* dst, int64_t row_bytes, void* stream);

/*
 * Per-expert retention quota q_e = min(ceil(num/den * n_e), cap), computed
 * in exact integer arithmetic; cap <= 0 means no cap. LRMoE Sec. 3.1: quotas
 * satisfy 0 <= K_e <= N_e with retention rate rho = sum_e K_e / N, fixed for
 * the invocation. Needs 0 <= num <= den, den > 0.
 *   counts [E] int32 (read), quota [E] int32 (written).
 */
lrm_status lrm_quota_from_rate(const int32_t* counts, int32_t E, int32_t num,
                               int32_t den, int32_t cap, int32_t* quota,
                               void* stream);

/*
 * Load Recalibration Metric of every routed pair, LRMoE Sec. 3.2 Prop. 3.1
 * Eq. 3 and Sec. 7.1 Eq. 12: R_u = alpha_u^2 * ||g_t||^2 * ||phi_u||^2, the
 * squared Frobenius norm of the pair's rank-one FC2 weight-gradient
 * contribution (alpha_u g_t) phi_u^T; g_t is the cotangent at the MoE output
 * before the routing weight (Sec. 7.1 Eq. 5). FP32 accumulation.
 *   g     [T,D] dtype          : output cotangent (read).
 *   phi   [N,H] dtype          : saved FC2 input, dispatch order (read).
 *   alpha [T,K] float          : routing weights (read).
 *   inv   [N]   int32          : from lrm_dispatch_permute (read).
 *   score [N]   float          : R in dispatch order (written).
 */
lrm_status lrm_score(const lrm_shape* shape, const void* g, const void* phi,
                     const float* alpha, const int32_t* inv, float* score,
                     void* ws, size_t ws_bytes, void* stream);

/*
 * The selection criteria LRMoE Sec. 4.7 (Table 2) compares LRM against,
 * computed like lrm_score and written to score [N] in dispatch order:
 *   LRM_METRIC_LRM       alpha_u^2 ||g_t||^2 ||phi_u||^2   (= lrm_score)
 *   LRM_METRIC_GRAD_SQ   ||g_t||_2^2       squared gradient norm
 *   LRM_METRIC_GRAD_ABS  sum_d |g_t,d|     absolute gradient magnitude
 *   LRM_METRIC_RANDOM    output p+1 of SplitMix64 seeded with `seed`, top 24
 *                        bits as a float in [0,1): random selection
 * The gradient-only criteria read g only (alpha and phi may be NULL); the
 * random one reads neither (g may be NULL too). All are non-negative, so
 * lrm_select_quota applies to them unchanged.
 */
typedef enum lrm_metric {
  LRM_METRIC_LRM = 0,
  LRM_METRIC_GRAD_SQ = 1,
  LRM_METRIC_GRAD_ABS = 2,
  LRM_METRIC_RANDOM = 3
} lrm_metric;
lrm_status lrm_score_variant(const lrm_shape* shape, int32_t metric, uint64_t seed,
                             const void* g, const void* phi, const float* alpha,
                             const int32_t* inv, float* score, void* ws,
                             size_t ws_bytes, void* stream);

/*
 * Per-expert top-q selection, LRMoE Alg. 1 (TopK per expert) and Sec. 7.2
 * Prop. 7.1 (keeping the largest scores inside each expert is optimal for
 * fixed per-expert quotas). Inside each segment [off[e], off[e+1]) the q_e
 * largest scores are kept; equal scores are broken by the lower pair index,
 * which inside a segment is the lower dispatch position. Scores must be
 * non-negative and not NaN (they are sums of squares).
 *   score   [N]   float (read), off [E+1] int32 (read), quota [E] int32 (read).
 *   keep    [N]   uint8 : 1 if retained, dispatch order (written).
 *   sel_off [E+1] int32 : exclusive prefix of the quotas (written).
 *   sel_pos [N]   int32 : capacity N; the first M = sel_off[E] entries are
 *                         the retained dispatch positions, ascending inside
 *                         each expert (written).
 * Quotas outside [0, n_e] are clamped and flag LRM_DEVERR_QUOTA.
 */
lrm_status lrm_select_quota(const lrm_shape* shape, const float* score,
                            const int32_t* off, const int32_t* quota,
                            uint8_t* keep, int32_t* sel_off, int32_t* sel_pos,
                            void* ws, size_t ws_bytes, void* stream);

/*
 * Physical compaction, LRMoE Sec. 3.1 (compact runtime) and Sec. 3.4 Fig. 4:
 * retained gradient rows and their saved state are gathered into contiguous
 * expert-major segments, with no zero-masked rows. For retained row
 * j < M = sel_off[E]: i = sel_pos[j], p = perm[i], t = p / K:
 *   dy_c[j]  = alpha[p] * g[t]   (product in float32, rounded once to dtype)
 *   x_c[j]   = x[t],  ab_c[j] = ab[i],  phi_c[j] = phi[i],  tok_c[j] = t
 *   row_of_pos[i] = j, and -1 at every position with keep[i] == 0.
 * Inputs: perm [N], keep [N], sel_off [E+1], sel_pos [N], alpha [T,K],
 *   x [T,D], g [T,D], ab [N,2H] (gate|up pre-activations, dispatch order),
 *   phi [N,H] (dispatch order).
 * Outputs (capacity N rows each, first M written): dy_c [N,D], x_c [N,D],
 *   ab_c [N,2H], phi_c [N,H], tok_c [N] int32; row_of_pos [N] int32.
 * Rows [M, min(M + 64, N)) of dy_c are written as zeros: the weight-gradient
 * products read them as padding past the last group.
 * x_c, ab_c and phi_c may each be NULL: that copy is skipped and its source
 * may be NULL too (see lrm_expert_fc1_recompute, which rebuilds [a | b], and
 * lrm_expert_bwd_gathered, which reads x, ab and phi rows in place). A
 * non-NULL destination with a NULL source is an error.
 * M is read from sel_off[E] on the device: a value outside [0, N] (sel_off
 * not produced by a selection call) is clamped into that range and flags
 * LRM_DEVERR_INDEX in the workspace error word; out-of-range sel_pos or perm
 * entries are skipped and flag the same bit.
 */
lrm_status lrm_compact(const lrm_shape* shape, const int32_t* perm,
                       const uint8_t* keep, const int32_t* sel_off,
                       const int32_t* sel_pos, const float* alpha, const void* x,
                       const void* g, const void* ab, const void* phi, void* dy_c,
                       void* x_c, void* ab_c, void* phi_c, int32_t* tok_c,
                       int32_t* row_of_pos, void* ws, size_t ws_bytes,
                       void* stream);

/*
 * SwiGLU expert backward over the retained rows, LRMoE Alg. 1
 * (PackedExpertBackward) and Sec. 3.4: four variable-size grouped products
 * per expert e over its m_e = sel_off[e+1] - sel_off[e] compacted rows J
 * (m_e is the row dimension of the data-gradient products and the reduction
 * dimension of the weight-gradient products; no padding):
 *   dphi       = dy_c[J] W_down[e]^T,  then the SwiGLU gradient
 *                da = dphi*b*s*(1 + a*(1-s)), db = dphi*a*s, s = sigmoid(a),
 *                (a, b) = ab_c[J] halves  -> dab_c[J] = [da | db]   (dtype)
 *   dW_down[e] = phi_c[J]^T dy_c[J]                               (H x D)
 *   dW_gate[e] = x_c[J]^T da,  dW_up[e] = x_c[J]^T db             (D x H)
 *   dx_c[J]    = da W_gate[e]^T + db W_up[e]^T                    (float32)
 * then the scatter back to tokens (Sec. 3.1: zero-initialised dense buffer):
 *   dx[t] = sum over kept slots k, ascending, of dx_c[row_of_pos[inv[t*K+k]]]
 * (deterministic, no atomics). BF16 runs on tcgen05 tensor cores with FP32
 * accumulation in tensor memory; F32 runs on CUDA cores.
 *   w_gate, w_up [E,D,H] dtype; w_down [E,H,D] dtype (read).
 *   dy_c, x_c [N,D]; ab_c [N,2H]; phi_c [N,H]  (read, first M rows used).
 *   inv [N], row_of_pos [N] int32 (read).
 *   dab_c [N,2H] dtype, dx_c [N,D] float : intermediates (first M rows written).
 *   dw_gate, dw_up [E,D,H] float; dw_down [E,H,D] float : OVERWRITTEN
 *     (zero for experts with no retained rows).
 *   dx [T,D] float : overwritten.
 * Pipeline waits are bounded; a timeout flags LRM_DEVERR_TIMEOUT.
 */
lrm_status lrm_expert_bwd_grouped(const lrm_shape* shape, const int32_t* sel_off,
                                  const void* w_gate, const void* w_up,
                                  const void* w_down, const void* dy_c,
                                  const void* x_c, const void* ab_c,
                                  const void* phi_c, const int32_t* inv,
                                  const int32_t* row_of_pos, void* dab_c,
                                  float* dx_c, float* dw_gate, float* dw_up,
                                  float* dw_down, float* dx, void* ws,
                                  size_t ws_bytes, void* stream);

/*
 * Self-test of the failure detection in the grouped GEMMs (no counterpart on
 * the pages). Every pipeline wait in those kernels is bounded; this launches
 * one grouped-GEMM CTA whose copy warp is told to deliver nothing, so the MMA
 * warp's wait for its first operand stage runs out after 20 ms. The CTA then
 * ORs LRM_DEVERR_TIMEOUT into the error word, frees its tensor memory and
 * returns; the CUDA context stays usable. It clears the error word first and
 * writes only the first 256 bytes of ws. Read the result with
 * lrm_get_device_error (expect LRM_DEVERR_TIMEOUT).
 */
lrm_status lrm_selftest_wait_timeout(void* ws, size_t ws_bytes, void* stream);

/*
 * lrm_dispatch_permute for callers that cannot allocate device memory (the
 * paper has no counterpart; this is a deployment variant). Some callers are
 * handed only their input and output tensors, e.g. a plugin inside a host
 * whose memory manager owns the whole device budget; a cudaMalloc there
 * would bypass that accounting and can stall the whole device. This entry
 * point allocates nothing. Up to 2^17 routed pairs it runs the one-cluster
 * dispatch, which needs no scratch; above that, the per-chunk tables of the
 * three-launch dispatch live in one file-scope device array of
 * 2 * LRM_NOALLOC_MAX_CHUNK_ENTRIES int32 (512 KiB), which every GPU that
 * loads the library holds until the process exits.
 *  - Same outputs as lrm_dispatch_permute (bit for bit). dev_err may be
 *    NULL; otherwise LRM_DEVERR_EXPERT_ID is ORed into *dev_err (a 4-byte
 *    device word the caller clears).
 *  - Limit: E * ceil(T*K / 2048) <= LRM_NOALLOC_MAX_CHUNK_ENTRIES, else
 *    LRM_ERR_WORKSPACE is returned before anything is launched (the built-in
 *    scratch is too small; use lrm_dispatch_permute with a workspace).
 *  - The first call on each device that needs the array (more than 2^17
 *    pairs) looks up its device address with cudaGetSymbolAddress (once,
 *    with that device current); make that first call before any stream
 *    capture.
 *  - All calls share the one array: calls whose kernels overlap on the GPU
 *    (different streams, or several host threads) race and corrupt each
 *    other's results; serialise them. Every table entry a call reads is
 *    written earlier in the same call, so stale contents are harmless.
 */
#define LRM_NOALLOC_MAX_CHUNK_ENTRIES 65536
lrm_status lrm_dispatch_permute_noalloc(const lrm_shape* shape,
                                        const int32_t* topk_idx, int32_t* perm,
                                        int32_t* inv, int32_t* counts,
                                        int32_t* off, int32_t* dev_err,
                                        void* stream);

/*
 * The five sub-steps of lrm_expert_bwd_grouped as separate calls, same
 * arithmetic, arguments and layouts as documented there (LRMoE Sec. 3.4:
 * both layers' data- and weight-gradient products run over the retained
 * rows). Issue them in this order on one stream; each reads only
 * what the earlier ones wrote.
 *   lrm_expert_fc2_dgrad : dab_c = SwiGLU-grad(dy_c W_down[e]^T, ab_c); also
 *                          zeroes rows [M, min(M + 64, N)) of dab_c (padding
 *                          read by lrm_expert_fc1_wgrad past the last group)
 *   lrm_expert_fc2_wgrad : dW_down[e] = phi_c^T dy_c        (overwritten)
 *   lrm_expert_fc1_wgrad : dW_gate[e], dW_up[e] = x_c^T dab_c (overwritten)
 *   lrm_expert_fc1_dgrad : dx_c = dab_c [W_gate | W_up][e]^T
 *   lrm_scatter_dx       : dx[t] = sum of the token's kept dx_c rows
 */
lrm_status lrm_expert_fc2_dgrad(const lrm_shape* shape, const int32_t* sel_off,
                                const void* w_down, const void* dy_c,
                                const void* ab_c, void* dab_c, void* ws,
                                size_t ws_bytes, void* stream);
lrm_status lrm_expert_fc2_wgrad(const lrm_shape* shape, const int32_t* sel_off,
                                const void* phi_c, const void* dy_c,
                                float* dw_down, void* ws, size_t ws_bytes,
                                void* stream);
lrm_status lrm_expert_fc1_wgrad(const lrm_shape* shape, const int32_t* sel_off,
                                const void* x_c, const void* dab_c,
                                float* dw_gate, float* dw_up, void* ws,
                                size_t ws_bytes, void* stream);
lrm_status lrm_expert_fc1_dgrad(const lrm_shape* shape, const int32_t* sel_off,
                                const void* w_gate, const void* w_up,
                                const void* dab_c, float* dx_c, void* ws,
                                size_t ws_bytes, void* stream);
lrm_status lrm_scatter_dx(const lrm_shape* shape, const float* dx_c,
                          const int32_t* inv, const int32_t* row_of_pos,
                          float* dx, void* ws, size_t ws_bytes, void* stream);

/*
 * Forward expert pass: the pass that produces the saved state the backward
 * reads. LRMoE Sec. 3.1 (design overview) and Alg. 1
 * (FullForwardAndSaveContext): every routed pair runs through its expert,
 * the outputs are combined, and [a | b] and phi are kept per pair. LLEP
 * Sec. 2.1: token rows are re-indexed into per-expert groups (the
 * lrm_dispatch_permute order), one product per expert and group, and the
 * MoE output is the routing-weighted sum h_t = sum_k alpha_tk y_(t,k).
 * SwiGLU experts: a = x W_gate[e], b = x W_up[e], phi = SiLU(a) * b,
 * y = phi W_down[e]. FP32 accumulation; [a | b], phi and y are rounded once
 * to the layer dtype (phi from the unrounded a and b).
 * Groups come from `off` (lrm_dispatch_permute), read on the device; every
 * routed row is processed. BF16 layers need D and H multiples of 64.
 *
 * lrm_gather_tokens: x_disp[pos] = x[perm[pos] / K].
 *   perm [N] int32 (read); x [T,D] dtype (read); x_disp [N,D] dtype (written).
 *   perm entries outside [0,N) skip the row and flag LRM_DEVERR_INDEX.
 * lrm_expert_fc1_fwd: ab [N,2H] = [a | b] and phi [N,H] (dtype, written)
 *   from x_disp [N,D] and W_gate, W_up [E,D,H] (dtype, read).
 * lrm_expert_fc2_fwd: y [N,D] dtype (written) from phi [N,H] and
 *   W_down [E,H,D] (dtype, read).
 * lrm_combine: out [T,D] float (written) = sum over slots k ascending of
 *   alpha[t,k] * y[inv[t*K+k]]; alpha [T,K] float, inv [N] int32 (read).
 *   Needs K <= 32.
 * lrm_expert_fwd_grouped: the four in order, on one stream.
 * Buffers are caller-owned device memory, 16-byte aligned, not overlapping.
 * Sizes whose off[E] exceeds N, or non-monotone off, process no rows and
 * flag LRM_DEVERR_INDEX. Host argument errors return before any launch.
 */
lrm_status lrm_gather_tokens(const lrm_shape* shape, const int32_t* perm, const void* x,
                             void* x_disp, void* ws, size_t ws_bytes, void* stream);
lrm_status lrm_expert_fc1_fwd(const lrm_shape* shape, const int32_t* off,
                              const void* x_disp, const void* w_gate, const void* w_up,
                              void* ab, void* phi, void* ws, size_t ws_bytes,
                              void* stream);
lrm_status lrm_expert_fc2_fwd(const lrm_shape* shape, const int32_t* off, const void* phi,
                              const void* w_down, void* y, void* ws, size_t ws_bytes,
                              void* stream);
lrm_status lrm_combine(const lrm_shape* shape, const void* y, const float* alpha,
                       const int32_t* inv, float* out, void* ws, size_t ws_bytes,
                       void* stream);
lrm_status lrm_expert_fwd_grouped(const lrm_shape* shape, const int32_t* perm,
                                  const int32_t* inv, const int32_t* off, const float* alpha,
                                  const void* x, const void* w_gate, const void* w_up,
                                  const void* w_down, void* x_disp, void* ab, void* phi,
                                  void* y, float* out, void* ws, size_t ws_bytes,
                                  void* stream);

/*
 * Retained-only recompute of [a | b] in the backward (RelayMoE Sec. 3.3,
 * memory-efficient MoE recomputation: the backward rebuilds the expert
 * intermediates it consumes; LRMoE Sec. 3.1: FC1 and the activation use the
 * retained identities). ab_c [M,2H] dtype (written, rows of sel_off's
 * segments) = [x_c W_gate[e] | x_c W_up[e]] from x_c [N,D] (compacted rows,
 * read) with the layer's FP32 accumulation and one rounding, the same as
 * lrm_expert_fc1_fwd over the routed rows. With it the saved state needs no
 * [a | b]: lrm_compact then takes ab = ab_c = NULL and copies none.
 */
lrm_status lrm_expert_fc1_recompute(const lrm_shape* shape, const int32_t* sel_off,
                                    const void* x_c, const void* w_gate, const void* w_up,
                                    void* ab_c, void* ws, size_t ws_bytes, void* stream);

/*
 * The expert backward with its row operands read in place instead of from
 * compacted copies. LRMoE Sec. 3.1 (compact runtime) asks that the products
 * run over the retained rows only, in a consistent pair order, with no
 * zero-masked rows; here the compaction writes only the gradient rows
 * dy_c = alpha * g (lrm_compact with x_c = ab_c = phi_c = NULL) and the
 * products gather the rest by index:
 *   FC2 dgrad + SwiGLU grad  reads [a | b] row sel_pos[j] of ab  [N,2H];
 *   FC2 wgrad                reads phi row sel_pos[j] of phi     [N,H];
 *   FC1 wgrad                reads x row tok_c[j] of x           [T,D];
 * (j = compacted row; ab and phi in dispatch order as lrm_score reads them).
 * The FC1 dgrad product and the dx scatter are those of
 * lrm_expert_bwd_grouped. The results equal the compacted form's bit for
 * bit: the same tiles and reduction order, only the operand source differs.
 * parts: an OR of LRM_BWD_* selecting the sub-steps to run, in this order.
 * Other arguments as lrm_expert_bwd_grouped. Row indices outside their
 * source are read as zero rows (FC2 / FC1 wgrad) or skipped and flagged
 * LRM_DEVERR_INDEX (FC2 dgrad).
 */
enum {
  LRM_BWD_FC2_DGRAD = 1,
  LRM_BWD_FC2_WGRAD = 2,
  LRM_BWD_FC1_WGRAD = 4,
  LRM_BWD_FC1_DGRAD = 8,
  LRM_BWD_SCATTER_DX = 16,
  LRM_BWD_ALL = 31
};
lrm_status lrm_expert_bwd_gathered(const lrm_shape* shape, int32_t parts,
                                   const int32_t* sel_off, const int32_t* sel_pos,
                                   const int32_t* tok_c, const void* w_gate,
                                   const void* w_up, const void* w_down, const void* dy_c,
                                   const void* x, const void* ab, const void* phi,
                                   const int32_t* inv, const int32_t* row_of_pos,
                                   void* dab_c, float* dx_c, float* dw_gate, float* dw_up,
                                   float* dw_down, float* dx, void* ws, size_t ws_bytes,
                                   void* stream);

/*
 * lrm_quota_from_rate and lrm_select_quota in one launch: the quotas
 * q_e = min(ceil(num/den * n_e), cap) (cap <= 0: none; exact integers, as
 * lrm_quota_from_rate) are computed from off inside the selection and also
 * written to quota [E] int32. Needs 0 <= num <= den, den > 0. Other
 * arguments, outputs and error behaviour as lrm_select_quota.
 */
lrm_status lrm_select_rate(const lrm_shape* shape, const float* score, const int32_t* off,
                           int32_t num, int32_t den, int32_t cap, int32_t* quota,
                           uint8_t* keep, int32_t* sel_off, int32_t* sel_pos, void* ws,
                           size_t ws_bytes, void* stream);

/*
 * ---------------------------------------------------------------------------
 * What a training step needs around the expert passes: the router, the
 * routing weights' gradient, the norm in front of the layer, the optimizer.
 * The descriptors below are HOST structs, read during the call only.
 * ---------------------------------------------------------------------------
 */

/*
 * Router: top-K of every token's logits, with the balance loss and the z-loss.
 * A token takes part if its mask byte is not 0 (mask NULL: all) and at least
 * one of its logits is above -inf. For those tokens, p_t = softmax(x_t) and
 * lse_t = log sum_e exp(x_te); n is their number (at least 1 in the losses):
 *   topk_idx[t] = the K largest logits, descending, equal ones by the lower
 *     expert id (NaN ranks as -inf, -0 as 0)
 *   alpha[t,k]  = p at topk_idx[t,k]; renorm != 0: divided by its sum over k
 *   counts[e]   = number of (t, k) with topk_idx[t,k] = e
 *   prob_sum[e] = sum_t p_te
 *   loss[0] = balance_coef * E / (n^2 K) * sum_e counts[e] prob_sum[e]
 *   loss[1] = z_coef / n * sum_t lse_t^2
 * Tokens that take no part get alpha = 0 and K valid, distinct ids (of their
 * logits, by the same rule); they count nowhere. In a token that takes part,
 * NaN and +inf logits make its weights and the statistics NaN. FP32 arithmetic: alpha,
 * the losses and float32 gradients keep its accuracy at any distance from the row's
 * largest logit; prob_sum is off by up to 7e-8 of an expert's share for each unit that
 * it stands below the largest (shares under 2^-126 count as 0). The statistics are
 * added in a fixed order (same inputs, same bits).
 *   logits [T,E] dtype (read), rows `stride` elements apart (stride >= E).
 *   mask [T] uint8 (read) or NULL, any alignment.
 *   topk_idx [T,K] int32, alpha [T,K] float (written).
 *   counts [E] int32, prob_sum [E] float, loss [2] float (written), or all
 *     three NULL: no statistics (the serving form; balance_coef, z_coef unused).
 * Limits: E <= 1024, K <= 32, T*K < 2^31, else LRM_ERR_UNSUPPORTED.
 * ws: lrm_router_workspace_bytes, header as everywhere (zeroed once with
 * lrm_clear_device_error).
 */
typedef struct lrm_router {
  int32_t T, E, K;
  int32_t dtype;      /* lrm_dtype of logits and dlogits */
  int64_t stride;     /* elements from one row of logits to the next */
  int32_t renorm;
  float balance_coef, z_coef;
} lrm_router;
size_t lrm_router_workspace_bytes(const lrm_router* router);
lrm_status lrm_route(const lrm_router* router, const void* logits, const uint8_t* mask,
                     int32_t* topk_idx, float* alpha, int32_t* counts, float* prob_sum,
                     float* loss, void* ws, size_t ws_bytes, void* stream);

/*
 * Gradient of the router with respect to its logits, of
 *   sum alpha dalpha + dloss[0] loss[0] + dloss[1] loss[1],
 * the choices and counts taken as constants:
 *   renorm: dx at the choices  = alpha (dalpha - sum_k alpha dalpha)
 *   else:   dx = p (dp - sum_e p dp), dp = dalpha at the choices, 0 elsewhere
 *   balance: + p (c - sum_e p c), c_e = dloss[0] balance_coef E counts[e] / (n^2 K)
 *   z:       + p dloss[1] 2 z_coef lse / n
 * Tokens that take no part get zeros, whatever their dalpha. n = sum counts / K.
 *   logits, mask as lrm_route (read); topk_idx [T,K], counts [E] from it (read).
 *   dalpha [T,K] float (read) or NULL (0); dloss [2] float (read) or NULL (1, 1).
 *   dlogits [T,E] dtype, contiguous (written).
 * Ids outside [0,E) are skipped and flag LRM_DEVERR_EXPERT_ID.
 */
lrm_status lrm_route_bwd(const lrm_router* router, const void* logits, const uint8_t* mask,
                         const int32_t* topk_idx, const int32_t* counts, const float* dalpha,
                         const float* dloss, void* dlogits, void* ws, size_t ws_bytes,
                         void* stream);

/*
 * Gradient of the routing weights through lrm_combine, for every routed pair:
 *   dalpha[t,k] = <g_t, y[inv[t*K+k]]>   (FP32 accumulation)
 *   g [T,D] dtype (cotangent at the MoE output), y [N,D] dtype (expert outputs
 *   in dispatch order, as lrm_expert_fc2_fwd leaves them), inv [N] int32 (read);
 *   dalpha [T,K] float (written).
 * inv entries outside [0,N) give 0, whatever g holds, and flag LRM_DEVERR_INDEX.
 */
lrm_status lrm_gate_grad(const lrm_shape* shape, const void* g, const void* y,
                         const int32_t* inv, float* dalpha, void* ws, size_t ws_bytes,
                         void* stream);

/*
 * Root-mean-square norm with the residual's addition and an 8-bit output.
 *   h = x + res (res NULL: h = x),  rstd = 1 / sqrt(mean_d h^2 + eps),
 *   y = h * rstd * w
 *   q = e4m3(y / scale), scale = max(amax, 2^-100) / 448 with amax the largest
 *     |y| of each q_cols columns of a row (the last group may be shorter), or
 *     of the whole row for q_cols = 0
 * FP32 arithmetic on the unrounded sum; h and y are rounded once to dtype, q is
 * taken from the unrounded y. NaN and infinities stay in their row (NaN is
 * ignored by amax and becomes the e4m3 NaN).
 *   x [T,D] dtype, rows x_stride elements apart; res [T,D] dtype or NULL, rows
 *     res_stride apart; w [D] dtype (read).
 *   h [T,D] dtype or NULL; y [T,D] dtype or NULL; q [T,D] e4m3 bytes and
 *     q_scale [T, ceil(D / q_cols)] float (one column for q_cols = 0), or both
 *     NULL; rstd [T] float or NULL (written, contiguous). y or q is required.
 * h or y may be x or res themselves (the same pointer; LRM_ERR_INVALID_ARG where
 * that input's rows are not contiguous); no other overlap is allowed.
 * Limits: D a multiple of 8 up to 16384, strides multiples of 8, q_cols one of
 * 0, 32, 64, 128, 256, else LRM_ERR_UNSUPPORTED.
 */
typedef struct lrm_norm {
  int32_t T, D;
  int32_t dtype;       /* of x, res, w, h, y */
  int32_t grad_dtype;  /* of dy, dh, dx */
  int32_t q_cols;
  float eps;
  int64_t x_stride, res_stride;
} lrm_norm;
size_t lrm_norm_workspace_bytes(const lrm_norm* norm);
lrm_status lrm_add_rmsnorm(const lrm_norm* norm, const void* x, const void* res, const void* w,
                           void* h, void* y, void* q, float* q_scale, float* rstd,
                           void* stream);

/*
 * Its gradients, with xhat = h * rstd:
 *   dx = rstd * (w dy - xhat * mean_d(w dy xhat)) + dh
 *   dw = sum_t dy * xhat
 * dx is the gradient of x and of res alike; dh is what reaches the stored sum h
 * from elsewhere (the residual stream), NULL for none.
 *   dy, dh [T,D] grad_dtype, h [T,D] dtype, w [D] dtype, rstd [T] float (read);
 *   dx [T,D] grad_dtype, dw [D] float (overwritten). All contiguous; dx may be
 *   dy or dh itself. The strides and q_cols of the descriptor are not used.
 * Rows are added in a fixed order (same inputs, same bits).
 * ws: lrm_norm_workspace_bytes.
 */
lrm_status lrm_add_rmsnorm_bwd(const lrm_norm* norm, const void* dy, const void* dh,
                               const void* h, const void* w, const float* rstd, void* dx,
                               float* dw, void* ws, size_t ws_bytes, void* stream);

/*
 * One AdamW step (decoupled weight decay) over `count` tensors:
 *   g' = grad * (*grad_scale),  m = beta1 m + (1 - beta1) g',
 *   v = beta2 v + (1 - beta2) g'^2,
 *   p = p (1 - lr weight_decay)
 *       - lr / (1 - beta1^step) * m / (sqrt(v) / sqrt(1 - beta2^step) + eps)
 * FP32 arithmetic. p is master where one is given (param then gets it rounded),
 * else param itself, updated in FP32 and rounded once.
 * LRM_STATE_F32: m, v float [n]. LRM_STATE_F8: m holds e4m3(m / scale) and v
 * holds e4m3(sqrt(v) / scale), with one scale = max(amax, 2^-100) / 448 for
 * each 256 consecutive values; a positive root is never stored as 0. Zero
 * codes and scales are a valid start. The step uses the unrounded new moments.
 * A NaN gradient makes its own value and moments NaN; an infinite one also the
 * 8-bit moments of its block.
 * Buffers are the caller's, param, grad, master, m, v 16-byte aligned, the scales
 * 4-byte, not overlapping. `step` counts from 1. It is read on the host: a captured graph
 * replays the bias correction of the step it was captured with.
 */
typedef enum lrm_state { LRM_STATE_F32 = 0, LRM_STATE_F8 = 1 } lrm_state;
typedef struct lrm_adamw_tensor {
  void* param;         /* [n] param_dtype, read and written */
  const void* grad;    /* [n] grad_dtype */
  float* master;       /* [n] float or NULL; only beside an LRM_BF16 param */
  void *m, *v;         /* [n] */
  float *m_scale, *v_scale; /* [ceil(n / 256)], LRM_STATE_F8 only */
  int64_t n;
  int32_t param_dtype, grad_dtype;
  int32_t state;       /* lrm_state */
  int32_t reserved;
  double weight_decay;
} lrm_adamw_tensor;
typedef struct lrm_adamw {
  double lr, beta1, beta2, eps;
  int64_t step;
  const float* grad_scale; /* device scalar, NULL: 1 */
} lrm_adamw;
lrm_status lrm_adamw_step(const lrm_adamw* adamw, const lrm_adamw_tensor* tensors,
                          int32_t count, void* stream);

/*
 * ---------------------------------------------------------------------------
 * Training under tight memory: a router with groups, the saved state in 8 bits,
 * the norms around a block. Descriptors are HOST structs, read during the call only.
 * ---------------------------------------------------------------------------
 */

/*
 * Router over groups of experts. The E experts stand in `groups` groups of E / groups
 * consecutive ones. A logit of -inf closes its expert to the token. A token takes part
 * if its mask byte is not 0 (mask NULL: all) and at least one of its logits is above
 * -inf (NaN is). For every token:
 *   s_te     = sigmoid(x_te) (LRM_SIGMOID) or softmax(x_t)_e (LRM_SOFTMAX)
 *   key_te   = s_te + bias_e, compared with 64 bits; without a bias: x_te
 *   a group's score = the sum of the group_top largest s + bias of its open experts
 *     (fewer open ones: of those; none: below every other group)
 *   the top_groups groups of the largest scores are kept, equal ones by the lower id
 *   topk_idx = the K largest keys of the kept groups' experts, descending, equal ones by
 *     the lower id; closed experts and NaN come last
 *   alpha    = scale * s at the choices; renorm != 0: divided by their sum before (0
 *     where that is 0). The bias is in the choices only, not in the weights.
 * and over the n tokens that take part (at least 1 in the loss), share_te = s_te / sum_e s_te:
 *   counts[e] = number of (t, k) with topk_idx[t,k] = e, prob_sum[e] = sum_t share_te
 *   loss[0]   = balance_coef * E / (n^2 K) * sum_e counts[e] prob_sum[e]
 * Tokens that take no part get alpha = 0 and K valid, distinct ids; they count nowhere.
 * In a token that takes part a NaN makes the softmax's weights NaN and, where the
 * sigmoid's choices hold it, its weight (renorm: all of the token's); both make its
 * shares NaN. Rows of the softmax that hold NaN
 * or +inf get some K valid, distinct ids of the kept groups. FP32 arithmetic; a choice
 * that 32 bits cannot tell is looked at with 64. Statistics are added in a fixed order.
 *   logits [T,E] dtype (read), rows `stride` elements apart (stride >= E).
 *   bias [E] float (read) or NULL; finite. mask [T] uint8 (read) or NULL.
 *   topk_idx [T,K] int32, alpha [T,K] float (written).
 *   counts [E] int32, prob_sum [E] float, loss [1] float (written), or all three
 *     NULL: no statistics (the serving form).
 * Limits: E <= 1024, K <= 32, groups <= 32 dividing E, 1 <= top_groups <= groups,
 * K <= top_groups * E / groups, group_top 1 or 2, T*K < 2^31, else
 * LRM_ERR_UNSUPPORTED (LRM_ERR_INVALID_ARG for sizes below 1).
 * ws: lrm_group_router_workspace_bytes, header as everywhere (zeroed once with
 * lrm_clear_device_error).
 */
typedef enum lrm_score_fn { LRM_SIGMOID = 0, LRM_SOFTMAX = 1 } lrm_score_fn;
typedef struct lrm_group_router {
  int32_t T, E, K;
  int32_t dtype;      /* lrm_dtype of logits and dlogits */
  int64_t stride;     /* elements from one row of logits to the next */
  int32_t score_fn;   /* lrm_score_fn */
  int32_t groups, top_groups, group_top;
  int32_t renorm;
  float scale, balance_coef;
} lrm_group_router;
size_t lrm_group_router_workspace_bytes(const lrm_group_router* router);
lrm_status lrm_group_route(const lrm_group_router* router, const void* logits,
                           const float* bias, const uint8_t* mask, int32_t* topk_idx,
                           float* alpha, int32_t* counts, float* prob_sum, float* loss,
                           void* ws, size_t ws_bytes, void* stream);

/*
 * Its gradient with respect to the logits, of sum alpha dalpha + dloss[0] loss[0], the
 * choices and counts taken as constants. With ds the gradient of the scores,
 *   renorm: ds at the choices = scale (dalpha - sum_k a dalpha) / sum_k s, a = s / sum_k s
 *   else:   ds at the choices = scale dalpha
 *   balance: + (c_e - sum_e share c) / sum_e s,
 *            c_e = dloss[0] balance_coef E counts[e] / (n^2 K), n = sum counts / K
 *   sigmoid: dx = ds s (1 - s);  softmax: dx = s (ds - sum_e s ds)
 * Tokens that take no part get zeros, whatever their dalpha.
 *   logits, mask as lrm_group_route (read); topk_idx [T,K], counts [E] from it (read).
 *   dalpha [T,K] float (read) or NULL (0); dloss [1] float (read) or NULL (1).
 *   dlogits [T,E] dtype, contiguous (written).
 * Ids outside [0,E) are skipped and flag LRM_DEVERR_EXPERT_ID. A token's ids have to be
 * distinct, as lrm_group_route's are.
 */
lrm_status lrm_group_route_bwd(const lrm_group_router* router, const void* logits,
                               const uint8_t* mask, const int32_t* topk_idx,
                               const int32_t* counts, const float* dalpha, const float* dloss,
                               void* dlogits, void* ws, size_t ws_bytes, void* stream);

/*
 * One step of the selection bias towards even loads, without a gradient:
 *   out[e] = bias[e] + rate * sign(sum counts - E counts[e])
 * counts [E] int32, bias [E] float (read), out [E] float (written; may be bias).
 */
typedef struct lrm_bias {
  int32_t E;
  float rate;
} lrm_bias;
lrm_status lrm_bias_step(const lrm_bias* step, const int32_t* counts, const float* bias,
                         float* out, void* stream);

/*
 * The saved state [a | b] of a forward expert pass in 8 bits (LRMoE Sec. 3.1 keeps it per
 * routed pair in the layer's type; this is a memory-saving variant): 2H + 8 ceil(H / cols)
 * + 4 bytes a pair in the place of 6H in bfloat16, phi = SiLU(a) * b being rebuilt from it.
 *   q [rows,2H] e4m3 bytes: a row's a and b, each by groups of `cols` columns (the last
 *     one may be shorter): q = e4m3(v / scale), scale = max(amax, 2^-100) / 448
 *   scale [rows, 2 ceil(H / cols)] float: the groups of a, then those of b
 *   phi_sq [rows] float: |phi|^2 of the unquantised a and b, for the pairs' scores: the
 *     selection is that of the exact state
 * NaN and infinities stay in their group (and their row's phi_sq).
 * lrm_pack_state: q, scale, phi_sq (written) from ab [rows,2H] dtype (read), in any row
 * order; lrm_score_packed and lrm_compact_packed take dispatch order.
 * Limits: H a multiple of 8, cols 32, 64 or 128, else LRM_ERR_UNSUPPORTED.
 */
typedef struct lrm_packed {
  uint8_t* q;
  float* scale;
  float* phi_sq;
  int64_t rows; /* routed pairs */
  int32_t H, cols;
  int32_t dtype; /* lrm_dtype of ab */
  int32_t reserved;
} lrm_packed;
lrm_status lrm_pack_state(const lrm_packed* packed, const void* ab, void* stream);

/*
 * lrm_score from a packed state: R_u = alpha_u^2 * ||g_t||^2 * phi_sq_u (no phi is read).
 * packed->rows, H and dtype have to be the shape's T*K, H and dtype. Other arguments as
 * lrm_score.
 */
lrm_status lrm_score_packed(const lrm_shape* shape, const lrm_packed* packed, const void* g,
                            const float* alpha, const int32_t* inv, float* score, void* ws,
                            size_t ws_bytes, void* stream);

/*
 * lrm_compact from a packed state: for retained row j < M, i = sel_pos[j], p = perm[i],
 * t = p / K, with (a, b) = q * scale of row i in float32,
 *   dy_c[j] = alpha[p] * g[t],  ab_c[j] = [a | b],  phi_c[j] = SiLU(a) * b,
 *   x_c[j] = x[t],  tok_c[j] = t,  row_of_pos[i] = j (-1 where keep[i] == 0),
 * each rounded once to dtype. The rows serve lrm_expert_bwd_grouped, or
 * lrm_expert_bwd_compacted with x read in place (then x_c NULL: no copy).
 *   x [T,D] dtype where x_scale is NULL; else e4m3 bytes [T,D] with x_scale
 *     [T, ceil(D / x_cols)] float, x_cols one of 0 (a scale a row), 32, 64, 128, 256: what
 *     lrm_add_rmsnorm and lrm_block_norm write (read where x_c is given).
 * Other arguments, the 64 zero rows after dy_c's and the checks of indices as lrm_compact.
 */
lrm_status lrm_compact_packed(const lrm_shape* shape, const lrm_packed* packed,
                              const int32_t* perm, const uint8_t* keep, const int32_t* sel_off,
                              const int32_t* sel_pos, const float* alpha, const void* x,
                              const float* x_scale, int32_t x_cols, const void* g, void* dy_c,
                              void* x_c, void* ab_c, void* phi_c, int32_t* tok_c,
                              int32_t* row_of_pos, void* ws, size_t ws_bytes, void* stream);

/*
 * lrm_expert_bwd_grouped over compacted dy_c, ab_c and phi_c, with the rows of x [T,D]
 * read in place by tok_c in the FC1 weight gradient, as lrm_expert_bwd_gathered does.
 */
lrm_status lrm_expert_bwd_compacted(const lrm_shape* shape, const int32_t* sel_off,
                                    const int32_t* tok_c, const void* w_gate, const void* w_up,
                                    const void* w_down, const void* dy_c, const void* x,
                                    const void* ab_c, const void* phi_c, const int32_t* inv,
                                    const int32_t* row_of_pos, void* dab_c, float* dx_c,
                                    float* dw_gate, float* dw_up, float* dw_down, float* dx,
                                    void* ws, size_t ws_bytes, void* stream);

/*
 * The norm behind a block, its gate, the scaled residual and the norm in front of the next:
 *   u = block * block_rstd * w_post, block_rstd = 1 / sqrt(mean_d block^2 + eps)
 *       (w_post NULL: u = block)
 *   h = residual_scale * res + gate * u
 *   y = h * rstd * w, rstd = 1 / sqrt(mean_d h^2 + eps); q, q_scale as lrm_add_rmsnorm
 * gate: LRM_GATE_NONE (1), LRM_GATE_COLUMN (gate [D]) or LRM_GATE_TOKEN (gate [T]).
 * FP32 arithmetic on unrounded values; h and y are rounded once to dtype.
 *   block [T,D] block_dtype, rows block_stride apart: LRM_F32 (what lrm_combine writes)
 *     or dtype; res [T,D] dtype, rows res_stride apart; w, w_post, gate dtype (read).
 *   h [T,D] dtype, y [T,D] dtype or NULL, q and q_scale or both NULL, rstd [T] float or
 *     NULL, block_rstd [T] float or NULL (written, contiguous). y or q is required.
 * h may be res itself where that is contiguous; no other overlap is allowed.
 * Limits: D a multiple of 8 up to 8192, strides multiples of 8, q_cols one of 0, 32, 64,
 * 128, 256, else LRM_ERR_UNSUPPORTED.
 */
typedef enum lrm_gate { LRM_GATE_NONE = 0, LRM_GATE_COLUMN = 1, LRM_GATE_TOKEN = 2 } lrm_gate;
typedef struct lrm_block {
  int32_t T, D;
  int32_t dtype;       /* of res, w, w_post, gate, h, y, dblock */
  int32_t block_dtype; /* of block */
  int32_t grad_dtype;  /* of dy, dh, dres */
  int32_t gate;        /* lrm_gate */
  int32_t q_cols;
  float eps, residual_scale;
  int64_t block_stride, res_stride;
} lrm_block;
size_t lrm_block_workspace_bytes(const lrm_block* block);
lrm_status lrm_block_norm(const lrm_block* desc, const void* block, const void* res,
                          const void* w, const void* w_post, const void* gate, void* h, void* y,
                          void* q, float* q_scale, float* rstd, float* block_rstd,
                          void* stream);

/*
 * Its gradients, with xhat = h * rstd, ohat = block * block_rstd:
 *   dhs    = rstd * (w dy - xhat * mean_d(w dy xhat)) + dh
 *   dres   = residual_scale * dhs,  dw = sum_t dy * xhat
 *   du     = gate * dhs,  dgate = sum dhs * u (over t for a gate of columns, over d for
 *            one of tokens),  dw_post = sum_t du * ohat
 *   dblock = block_rstd * (w_post du - ohat * mean_d(w_post du ohat)); w_post NULL: du
 *   dy, dh [T,D] grad_dtype (dh NULL: none), h [T,D] dtype, block [T,D] block_dtype, w,
 *     w_post, gate as in the forward call, rstd, block_rstd [T] float (read).
 *   dres [T,D] grad_dtype, dblock [T,D] dtype, dw [D], dw_post [D] (with w_post), dgate [D]
 *     or [T] (with a gate) float (overwritten). All contiguous; dres may be dy or dh
 *     itself, no other overlap. Strides and q_cols are not used.
 * Rows are added in a fixed order (same inputs, same bits). ws: lrm_block_workspace_bytes.
 */
lrm_status lrm_block_norm_bwd(const lrm_block* desc, const void* dy, const void* dh,
                              const void* h, const void* block, const void* w,
                              const void* w_post, const void* gate, const float* rstd,
                              const float* block_rstd, void* dres, void* dblock, float* dw,
                              float* dw_post, float* dgate, void* ws, size_t ws_bytes,
                              void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LRM_H_ */
