/*
 * gdr.h -- C ABI of the chunked gated delta-rule forward pass on GB300 (sm_103a).
 *
 * The operation.  For every (sequence, head) unit, with per-token inputs
 * q_t, k_t in R^dk, v_t in R^dv, a gate logit a_t and a write strength
 * beta_t, the library computes
 *
 *     g_t   = -b * sigmoid(a_t)        (bounded gate, GDR_GATE_BOUNDED)
 *           = -softplus(a_t)           (unbounded gate, GDR_GATE_SOFTPLUS)
 *     H_t   = exp(g_t) H_{t-1} + beta_t k_t (v_t - exp(g_t) H_{t-1}^T k_t)^T
 *     o_t   = H_t^T q_t
 *
 * with H the dk x dv fp32 state (H = S^T for the dv x dk delta-rule state
 * S_t = alpha_t S_{t-1}(I - beta_t k_t k_t^T) + beta_t v_t k_t^T, o_t = S_t q_t,
 * alpha_t = exp(g_t)),
 * starting from h0 and ending in hT.  The bounded gate is the scaled-sigmoid
 * log-decay the pages introduce in place of the unbounded negative softplus
 * ("Deep Dive: The Next Generation of Ultra-Long Context Sparse MoE LLMs",
 * §3.3; "Core Technologies Behind Ultra-Long-Context Sparse MoE Large
 * Models", §2.2; "How Trillion-Scale Sparse MoE Models Achieve Million-Token
 * Long Context Capabilities", §3.2; "Evaluating Next-Gen Sparse MoE and
 * Long-Context LLMs", §2.3); the pages fix b = 5 there, b is a parameter
 * here.  The state update is the delta-rule write with data-dependent decay
 * of the incremental linear-attention layer ("Evaluating Next-Gen Sparse MoE
 * and Long-Context LLMs", §2.2).  It is computed chunk-parallel: the
 * sequence is cut into tiles of `chunk` tokens, each tile is a set of dense
 * products, and the state is passed from tile to tile ("Deep Dive ...",
 * §3.2; "Core Technologies ...", §2.1).  The result does not depend on
 * `chunk` beyond rounding.
 *
 * Layouts (row-major, contiguous, element type = dtype unless stated):
 *   dense  (cu_seqlens == NULL): q,k [B,T,H,dk]  v,out [B,T,H,dv]  a,beta [B,T,H]
 *   varlen (cu_seqlens != NULL): the same tensors with a leading 1 instead of B
 *          and T = total tokens; cu_seqlens holds N+1 int32 offsets (device
 *          memory), cu[0] = 0, non-decreasing, cu[N] = T; B is then N.
 *          Tiles restart at every sequence start; a partial last tile is masked.
 *   h0, hT : [N,H,dk,dv] fp32 (N = B for dense input).  h0 == NULL means zero.
 *          hT may be NULL (not written) and may alias h0 (in-place carry).
 *   beta is a probability (used as given, not passed through a sigmoid).
 *   q and k are used as given: no scaling, no normalisation.
 *
 * Segments of the tensor-core path.  A long sequence is cut into segments
 * whose state transitions are computed in parallel and chained.  A transition
 * skips what enters its segment so early that it reaches the segment's end
 * attenuated below 2^-64 of the state: the bound multiplies, per token, the
 * decay exp(g_t) by the erase factor's norm max(1, |1 - beta_t |k_t|^2|), so
 * it holds for any keys and write strengths (with unit keys and beta in
 * [0, 1] the erase factors are 1 and the decay alone sets it).  Where no such
 * point lies inside a segment the full transition is used.  The environment
 * variable GDR_TC_EXACT=1 turns the skipping off.
 *
 * Ownership and concurrency.  All tensor pointers of gdr_chunk_fwd* and of
 * the stage calls are DEVICE pointers owned by the caller; the library
 * retains none of them.  Calls are asynchronous on `stream` (NULL = the
 * legacy default stream).  Scratch memory comes from `workspace` if given,
 * else from a cache the library keeps per device (grown with cudaMalloc,
 * freed by gdr_release).  Calls that share the internal cache must not
 * overlap on the GPU: issue them on one stream, or pass each stream its own
 * workspace.  Nor may several host threads issue them at once, since the first
 * call that needs more scratch than any before it replaces the cache's buffer;
 * a call captured into a graph, which keeps its pointers, is given a workspace.
 *
 * Errors.  Arguments are checked before anything is launched: unsupported
 * sizes return GDR_ERR_UNSUPPORTED, malformed ones GDR_ERR_INVALID_ARG.  A
 * failed CUDA call returns GDR_ERR_CUDA.  Conditions only the device can see
 * (cu_seqlens that are not a valid offset list, a bounded wait that gave
 * up) set a per-device status word; gdr_get_status() reads and clears it.
 */
#ifndef GDR_H_
#define GDR_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define GDR_API __attribute__((visibility("default")))
#else
#define GDR_API
#endif

struct CUstream_st;
typedef struct CUstream_st *gdr_stream_t; /* the same type as cudaStream_t */

typedef enum {
    GDR_OK = 0,
    GDR_ERR_INVALID_ARG = 1,  /* null required pointer, negative size, ...     */
    GDR_ERR_UNSUPPORTED = 2,  /* valid but not implemented (e.g. dk = 96)       */
    GDR_ERR_CUDA = 3,         /* a CUDA runtime call failed                      */
    GDR_ERR_TIMEOUT = 4,      /* a bounded device-side wait ran out              */
    GDR_ERR_NO_WORKSPACE = 5, /* caller workspace smaller than required          */
    GDR_ERR_BAD_SEQLENS = 6,  /* cu_seqlens is not 0 = c0 <= c1 <= ... <= cN = T */
    GDR_ERR_BOUNDS = 7        /* checking build (GDR_DEBUG) only: a device-side index
                                 check failed and its access was skipped           */
} gdr_status_t;

typedef enum { GDR_BF16 = 0, GDR_F32 = 1 } gdr_dtype_t;

typedef enum {
    GDR_GATE_BOUNDED = 0, /* g = -b * sigmoid(a), g in [-b, 0]   */
    GDR_GATE_SOFTPLUS = 1 /* g = -softplus(a),    g in (-inf, 0) */
} gdr_gate_t;

typedef enum {
    GDR_PATH_AUTO = 0, /* tensor-core path where supported and q, k, v are 16-byte
                          aligned (TMA tiles), else SIMT                            */
    GDR_PATH_SIMT = 1, /* fp32 CUDA-core path (any supported shape and dtype)     */
    GDR_PATH_TC = 2    /* tcgen05 path; GDR_ERR_UNSUPPORTED where it does not apply
                          (shape, dtype, or q, k, v not 16-byte aligned)            */
} gdr_path_t;

/*
 * The forward pass with the defaults: dtype bf16, bounded gate with bound b,
 * automatic path, internal workspace.
 *   q,k,v,a,beta : inputs, layouts above (bf16)
 *   h0           : initial state or NULL (zero)
 *   out          : output, bf16, layout above; must not alias an input
 *   hT           : final state or NULL
 *   cu_seqlens   : NULL (dense) or N+1 int32 device offsets (varlen)
 *   B, T, H      : batch (or N), tokens per sequence (or total), heads
 *   dk, dv       : key / value width, each 64 or 128
 *   chunk        : tile length, 16, 32 or 64.  The CUDA-core path tiles by
 *                  chunk; the tensor-core path (bf16, dk = dv = 128) tiles by
 *                  16 tokens for every chunk, since the result does not depend
 *                  on the tile length beyond rounding (its in-tile decays are
 *                  pairwise, bounded for any tile length and gate)
 *   b            : gate bound, > 0 and finite
 * Supported sizes: B, H >= 1, T >= 0 (T = 0 copies h0 to hT, or zeroes hT).
 */
GDR_API gdr_status_t gdr_chunk_fwd(const void *q, const void *k, const void *v, const void *a,
                           const void *beta, const float *h0, void *out, float *hT,
                           const int32_t *cu_seqlens, int B, int64_t T, int H, int dk,
                           int dv, int chunk, float b, gdr_stream_t stream);

/*
 * The forward pass with every option.
 *   dtype       : element type of q, k, v, a, beta and out
 *   gate        : gate form; b is ignored for GDR_GATE_SOFTPLUS
 *   path        : kernel family (see gdr_path_t)
 *   workspace   : device scratch of workspace_bytes >= gdr_chunk_fwd_workspace_size(...),
 *                 or NULL for the internal per-device cache
 */
GDR_API gdr_status_t gdr_chunk_fwd_ex(const void *q, const void *k, const void *v, const void *a,
                              const void *beta, const float *h0, void *out, float *hT,
                              const int32_t *cu_seqlens, int B, int64_t T, int H, int dk,
                              int dv, int chunk, float b, gdr_dtype_t dtype, gdr_gate_t gate,
                              gdr_path_t path, void *workspace, size_t workspace_bytes,
                              gdr_stream_t stream);

/* Scratch bytes gdr_chunk_fwd_ex needs for these sizes (0 on invalid sizes).
 * B is N (the sequence count) for varlen input.  For GDR_PATH_AUTO it covers
 * both paths, since the pointers' alignment decides between them. */
GDR_API size_t gdr_chunk_fwd_workspace_size(int B, int64_t T, int H, int dk, int dv, int chunk,
                                    gdr_dtype_t dtype, gdr_path_t path);

/*
 * The forward pass on HOST buffers: inputs are copied to the device, the
 * pass runs, out (and hT) are copied back, and the call returns after the
 * copies have finished (it synchronises `stream`).  Same arguments and
 * layouts as gdr_chunk_fwd_ex except that every tensor pointer, including
 * cu_seqlens, is host memory (pinned memory gives full copy bandwidth).
 * Device buffers come from the internal per-device cache.
 * From 2^21 (token, head) units up, the call is pipelined: the tokens are cut
 * into up to 8 pieces (dense input: tile-aligned token ranges of every
 * sequence, the state carried from piece to piece; packed input: groups of
 * whole sequences, when cu_seqlens is well formed) and a piece's copies in
 * and out overlap the neighbouring pieces' passes, on two internal copy
 * streams.  The result then differs from gdr_chunk_fwd_ex's only by the
 * rounding of the different segment split.
 */
GDR_API gdr_status_t gdr_chunk_fwd_host(const void *q, const void *k, const void *v, const void *a,
                                const void *beta, const float *h0, void *out, float *hT,
                                const int32_t *cu_seqlens, int B, int64_t T, int H, int dk,
                                int dv, int chunk, float b, gdr_dtype_t dtype, gdr_gate_t gate,
                                gdr_path_t path, gdr_stream_t stream);

/*
 * The forward pass without any device allocation by the library.  The pages
 * have no counterpart to this call; it exists for callers that must not
 * allocate device memory when they run the pass (during CUDA graph capture,
 * inside engines that pre-reserve all device memory, in allocation-free
 * latency loops).  It runs the fp32 CUDA-core path on DENSE input only (no
 * cu_seqlens) and keeps its scratch in one statically allocated 32 MiB device
 * array that every GPU loading the library holds until exit.
 *   Arguments, layouts and ownership are those of gdr_chunk_fwd_ex.
 *   Limit: sizes whose scratch (4 * B*T*H * (1 + dk + dv) bytes plus
 *   24 * (B+1) bytes, each part rounded up to 256) exceeds 32 MiB return
 *   GDR_ERR_NO_WORKSPACE before anything is launched -- about 32K
 *   (token, head) pairs at dk = dv = 128.
 *   The first call on a device looks up the array's device address once
 *   (cudaGetSymbolAddress); make that first call before any stream capture.
 *   Every call reuses the same array, so calls that overlap on the GPU (on
 *   different streams, or from several threads) race and must be
 *   serialised by the caller.  Nothing in the array needs clearing between
 *   calls: each call writes every scratch element before reading it.
 */
GDR_API gdr_status_t gdr_chunk_fwd_noalloc(const void *q, const void *k, const void *v,
                                           const void *a, const void *beta, const float *h0,
                                           void *out, float *hT, int B, int64_t T, int H, int dk,
                                           int dv, int chunk, float b, gdr_dtype_t dtype,
                                           gdr_gate_t gate, gdr_stream_t stream);

/*
 * Stage 1 alone: the gate and its in-tile cumulative sum.
 *   G[h, r] = sum over tokens r' of r's tile with r' <= r of g(a[r', h]),
 * written head-major as G [H, B*T] fp32 (token rows packed as in a).
 * Tiles restart at every sequence start ("Deep Dive ...", §3.2-3.3).
 */
GDR_API gdr_status_t gdr_gate_cumsum(const void *a, float *G, const int32_t *cu_seqlens, int B,
                             int64_t T, int H, int chunk, float b, gdr_dtype_t dtype,
                             gdr_gate_t gate, gdr_stream_t stream);

/*
 * Stage 2 alone: the per-tile WY / UT representation.  With G from
 * gdr_gate_cumsum (layout above), per tile of length C
 *   A_ij = beta_i exp(G_i - G_j) (k_i . k_j) for j < i,  T = (I + A)^{-1},
 *   W = T diag(beta exp(G)) K  [C x dk],  U = T diag(beta) V  [C x dv],
 * written fp32 in the layouts of k and v: W [B,T,H,dk], U [B,T,H,dv].
 */
GDR_API gdr_status_t gdr_wy_repr(const void *k, const void *v, const void *beta, const float *G,
                         float *W, float *U, const int32_t *cu_seqlens, int B, int64_t T,
                         int H, int dk, int dv, int chunk, gdr_dtype_t dtype,
                         gdr_stream_t stream);

/*
 * The recurrent (token-by-token) form, for decoding: advances each sequence's
 * state over T tokens and writes their outputs; T = 1 is one decode step of
 * an inference engine that keeps a constant-size state per sequence instead
 * of a cache that grows with the context ("Evaluating Next-Gen Sparse MoE and
 * Long-Context LLMs", §2.2: the state is updated token by token; §4, §5:
 * chunked prefill and constant-state layers on the inference side).  A prompt
 * is prefilled with gdr_chunk_fwd_ex (its hT is the state), then decoded here.
 *
 *   q, k   [N, T, H, dk]   v, out [N, T, H, dv]   a, beta [N, T, H]   (dtype)
 *   state  [N, H, dk, dv]  fp32, read as the entering state and overwritten
 *          with the state after the last token (same layout as h0 / hT)
 * Per token: alpha = exp(g(a)), H <- alpha H + beta k (v - alpha H^T k)^T,
 * o = H^T q (the same recurrence as gdr_chunk_fwd_ex, computed without tiles).
 * Device pointers owned by the caller; nothing is retained or allocated.
 * dk, dv in {64, 128}; N, H >= 1; T >= 0 (T = 0 leaves state untouched).
 * out must not alias any input or state; state must be 16-byte aligned (it
 * is read and written as float4).  Returns GDR_ERR_INVALID_ARG or
 * GDR_ERR_UNSUPPORTED before any launch, GDR_ERR_CUDA on a launch failure;
 * the call is asynchronous on `stream`.
 */
GDR_API gdr_status_t gdr_recurrent_fwd(const void *q, const void *k, const void *v, const void *a,
                               const void *beta, float *state, void *out, int N, int64_t T,
                               int H, int dk, int dv, float b, gdr_dtype_t dtype,
                               gdr_gate_t gate, gdr_stream_t stream);

/*
 * Per-channel (vector) decay: the forward pass of gdr_chunk_fwd_ex with one
 * gate input per key channel.  Token t decays row i of the dk x dv state by
 * exp(g(a[t, h, i])) before the delta-rule write:
 *     H_t = (I - beta k k^T) diag(exp(g(a_t))) H_{t-1} + beta k v^T,  o_t = H_t^T q_t,
 * g(a) = -b sigmoid(a) (the bounded gate).  Inside each 16-token tile the
 * pairwise decays exp(G_i - G_j) are split into the factors exp(G_i) and
 * exp(-G_j), which turns every in-tile product into a plain matrix product;
 * the bound keeps exp(-G) finite ("Deep Dive: The Next Generation of
 * Ultra-Long Context Sparse MoE LLMs", §2.1-2.2; "How Trillion-Scale Sparse
 * MoE Models Achieve Million-Token Long Context Capabilities", §3.2).
 *   a    [B, T, H, dk] in dtype (varlen: [1, T, H, dk]); every other argument as
 *        for gdr_chunk_fwd_ex.
 * chunk must be 16 and 0 < b <= 5 (exp(16 b) must stay below FLT_MAX):
 * GDR_ERR_UNSUPPORTED otherwise; b <= 0 is GDR_ERR_INVALID_ARG.  Only the
 * bounded gate is taken (an unbounded one can overflow exp(-G)).  bf16 with
 * dk = dv = 128 runs a fused tensor-core kernel when q, k, v, a and `out` are
 * 16-byte aligned; other shapes, fp32 and unaligned pointers run the CUDA-core
 * kernels (same results within the stated tolerances).  Scratch
 * comes from the internal per-device cache; asynchronous on `stream`.
 */
GDR_API gdr_status_t gdr_chunk_fwd_vec(const void *q, const void *k, const void *v, const void *a,
                               const void *beta, const float *h0, void *out, float *hT,
                               const int32_t *cu_seqlens, int B, int64_t T, int H, int dk, int dv,
                               int chunk, float b, gdr_dtype_t dtype, gdr_stream_t stream);

/*
 * Backward of the per-channel decay form (gdr_chunk_fwd_vec): gradients of
 * <dout, out> + <dhT, hT> with respect to q, k, v, a, beta and h0, as for
 * gdr_chunk_bwd, except that a and da are [tokens, H, dk] (one gate input and one
 * gradient per key channel).  It runs the chunked tensor-core form only: bf16,
 * dk = dv = 128, chunk 16, 0 < b <= 5 (GDR_ERR_UNSUPPORTED otherwise); the
 * bounded gate is implied.  Errors, ownership and streams as for gdr_chunk_bwd.
 */
GDR_API gdr_status_t gdr_chunk_bwd_vec(const void *q, const void *k, const void *v, const void *a,
                               const void *beta, const float *h0, const void *dout,
                               const float *dhT, void *dq, void *dk_out, void *dv_out, void *da,
                               void *dbeta, float *dh0, const int32_t *cu_seqlens, int B,
                               int64_t T, int H, int dk, int dv, int chunk, float b,
                               gdr_dtype_t dtype, gdr_stream_t stream);

/* Bias-update rule of the quantile-balancing router (see gdr_router_bias_update). */
typedef enum { GDR_QB_SIGN = 0, GDR_QB_PROPORTIONAL = 1 } gdr_qb_mode_t;

/*
 * Routing step of aux-loss-free quantile balancing ("Deep Dive: The Next
 * Generation of Ultra-Long Context Sparse MoE LLMs", §4.2; "Core Technologies
 * Behind Ultra-Long-Context Sparse MoE Large Models", §3.2): every token t
 * picks the k experts of largest score logits[t, e] + bias[e], the sum taken
 * in binary32; equal scores go to the lower expert index.  The bias only
 * steers the selection: topk_logit returns the unbiased logits.
 *   logits     [T, E] in dtype (bf16 or fp32), 16-byte aligned (device)
 *   bias       [E] fp32 (device)
 *   topk_idx   [T, k] int32, experts in descending score order (device, written)
 *   topk_logit [T, k] fp32 logits of the picked experts, or NULL
 *   load       [E] int64: this call's per-expert counts are ADDED (a window may
 *              span several calls; zero it at the window start), or NULL
 * 1 <= E <= 2048 with E % 4 == 0 and 1 <= k <= min(E, 32): GDR_ERR_UNSUPPORTED
 * otherwise.  NaN logits or biases give an unspecified (but in-bounds)
 * selection.  Outputs must not overlap inputs: GDR_ERR_INVALID_ARG.
 * Asynchronous on `stream`; the counts are exact (integer atomics).
 */
GDR_API gdr_status_t gdr_router_topk(const void *logits, const float *bias, int32_t *topk_idx,
                             float *topk_logit, int64_t *load, int64_t T, int E, int k,
                             gdr_dtype_t dtype, gdr_stream_t stream);

/*
 * Bias step of quantile balancing (the four pages print it in two forms;
 * "Core Technologies ...", §3.2, "How Trillion-Scale Sparse MoE Models Achieve
 * Million-Token Long Context Capabilities", §4.3, "Evaluating Next-Gen Sparse
 * MoE and Long-Context LLMs", §3.2).  Q(q) is the q-quantile of the E loads by
 * linear interpolation between order statistics (sorted x, p = q (E - 1),
 * i = floor p: Q = x_i + (p - i)(x_{i+1} - x_i)), in binary64.
 *   GDR_QB_SIGN:         bias[e] -= eta if load[e] > Q(q_hi), else
 *                        bias[e] += eta if load[e] < Q(q_lo)   (binary32 steps;
 *                        q_lo = q_hi is the single-threshold form)
 *   GDR_QB_PROPORTIONAL: bias[e] += eta (Q(q_hi) - load[e]) / Q(q_hi) in
 *                        binary64, rounded to binary32; no change if Q(q_hi) = 0
 *   load [E] int64 (device), bias [E] fp32 (device, updated in place),
 *   thresholds [2] fp64 = {Q(q_lo), Q(q_hi)} (device, written) or NULL.
 * 1 <= E <= 2048 (GDR_ERR_UNSUPPORTED otherwise); q_lo, q_hi in [0, 1] and eta
 * finite (GDR_ERR_INVALID_ARG otherwise).  Asynchronous on `stream`.
 */
GDR_API gdr_status_t gdr_router_bias_update(const int64_t *load, float *bias, double *thresholds,
                                    int E, gdr_qb_mode_t mode, double q_lo, double q_hi,
                                    float eta, gdr_stream_t stream);

/*
 * The backward pass: gradients of  L = <dout, out> + <dhT, hT>  with respect to
 * q, k, v, a, beta and h0, for the forward of gdr_chunk_fwd_ex on the same
 * inputs (same layouts, dtype, gate, b and cu_seqlens; B is N for varlen).
 * The pages train the layer in bf16 mixed precision ("Core Technologies ...",
 * §2.3; "Deep Dive ...", §3.3) but print no backward; the adjoints here are
 * those of the recurrence H_t = alpha H_{t-1} + beta k (v - alpha H^T k)^T,
 * o = H_t^T q, written out per token:
 *   dout [tokens, H, dv] (dtype) or NULL (zero);  dhT [N, H, dk, dv] fp32 or NULL
 *   dq, dk [tokens, H, dk], dv [tokens, H, dv], da, dbeta [tokens, H]  (dtype, all
 *   written);  dh0 [N, H, dk, dv] fp32 (written when not NULL)
 * `chunk` is validated like the forward's; the pass works on 16-token tiles
 * either way.  bf16 with dk = dv = 128 and the bounded gate with b <= 5 runs
 * the chunked tensor-core form: the states at tile boundaries are stored in
 * bf16, and each tile's gradients come from dense products.  Every other case
 * runs token by token, from fp32 checkpoints every 16 tokens with the tokens
 * between them recomputed.  Device pointers owned
 * by the caller; scratch comes from the internal per-device cache.  Outputs
 * must not alias inputs; dhT and dh0 must be 16-byte aligned (copied as
 * float4), GDR_ERR_INVALID_ARG otherwise.  The result is deterministic (no
 * atomics).  Errors as for gdr_chunk_fwd_ex; asynchronous on `stream`.  The
 * chunked form runs its two state chains (forward and adjoint, independent of
 * each other) concurrently: the adjoint chain on a second stream the library
 * keeps per device (freed by gdr_release), forked from and joined back to
 * `stream` with events, so the call is ordered on `stream` as a whole.  Both
 * chains run on the tcgen05 tensor cores with the state in tensor memory when
 * q, k, v, dout (and a per-channel a) are 16-byte aligned, and on warp-level
 * tensor-core kernels otherwise; their waits are bounded like the forward's
 * (GDR_ERR_TIMEOUT in the status word).
 */
GDR_API gdr_status_t gdr_chunk_bwd(const void *q, const void *k, const void *v, const void *a,
                           const void *beta, const float *h0, const void *dout,
                           const float *dhT, void *dq, void *dk_out, void *dv_out, void *da,
                           void *dbeta, float *dh0, const int32_t *cu_seqlens, int B,
                           int64_t T, int H, int dk, int dv, int chunk, float b,
                           gdr_dtype_t dtype, gdr_gate_t gate, gdr_stream_t stream);

/*
 * Linear attention with one constant decay per head, for prompts: per (sequence, head)
 *     S_t = exp(log_decay[h]) S_{t-1} + k_t v_t^T,    o_t = scale * S_t^T q_t
 * with the dk x dv fp32 state S, from h0 to hT -- the incremental linear-attention layer
 * ("Evaluating Next-Gen Sparse MoE and Long-Context LLMs", §2.2) without the delta rule's
 * erase step and with a decay that does not depend on the data.  It is computed in
 * chunks ("Deep Dive ...", §3.2): inside a tile of 128 tokens the pairwise decays
 * exp((i - j) log_decay) weigh a dense causal product, and the state passes from tile to
 * tile.
 *   q, k       [B, T, H, dk]   v, out [B, T, H, dv]   (dtype; packed input as for
 *              gdr_chunk_fwd: a leading 1, cu_seqlens with B + 1 offsets, T in all)
 *   log_decay  [H] fp32 (device), natural logarithms, meant to be <= 0; -inf keeps
 *              nothing of earlier tokens; above 0 the state grows, which nothing limits
 *   h0, hT     [N, H, dk, dv] fp32, 16-byte aligned, or NULL (zero / not written); hT
 *              may be h0 (carried in place)
 *   scale      finite; multiplies the outputs only, not the state
 *   path       GDR_PATH_AUTO: the tcgen05 kernel for bf16 tensors that are 16-byte
 *              aligned, else (and for sequences of at most 8 tokens; packed: 8 in all) the
 *              fp32 CUDA-core kernel; GDR_PATH_TC refuses (GDR_ERR_UNSUPPORTED) what the
 *              former cannot take
 *   workspace  16-byte aligned device scratch of gdr_decay_workspace_size(...) bytes, or
 *              NULL: the internal per-device cache (calls that share it must not
 *              overlap on the GPU)
 * dk, dv in {64, 128}; B, H >= 1; T >= 0; sequences of no tokens pass h0 on to hT.
 * Magnitudes.  On the CUDA cores products scale k v below 2^104 and outputs above 2^-104
 * keep clear of fp32's limits.  On the tensor cores |scale q.k| and |out / scale| have to stay
 * below 2^62 (in gdr_decay_bwd |scale v.dout| and the gradients too), and an output takes 2^-64
 * of the entering state's part where the decay leaves less of it than that.
 * States are accumulated in fp32; on the tensor cores the writes enter them with 24
 * significant bits, while the in-tile weights and the state are rounded to bf16 where
 * they are multiplied for a (bf16) output.  A NaN or infinity in a token stays in the state,
 * however fast the head forgets: it reaches the outputs after it and hT (on the tensor
 * cores as a NaN, and also the outputs of its own 128-token tile; a call whose cut
 * sequence has one that the decay leaves nothing of runs that sequence's head twice);
 * other heads and sequences never.  Outputs must not overlap inputs.  Bad offsets:
 * GDR_ERR_BAD_SEQLENS in the status word, nothing is written.  Asynchronous on `stream`;
 * deterministic.
 */
GDR_API gdr_status_t gdr_decay_fwd(const void *q, const void *k, const void *v, const float *log_decay,
                           const float *h0, void *out, float *hT, const int32_t *cu_seqlens, int B,
                           int64_t T, int H, int dk, int dv, float scale, gdr_dtype_t dtype,
                           gdr_path_t path, void *workspace, size_t workspace_bytes,
                           gdr_stream_t stream);

/*
 * The gradients of <dout, out> + <dhT, hT> of gdr_decay_fwd with respect to q, k, v and
 * h0 (log_decay is a constant of the layer and gets none).  With dS_t the gradient of S_t,
 *     dS_t = exp(log_decay) dS_{t+1} + scale q_t dout_t^T   (dS_T holds dhT too)
 *     dq_t = scale S_t dout_t,  dk_t = dS_t v_t,  dv_t = dS_t^T k_t,
 *     dh0 = exp(log_decay) dS_1
 *   dout [.., H, dv] (dtype);  dhT [N, H, dk, dv] fp32 or NULL (zero)
 *   dq, dk [.., H, dk], dv [.., H, dv] (dtype);  dh0 [N, H, dk, dv] fp32 or NULL
 * The states are recomputed, nothing is kept from the forward pass.  dhT and dh0 must be
 * 16-byte aligned; everything else as for gdr_decay_fwd.
 */
GDR_API gdr_status_t gdr_decay_bwd(const void *q, const void *k, const void *v, const float *log_decay,
                           const float *h0, const void *dout, const float *dhT, void *dq,
                           void *dk_out, void *dv_out, float *dh0, const int32_t *cu_seqlens, int B,
                           int64_t T, int H, int dk, int dv, float scale, gdr_dtype_t dtype,
                           gdr_path_t path, void *workspace, size_t workspace_bytes,
                           gdr_stream_t stream);

/* Scratch bytes of gdr_decay_fwd (backward = 0) or gdr_decay_bwd (backward = 1) for these
 * sizes; B is the number of sequences and T the total of tokens where packed = 1.  0 on
 * invalid sizes, and where no scratch is needed. */
GDR_API size_t gdr_decay_workspace_size(int B, int64_t T, int H, int dk, int dv, int packed,
                                int backward, gdr_dtype_t dtype, gdr_path_t path);

/*
 * The same recurrence token by token, for decoding: advances each sequence's state over T
 * tokens (T = 1: one step) in place.  q, k [N, T, H, dk], v, out [N, T, H, dv] (dtype),
 * log_decay [H] fp32, state [N, H, dk, dv] fp32, 16-byte aligned, updated in place.
 * Nothing is allocated.  T = 0 leaves the state untouched.  Errors as for
 * gdr_recurrent_fwd; asynchronous on `stream`.
 */
GDR_API gdr_status_t gdr_decay_recurrent_fwd(const void *q, const void *k, const void *v,
                                     const float *log_decay, float *state, void *out, int N,
                                     int64_t T, int H, int dk, int dv, float scale,
                                     gdr_dtype_t dtype, gdr_stream_t stream);

/*
 * Layer norm over the last axis: row r of x (D elements) becomes
 *     y = (x - mean) * rstd * weight[r % G] + bias[r % G],
 *     mean = sum(x) / D,   rstd = 1 / sqrt(sum((x - mean)^2) / D + eps)
 * G = 1 is one weight for all rows; G = H norms every head of a [.., H, D] tensor with its
 * own weight, as the outputs of an attention without a normaliser need.
 *   x, y         [rows, D] in dtype (y may be x)
 *   weight, bias [G, D] fp32, or NULL (1 / 0)
 *   mean, rstd   [rows] fp32, or NULL: what the backward pass reads
 * rows >= 0 and a multiple of G; 1 <= D <= 16384 (GDR_ERR_UNSUPPORTED above); eps >= 0 and
 * finite.  fp32 inside; any alignment of elements.  Asynchronous on `stream`.
 */
GDR_API gdr_status_t gdr_layer_norm_fwd(const void *x, const float *weight, const float *bias, void *y,
                                float *mean, float *rstd, int64_t rows, int G, int D, float eps,
                                gdr_dtype_t dtype, gdr_stream_t stream);

/*
 * Its backward pass, from the forward's mean and rstd; xh = (x - mean) rstd:
 *     dx = rstd (w dy - mean_D(w dy) - xh mean_D(w dy xh))
 *     dweight[g] = sum over rows r with r % G = g of dy xh,  dbias[g] = sum of dy
 *   dy, x, dx [rows, D] in dtype (dx may be dy or x); weight [G, D] fp32 or NULL (1)
 *   dweight, dbias [G, D] fp32, or NULL (not wanted)
 * The sums over rows are fp32 in a fixed order (no atomics).  Scratch comes from the
 * internal per-device cache: calls that share it must not overlap on the GPU.  Sizes and
 * errors as above; asynchronous on `stream`.
 */
GDR_API gdr_status_t gdr_layer_norm_bwd(const void *dy, const void *x, const float *mean,
                                const float *rstd, const float *weight, void *dx, float *dweight,
                                float *dbias, int64_t rows, int G, int D, gdr_dtype_t dtype,
                                gdr_stream_t stream);

/*
 * The same with the caller's scratch: 16-byte aligned device memory of
 * gdr_layer_norm_bwd_workspace_size(...) bytes (GDR_ERR_NO_WORKSPACE if it is less), or NULL
 * for the cache.  A call on a stream of its own, beside other calls that need scratch, is
 * given one.
 */
GDR_API gdr_status_t gdr_layer_norm_bwd_ex(const void *dy, const void *x, const float *mean,
                                const float *rstd, const float *weight, void *dx, float *dweight,
                                float *dbias, int64_t rows, int G, int D, gdr_dtype_t dtype,
                                void *workspace, size_t workspace_bytes, gdr_stream_t stream);

/* Scratch bytes of gdr_layer_norm_bwd for these sizes (none where neither dweight nor dbias
 * is wanted); 0 on invalid sizes. */
GDR_API size_t gdr_layer_norm_bwd_workspace_size(int64_t rows, int G, int D, gdr_dtype_t dtype);

/* What weighs the inputs of the gated scan. */
typedef enum {
    GDR_SOURCE_PLAIN = 0,   /* 1                                                     */
    GDR_SOURCE_CONVEX = 1,  /* 1 - alpha: the state is a weighted mean of its inputs */
    GDR_SOURCE_VARIANCE = 2 /* sqrt(1 - alpha^2): unit inputs leave a unit state     */
} gdr_source_t;

/*
 * Gated scan, one decay per token and channel: the recurrence of a layer whose state is a
 * vector, with the library's gates.  Per (sequence, channel)
 *     alpha_t = exp(g(a_t)),   h_t = alpha_t h_{t-1} + w(alpha_t) x_t
 * from h0 to hT; every h_t is an output.  The bounded gate is that of the incremental
 * linear-attention layer ("Deep Dive: The Next Generation of Ultra-Long Context Sparse MoE
 * LLMs", §3.3), whose decay here acts on a diagonal state.
 *   x, a, out  [B, T, D] in dtype (packed: [1, T, D], cu_seqlens with B + 1 offsets, T in all)
 *   h0, hT     [N, D] fp32, or NULL (zero / not written); hT may be h0 (carried in place)
 *   states     [total / 128, D] fp32, or NULL: row i is the state behind token 128 i + 127 of
 *              the token axis (all B T tokens one after the other), which the backward pass
 *              starts from.  total / 128 is rounded down.
 *   b          bound of the bounded gate, > 0 and finite, one for all channels and without a
 *              gradient (not looked at for softplus)
 * 1 <= D <= 2^22; B >= 1; T >= 0; at most 2^31 - 4097 tokens in all and 2^40 elements; sequences of no
 * tokens pass h0 on to hT.  Element alignment is enough (16-byte pointers with D a multiple of
 * 16 bytes are read fastest).  fp32 inside.  A NaN or an infinity stays in its channel's state
 * to the end of the sequence (an infinity may become a NaN); other channels and sequences
 * never see it.  The decays of a stretch of tokens are multiplied in fp32 before they meet the state, so
 * that what is left of a state (backward: of a gradient) behind it may be off by 2^-150 of that state,
 * besides the roundings in proportion.  Outputs must not overlap inputs.  Bad offsets: GDR_ERR_BAD_SEQLENS in the
 * status word, nothing is written; waits are bounded (GDR_ERR_TIMEOUT).  No scratch; asynchronous
 * on `stream`; deterministic.
 */
GDR_API gdr_status_t gdr_gated_scan_fwd(const void *x, const void *a, const float *h0, void *out, float *hT,
                                float *states, const int32_t *cu_seqlens, int B, int64_t T, int D, float b,
                                gdr_dtype_t dtype, gdr_gate_t gate, gdr_source_t source,
                                gdr_stream_t stream);

/*
 * The gradients of <dout, out> + <dhT, hT> of gdr_gated_scan_fwd with respect to x, a and h0.
 * With l_t the gradient of h_t,
 *     l_t = dout_t + alpha_{t+1} l_{t+1} (the last token's holds dhT too)
 *     dx_t = w l_t,  da_t = l_t (alpha_t h_{t-1} + w'(g_t) x_t) g'(a_t),  dh0 = alpha_1 l_1
 *   dout, dx, da [.., D] (dtype);  dhT [N, D] fp32 or NULL (zero);  dh0 [N, D] fp32 or NULL
 *   states       as the forward pass wrote them for the same inputs, or NULL: they are computed
 *                again, into the workspace
 *   workspace    device scratch of gdr_gated_scan_bwd_workspace_size(...) bytes, 16-byte
 *                aligned, or NULL: the internal per-device cache (calls that share it must not
 *                overlap on the GPU).  Not looked at where states are given.
 * Everything else as for gdr_gated_scan_fwd.
 */
GDR_API gdr_status_t gdr_gated_scan_bwd(const void *x, const void *a, const float *h0, const float *states,
                                const void *dout, const float *dhT, void *dx, void *da, float *dh0,
                                const int32_t *cu_seqlens, int B, int64_t T, int D, float b,
                                gdr_dtype_t dtype, gdr_gate_t gate, gdr_source_t source, void *workspace,
                                size_t workspace_bytes, gdr_stream_t stream);

/* Scratch bytes of gdr_gated_scan_bwd without states; B sequences of T tokens, packed = 1: T
 * tokens in all.  0 on invalid sizes, and where no scratch is needed. */
GDR_API size_t gdr_gated_scan_bwd_workspace_size(int B, int64_t T, int D, int packed);

/*
 * The same recurrence token by token, for decoding: advances each sequence's state over T
 * tokens (T = 1: one step) in place.  x, a, out [N, T, D] (dtype), state [N, D] fp32.  Nothing
 * is allocated.  T = 0 leaves the state untouched.  Asynchronous on `stream`.
 */
GDR_API gdr_status_t gdr_gated_scan_recurrent_fwd(const void *x, const void *a, float *state, void *out, int N,
                                          int64_t T, int D, float b, gdr_dtype_t dtype, gdr_gate_t gate,
                                          gdr_source_t source, gdr_stream_t stream);

/* The norm of gdr_add_norm_* and gdr_norm_gate_*: with the mean taken off, or without. */
typedef enum { GDR_NORM_LAYER = 0, GDR_NORM_RMS = 1 } gdr_norm_kind_t;
/* The activation of gdr_norm_gate_*: z sigmoid(z), or sigmoid(z). */
typedef enum { GDR_ACT_SILU = 0, GDR_ACT_SIGMOID = 1 } gdr_act_t;

/*
 * The norm in front of a block, with the residual stream's sum: row r becomes
 *     sum = residual + scale x,   y = N(sum) = (sum - mean) rstd weight[r % G] + bias[r % G]
 *     mean = sum over the row / D (GDR_NORM_LAYER) or 0 (GDR_NORM_RMS),
 *     rstd = 1 / sqrt(sum((sum - mean)^2) / D + eps)
 * The norm is that of the sum as it is stored, rounded to dtype.
 *   x, residual, sum, y  [rows, D] in dtype (sum may be residual, and y may be x)
 *   weight, bias         [G, D] fp32, or NULL (1 / 0); G as for gdr_layer_norm_fwd
 *   mean, rstd           [rows] fp32, or NULL: what the backward pass reads; mean must be NULL
 *                        for GDR_NORM_RMS
 * rows >= 0 and a multiple of G; 1 <= D <= 16384 (GDR_ERR_UNSUPPORTED above); eps >= 0 and
 * scale finite.  fp32 inside; any alignment of elements.  Asynchronous on `stream`.
 */
GDR_API gdr_status_t gdr_add_norm_fwd(const void *x, const void *residual, const float *weight, const float *bias,
                              void *sum, void *y, float *mean, float *rstd, int64_t rows, int G, int D,
                              float scale, float eps, gdr_norm_kind_t kind, gdr_dtype_t dtype,
                              gdr_stream_t stream);

/*
 * Its backward pass, from the forward's sum and statistics; xh = (sum - mean) rstd, n = weight dy:
 *     dresidual = dsum + rstd (n - mean_D(n) - xh mean_D(n xh))   (mean_D(n): GDR_NORM_LAYER alone)
 *     dx = scale dresidual
 *     dweight[g] = sum over rows r with r % G = g of dy xh,  dbias[g] = sum of dy
 *   dy, dsum, sum, dx, dresidual [rows, D] in dtype; dsum (the gradient along the residual
 *   stream) NULL: zero; dx NULL: not wanted; dx and dresidual may each be one of the inputs
 *   dweight, dbias [G, D] fp32, or NULL (not wanted); mean NULL exactly for GDR_NORM_RMS
 *   workspace as for gdr_layer_norm_bwd_ex, of gdr_block_norm_bwd_workspace_size(...) bytes
 * The sums over rows are fp32 in a fixed order (no atomics).  Asynchronous on `stream`.
 */
GDR_API gdr_status_t gdr_add_norm_bwd(const void *dy, const void *dsum, const void *sum, const float *mean,
                              const float *rstd, const float *weight, void *dx, void *dresidual,
                              float *dweight, float *dbias, int64_t rows, int G, int D, float scale,
                              gdr_norm_kind_t kind, gdr_dtype_t dtype, void *workspace,
                              size_t workspace_bytes, gdr_stream_t stream);

/*
 * The norm behind a block, with its gate and the residual stream:
 *     y = [residual +] scale N(x) act(gate),   N as above with x for sum
 *   x, gate, residual, y [rows, D] in dtype; residual NULL: none; y may be one of the inputs
 * Everything else as for gdr_add_norm_fwd.
 */
GDR_API gdr_status_t gdr_norm_gate_fwd(const void *x, const void *gate, const float *weight, const float *bias,
                               const void *residual, void *y, float *mean, float *rstd, int64_t rows,
                               int G, int D, float scale, float eps, gdr_norm_kind_t kind, gdr_act_t act,
                               gdr_dtype_t dtype, gdr_stream_t stream);

/*
 * Its backward pass (the residual's gradient is dy itself); xh = (x - mean) rstd,
 * d = scale dy act(gate), n = weight d:
 *     dx = rstd (n - mean_D(n) - xh mean_D(n xh))   (mean_D(n): GDR_NORM_LAYER alone)
 *     dgate = scale dy (xh weight + bias) act'(gate)
 *     dweight[g] = sum over rows r with r % G = g of d xh,  dbias[g] = sum of d
 *   dy, x, gate, dx, dgate [rows, D] in dtype; dx and dgate may each be one of the inputs
 * Everything else as for gdr_add_norm_bwd.
 */
GDR_API gdr_status_t gdr_norm_gate_bwd(const void *dy, const void *x, const void *gate, const float *mean,
                               const float *rstd, const float *weight, const float *bias, void *dx,
                               void *dgate, float *dweight, float *dbias, int64_t rows, int G, int D,
                               float scale, gdr_norm_kind_t kind, gdr_act_t act, gdr_dtype_t dtype,
                               void *workspace, size_t workspace_bytes, gdr_stream_t stream);

/* Scratch bytes of gdr_add_norm_bwd and gdr_norm_gate_bwd for these sizes (none where neither
 * dweight nor dbias is wanted); 0 on invalid sizes. */
GDR_API size_t gdr_block_norm_bwd_workspace_size(int64_t rows, int G, int D, gdr_dtype_t dtype);

/* Synchronise `stream`, then read and clear the current device's status word.
 * Returns GDR_OK, GDR_ERR_BAD_SEQLENS, GDR_ERR_TIMEOUT or GDR_ERR_CUDA. */
GDR_API gdr_status_t gdr_get_status(gdr_stream_t stream);

/* Static description of a status code (never NULL). */
GDR_API const char *gdr_status_string(gdr_status_t status);

/* Free the internal per-device caches of every device (synchronises them). */
GDR_API void gdr_release(void);

/* Number of kernels this library has launched so far in this process. */
GDR_API uint64_t gdr_launch_count(void);

/*
 * Per-kernel timing.  While enabled, every kernel the library launches is
 * bracketed by a pair of CUDA events recorded on its launch stream.
 * gdr_profile_read synchronises those events, writes for up to `max`
 * distinct kernels its name (a static string), the summed device time in
 * milliseconds and the launch count, returns the number of distinct kernels
 * seen (which may exceed `max`), and clears the record.  Enabling adds two
 * event records per launch and nothing else.
 */
GDR_API void gdr_profile_enable(int on);
GDR_API int gdr_profile_read(const char **names, double *total_ms, int *launches, int max);
/* Restrict the timing to the launches of one kernel, named as gdr_profile_read
 * reports it (NULL or "": every kernel, the default), so that a measurement of
 * that kernel puts no events between the other launches.  The name is copied. */
GDR_API void gdr_profile_select(const char *name);

#ifdef __cplusplus
}
#endif
#endif /* GDR_H_ */
