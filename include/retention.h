/*
 * retention.h - C ABI of the MI355X (gfx950) multi-scale retention library, libretention.so.
 *
 * Retention is the sequence mixer of RetNet: for each (batch b, head h) with a fixed decay gamma_h,
 *     S_n = gamma S_{n-1} + k_n^T v_n,   o_n = q_n S_n            (state S: d_k x d_v, S before token 0 given)
 * with q and k first rotated by their absolute position (xPos/rotary form). Sources: "Hybrid Architectures:
 * RetNet and the Three Computation Paradigms" (sections 2, 4, 6 and 7) and the RetNet paper summary
 * (Eq. 5 parallel, Eq. 6 recurrent, Eq. 7 chunkwise; the paper's ParallelRetention / RecurrentRetention /
 * ChunkwiseRetention interfaces, whose precomputed decay tensors are replaced here by gamma itself).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * Layouts (row-major, contiguous, device memory):
 *     q, k  [B, N, H, d_k]      v, o  [B, N, H, d_v]      state [B, H, d_k, d_v] (fp32, d_v fastest)
 *     decode step: q, k [B, H, d_k], v, o [B, H, d_v]
 * dtypes: q/k/v in `in_dt`, o in `out_dt`; supported pairs are (F32, F32), (BF16, BF16) and (BF16, F32).
 *     Products accumulate in fp32 and the state is always fp32. On the BF16 path the rotated q and k, the
 *     masked scores and the copy of the state used for q.S are rounded to bf16 (nearest-even) as MFMA
 *     operands; the carried state is never rounded.
 * gamma: HOST float[H], 0 < gamma <= 1 (per-head decay; multi-scale schedule 1 - 2^(-5-h) in the pages).
 * theta: HOST double[d_k/2] rotation frequencies, or NULL for no rotation. Pair (2i, 2i+1) of q and of k at
 *     absolute position p is turned by the angle +p*theta_i, so q'.k' depends on positions only through
 *     n - m (the conjugate-transpose reading of the paper summary's rotation; blog section 6.8).
 * pos0 / pos: absolute position of the first token (0 for a fresh sequence).
 * stream: a hipStream_t (NULL = the null stream). Every call only enqueues work and never synchronises.
 * Ownership: the caller owns every buffer. The library allocates no device memory; gamma/theta are read
 *     during the call and copied into kernel arguments.
 * Alignment: device pointers must be 16-byte aligned.
 * Errors: a non-zero status is returned before anything is enqueued, and ret_last_error() gives a detail
 *     string for the calling thread. RET_ERR_INVALID_ARG: null pointer, non-positive size, gamma outside
 *     (0, 1] or NaN, odd d_k with theta, misalignment, o aliasing an input, bad dtype pair.
 *     RET_ERR_UNSUPPORTED: a shape outside the kernels' tiling (listed per call). RET_ERR_HIP: a launch failed
 *     (device faults surface at the caller's next synchronisation). There is no fallback path.
 * NaN/Inf in inputs propagate into outputs; nothing traps.
 */
#ifndef RETENTION_H
#define RETENTION_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define RET_ABI_VERSION 8

typedef enum { RET_F32 = 0, RET_BF16 = 1 } ret_dtype_t;

typedef enum {
    RET_OK = 0,
    RET_ERR_INVALID_ARG = -1,
    RET_ERR_UNSUPPORTED = -2,
    RET_ERR_WORKSPACE = -3,
    RET_ERR_HIP = -4
} ret_status_t;

/* ABI version of the loaded library (RET_ABI_VERSION at build time). */
int ret_abi_version(void);

/* Digest of the sources the library was built from (for detecting a stale build). */
const char* ret_source_digest(void);

/* Static text for a status code. */
const char* ret_status_string(int status);

/* Detail for the last non-OK status returned on the calling thread ("" if none). */
const char* ret_last_error(void);

/*
 * Parallel form: O = (Q K^T (.) D) V, D[n][m] = gamma^(n-m) for n >= m and 0 otherwise, per (b, h), over the
 * whole sequence (blog sections 4.2-4.3; paper summary Eq. 5). No state in or out. Cost O(N^2 d).
 * Supported: F32 input: d_k in {16, 32, 64}, d_v a multiple of 16. BF16 input: d_k in {32, 64, 128, 256},
 * d_v a multiple of 64. N >= 1 (any length).
 */
ret_status_t ret_parallel_fwd(const void* q, const void* k, const void* v, void* o, int B, int N, int H, int dk,
                              int dv, ret_dtype_t in_dt, ret_dtype_t out_dt, const float* gamma,
                              const double* theta, int64_t pos0, void* stream);

/*
 * Workspace (device bytes) that ret_chunkwise_fwd can use, for the given shape and input dtype:
 *  - segment states: each sequence is split into segments that run in parallel, and the state entering a
 *    segment is built from the end states of the segments before it (a scan of the chunk state over
 *    segments; BF16 input: counters, flags and two d_k x 64 fp32 slots per segment and d_v tile of 64);
 *  - BF16 input with rotation and d_v >= 256: bf16 copies of q and k rotated once (2 * B*N*H*d_k*2 bytes),
 *    so the d_v tiles of a head do not each rotate the same rows. They start past the chain's first 64 KB
 *    (header, counters, flags), which are reserved even when the plan has a single segment.
 * 0 means the call runs one segment per (b, h) and needs none. A smaller workspace is allowed: the call then
 * first drops the rotated copies, then uses fewer segments; the results are the same up to rounding order.
 * The workspace must be zero-filled before its first use. Every call leaves it in a state the next call
 * accepts: the header (first 256 bytes) zero except a sticky error word, counters and flags zero (they occupy
 * the first 64 KB, ahead of every shape's state slots, while units x segments stays below about 16,000; beyond
 * that, zero-fill the workspace again before a call of another shape). Calls sharing a workspace must not
 * overlap in time (on one stream they do not). The library never frees it.
 */
size_t ret_chunkwise_workspace_bytes(int B, int N, int H, int dk, int dv, int chunk, ret_dtype_t in_dt);

/*
 * Synchronises `stream` and reports whether any call that used this workspace had to abandon a wait for
 * the state of an earlier segment (a sticky flag in the workspace). A wait gives up after about 0.17 s without
 * any progress of the segments it waits for (a flag rising resets the limit); the segment that gave up then
 * takes NaN for its entering state, so its outputs, and whatever is computed from its state (the final state,
 * later segments' entering states where its state enters them), come out NaN rather than silently wrong. RET_OK if no wait gave up (or workspace is NULL), RET_ERR_HIP with detail
 * otherwise.
 */
ret_status_t ret_chunkwise_check(const void* workspace, void* stream);

/*
 * Chunkwise recurrent form with chunk size `chunk` (blog section 7.2; paper summary Eq. 7). For chunk i of
 * length L (the last chunk may be shorter):
 *     O_[i] = (Q_[i] K_[i]^T (.) D) V_[i] + (Q_[i] R_{i-1}) (.) xi,   xi_j = gamma^(j+1)
 *     R_i   = gamma^L R_{i-1} + K_[i]^T (V_[i] (.) zeta),             zeta_j = gamma^(L-1-j)
 * with R_{-1} = state_in (NULL = zeros). state_out (may be NULL, may equal state_in) receives the state after
 * the last token, so a sequence can resume with pos0 = N and state_in = state_out, or hand over to
 * ret_recurrent_step. Results equal the recurrent and parallel forms up to rounding.
 * workspace: device memory of `workspace_bytes` (see ret_chunkwise_workspace_bytes), or NULL with 0.
 * Supported: F32 input: d_k in {16, 32, 64}, d_v a multiple of 16, chunk in {16, 32, 64}. BF16 input:
 * d_k in {32, 64, 128, 256}, d_v a multiple of 64, chunk in {32, 64, 128, 256, 512}. N >= 1. BF16 chunks
 * longer than 64 tokens are computed as runs of 64-token chunks, which the chunkwise form allows (any chunk
 * size gives the same result up to rounding). Kernels that read a chunk address it with 32-bit offsets:
 * chunk * H * max(d_k, d_v) * 4 must stay below 2^31 (RET_ERR_UNSUPPORTED otherwise).
 */
ret_status_t ret_chunkwise_fwd(const void* q, const void* k, const void* v, void* o, int B, int N, int H, int dk,
                               int dv, ret_dtype_t in_dt, ret_dtype_t out_dt, const float* gamma,
                               const double* theta, int64_t pos0, int chunk, const float* state_in,
                               float* state_out, void* workspace, size_t workspace_bytes, void* stream);

/*
 * One recurrent (decode) step at absolute position `pos` (blog section 2.1; paper summary Eq. 6):
 *     S <- gamma S + k'^T v,   o = q' S      (update, then read; the token sees itself)
 * `state` [B, H, d_k, d_v] fp32 is updated in place. q, k [B, H, d_k], v, o [B, H, d_v].
 * Supported: d_k in {16, 32, 64, 128, 256}, d_v a multiple of 4 and <= 512.
 */
ret_status_t ret_recurrent_step(const void* q, const void* k, const void* v, void* o, float* state, int B, int H,
                                int dk, int dv, ret_dtype_t in_dt, ret_dtype_t out_dt, const float* gamma,
                                const double* theta, int64_t pos, void* stream);

/*
 * The decode step of ret_recurrent_step with one position per sequence: sequence b is at absolute position
 * pos[b] (a batch of sequences at different lengths; the pages decode one token per step at its own position,
 * paper summary Eq. 6 and "Overall RetNet Architecture and Training/Inference Protocol"). pos: device int64[B],
 * 8-byte aligned, read by the kernel when it runs (a captured graph can advance it on the device); unused
 * without theta. The rotation factors are evaluated on the device (fp64 angle reduced by pi/2, fp32 sine and
 * cosine; angle error about pos * 2^-52 rad) rather than on the host, so results may differ from
 * ret_recurrent_step in the last bits. Otherwise as ret_recurrent_step.
 */
ret_status_t ret_recurrent_step_positions(const void* q, const void* k, const void* v, void* o, float* state, int B,
                                          int H, int dk, int dv, ret_dtype_t in_dt, ret_dtype_t out_dt,
                                          const float* gamma, const double* theta, const int64_t* pos,
                                          void* stream);

/*
 * Multi-scale retention epilogue ("Hybrid Architectures: RetNet and the Three Computation Paradigms",
 * sections 8.4 and 9.1; paper summary, "Gating mechanism"):
 *     y = swish(gate) (.) GroupNorm_h(o),   swish(x) = x * sigmoid(x)
 * o, gate, y: [rows, H, d_v] device arrays, row-major (rows = B*N tokens of a chunkwise or parallel call, or B
 * for one decode step). GroupNorm has one group per head: each (row, head) vector of d_v values is
 * standardized by its own mean and biased variance, (x - mean) / sqrt(var + eps), then multiplied by
 * gn_weight[h * d_v + c] and shifted by gn_bias[h * d_v + c] (device float[H * d_v] each; NULL means 1 and 0).
 * gate: the gate projection X W_G, or NULL for no gate; the projections themselves are the caller's.
 * o_dt, gate_dt, y_dt: F32 or BF16 each. y may equal o or gate (in place); other overlaps are not allowed.
 * Every pointer 16-byte aligned. rows = 0 does nothing. Supported: d_v in {16, 32, 64, 128, 256, 512} and
 * rows * H < 2^31.
 * eps >= 0 and finite (RET_ERR_INVALID_ARG otherwise). Asynchronous on `stream`.
 */
ret_status_t ret_msr_epilogue(const void* o, const void* gate, const float* gn_weight, const float* gn_bias,
                              void* y, int64_t rows, int H, int dv, ret_dtype_t o_dt, ret_dtype_t gate_dt,
                              ret_dtype_t y_dt, float eps, void* stream);

/*
 * Chunkwise retention followed by the multi-scale retention epilogue, into y [B, N, H, d_v]:
 *     y = swish(gate) (.) GroupNorm_h(O),   O = ret_chunkwise_fwd's output, rounded to out_dt
 * Arguments as ret_chunkwise_fwd (with y in the place of o) and ret_msr_epilogue (gate [B, N, H, d_v] or
 * NULL, gate_dt, gn_weight, gn_bias, eps). Where the kernel holds whole head rows (bf16 input and output,
 * d_v = 64, the on-chip kernel: segments of at most 256 tokens) the epilogue is applied before the outputs are
 * stored, which saves writing and reading O; otherwise ret_msr_epilogue runs over y in place. Either way the
 * result equals the two calls in sequence up to rounding. gate must not alias q, k, v or y. Every check of
 * either call is made before anything is launched, except those of the chunkwise plan itself.
 */
ret_status_t ret_chunkwise_msr_fwd(const void* q, const void* k, const void* v, const void* gate, void* y, int B,
                                   int N, int H, int dk, int dv, ret_dtype_t in_dt, ret_dtype_t out_dt,
                                   ret_dtype_t gate_dt, const float* gamma, const double* theta, int64_t pos0,
                                   int chunk, const float* state_in, float* state_out, const float* gn_weight,
                                   const float* gn_bias, float eps, void* workspace, size_t workspace_bytes,
                                   void* stream);

/*
 * Gradients of chunkwise retention, for training with the chunkwise form (paper summary, "Overall RetNet
 * Architecture and Training/Inference Protocol"). With O the output of ret_chunkwise_fwd from a zero state
 * (state_in NULL) and dout = dL/dO [B, N, H, d_v], writes dq, dk [B, N, H, d_k] and dv [B, N, H, d_v]; the
 * gradients with respect to q and k are taken through their rotation. They follow from the parallel form
 * ("Hybrid Architectures: RetNet and the Three Computation Paradigms", section 4.3; paper summary Eq. 5):
 *     dq'_n = sum_{m<=n} gamma^(n-m) (dO_n . v_m) k'_m,    dk'_m = sum_{n>=m} gamma^(n-m) (dO_n . v_m) q'_n,
 *     dv_m  = sum_{n>=m} gamma^(n-m) (q'_n . k'_m) dO_n,   dq, dk = dq', dk' turned back by the rotation's
 *     transpose,
 * each a retention (the last two over the reversed sequence) that the chunkwise kernels compute.
 * in_dt: BF16 or F32 (q, k, v, dout); out_dt: F32 or BF16 (dq, dk, dv; F32 for F32 input). No gradient for a
 * state in or out.
 * workspace: device memory of ret_chunkwise_bwd_workspace_bytes for the input dtype (zero-filled once by the
 * caller, like the chunkwise workspace; every call leaves its chain part zeroed again; ret_chunkwise_check
 * accepts it and reports a segment-chain wait that gave up). dq, dk, dv must not alias the inputs or each
 * other. Errors: RET_ERR_INVALID_ARG (as ret_chunkwise_fwd, a null or aliased gradient), RET_ERR_UNSUPPORTED
 * (shape), RET_ERR_WORKSPACE (missing or smaller than the query). Supported wherever the forward supports
 * (d_k, d_v) and (w, d_k) for the input dtype, with w = d_v or, when d_v is too wide for a retention's d_k,
 * w = d_v / 2 (dq' and dk' are then sums of two retentions over the halves of d_v): BF16 d_k in {64, 128, 256}
 * and d_v in {64, 128, 256, 512} (the paper's d_k = 256, d_v = 512 included), every BF16 chunk size; F32 d_k in
 * {16, 32, 64}, d_v in {16, 32, 64, 128}, chunk in {16, 32, 64}. The workspace query returns 0 for other
 * shapes. Asynchronous on `stream`.
 */
size_t ret_chunkwise_bwd_workspace_bytes(int B, int N, int H, int dk, int dv, int chunk, ret_dtype_t in_dt);
ret_status_t ret_chunkwise_bwd(const void* q, const void* k, const void* v, const void* dout, void* dq, void* dk_out,
                               void* dv_out, int B, int N, int H, int dk, int dv, ret_dtype_t in_dt,
                               ret_dtype_t out_dt, const float* gamma, const double* theta, int64_t pos0, int chunk,
                               void* workspace, size_t workspace_bytes, void* stream);

/*
 * Kernel launch records for measurement tools: a caller-owned object, passed in ret_options_t.timer. While a
 * call holds one, every kernel it launches is bracketed by a pair of HIP events on the launch stream and
 * recorded in it (the library keeps no timing state of its own). ret_timer_query synchronises those events and
 * returns the total milliseconds and launch count recorded for kernels whose name equals `kernel` ("" or NULL =
 * all). Kernel names: "ret_chunk_seg", "ret_chunk_fused", "ret_chunk_fused_local", "ret_chunk_fused_scan",
 * "ret_chunk_wide", "ret_chunk_dma_local", "ret_chunk_dma_scan", "ret_chunk_dma" and "ret_rotate_qk" (bf16 input),
 * "ret_chunk_full", "ret_chunk_local", "ret_segment_scan" (fp32 input), "ret_parallel", "ret_recurrent_step",
 * "ret_msr_epilogue", "ret_permute_rotate" (gradients), "ret_norm_zseg", "ret_norm_rows", "ret_norm_scale",
 * "ret_norm_step" (score normalizations); the entry points after them name theirs. A timer must not be attached to calls that are being captured into a
 * graph. One timer may be shared by calls on several threads.
 */
typedef struct ret_timer ret_timer_t;
ret_timer_t* ret_timer_create(void);   /* NULL if out of host memory */
void ret_timer_destroy(ret_timer_t* t);
int ret_timer_query(ret_timer_t* t, const char* kernel, double* total_ms, int64_t* launches);
void ret_timer_reset(ret_timer_t* t);

/*
 * Options of the *_ex entry points: the plan the library would otherwise choose, for measurements and for
 * tests that compare kernels and plans (every choice gives the result of the default plan up to rounding
 * order), and an optional timer. NULL options, or ret_options_default(), mean the library's own plan.
 *   segments     > 0: segments per sequence of the chained chunkwise kernels (capped at one per chunk); 0: planner
 *   target_wgs   > 0: workgroups the segment planner aims for; 0: the kernel's default
 *   prerotate    -1: planner; 0: q and k rotated while staging; 1: rotated once up front into the workspace
 *   onchip       -1 or 1: the on-chip segment kernel where segments fit (d_k <= 64, <= 256 tokens); 0: never
 *   variant      0: default kernel of the shape; d_v a multiple of 128: 3 = the wide-head kernel (32-token steps,
 *                q and k rotated once up front; the default for d_k = 256 where d_v is not a multiple of 256);
 *                d_k = 256: 5 = the LDS-loading wide-head kernels (d_v a multiple of 256, the default there:
 *                local passes, a scan, the full pass; gives way to 4 when q and k need rotating and the workspace
 *                has no room for rotated copies), 1 = 256 threads whose waves own 32 columns, 2 = 256 threads
 *                with d_v tiles of 64, 4 = 512 threads x 16 columns; d_k = 128: 4 = 512 threads x 16 columns
 *                (d_v tiles of 128, the default where d_v is a multiple of 128), 1 = 256 threads whose waves
 *                own 32 columns, 2 = 256 threads with d_v tiles of 64
 *   step_cw, step_wr, step_pairs   decode tile: columns per workgroup (16, 32, 64), rows per wave (16, 32, 64),
 *                pairs (0 planner, 1 one (b, h) per workgroup, 2 grouped); 0 = default
 *   bwd_direct   -1 or 1: gradients by the reversed traversal, with d_v blocks of dO and V read in place, where
 *                the kernels have them; 0: through reordered copies
 *   step_cache   0: the decode step streams the state (non-temporal loads and stores, one (b, h) per
 *                workgroup): right when each step's state has left the caches by the next step, as with a state
 *                per layer of a model; 1: the state's accesses may stay cached (grouped workgroups), faster when
 *                the same state is stepped again while it still fits the 256 MB Infinity Cache
 *   chain_spin   segment-chain wait limit in device clock ticks (100 MHz) without progress before a wait gives
 *                up; 0 = default (2^24 ticks, ~0.17 s); negative: every wait gives up at once (for testing the
 *                give-up path: the affected outputs become NaN and ret_chunkwise_check reports it)
 *   timer        launch records, or NULL
 */
typedef struct {
    int segments;
    int target_wgs;
    int prerotate;
    int onchip;
    int variant;
    int step_cw, step_wr, step_pairs;
    int bwd_direct;
    int step_cache;
    long long chain_spin;
    ret_timer_t* timer;
} ret_options_t;
void ret_options_default(ret_options_t* o);

/* ret_chunkwise_workspace_bytes, ret_chunkwise_bwd_workspace_bytes, ret_chunkwise_fwd, ret_chunkwise_msr_fwd,
 * ret_chunkwise_bwd, ret_recurrent_step and ret_recurrent_step_positions with options (NULL = defaults);
 * otherwise identical. A call planned with options wants the workspace its _ex query returns for them. */
size_t ret_chunkwise_workspace_bytes_ex(int B, int N, int H, int dk, int dv, int chunk, ret_dtype_t in_dt,
                                        const ret_options_t* opts);
size_t ret_chunkwise_bwd_workspace_bytes_ex(int B, int N, int H, int dk, int dv, int chunk, ret_dtype_t in_dt,
                                            const ret_options_t* opts);
ret_status_t ret_chunkwise_fwd_ex(const void* q, const void* k, const void* v, void* o, int B, int N, int H, int dk,
                                  int dv, ret_dtype_t in_dt, ret_dtype_t out_dt, const float* gamma,
                                  const double* theta, int64_t pos0, int chunk, const float* state_in,
                                  float* state_out, void* workspace, size_t workspace_bytes, void* stream,
                                  const ret_options_t* opts);
ret_status_t ret_chunkwise_msr_fwd_ex(const void* q, const void* k, const void* v, const void* gate, void* y, int B,
                                      int N, int H, int dk, int dv, ret_dtype_t in_dt, ret_dtype_t out_dt,
                                      ret_dtype_t gate_dt, const float* gamma, const double* theta, int64_t pos0,
                                      int chunk, const float* state_in, float* state_out, const float* gn_weight,
                                      const float* gn_bias, float eps, void* workspace, size_t workspace_bytes,
                                      void* stream, const ret_options_t* opts);
ret_status_t ret_chunkwise_bwd_ex(const void* q, const void* k, const void* v, const void* dout, void* dq,
                                  void* dk_out, void* dv_out, int B, int N, int H, int dk, int dv, ret_dtype_t in_dt,
                                  ret_dtype_t out_dt, const float* gamma, const double* theta, int64_t pos0,
                                  int chunk, void* workspace, size_t workspace_bytes, void* stream,
                                  const ret_options_t* opts);
/*
 * ret_chunkwise_bwd after the forward, for a training step: fwd_workspace (fwd_workspace_bytes) is the workspace of
 * a ret_chunkwise_fwd call on the same q, k, v, gamma, theta, pos0 and chunk with no state_in (and the same
 * options), passed unchanged since that call. Where that call ran the LDS-loading d_k = 256 kernels (d_v a
 * multiple of 256, several segments, N a multiple of 32) it left there the rotated copies of q and k and the
 * state entering each segment, which the gradients need too: they are read instead of recomputed (the dq'
 * retentions enter their segments with those states, transposed); where it ran the streaming kernel's split
 * launches (d_k = d_v = 128, several segments) it left the states, read the same way. Otherwise, or with
 * fwd_workspace NULL, the call is ret_chunkwise_bwd_ex. Same results as ret_chunkwise_bwd_ex (bit for bit on the
 * LDS-loading kernels, whose forward ran the same products; to rounding on the streaming kernel, whose forward
 * formed the states in another order); a forward workspace from another call gives wrong gradients, which the
 * library cannot detect. fwd_workspace is only read.
 */
ret_status_t ret_chunkwise_bwd_saved_ex(const void* q, const void* k, const void* v, const void* dout, void* dq,
                                        void* dk_out, void* dv_out, int B, int N, int H, int dk, int dv,
                                        ret_dtype_t in_dt, ret_dtype_t out_dt, const float* gamma, const double* theta,
                                        int64_t pos0, int chunk, const void* fwd_workspace, size_t fwd_workspace_bytes,
                                        void* workspace, size_t workspace_bytes, void* stream,
                                        const ret_options_t* opts);
ret_status_t ret_recurrent_step_ex(const void* q, const void* k, const void* v, void* o, float* state, int B, int H,
                                   int dk, int dv, ret_dtype_t in_dt, ret_dtype_t out_dt, const float* gamma,
                                   const double* theta, int64_t pos, void* stream, const ret_options_t* opts);
ret_status_t ret_recurrent_step_positions_ex(const void* q, const void* k, const void* v, void* o, float* state,
                                             int B, int H, int dk, int dv, ret_dtype_t in_dt, ret_dtype_t out_dt,
                                             const float* gamma, const double* theta, const int64_t* pos,
                                             void* stream, const ret_options_t* opts);

/*
 * Retention score normalizations ("Hybrid Architectures: RetNet and the Three Computation Paradigms", section
 * 8.5; RetNet paper summary, "Retention Score Normalization"), selected by `norm` (any combination, 0 = none):
 *   RET_NORM_SCALE   scores Q K^T divided by sqrt(d_k)
 *   RET_NORM_DECAY   each row of the decay matrix divided by the square root of its sum, sum_{i<=p} gamma^i
 *   RET_NORM_SCORES  each row of the (scaled) scores divided by max(|row sum|, 1)
 * The pages state them for the parallel form. Each is a positive factor per output row, so the normalized
 * output of the row at absolute position p is the plain one times c_p / den_p, with c_p the product of the
 * first two factors and den_p = max(|c_p q'_p . z_p|, 1) under RET_NORM_SCORES, where z_p = gamma z_{p-1} + k'_p
 * is the decayed sum of the rotated keys (q'_p . z_p is the row sum of the scores). Rows refer to the whole
 * sequence from its first token at position 0: a call that resumes at pos0 passes the key sum z [B, H, d_k]
 * (fp32) of the tokens before it, as it passes the state. GroupNorm cancels every factor (section 8.4).
 */
#define RET_NORM_SCALE 1
#define RET_NORM_DECAY 2
#define RET_NORM_SCORES 4

/*
 * Chunkwise form (as ret_chunkwise_fwd, options as the _ex calls) with the score normalizations. z_in: the key
 * sum before token 0 ([B, H, d_k] fp32 device, or NULL = zeros); z_out: the key sum after the last token (or
 * NULL; may equal z_in). pos0 >= 0. The workspace is required: ret_chunkwise_normalized_workspace_bytes (0 for
 * an unsupported shape) bytes, zero-filled before first use like the chunkwise workspace. Supported: as
 * ret_chunkwise_fwd, B*N*H*d_v < 2^35. RET_ERR_INVALID_ARG also for norm outside 0..7 and misaligned z buffers,
 * RET_ERR_WORKSPACE for a missing or short workspace. Kernels: the chunkwise kernels, then "ret_norm_zseg",
 * "ret_segment_scan", "ret_norm_rows" and "ret_norm_scale" (the output scaled in place).
 */
size_t ret_chunkwise_normalized_workspace_bytes(int B, int N, int H, int dk, int dv, int chunk, ret_dtype_t in_dt,
                                                const ret_options_t* opts);
ret_status_t ret_chunkwise_normalized_fwd(const void* q, const void* k, const void* v, void* o, int B, int N, int H,
                                          int dk, int dv, ret_dtype_t in_dt, ret_dtype_t out_dt, const float* gamma,
                                          const double* theta, int64_t pos0, int chunk, int norm,
                                          const float* state_in, float* state_out, const float* z_in, float* z_out,
                                          void* workspace, size_t workspace_bytes, void* stream,
                                          const ret_options_t* opts);

/*
 * One decode step (as ret_recurrent_step) with the score normalizations: the state S and the key sum z
 * ([B, H, d_k] fp32 device, required) are both updated in place, S <- gamma S + k'^T v, z <- gamma z + k', and
 * o = c_p (q' S) / den_p at position p = pos >= 0. Kernels: "ret_recurrent_step", then "ret_norm_step".
 */
ret_status_t ret_recurrent_step_normalized(const void* q, const void* k, const void* v, void* o, float* state,
                                           float* z, int B, int H, int dk, int dv, ret_dtype_t in_dt,
                                           ret_dtype_t out_dt, const float* gamma, const double* theta, int64_t pos,
                                           int norm, void* stream, const ret_options_t* opts);

/*
 * For callers that cannot allocate device memory (code under HIP graph capture, tight serving loops, harnesses
 * that forbid allocation): ret_chunkwise_fwd (arguments as there, defaults for the options) with the workspace
 * taken from a device array the library owns, RET_NOALLOC_SCRATCH_BYTES on every GPU it runs on, held until the
 * process ends. The call allocates nothing; the first call on a device looks up the array's address and zeroes
 * its first 64 KB with a fill kernel on `stream`. The call uses the library's segment plan for the shape, with
 * the rotated copies of q and k only where they fit beside the chain (otherwise staging rotates: the same result
 * up to rounding). RET_ERR_WORKSPACE (before anything is enqueued) when the plan's segment chain needs more than
 * the array, or more counters and flags than its zeroed region holds. Every call on a GPU shares that GPU's
 * array and leaves its counters and flags zero: calls that overlap in time on one GPU (different streams or
 * threads) race and must not be made. The array is not visible to ret_chunkwise_check; a segment-chain wait
 * that gives up shows as NaN outputs.
 */
#define RET_NOALLOC_SCRATCH_BYTES (128u << 20)
ret_status_t ret_chunkwise_fwd_noalloc(const void* q, const void* k, const void* v, void* o, int B, int N, int H,
                                       int dk, int dv, ret_dtype_t in_dt, ret_dtype_t out_dt, const float* gamma,
                                       const double* theta, int64_t pos0, int chunk, const float* state_in,
                                       float* state_out, void* stream);

/*
 * Gradients of ret_msr_epilogue, y = swish(gate) (.) n with n = w xh + b and xh the standardized head row of o:
 *     dn = dy (.) swish(gate),  dgate = dy (.) n (.) swish'(gate),  swish'(x) = s + x s (1 - s), s = sigmoid(x)
 *     do = rstd (a - mean(a) - xh mean(a xh)),  a = w (.) dn, the means over the d_v values of a head
 *     dweight[h d_v + c] = sum over rows of dn xh,  dbias = sum over rows of dn
 * dy, o, gate, dout, dgate: [rows, H, d_v], each F32 or BF16; gate, gn_weight, gn_bias as the forward call had them
 * (NULL where it had NULL). dgate, dweight, dbias (device float[H * d_v]) may each be NULL: not wanted. rows = 0 writes
 * zeros to dweight and dbias. dout and dgate may take the place of dy, o or gate (same start and dtype); no other
 * overlap (RET_ERR_INVALID_ARG). workspace: ret_msr_epilogue_bwd_workspace_bytes device bytes when dweight or dbias is
 * wanted (RET_ERR_WORKSPACE if short), of any content; calls sharing one must not overlap in time. The sums are added
 * in a fixed order: the same call gives the same bits. Pointers 16-byte aligned; supported: d_v in {16, 32, 64, 128,
 * 256, 512}, H * d_v < 2^27. Kernels: "ret_msr_epilogue_bwd", "ret_column_sums". opts: the timer, or NULL.
 */
size_t ret_msr_epilogue_bwd_workspace_bytes(int64_t rows, int H, int dv);
ret_status_t ret_msr_epilogue_bwd(const void* dy, const void* o, const void* gate, const float* gn_weight,
                                  const float* gn_bias, void* dout, void* dgate, float* dweight, float* dbias,
                                  int64_t rows, int H, int dv, ret_dtype_t dy_dt, ret_dtype_t o_dt,
                                  ret_dtype_t gate_dt, ret_dtype_t do_dt, ret_dtype_t dgate_dt, float eps,
                                  void* workspace, size_t workspace_bytes, void* stream, const ret_options_t* opts);

/*
 * Layer norm, the pre-norm of a retention or gated-delta block, with the residual stream's addition:
 *     s = x + residual (rounded to x_dt; s = x without one),  y = w (.) (s - mean) rstd + b,  rstd = 1/sqrt(var + eps)
 * over the last axis of x [rows, D] (biased variance, statistics in fp32). residual, sum_out: as x, or NULL; sum_out
 * receives s, the stream the next block adds to. weight, bias: device float[D], NULL means 1 and 0. mean, rstd: device
 * float[rows], or NULL; the gradients want them. x_dt, y_dt: F32 or BF16 each. y and sum_out may take the place of x or
 * residual (same start and dtype); no other overlap. Pointers 16-byte aligned (mean and rstd 4: a slice of the rows'
 * statistics will do); rows = 0 does nothing; 1 <= D <= 16384 (rows with D a multiple of 8 move as 16-byte vectors).
 * Kernel: "ret_layer_norm".
 */
ret_status_t ret_layer_norm_fwd(const void* x, const void* residual, const float* weight, const float* bias, void* y,
                                void* sum_out, float* mean, float* rstd, int64_t rows, int D, ret_dtype_t x_dt,
                                ret_dtype_t y_dt, float eps, void* stream, const ret_options_t* opts);

/*
 * Gradients of ret_layer_norm_fwd: x [rows, D] is what was normalized (s where there was a residual), mean and rstd are
 * the forward call's.
 *     dx = rstd (a - mean(a) - xh mean(a xh)) + dsum,  a = w (.) dy,  xh = (x - mean) rstd
 *     dweight = sum over rows of dy xh,  dbias = sum over rows of dy     (device float[D]; NULL: not wanted)
 * dsum ([rows, D] in dx_dt, or NULL) is the gradient that reaches s past the norm; dx is then the gradient of x and of
 * residual alike. dx may take the place of dy, x or dsum (same start and dtype); no other overlap. rows = 0 writes zeros
 * to dweight and dbias. workspace: as ret_msr_epilogue_bwd's. Kernels: "ret_layer_norm_bwd", "ret_column_sums".
 */
size_t ret_layer_norm_bwd_workspace_bytes(int64_t rows, int D);
ret_status_t ret_layer_norm_bwd(const void* dy, const void* x, const float* weight, const float* mean,
                                const float* rstd, const void* dsum, void* dx, float* dweight, float* dbias,
                                int64_t rows, int D, ret_dtype_t x_dt, ret_dtype_t dy_dt, ret_dtype_t dx_dt,
                                void* workspace, size_t workspace_bytes, void* stream, const ret_options_t* opts);

/*
 * The gated delta rule: the state decays per token and each token writes the difference between its value and what the
 * state already holds for its key. Per batch b and value head h, alpha_t = exp(g_t):
 *     S'_t = alpha_t S_{t-1},  u_t = beta_t (v_t - S'_t^T k_t),  S_t = S'_t + k_t u_t^T,  o_t = scale S_t^T q_t
 * Layouts: q, k [B, N, Hk, d_k] with H a multiple of Hk (value head h reads key head h / (H / Hk)), v, o
 * [B, N, H, d_v], g, beta [B, N, H], state [B, H, d_k, d_v] fp32; a step has no N axis. dtypes: q, k, v in in_dt, o in
 * out_dt, g and beta in gate_dt; F32 input takes F32 output and gates, BF16 input either. g is the natural logarithm of
 * the decay (g <= 0 as a rule; values below -200, -inf included, clear the state); beta usually lies in [0, 1] and k has
 * unit length, which keeps the state bounded; neither is checked. scale = 0 means 1 / sqrt(d_k).
 *
 * ret_gated_delta_fwd computes a whole sequence in chunks of 64 tokens. state_in (NULL: zeros), state_out (NULL: not
 * wanted; may equal state_in): the state before token 0 and after the last token, so that a sequence can be resumed or
 * handed to ret_gated_delta_step. lengths (device int32[B], or NULL): sequence b has lengths[b] tokens (0 .. N, other
 * values are taken as the nearest of these); inputs past them are not used, outputs past them are zero, and state_out
 * is the state after lengths[b] tokens. Products accumulate in fp32; on BF16 input everything the kernels compute and
 * multiply again (the state among it) is split in two bf16 parts, which leaves an error of about 6e-6 in the 2-norm of
 * the outputs (before their own rounding) and of the state, 5e-7 on F32 input. A NaN or infinity of a token can reach
 * the outputs of its own chunk's earlier tokens.
 * workspace: ret_gated_delta_workspace_bytes device bytes (0 for an unsupported shape), of any content; calls sharing
 * one must not overlap in time. Supported: d_k in {32, 64, 128, 256} (BF16) or {16, 32, 64, 128} (F32), d_v a multiple
 * of 16, B*H <= 65535, N >= 1, H * max(d_k, d_v) < 2^22, d_k * d_v < 2^28, and no launch of 2^32 work-items (512 per
 * sequence, value head, segment and 128 columns of d_v). Written buffers must not overlap other buffers. Pointers
 * 16-byte aligned; those of g, beta and lengths (and of dg and dbeta) like one of their elements, so that one token's
 * gates can be a slice of a sequence's. opts: segments (> 0: segments per sequence that run in parallel, joined by
 * their transitions) and timer.
 * Kernels: "ret_delta_prep", "ret_delta_local", "ret_delta_scan", "ret_delta_full".
 *
 * ret_gated_delta_step computes one token of every sequence, the state updated in place; d_k in {16, 32, 64, 128, 256},
 * d_v a multiple of 16, B*H <= 131072 and otherwise the limits above; fp32 arithmetic for either input dtype. Kernel:
 * "ret_delta_step".
 */
size_t ret_gated_delta_workspace_bytes(int B, int N, int H, int Hk, int dk, int dv, ret_dtype_t in_dt,
                                       const ret_options_t* opts);
ret_status_t ret_gated_delta_fwd(const void* q, const void* k, const void* v, const void* g, const void* beta, void* o,
                                 int B, int N, int H, int Hk, int dk, int dv, ret_dtype_t in_dt, ret_dtype_t out_dt,
                                 ret_dtype_t gate_dt, float scale, const int32_t* lengths, const float* state_in,
                                 float* state_out, void* workspace, size_t workspace_bytes, void* stream,
                                 const ret_options_t* opts);
ret_status_t ret_gated_delta_step(const void* q, const void* k, const void* v, const void* g, const void* beta, void* o,
                                  float* state, int B, int H, int Hk, int dk, int dv, ret_dtype_t in_dt,
                                  ret_dtype_t out_dt, ret_dtype_t gate_dt, float scale, void* stream,
                                  const ret_options_t* opts);

/*
 * Gradients of ret_gated_delta_fwd: with dout = dL/do [B, N, H, d_v] in in_dt and, optionally, dstate_out =
 * dL/dstate_out [B, H, d_k, d_v] fp32, writes dq, dk [B, N, Hk, d_k] (summed over the value heads that share a key
 * head), dv [B, N, H, d_v] in out_dt, dg, dbeta [B, N, H] in gate_dt and, unless NULL, dstate_in. The other arguments
 * are the forward call's. Gradients of the padding past lengths[b] are zero. On BF16 input with BF16 outputs and gates,
 * dq, dk, dbeta and dg come from states and writes rounded once to BF16: their error is about 0.003 of the tensor's
 * 2-norm with their own rounding (tested up to 0.0051); dg's, a difference of sums, up to 0.008 (tested up to 0.011),
 * and single values that are small beside the rest can be off by more than themselves. With F32 outputs or gates these
 * are kept in two BF16 parts, at a sixth to a third more time: 1e-5 (tested up to 2e-5), dg 2e-5 (8e-5), before a BF16
 * output's own rounding. dv and dstate_in are as precise as the forward's results. workspace:
 * ret_gated_delta_bwd_workspace_bytes (it holds the state entering and the state gradient leaving every chunk of 64
 * tokens, on BF16 input room for both parts). Same limits as the forward. Sums have one order: the same call gives the
 * same bits.
 * Kernels: "ret_delta_prep", "ret_delta_local", "ret_delta_scan", "ret_delta_states", "ret_delta_local_bwd",
 * "ret_delta_full_bwd", "ret_delta_grad".
 */
size_t ret_gated_delta_bwd_workspace_bytes(int B, int N, int H, int Hk, int dk, int dv, ret_dtype_t in_dt,
                                           const ret_options_t* opts);
ret_status_t ret_gated_delta_bwd(const void* q, const void* k, const void* v, const void* g, const void* beta,
                                 const void* dout, void* dq, void* dk_out, void* dv_out, void* dg, void* dbeta, int B,
                                 int N, int H, int Hk, int dk, int dv, ret_dtype_t in_dt, ret_dtype_t out_dt,
                                 ret_dtype_t gate_dt, float scale, const int32_t* lengths, const float* state_in,
                                 const float* dstate_out, float* dstate_in, void* workspace, size_t workspace_bytes,
                                 void* stream, const ret_options_t* opts);

/*
 * Root-mean-square norm, the pre-norm without a mean, with the residual stream's addition and an output in 8 bits:
 *     s = x + residual (rounded to x_dt; s = x without one),  y = w (.) s rstd,  rstd = 1 / sqrt(mean(s^2) + eps)
 * over the last axis of x [rows, D]; the statistic in fp32, of any finite values (a row whose squares leave the range is scaled
 * first; where the root is below 2^-128, rstd is infinite). residual, weight, sum_out, rstd as in ret_layer_norm_fwd. At
 * least one of y (y_dt) and y8 is wanted. y8 [rows, D] holds y in e4m3 (OCP, 1 byte a value) divided by its scale, rounded to
 * nearest even, for a product in 8 bits: y = y8 scale. group = 0: one scale a row, scales float[rows]; group = 32, 64 or 128:
 * one for every group columns, scales float[rows, ceil(D / group)]. scale = max |y| / 448 over its columns, at least 2^-126;
 * y is taken before its rounding to y_dt. A NaN makes its scale NaN. y and sum_out may take the place of x or residual (same
 * start and dtype); no other overlap. Pointers 16-byte aligned (rstd and scales 4); rows = 0 does nothing; 1 <= D <= 16384.
 * Kernel: "ret_rms_norm".
 */
ret_status_t ret_rms_norm_fwd(const void* x, const void* residual, const float* weight, void* y, void* sum_out,
                              float* rstd, void* y8, float* scales, int group, int64_t rows, int D, ret_dtype_t x_dt,
                              ret_dtype_t y_dt, float eps, void* stream, const ret_options_t* opts);

/*
 * Gradients of ret_rms_norm_fwd's y: x [rows, D] is what was normalized (s where there was a residual), rstd the forward
 * call's.
 *     dx = rstd (a - xh mean(a xh)) + dsum,  a = w (.) dy,  xh = x rstd,  dweight = sum over rows of dy xh
 * dsum, dweight, workspace and the places dx may take as in ret_layer_norm_bwd. Kernels: "ret_rms_norm_bwd",
 * "ret_column_sums".
 */
size_t ret_rms_norm_bwd_workspace_bytes(int64_t rows, int D);
ret_status_t ret_rms_norm_bwd(const void* dy, const void* x, const float* weight, const float* rstd, const void* dsum,
                              void* dx, float* dweight, int64_t rows, int D, ret_dtype_t x_dt, ret_dtype_t dy_dt,
                              ret_dtype_t dx_dt, void* workspace, size_t workspace_bytes, void* stream,
                              const ret_options_t* opts);

/*
 * Short causal convolution along the tokens, channel by channel (before a selective scan, or before q, k and v of a gated
 * delta rule), with its activation:
 *     y_t[d] = act(bias[d] + sum_{j < W} weight[d][j] x_{t - W + 1 + j}[d])
 * x, y [B, N, D]; weight float[D, W], bias float[D] or NULL (0); act RET_ACT_NONE or RET_ACT_SILU. Tokens before the first
 * are state_in [B, W - 1, D] in in_dt, oldest first (NULL: zeros); state_out (as state_in, may equal it; NULL: not wanted)
 * receives the last W - 1 inputs. lengths (device int32[B], or NULL) as in ret_gated_delta_fwd: inputs past them are not used, outputs
 * past them are zero, and state_out is the state after lengths[b] tokens. x_ld: elements from a token's row of x to the next
 * token's (0: D), so that x can be a slice of a wider projection's rows; sequence b starts at row b N.
 * dtypes: x and the states in in_dt, y in out_dt; pairs as in ret_chunkwise_fwd; arithmetic in fp32. Supported: W in
 * {2, 3, 4}, N <= 2^31 - 17, B N <= 2^40, D <= 2^28, x_ld <= 2^32, and no launch of 2^32 work-items. Pointers 16-byte
 * aligned, x and lengths like one of their elements (rows move as vectors of 4 elements where D and x_ld are multiples of 8
 * and x is 16-byte aligned, else one by one). Written buffers must not overlap others. Kernel: "ret_short_conv".
 *
 * ret_short_conv_step computes one token of every sequence: x, y [B, D] (x_ld from sequence to sequence), state [B, W - 1, D]
 * moved on in place. Kernel: "ret_short_conv_step".
 */
#define RET_ACT_NONE 0
#define RET_ACT_SILU 1
ret_status_t ret_short_conv_fwd(const void* x, int64_t x_ld, const float* weight, const float* bias, void* y, int B, int N,
                                int D, int W, ret_dtype_t in_dt, ret_dtype_t out_dt, int act, const int32_t* lengths,
                                const void* state_in, void* state_out, void* stream, const ret_options_t* opts);
ret_status_t ret_short_conv_step(const void* x, int64_t x_ld, const float* weight, const float* bias, void* y, void* state,
                                 int B, int D, int W, ret_dtype_t in_dt, ret_dtype_t out_dt, int act, void* stream,
                                 const ret_options_t* opts);

/*
 * Gradients of ret_short_conv_fwd: with dy [B, N, D] in in_dt and, optionally, dstate_out = dL/dstate_out [B, W - 1, D] in
 * out_dt, writes dx [B, N, D] (contiguous) and, unless NULL, dstate_in in out_dt and dweight float[D, W], dbias float[D]. The
 * other arguments are the forward call's. workspace: ret_short_conv_bwd_workspace_bytes device bytes when dweight or dbias is
 * wanted, of any content; calls sharing one must not overlap in time. Sums have one order: the same call gives the same bits.
 * Kernels: "ret_short_conv_bwd", "ret_column_sums".
 */
size_t ret_short_conv_bwd_workspace_bytes(int B, int N, int D, int W);
ret_status_t ret_short_conv_bwd(const void* dy, const void* x, int64_t x_ld, const float* weight, const float* bias,
                                void* dx, float* dweight, float* dbias, int B, int N, int D, int W, ret_dtype_t in_dt,
                                ret_dtype_t out_dt, int act, const int32_t* lengths, const void* state_in,
                                const void* dstate_out, void* dstate_in, void* workspace, size_t workspace_bytes,
                                void* stream, const ret_options_t* opts);

/*
 * The selective scan: a state of S numbers per channel with its own decays, whose step length, write and read depend on the
 * token. Per batch b and channel d, with group g = d / (D / G):
 *     dt_t = softplus(dt[t][d] + dt_bias[d]),  h_t[s] = exp(dt_t A[d][s]) h_{t-1}[s] + dt_t u_t b_t[g][s],
 *     y_t = (sum_s c_t[g][s] h_t[s] + d_skip[d] u_t) silu(z_t)
 * Layouts: u, dt, z, y [B, N, D], b, c [B, N, G, S], A float[D, S] (negative as a rule), d_skip, dt_bias float[D], states
 * [B, D, S] fp32; a step has no N axis. softplus = 0: dt + dt_bias is the step length itself. NULL d_skip, dt_bias: 0; NULL
 * z: no gate. z_ld, b_ld, c_ld: elements from a token's row to the next token's (0: contiguous), so that z, b and c can be
 * slices of wider projections' rows; sequence b starts at row b N. dtypes: u, dt, z, b, c in in_dt, y in out_dt; pairs as in
 * ret_chunkwise_fwd. All arithmetic is fp32, nothing is rounded before the output. Tokens are joined by the products of their
 * decays, which may vanish; where dt_t A > 0 makes the product over some tokens exceed fp32's range, states and outputs are
 * not finite even if the states would be.
 *
 * ret_selective_scan_fwd computes whole sequences. state_in (NULL: zeros), state_out (NULL: not wanted; may equal state_in),
 * lengths: as in ret_gated_delta_fwd. A NaN or infinity reaches only later tokens of its sequence. workspace:
 * ret_selective_scan_workspace_bytes device bytes (0 for an unsupported shape), of any content; calls sharing one must not
 * overlap in time. Supported: S in {8, 16, 32, 64}, G = 1 or D / G a multiple of 16, D and z_ld, b_ld, c_ld below 2^22,
 * B N <= 2^36, and no launch of 2^32 work-items (512 a sequence, segment and 16 channels) or, in segments, 65536 sequences.
 * Written buffers must not overlap others. Pointers: A and the states 16-byte aligned, the others like one of their elements.
 * opts: segments (> 0: segments per sequence that run in parallel), variant (1: waves that walk their tokens one by one, 2:
 * workgroups that do chunks of 128 tokens, 32 and 16 at 32 and 64 states) and timer. Kernels: "ret_scan_local",
 * "ret_scan_join", "ret_scan_walk", "ret_scan_chunks".
 *
 * ret_selective_scan_step computes one token of every sequence, the state updated in place. Kernel: "ret_scan_step".
 */
size_t ret_selective_scan_workspace_bytes(int B, int N, int D, int S, int G, ret_dtype_t in_dt,
                                          const ret_options_t* opts);
ret_status_t ret_selective_scan_fwd(const void* u, const void* dt, const float* A, const void* b, int64_t b_ld,
                                    const void* c, int64_t c_ld, const float* d_skip, const void* z, int64_t z_ld,
                                    const float* dt_bias, void* y, int B, int N, int D, int S, int G, ret_dtype_t in_dt,
                                    ret_dtype_t out_dt, int softplus, const int32_t* lengths, const float* state_in,
                                    float* state_out, void* workspace, size_t workspace_bytes, void* stream,
                                    const ret_options_t* opts);
ret_status_t ret_selective_scan_step(const void* u, const void* dt, const float* A, const void* b, int64_t b_ld,
                                     const void* c, int64_t c_ld, const float* d_skip, const void* z, int64_t z_ld,
                                     const float* dt_bias, void* y, float* state, int B, int D, int S, int G,
                                     ret_dtype_t in_dt, ret_dtype_t out_dt, int softplus, void* stream,
                                     const ret_options_t* opts);

/*
 * Gradients of ret_selective_scan_fwd: with dy = dL/dy [B, N, D] in in_dt and, optionally, dstate_out = dL/dstate_out fp32,
 * writes du, ddt [B, N, D] (ddt: that of dt before dt_bias and softplus), db, dc [B, N, G, S] (summed over the channels of a
 * group) in out_dt, contiguous, and, unless NULL, dz (out_dt), dA float[D, S], dd_skip, ddt_bias float[D] and dstate_in. The
 * other arguments are the forward call's. Gradients of the padding past lengths[b] are zero, and it has no part in any other,
 * whatever the states are; a step that softplus underflows to 0 has no gradient through its decay. workspace:
 * ret_selective_scan_bwd_workspace_bytes (the states entering and the gradients leaving chunks of 128 tokens (32 and 16 at 32
 * and 64 states), partial sums of db and dc over up to 512 channels and of dA over a chunk). Limits as the forward's in
 * segments. Sums have one order: the same call gives the same bits. opts: the timer. Kernels: "ret_scan_local_bwd",
 * "ret_scan_join_bwd", "ret_scan_grad", "ret_scan_sums".
 */
size_t ret_selective_scan_bwd_workspace_bytes(int B, int N, int D, int S, int G, ret_dtype_t in_dt);
ret_status_t ret_selective_scan_bwd(const void* u, const void* dt, const float* A, const void* b, int64_t b_ld,
                                    const void* c, int64_t c_ld, const float* d_skip, const void* z, int64_t z_ld,
                                    const float* dt_bias, const void* dy, void* du, void* ddt, float* dA, void* db,
                                    void* dc, float* dd_skip, void* dz, float* ddt_bias, int B, int N, int D, int S, int G,
                                    ret_dtype_t in_dt, ret_dtype_t out_dt, int softplus, const int32_t* lengths,
                                    const float* state_in, const float* dstate_out, float* dstate_in, void* workspace,
                                    size_t workspace_bytes, void* stream, const ret_options_t* opts);

#ifdef __cplusplus
}
#endif

#endif /* RETENTION_H */
