/*
 * moe.h -- C ABI of the DWDP-style MoE layer on one MI355X (gfx950): the forward pass, and
 * the gradients of its steps.
 *
 * The layer follows the pattern of "DWDP: Distributed Weight Data Parallelism
 * for High-Performance LLM Inference on NVL72" (arXiv 2604.01621v1, abstract)
 * and its explainer (viz: "Distributed Weight Data Parallelism cuts LLM
 * inference stalls"): every GPU stays data-parallel and holds a share of the
 * MoE experts; the missing ("remote") experts are pulled on a copy engine into
 * an alternate buffer while compute runs ("stay data-parallel" and
 * prefetch-schedule panels), and local plus remote weights reach the grouped
 * GEMM as one contiguous buffer (contiguous-buffer panel).  On one GPU the
 * peers' share is a separate device pool (or pinned host memory).
 *
 * The pages do not define the MoE layer's arithmetic; the library computes the
 * plain top-k softmax-gated mixture of SwiGLU experts: route -> permute ->
 * grouped SwiGLU -> combine, with the weight merge and prefetch in between.
 *
 * Conventions shared by every call
 * --------------------------------
 * - Pointers named *_host are host memory; every other pointer is device
 *   memory (or pinned host memory where stated).  The caller owns all memory,
 *   streams and events; the library allocates nothing (the moe_vmm_* set-up
 *   calls excepted, whose purpose is to allocate) and keeps no state except
 *   the thread-local text returned by moe_last_error().
 * - Every call only enqueues work on the stream it is given and returns; none
 *   synchronises the device.  A return value < 0 means nothing was enqueued
 *   (MOE_ERR_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE) or a HIP call failed
 *   part-way (MOE_ERR_HIP); moe_last_error() then holds a description.
 * - Data errors found on the device set bits of a caller-provided int32
 *   status word (MOE_STATUS_*), which the caller reads after a sync.  The
 *   kernels only OR bits into it; the caller clears it.
 * - Sizes are int (T, E, k, H, I, R = T*k all < 2^31); byte counts are
 *   int64_t / size_t.
 *
 * Layouts
 * -------
 * - logits  f32[T][E], row-major.
 * - x       [T][H] row-major, f32 (MOE_F32) or bf16 (MOE_BF16).
 * - topk_idx i32[T][k], topk_w f32[T][k]: slot j of token t is assignment
 *   a = t*k + j.
 * - Expert block (one expert, row-major, dtype elements, output-major):
 *     [ Wg : I rows x H cols ][ Wu : I rows x H cols ][ Wd : H rows x I cols ]
 *   so that g = x Wg^T, u = x Wu^T, y = h Wd^T.  expert_bytes = 3*H*I*elem.
 * - Permuted rows: the rows of expert e are [offsets[e], offsets[e+1]), in
 *   ascending assignment index (a stable counting sort by expert id).
 */
#ifndef MOE_H_
#define MOE_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef void* moe_stream_t; /* a hipStream_t; NULL is the null stream */
typedef void* moe_event_t;  /* a hipEvent_t */

typedef enum { MOE_F32 = 0, MOE_BF16 = 1 } moe_dtype;

enum {
  MOE_OK = 0,
  MOE_ERR_ARG = -1,         /* invalid argument; nothing enqueued */
  MOE_ERR_UNSUPPORTED = -2, /* valid, but outside what the kernels support; nothing enqueued */
  MOE_ERR_WORKSPACE = -3,   /* workspace missing or too small; nothing enqueued */
  MOE_ERR_HIP = -4,         /* a HIP runtime call failed; see moe_last_error() */
  MOE_ERR_STATUS = -5       /* debug mode only: the call's kernels set a status bit */
};

/*
 * Debug mode: with MOE_DEBUG_SYNC set in the environment (to anything but "" or "0"),
 * every call that enqueues work synchronises its stream before returning.  A kernel that
 * failed then returns MOE_ERR_HIP, and a set bit of the call's status word (when it takes
 * one) MOE_ERR_STATUS, each with a description in moe_last_error(); the failing call is
 * the one that returns.  Off by default: the calls then only enqueue.
 */

/* bits of the device status word */
#define MOE_STATUS_NONFINITE_LOGIT 1 /* a router logit was NaN or +-inf */
#define MOE_STATUS_EXPERT_ABSENT 2   /* a routed expert has no slot in the merged buffer */
#define MOE_STATUS_BAD_EXPERT_ID 4   /* a top-k id outside [0, E) reached the permutation */

/* copy-engine selection for moe_merge_weights / moe_prefetch_layer */
#define MOE_COPY_SDMA 0 /* device-to-device copies on the SDMA engines, no compute units */
#define MOE_COPY_ANY 1  /* let the runtime choose (it may use a copy kernel on the CUs) */
/* The library's own streaming copy kernel for device-to-device runs, on at most n
 * workgroups of 1024 threads (n = 0: as many as the copy can use).  A small n holds the
 * pull to at most n compute units at a time, leaving the rest to a grouped GEMM running
 * beside it (one workgroup per CU).  Each workgroup moves only ~20-25 GB/s, though, so on
 * MI355X the unbounded copy (n = 0) is the faster choice even beside a GEMM.  Host-memory
 * sources still use the runtime copy. */
#define MOE_COPY_KERNEL 2
#define MOE_COPY_KERNEL_ON(n) (MOE_COPY_KERNEL | ((n) << 8))

/* Limits of the kernels (MOE_ERR_UNSUPPORTED beyond them). */
#define MOE_MAX_E 1024
#define MOE_MAX_K 64

/*
 * A pool of consecutive experts [first_expert, first_expert + n_experts):
 * n_experts contiguous expert blocks of expert_bytes each, in device memory
 * or in pinned host memory.  The local pool is this rank's resident share;
 * the remote pool stands in for the peers' shares (DWDP abstract: MoE weights
 * are offloaded across peer GPUs and missing experts fetched on demand).
 * An empty pool (n_experts == 0: every expert local, or none) may have base NULL.
 */
typedef struct moe_pool {
  const void* base;
  int64_t expert_bytes;
  int32_t first_expert;
  int32_t n_experts;
} moe_pool;

/*
 * One half of the double buffer: n_slots expert blocks in ONE contiguous
 * device allocation (DWDP explainer, contiguous-buffer panel) plus the device
 * slot map slot_of[E] (slot of expert e, or -1) that the grouped GEMM reads.
 * The caller allocates base (n_slots * expert_bytes bytes) and slot_of
 * (E int32); the merge call writes slot_of on its stream.
 */
typedef struct moe_wbuf {
  void* base;
  int64_t expert_bytes;
  int32_t n_slots;
  int32_t n_experts; /* E: length of slot_of */
  int32_t* slot_of;  /* device int32[E] */
} moe_wbuf;

/*
 * moe_route -- top-k routing with weights renormalised over the chosen k.
 *
 * For each token t: topk_idx[t][0..k-1] are the k experts with the largest
 * logits, in order of (logit descending, expert id ascending), so +0 and -0
 * tie and ties go to the smaller id; topk_w[t][j] = exp(l_j - l_0) /
 * sum_{i<k} exp(l_i - l_0), which equals the softmax over all E experts
 * renormalised over the chosen k.  Routing exists on the pages only as the
 * "weight-level imbalance" its skew causes (DWDP explainer); the rule is the
 * plain top-k softmax gate.
 *   logits   device f32[T][E]          (read)
 *   topk_idx device i32[T][k]          (written)
 *   topk_w   device f32[T][k]          (written)
 *   status   device i32, may be NULL   (MOE_STATUS_NONFINITE_LOGIT is ORed in
 *            when a token has a non-finite logit; that token's outputs are
 *            then unspecified)
 * Errors: MOE_ERR_ARG for null outputs, T < 0, k < 1 or k > E;
 * MOE_ERR_UNSUPPORTED for E > MOE_MAX_E or k > MOE_MAX_K.  T = 0 is a no-op.
 */
int moe_route(const float* logits, int T, int E, int k, int32_t* topk_idx, float* topk_w,
              int32_t* status, moe_stream_t stream);

/* Workspace bytes moe_permute needs for (T, E, k). */
int moe_permute_workspace_size(int T, int E, int k, size_t* bytes);

/*
 * moe_permute -- counts, offsets, the stable expert-major permutation and the
 * row gather that put the tokens in expert-contiguous order for the grouped
 * GEMM (the grouped GEMM of the DWDP explainer's contiguous-buffer panel
 * consumes rows grouped by expert).
 *   topk_idx device i32[T*k]     (read; a = t*k + j)
 *   x        device [T][H] dtype (read)
 *   counts   device i32[E]       counts[e] = #assignments routed to e
 *   offsets  device i32[E+1]     exclusive prefix sum; offsets[E] = T*k
 *   row_of   device i32[T*k]     row of assignment a
 *   src_of   device i32[T*k]     assignment held by row r (src_of[row_of[a]] = a)
 *   x_perm   device [T*k][H] dtype, x_perm[r] = x[src_of[r] / k]; may be NULL
 *            to skip the gather
 *   ws       device workspace of moe_permute_workspace_size() bytes
 *   status   device i32, may be NULL (MOE_STATUS_BAD_EXPERT_ID for an id
 *            outside [0, E); such assignments are dropped and the outputs
 *            are then unspecified)
 * Errors: MOE_ERR_ARG for null required pointers or bad sizes;
 * MOE_ERR_WORKSPACE when ws_bytes is too small; MOE_ERR_UNSUPPORTED for
 * E > MOE_MAX_E.
 */
int moe_permute(const int32_t* topk_idx, int T, int E, int k, const void* x, int H,
                moe_dtype dtype, int32_t* counts, int32_t* offsets, int32_t* row_of,
                int32_t* src_of, void* x_perm, void* ws, size_t ws_bytes, int32_t* status,
                moe_stream_t stream);

/*
 * moe_permute_noalloc -- moe_permute with no workspace argument and no allocation, for
 * callers that cannot allocate device memory: code under HIP graph capture, tight serving
 * loops, harnesses that forbid hipMalloc.  Its kernels use a file-scope device array of
 * 2 MiB (the most moe_permute's workspace can need for any T, k and E <= MOE_MAX_E) that
 * each GPU holds until the process ends; its address is looked up once per device.
 * Every call on a GPU shares that array: calls that overlap on one GPU (on different
 * streams, or from several threads) race and must be ordered by the caller.  Nothing in it
 * needs clearing: each call writes all of it that it reads.
 * Arguments and outputs: as moe_permute, without ws / ws_bytes.
 * Errors: as moe_permute; MOE_ERR_WORKSPACE if a size needed more than the array (not
 * reachable within the other limits); MOE_ERR_HIP if the array's address cannot be found.
 */
int moe_permute_noalloc(const int32_t* topk_idx, int T, int E, int k, const void* x, int H,
                        moe_dtype dtype, int32_t* counts, int32_t* offsets, int32_t* row_of,
                        int32_t* src_of, void* x_perm, int32_t* status, moe_stream_t stream);

/*
 * moe_merge_weights -- make the merged buffer: write the slot map for the
 * expert set ids_host (strictly ascending; slot = position in ids_host) and
 * copy every expert of that set that the local pool holds into its slot
 * (DWDP explainer, contiguous-buffer panel: local and remote expert weights
 * reach the grouped GEMM as one contiguous buffer; the copy is the
 * "buffer-merge overhead" of the iteration-latency panel).
 *   local     pool of this rank's resident experts (device or pinned host)
 *   ids_host  host i32[n_ids], read during the call only
 *   dst       merged buffer half; dst->slot_of is written on the stream
 *   wait_free if not NULL, the stream first waits for it (the last reader of
 *             this half is done)
 *   ready     if not NULL, recorded on the stream after the copies
 *   copy_mode MOE_COPY_SDMA, MOE_COPY_ANY or MOE_COPY_KERNEL_ON(n), n in [0, 65535]
 * Copies of consecutive ids in consecutive slots are coalesced, and a run
 * whose source bytes are its destination bytes is skipped: when the merged
 * range is stitched with the local-expert block at its head (moe_vmm_map
 * below) and that range is passed as the local pool, the merge copies nothing
 * and only writes the slot map.
 * Errors: MOE_ERR_ARG for unsorted or out-of-range ids, n_ids > n_slots,
 * mismatched expert_bytes or null pointers.
 */
int moe_merge_weights(const moe_pool* local, const int32_t* ids_host, int n_ids, moe_wbuf* dst,
                      moe_stream_t stream, moe_event_t wait_free, moe_event_t ready,
                      int copy_mode);

/*
 * moe_prefetch_layer -- pull the experts of ids_host that the remote pool
 * holds into their slots of dst (slot = position in ids_host, the same set
 * the merge of this half is given), asynchronously on copy_stream: the
 * one-GPU stand-in of the peer pull on the copy engine that fills the
 * alternate buffer while compute runs (DWDP explainer, "stay data-parallel"
 * and prefetch-schedule panels).  It does not write dst->slot_of.
 *   wait_free / ready / copy_mode as for moe_merge_weights.
 * Errors: as for moe_merge_weights.  For tests of a caller's error handling,
 * the environment variable MOE_INJECT_FAULT=prefetch makes the call return
 * MOE_ERR_HIP at once, with nothing enqueued (the ready event is not recorded).
 */
int moe_prefetch_layer(const moe_pool* remote, const int32_t* ids_host, int n_ids, moe_wbuf* dst,
                       moe_stream_t copy_stream, moe_event_t wait_free, moe_event_t ready,
                       int copy_mode);

/*
 * moe_prefetch_routed -- the routed pull with the expert set decided on the
 * device, so nothing is read back to the host between the routing and the
 * pull: on copy_stream, every expert e of the remote pool with counts[e] > 0
 * is copied into slot e of dst, and dst->slot_of[e] is set to e, or to -1 for
 * an expert with no tokens (whose slot keeps what it held).  The same pull
 * as moe_prefetch_layer (DWDP explainer, "stay data-parallel" and
 * prefetch-schedule panels) for the set that moe_permute's counts name.  The
 * slots of the experts outside the remote pool are the caller's: a
 * moe_merge_weights of ids 0 .. n_local - 1 before this call copies (or, for a
 * stitched half, maps) the local experts to slots 0 .. n_local - 1 and writes
 * -1 for every other expert.
 *   remote       pool of experts [first, first + n) in device memory; a pool
 *                in host memory is MOE_ERR_UNSUPPORTED (its pull stays on
 *                moe_prefetch_layer, whose copies the copy engine runs)
 *   counts       device i32[dst->n_experts], tokens per expert (moe_permute)
 *   dst          merged buffer half with n_slots >= first + n: slot = expert id
 *   counts_ready if not NULL, the stream first waits for it (the permute that
 *                writes counts is done)
 *   wait_free / ready as for moe_merge_weights
 *   max_blocks   bound on the copy's workgroups (0: the library's default)
 * Expert blocks and both bases must be 16-byte aligned (MOE_ERR_UNSUPPORTED
 * otherwise).  MOE_INJECT_FAULT=prefetch makes the call fail as for
 * moe_prefetch_layer.
 */
int moe_prefetch_routed(const moe_pool* remote, const int32_t* counts, moe_wbuf* dst,
                        moe_stream_t copy_stream, moe_event_t counts_ready,
                        moe_event_t wait_free, moe_event_t ready, int max_blocks);

/* Workspace bytes moe_grouped_swiglu needs for R = T*k rows. */
int moe_grouped_swiglu_workspace_size(int R, int E, int H, int I, moe_dtype dtype, size_t* bytes);

/*
 * moe_grouped_swiglu -- the grouped GEMM over the experts of the merged
 * buffer (DWDP explainer, contiguous-buffer panel), with the SwiGLU FFN of
 * each expert (Shazeer 2020, "GLU Variants Improve Transformer"):
 *   for the rows r of each expert e:  g = x_perm[r] Wg_e^T,  u = x_perm[r] Wu_e^T,
 *   h = silu(g) * u  (stored as bf16 for MOE_BF16, f32 for MOE_F32),
 *   y_perm[r] = h Wd_e^T  (always f32).
 * Accumulation is f32 (bf16 MFMA for MOE_BF16, f32 FMA for MOE_F32).
 *   x_perm  device [R][H] dtype
 *   offsets device i32[E+1] (from moe_permute)
 *   w       merged buffer; expert e is read at w->base + w->slot_of[e]*expert_bytes
 *   ws      device workspace of moe_grouped_swiglu_workspace_size() bytes
 *   y_perm  device f32[R][H]
 *   status  device i32, may be NULL (MOE_STATUS_EXPERT_ABSENT when an expert
 *           with rows has slot -1, or a slot outside [0, w->n_slots), which is
 *           never read; that expert's rows are then left unwritten)
 * Errors: MOE_ERR_ARG for null pointers or sizes that disagree with w;
 * MOE_ERR_UNSUPPORTED for E > MOE_MAX_E, H*I >= 2^31, or (MOE_BF16) H or I
 * not a multiple of 8; MOE_ERR_WORKSPACE when ws_bytes is too small.
 */
int moe_grouped_swiglu(const void* x_perm, const int32_t* offsets, int R, int E, int H, int I,
                       moe_dtype dtype, const moe_wbuf* w, void* ws, size_t ws_bytes,
                       float* y_perm, int32_t* status, moe_stream_t stream);

/*
 * moe_grouped_swiglu_range -- moe_grouped_swiglu restricted to the experts
 * [e_begin, e_end): only their rows of h and y_perm are written, the rows of
 * other experts are left untouched, and only their slots are read.  Lets the
 * compute stream start on the experts whose weights have arrived while the
 * copy stream is still pulling the rest (per-chunk readiness: one ready event
 * per chunk of the prefetch, each chunk's GEMM waiting only for its own
 * chunk).  Calls on one stream may share the workspace.
 * Errors: as moe_grouped_swiglu, plus MOE_ERR_ARG for a range outside [0, E].
 */
int moe_grouped_swiglu_range(const void* x_perm, const int32_t* offsets, int R, int E, int H, int I,
                             moe_dtype dtype, const moe_wbuf* w, int e_begin, int e_end, void* ws,
                             size_t ws_bytes, float* y_perm, int32_t* status, moe_stream_t stream);

/*
 * moe_grouped_swiglu_gathered -- moe_grouped_swiglu_range with the row gather
 * of moe_permute folded into the GEMM's operand loads: row r of the gate/up
 * GEMM is read from x[src_of[r] / k] instead of x_perm[r], so moe_permute may
 * be called with x_perm = NULL and the [T*k][H] copy is never written.
 *   x      device [T][H] dtype; src_of device i32[T*k] (from moe_permute); k >= 1
 *   other arguments as moe_grouped_swiglu_range.
 * Errors: as moe_grouped_swiglu_range, plus MOE_ERR_ARG for k < 1 or a null src_of,
 * and MOE_ERR_UNSUPPORTED when R > 4*E (prefill tiles) and x spans 4 GiB or more
 * ((R/k + 1) * H * 2 bytes): those tiles address x with 32-bit byte offsets.
 */
int moe_grouped_swiglu_gathered(const void* x, const int32_t* src_of, int k, const int32_t* offsets,
                                int R, int E, int H, int I, moe_dtype dtype, const moe_wbuf* w,
                                int e_begin, int e_end, void* ws, size_t ws_bytes, float* y_perm,
                                int32_t* status, moe_stream_t stream);

/*
 * moe_grouped_swiglu_combine -- the grouped SwiGLU GEMM with the row gather folded into its
 * operand loads (as moe_grouped_swiglu_gathered) and the combine folded into the down
 * GEMM's epilogue: each output row of assignment a = src_of[r] is scaled by topk_w[a] and
 * added into y[a / k] with a float atomic, so neither x_perm nor y_perm is written (the
 * groupedGEMM of the DWDP explainer's contiguous-buffer panel, producing the layer output).
 * y is cleared on the stream first.  The k terms of a token are added in whatever order
 * the tiles finish, so y agrees with moe_combine's fixed-order sum to rounding, not bit for
 * bit, and can differ in its last bits from run to run.  All experts of the buffer.
 *   x device [T][H] bf16; src_of device i32[T*k]; topk_w device f32[T][k]; y device f32[T][H]
 *   offsets, w, ws (moe_grouped_swiglu_workspace_size(T*k, ...)), status: as moe_grouped_swiglu.
 * Errors: as moe_grouped_swiglu_gathered; MOE_ERR_UNSUPPORTED for MOE_F32.
 */
int moe_grouped_swiglu_combine(const void* x, const int32_t* src_of, const float* topk_w, int T,
                               int k, const int32_t* offsets, int E, int H, int I, moe_dtype dtype,
                               const moe_wbuf* w, void* ws, size_t ws_bytes, float* y,
                               int32_t* status, moe_stream_t stream);

/*
 * moe_combine -- the weighted un-permute:
 *   y[t] = sum_{j=0..k-1} topk_w[t][j] * y_perm[row_of[t*k + j]], summed in j order, f32.
 * The pages give no combine rule of their own (like routing, the mixture only appears
 * through the DWDP explainer's imbalance panels); this is the output of the plain top-k
 * mixture of experts: each chosen expert's output weighted by its moe_route weight.  The
 * fixed j order makes the sum reproducible run to run.
 *   y_perm device f32[T*k][H]; row_of device i32[T*k]; topk_w device f32[T][k];
 *   y device f32[T][H] (must not alias y_perm).
 * Errors: MOE_ERR_ARG for null pointers or bad sizes.
 */
int moe_combine(const float* y_perm, const int32_t* row_of, const float* topk_w, int T, int k,
                int H, float* y, moe_stream_t stream);

/*
 * Training pass of the block: the layer norm in front of it and the gradients of the calls
 * above.  With dy the gradient of moe_combine's output y, one backward pass is
 *   moe_combine_backward         dy -> dy_perm, dtopk_w
 *   moe_route_backward           dtopk_w -> dlogits
 *   moe_grouped_swiglu_backward  dy_perm -> dx_perm, dw
 *   moe_permute_backward         dx_perm -> dx
 *   moe_layer_norm_backward      dx -> the block input's gradient, dgamma, dbeta
 * on the forward pass's own buffers (x_perm, y_perm, row_of, offsets, topk_idx, topk_w, mean,
 * rstd).  Sums and statistics are f32; outputs are rounded once.  No call uses atomics on its
 * outputs: the same inputs give the same bits.  dtype is that of x, x_perm and the weights.
 * Every call may be captured into a HIP graph; captured calls that may run at the same time
 * need workspaces of their own.  Outputs must not alias inputs.  Sizes whose launch would pass
 * 2^32 threads are MOE_ERR_UNSUPPORTED; no call has that limit below 4 million tokens or rows, except
 * moe_grouped_swiglu_backward, whose launch also grows with H, I and E.
 */

/*
 * moe_layer_norm -- y[t] = (x[t] - mean_t) * rstd_t * gamma + beta over rows of H, with
 * rstd_t = 1 / sqrt(var_t + eps) and var_t the mean square of x[t] - mean_t.
 *   x, y        device [T][H] dtype; any alignment of one element
 *   gamma, beta device f32[H]; beta may be NULL (no shift)
 *   mean, rstd  device f32[T] (written; what the backward pass reads); either may be NULL
 * Errors: MOE_ERR_ARG for null pointers, bad sizes or eps negative or NaN; MOE_ERR_UNSUPPORTED
 * for H > 2^26, or rows of more than 16384 elements by the millions (2^32 threads).  T = 0 is a no-op.
 */
int moe_layer_norm(const void* x, const float* gamma, const float* beta, int T, int H, float eps,
                   moe_dtype dtype, void* y, float* mean, float* rstd, moe_stream_t stream);

/* Workspace bytes moe_layer_norm_backward needs for dgamma or dbeta (none without both). */
int moe_layer_norm_backward_workspace_size(int T, int H, size_t* bytes);

/*
 * moe_layer_norm_backward -- the gradient of moe_layer_norm: with xh = (x - mean) * rstd and
 * a = dy * gamma,  dx = rstd * (a - mean_h(a) - xh * mean_h(a xh)),
 * dgamma = sum_t dy * xh,  dbeta = sum_t dy.
 *   dy, x, dx    device [T][H] dtype
 *   mean, rstd   device f32[T] (from moe_layer_norm)
 *   dgamma, dbeta device f32[H] (overwritten; zeros for T = 0); either may be NULL
 *   ws           device workspace of moe_layer_norm_backward_workspace_size() bytes; may be NULL
 *                when dgamma and dbeta are
 * Errors: as moe_layer_norm, plus MOE_ERR_WORKSPACE when ws_bytes is too small.
 */
int moe_layer_norm_backward(const void* dy, const void* x, const float* gamma, const float* mean,
                            const float* rstd, int T, int H, moe_dtype dtype, void* dx,
                            float* dgamma, float* dbeta, void* ws, size_t ws_bytes,
                            moe_stream_t stream);

/*
 * moe_combine_backward -- the gradient of moe_combine:
 *   dy_perm[row_of[t*k + j]] = topk_w[t][j] * dy[t]
 *   dtopk_w[t][j] = sum_h dy[t][h] * y_perm[row_of[t*k + j]][h]
 *   dy      device [T][H] dy_dtype (MOE_F32, or MOE_BF16 from a bf16 residual stream)
 *   y_perm  device f32[T*k][H]; may be NULL when dtopk_w is
 *   dy_perm device [T*k][H] dtype
 *   dtopk_w device f32[T][k]; may be NULL (the routing weights are not trained)
 * Rows that row_of does not name keep what they held; an index outside [0, T*k) (an assignment
 * that moe_permute dropped) writes no row, and its dtopk_w is 0.
 * Errors: MOE_ERR_ARG for null pointers or bad sizes; MOE_ERR_UNSUPPORTED for k > MOE_MAX_K,
 * T*k >= 2^31 or H > 2^26.
 */
int moe_combine_backward(const void* dy, moe_dtype dy_dtype, const float* y_perm,
                         const int32_t* row_of, const float* topk_w, int T, int k, int H,
                         moe_dtype dtype, void* dy_perm, float* dtopk_w, moe_stream_t stream);

/*
 * moe_permute_backward -- the gradient of moe_permute's row gather:
 *   dx[t] = sum_{j=0..k-1} dx_perm[row_of[t*k + j]], summed in j order in f32.
 *   dx_perm device [T*k][H] dtype; dx device [T][H] dtype
 * An index outside [0, T*k) adds nothing.
 * Errors: MOE_ERR_ARG for null pointers or bad sizes; MOE_ERR_UNSUPPORTED for T*k >= 2^31 or
 * H > 2^26.
 */
int moe_permute_backward(const void* dx_perm, const int32_t* row_of, int T, int k, int H,
                         moe_dtype dtype, void* dx, moe_stream_t stream);

/*
 * moe_route_backward -- the gradient of moe_route's weights with respect to the logits:
 *   dlogits[t][topk_idx[t][j]] = topk_w[t][j] * (dtopk_w[t][j] - sum_i topk_w[t][i] dtopk_w[t][i])
 * and zero for the experts that were not chosen (the choice itself has no gradient).  An id that
 * a token lists more than once gets the sum of its slots.
 *   topk_idx, topk_w, dtopk_w device [T][k]; dlogits device f32[T][E] (every element written)
 *   status device i32, may be NULL (MOE_STATUS_BAD_EXPERT_ID for an id outside [0, E), which is
 *          then left out of dlogits)
 * Errors: as moe_route.
 */
int moe_route_backward(const int32_t* topk_idx, const float* topk_w, const float* dtopk_w, int T,
                       int E, int k, float* dlogits, int32_t* status, moe_stream_t stream);

/* Workspace bytes moe_grouped_swiglu_backward needs for R = T*k rows. */
int moe_grouped_swiglu_backward_workspace_size(int R, int E, int H, int I, moe_dtype dtype,
                                               size_t* bytes);

/*
 * moe_grouped_swiglu_backward -- the gradient of moe_grouped_swiglu (of y_perm with respect to
 * x_perm and the weights): for the rows r of each expert e, with g, u, h as there (recomputed
 * from x_perm), dh = dy_perm[r] Wd_e, s = sigmoid(g):
 *   du = dh * g * s,  dg = dh * u * s * (1 + g * (1 - s))  (stored in dtype, as h is),
 *   dx_perm[r] = dg Wg_e + du Wu_e,
 *   dWg_e = sum_r dg^T x_perm[r],  dWu_e = sum_r du^T x_perm[r],  dWd_e = sum_r dy_perm[r]^T h.
 * Accumulation is f32 (MFMA).
 *   x_perm, dy_perm device [R][H] dtype
 *   offsets device i32[E+1] (from moe_permute)
 *   w       merged buffer, as for moe_grouped_swiglu
 *   ws      device workspace of moe_grouped_swiglu_backward_workspace_size() bytes
 *   dx_perm device [R][H] dtype; may be NULL (only the weights are trained)
 *   dw      device, n_slots expert blocks laid out as w's: the gradient of the expert in slot s
 *           is written (not added) at dw + s * expert_bytes, zeros for an expert without rows;
 *           blocks of slots that no expert maps to keep what they held (moe_clear_unmapped
 *           clears them).  No two experts may
 *           share a slot.  May be NULL (frozen experts).  Not both dx_perm and dw NULL.
 *   status  device i32, may be NULL (MOE_STATUS_EXPERT_ABSENT when an expert with rows has no
 *           slot in [0, n_slots): its rows of dx_perm are left unwritten)
 * Rows of dx_perm at or past offsets[E] are left as they were.  With R = 0 only dw is written.
 * Errors: MOE_ERR_ARG for null pointers or sizes that disagree with w; MOE_ERR_UNSUPPORTED for
 * E > MOE_MAX_E, H or I > 2^20, a weight matrix of 2^30 bytes or more, (MOE_BF16) H or I not a
 * multiple of 8, or a pointer not aligned to 16 bytes (MOE_F32: to 4), and sizes whose launch would
 * pass 2^32 threads; MOE_ERR_WORKSPACE when ws_bytes is too small.
 */
int moe_grouped_swiglu_backward(const void* x_perm, const void* dy_perm, const int32_t* offsets,
                                int R, int E, int H, int I, moe_dtype dtype, const moe_wbuf* w,
                                void* ws, size_t ws_bytes, void* dx_perm, void* dw,
                                int32_t* status, moe_stream_t stream);

/*
 * moe_clear_unmapped -- zeros for the expert blocks of dw (n_slots blocks laid out as w's) whose slot
 * no expert of w->slot_of maps to.  After moe_grouped_swiglu_backward on the same w and dw every
 * block then holds the gradient of what its slot holds, whichever experts earlier steps had there.
 *   w   merged buffer (base is not read; expert_bytes a multiple of 4); dw device, aligned to 4
 * Errors: MOE_ERR_ARG for null pointers or a bad buffer; MOE_ERR_UNSUPPORTED for more than MOE_MAX_E
 * experts, an unaligned dw, or sizes whose launch would pass 2^32 threads.
 */
int moe_clear_unmapped(const moe_wbuf* w, void* dw, moe_stream_t stream);

/*
 * The block in 8 bits, products by expert, and what stands around the block.
 *
 * 8-bit rows ("mx") are the OCP microscaling format MXFP8 with e4m3 elements: 32 consecutive values
 * of a row share a scale 2^s, kept as the byte s + 127 (255: the block is NaN), and are held as
 * e4m3(v / 2^s).  A matrix of
 * rows x cols is
 *   q       uint8 [rows][cols], cols a multiple of 32
 *   scales  uint8 [rows][pitch], pitch = moe_mx_scale_pitch(cols) = 16 * ceil(cols / 512): the bytes
 *           of the row's blocks, then zeros (whoever fills scales by other means writes the zeros too)
 * The quantisers here take the smallest s with max |v| <= 448 * 2^s, so that no value saturates; a
 * block of zeros has scale byte 0.  A value that is not finite becomes NaN; its block's scale is that
 * of the finite ones.  A decode step of an 8-bit block is
 *   moe_rms_norm         x + residual -> sum, y (for the router), q and scales
 *   moe_route, moe_permute (x_perm = NULL)
 *   moe_grouped_gemm_mx  gathered by src_of: gate and up as one matrix of 2 I rows -> [R][2 I]
 *   moe_mx_quantize      with swiglu -> q and scales [R][I]
 *   moe_grouped_gemm_mx  down -> y_perm f32
 *   moe_combine
 * Statistics and sums are f32 (of moe_grouped_gemm_mx with bf16 outputs see there), outputs are rounded
 * once, no call uses atomics on its outputs and the same inputs give the same bits.  Every call only
 * enqueues and may be captured into a HIP graph; captured calls that may run at the same time need
 * workspaces of their own.  Unless a call says otherwise, outputs must not overlap inputs.  Sizes whose
 * launch would pass 2^32 threads are
 * MOE_ERR_UNSUPPORTED.
 */

/* Bytes of the scales of a row of `cols` values. */
int moe_mx_scale_pitch(int cols, size_t* bytes);

/*
 * moe_mx_quantize -- rows to 8 bits: v = x[r], or with swiglu = 1 (x has 2 cols columns, gate then up)
 * v = silu(x[r][:cols]) * x[r][cols:].
 *   x       device [rows][cols] dtype ([rows][2 cols] with swiglu); any alignment of one element
 *   q, scales device, aligned to 16 bytes
 * Errors: MOE_ERR_ARG for null pointers, bad sizes or swiglu not 0 or 1; MOE_ERR_UNSUPPORTED for cols not
 * a multiple of 32 or above 2^26, an unaligned output, or a launch past 2^32 threads (a wave takes 512
 * columns of a row: 2^26 of them).  rows = 0 is a no-op.
 */
int moe_mx_quantize(const void* x, int rows, int cols, moe_dtype dtype, int swiglu, uint8_t* q,
                    uint8_t* scales, moe_stream_t stream);

/*
 * moe_rms_norm -- the root-mean-square norm with the residual's addition: s[t] = x[t] + residual[t],
 * rounded to dtype (s = x without a residual), rstd_t = 1 / sqrt(mean s[t]^2 + eps),
 * y[t] = s[t] * rstd_t * gamma, and the same in 8 bits (from f32, not from y's rounding).
 *   x, residual device [T][H] dtype; residual may be NULL
 *   gamma     device f32[H]
 *   sum       device [T][H] dtype (s: the stream after the addition); may be NULL, has to be without a
 *             residual; may be x or the residual itself (the addition in place)
 *   y         device [T][H] dtype; may be NULL when q is given
 *   q, scales device, 8-bit rows of H (H a multiple of 32), aligned to 16 bytes; both or neither
 *   rstd      device f32[T] (what the backward pass reads); may be NULL
 * Errors: MOE_ERR_ARG for null pointers, bad sizes, eps negative or NaN, a sum without a residual, or one
 * of q and scales; MOE_ERR_UNSUPPORTED for H > 2^26, q with H not a multiple of 32, or unaligned.
 * T = 0 is a no-op.
 */
int moe_rms_norm(const void* x, const void* residual, const float* gamma, int T, int H, float eps,
                 moe_dtype dtype, void* sum, void* y, uint8_t* q, uint8_t* scales, float* rstd,
                 moe_stream_t stream);

/* Workspace bytes moe_rms_norm_backward needs for dgamma (none without it). */
int moe_rms_norm_backward_workspace_size(int T, int H, size_t* bytes);

/*
 * moe_rms_norm_backward -- the gradient of moe_rms_norm with respect to x (and to the residual, which is
 * the same): with xh = s * rstd and a = dy * gamma,
 *   dx = dsum + rstd * (a - xh * mean_h(a xh)),   dgamma = sum_t dy * xh.
 *   dy      device [T][H] dtype, the gradient of y
 *   dsum    device [T][H] dtype, what reaches s past the norm; may be NULL (none); dx may be dsum itself
 *   s       device [T][H] dtype: the sum that moe_rms_norm wrote (x without a residual)
 *   dx      device [T][H] dtype
 *   dgamma  device f32[H] (overwritten; zeros for T = 0); may be NULL
 *   ws      device workspace of moe_rms_norm_backward_workspace_size() bytes; may be NULL when dgamma is
 * Errors: as moe_rms_norm, plus MOE_ERR_WORKSPACE when ws_bytes is too small.
 */
int moe_rms_norm_backward(const void* dy, const void* dsum, const void* s, const float* gamma,
                          const float* rstd, int T, int H, moe_dtype dtype, void* dx, float* dgamma,
                          void* ws, size_t ws_bytes, moe_stream_t stream);

/*
 * moe_grouped_gemm -- one product per expert over ragged rows: y[r] = x[r] W_e^T for the rows r of
 * expert e (offsets[e] <= r < offsets[e + 1]), accumulated in f32 (MFMA).
 *   x       device [R][K] dtype; or, with src_of (device i32[R], from moe_permute) not NULL, [ceil(R / top_k)][K]:
 *           row r is x[src_of[r] / top_k] (zeros where that is no row of x)
 *   offsets device i32[E+1] (from moe_permute)
 *   w       merged buffer; W_e [N][K] dtype is read at w_off bytes of expert e's block, so a block may hold
 *           other matrices too
 *   y       device [R][N] y_dtype (MOE_F32 for MOE_F32 operands)
 *   status  device i32, may be NULL (MOE_STATUS_EXPERT_ABSENT when an expert with rows has no slot in
 *           [0, n_slots): its rows of y are left unwritten)
 * Rows of y at or past offsets[E] are left as they were.
 * Errors: MOE_ERR_ARG for null pointers or sizes that disagree with w; MOE_ERR_UNSUPPORTED for E > MOE_MAX_E,
 * K or N > 2^20, a matrix of 2^30 bytes or more, a gathered x of 2^31 bytes or more, (MOE_BF16) K or N
 * not a multiple of 8, or pointers, w_off or expert_bytes not aligned to 16 bytes (MOE_F32: to 4).
 * R = 0 is a no-op.
 */
int moe_grouped_gemm(const void* x, const int32_t* src_of, int top_k, const int32_t* offsets, int R,
                     int E, int K, int N, moe_dtype dtype, const moe_wbuf* w, int64_t w_off,
                     moe_dtype y_dtype, void* y, int32_t* status, moe_stream_t stream);

/*
 * moe_grouped_gemm_backward -- its gradient, for x that is not gathered (moe_permute_backward gathers
 * dx back to the tokens): dx[r] = dy[r] W_e,  dW_e = sum_r dy[r]^T x[r].
 *   x, dy   device [R][K] and [R][N] dtype
 *   dx      device [R][K] dtype; may be NULL (only the weights are trained)
 *   dw      device, n_slots expert blocks laid out as w's: dW_e is written (not added) at w_off of
 *           the block of its expert's slot, zeros for an expert without rows; the rest of a block, and
 *           blocks that no expert maps to, keep what they held (moe_clear_unmapped).  No two experts may
 *           share a slot.  May be NULL (frozen experts).  Not both dx and dw NULL.
 *   status  as moe_grouped_gemm
 * Errors: as moe_grouped_gemm.  With R = 0 only dw is written.
 */
int moe_grouped_gemm_backward(const void* x, const void* dy, const int32_t* offsets, int R, int E, int K,
                              int N, moe_dtype dtype, const moe_wbuf* w, int64_t w_off, void* dx,
                              void* dw, int32_t* status, moe_stream_t stream);

/*
 * moe_grouped_gemm_mx -- moe_grouped_gemm on 8-bit rows and weights: W_e's elements [N][K] are read at
 * w_off of expert e's block and its scales [N][moe_mx_scale_pitch(K)] at s_off.  f32 outputs are f32 sums
 * of exact products: the values are expanded to bf16, which holds them (with scales below 2^-124 to the
 * nearest of its subnormals; values from 2^128 on are infinite).  bf16 outputs come from the 8-bit MFMA,
 * twice as fast at many rows, which adds eight consecutive products at once, each cut below 2^-13 of the
 * largest: in the 2-norm about 3e-5 of the result, a sixtieth of what bf16's rounding makes.  The cut is at
 * most 7 * 2^-13 of the sum over those eights of their largest |product|, whatever the products add up to:
 * an output whose products cancel can be off by more than its own rounding.  Of random values 1.2 % come
 * out as the neighbour of the nearest bf16 number.  Where that matters, take f32 outputs.
 *   x, x_scales device, 8-bit rows of K ([R], or with src_of [ceil(R / top_k)])
 *   other arguments as moe_grouped_gemm
 * Errors: as moe_grouped_gemm; MOE_ERR_UNSUPPORTED for K not a multiple of 32 or N not one of 8, or
 * pointers, w_off, s_off or expert_bytes not aligned to 16 bytes.
 */
int moe_grouped_gemm_mx(const uint8_t* x, const uint8_t* x_scales, const int32_t* src_of, int top_k,
                        const int32_t* offsets, int R, int E, int K, int N, const moe_wbuf* w,
                        int64_t w_off, int64_t s_off, moe_dtype y_dtype, void* y, int32_t* status,
                        moe_stream_t stream);

/*
 * moe_dropout_add -- dropout and the residual's addition, with a mask that is never stored:
 *   out[i] = residual[i] + (keep_i ? x[i] / (1 - p) : 0),  i < n.
 * keep_i: Philox4x32-10 with rng[0] (the seed) as key and (i / 4, rng[1] (the step)) as counter gives
 * four 32-bit words; i is kept where word i % 4 is at least floor(p * 2^32).  The mask depends on i, the
 * seed and the step alone.  rng is read on the device when the call runs, so a captured graph draws a
 * new mask on each replay if the program changes the step in between.
 *   x        device [n] x_dtype
 *   residual device [n] dtype; may be NULL (nothing is added)
 *   p        in [0, 1)
 *   rng      device u64[2]
 *   out      device [n] dtype; may be x (of the same type) or the residual itself
 * Any alignment of one element (rng: 8 bytes).  A dropped x counts for nothing, also where it is not finite.
 * Errors: MOE_ERR_ARG for null pointers, n < 0, p outside [0, 1) or NaN, or a bad dtype.  n = 0 is a no-op.
 */
int moe_dropout_add(const void* x, moe_dtype x_dtype, const void* residual, int64_t n, double p,
                    const uint64_t* rng, moe_dtype dtype, void* out, moe_stream_t stream);

/*
 * moe_dropout_add_backward -- its gradient with respect to x: dx[i] = keep_i ? dout[i] / (1 - p) : 0 with
 * the same rng (the residual's gradient is dout itself).
 *   dout device [n] dtype; dx device [n] x_dtype; dx may be dout itself when the types are the same
 * Errors: as moe_dropout_add.
 */
int moe_dropout_add_backward(const void* dout, moe_dtype dtype, int64_t n, double p, const uint64_t* rng,
                             moe_dtype x_dtype, void* dx, moe_stream_t stream);

/*
 * Multi-layer pipeline helpers (the block between two MoE layers).  The
 * explainer's prefetch-schedule panel hides the fetch of layer l+1's remote
 * experts behind layer l's MoE block and layer l+1's attention block; a
 * dense bf16 GEMM stands in for the attention block.
 *
 * moe_dense_gemm: out[M][N] = bf16(x[M][K] W[N][K]^T), bf16 in, f32 accumulate.
 *   K and N must be multiples of 8 and N*K below 2^31 (MOE_ERR_UNSUPPORTED otherwise).
 * moe_residual_add: out[i] = bf16(x[i] + y[i]) for i < n; x, out bf16, y f32;
 *   out may alias x.
 */
int moe_dense_gemm(const void* x, const void* w, int M, int N, int K, void* out,
                   moe_stream_t stream);
int moe_residual_add(const void* x, const float* y, int64_t n, void* out, moe_stream_t stream);

/*
 * Split-weight management by page stitching (set-up calls: these allocate and
 * map; never call them on the hot path).  The merged-buffer half of the
 * contiguous-buffer panel is built as one virtual range over physical blocks
 * placed back to back -- the local-expert block of the layer it serves, then
 * the half's own block for fetched experts -- so the local experts need no
 * copy (the "buffer-merge overhead" of the iteration-latency panel).
 *   moe_vmm_granularity: the allocation granularity on `device` (block sizes
 *                        must be multiples of it; an R1 expert block is 42 x 2 MiB)
 *   moe_vmm_create:      a physical block of `bytes` on `device` (no mapping)
 *   moe_vmm_map:         reserve one virtual range, map the n blocks back to
 *                        back, grant `device` read/write; *va is its base
 *   moe_vmm_unmap:       undo moe_vmm_map (same blocks sizes, in order)
 *   moe_vmm_release:     free a physical block once no range maps it
 * With such a range the expert set given to merge and prefetch must begin
 * with every expert of the stitched local block (their slots then coincide
 * with the block); a set that skips one would shift later experts into the
 * block and overwrite it.
 * Errors: MOE_ERR_ARG for empty or non-granular sizes, MOE_ERR_HIP from the runtime.
 */
typedef void* moe_phys_t; /* a hipMemGenericAllocationHandle_t */
int moe_vmm_granularity(int device, size_t* bytes);
int moe_vmm_create(int device, size_t bytes, moe_phys_t* phys);
int moe_vmm_map(int device, const moe_phys_t* phys, const size_t* bytes, int n, void** va);
int moe_vmm_unmap(void* va, const size_t* bytes, int n);
int moe_vmm_release(moe_phys_t phys);

/* Events and stream waits, so a caller without HIP headers can order the
 * copy stream against the compute stream.  timing != 0 makes a timing event. */
int moe_event_create(moe_event_t* ev, int timing);
int moe_event_destroy(moe_event_t ev);
int moe_event_record(moe_event_t ev, moe_stream_t stream);
int moe_event_elapsed_ms(moe_event_t start, moe_event_t stop, float* ms);
int moe_stream_wait_event(moe_stream_t stream, moe_event_t ev);

/* Thread-local text describing the last failed call on this thread ("" if none). */
const char* moe_last_error(void);
/* Library version string. */
const char* moe_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MOE_H_ */
