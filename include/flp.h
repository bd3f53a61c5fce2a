/*
 * flp.h - C ABI of the fused linear log-prob / cross-entropy LM head for
 * GB300 (sm_103a).
 *
 * Problem (Liger-Kernel v0.8.3 test/transformers page, the native SM100 fused
 * scaled linear cross-entropy commit, section "Summary": the classifier GEMM
 * fused with NLL/LSE and optional entropy; "Chunked Triton GRPO loss" of the
 * Liger-Kernel pull request 1294 page: the lm_head fused into the loss with an
 * online logsumexp so that the (N, V) logits are never materialised):
 *
 *   X  : bf16 [M, H], row-major, contiguous   (hidden states)
 *   W  : bf16 [V, H], row-major, contiguous   (classifier / lm_head weight,
 *                                              the nn.Linear layout)
 *   y  : int64 [M]                            (targets, ignore_index allowed)
 *   s  : fp32                                 (logit scale, 1/temperature)
 *
 *   z_ij      = s * sum_k X_ik W_jk   (fp32 accumulation; never stored in HBM)
 *   lse_i     = log sum_j exp(z_ij)
 *   logprob_i = z_{i,y_i} - lse_i
 *   entropy_i = lse_i - sum_j p_ij z_ij,   p_ij = exp(z_ij - lse_i)
 *
 * Backward (same Liger-Kernel pages: "Implementation > Backward" of the native
 * commit, "Kernel design notes" of pull request 1294): the logits are
 * recomputed tile by tile,
 *
 *   dZ_ij = s * [ g_lp_i (1[j = y_i] - p_ij) + g_ent_i p_ij (sum_k p_ik z_ik - z_ij) ]
 *
 * is rounded to bf16, and contracted into dX = dZ W and dW = dZ^T X with fp32
 * accumulation.
 *
 * Conventions shared by every entry point
 *  - Device pointers are CUDA device addresses owned by the caller; the library
 *    allocates no device memory and keeps no state between calls beyond cached
 *    device attributes.  Every call is asynchronous on `stream` (a
 *    cudaStream_t passed as void*, NULL for the legacy default stream) and
 *    launches only on the device that is current on the calling thread.
 *  - Argument errors are returned synchronously before anything is launched.
 *    Required: every pointer 16-byte aligned; H % 8 == 0 (row pitch of a TMA
 *    tensor, else FLP_ERR_UNSUPPORTED); M >= 0 (M == 0 is a no-op); V >= 1;
 *    workspace large enough (else FLP_ERR_WORKSPACE).
 *  - A row whose target equals ignore_index has logprob = 0, entropy = 0 and a
 *    zero gradient row; its lse is still written.  A target outside [0, V)
 *    that is not ignore_index yields logprob = NaN for that row and sets
 *    FLP_ERR_BAD_TARGET in the workspace's error word (read it with
 *    flp_get_error); the call itself still returns FLP_OK because the hot path
 *    never synchronises.
 *  - The workspace is caller-owned device memory of at least the queried size.
 *    Its contents need no initialisation; a call owns it until the work it
 *    queued on `stream` has finished.  Calls that run concurrently must use
 *    distinct workspaces.
 *  - Results are deterministic: no floating-point atomics are used, so two
 *    identical calls produce bit-identical outputs.
 */
#ifndef FLP_H
#define FLP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    FLP_OK = 0,
    FLP_ERR_INVALID_ARG = 1, /* null/misaligned pointer, negative size, bad flag */
    FLP_ERR_UNSUPPORTED = 2, /* shape or device the kernels do not handle (H % 8 != 0,
                                not an sm_103 device, size beyond int32 tiling) */
    FLP_ERR_WORKSPACE = 3,   /* workspace pointer null or smaller than required */
    FLP_ERR_CUDA = 4,        /* a CUDA runtime/driver call failed; see flp_last_error_message */
    FLP_ERR_BAD_TARGET = 5,  /* (error word) a target outside [0, V) that is not ignore_index */
    FLP_ERR_TIMEOUT = 6      /* (error word) a kernel's bounded wait expired; its outputs are invalid */
} flp_status;

typedef enum { FLP_F32 = 0, FLP_BF16 = 1 } flp_dtype;

/*
 * Workspace sizes, in bytes, for the given problem on the current device
 * (the Liger-Kernel native commit's "Summary" lists reusable workspace
 * configuration and query APIs).
 *   fwd_bytes : needed by flp_forward (per-split raw partials and the target
 *               logits; the SkyRL page "perf(megatron): autotune fused LM-head
 *               Triton kernels", section "Correctness", keeps raw and final
 *               results in separate buffers, and so does this library).
 *   bwd_bytes : needed by flp_backward with its default row waves of up to
 *               8192 rows (all M rows when M <= 8192); one wave's bf16 dZ,
 *               [wave rows, ceil(V/256)*256], dominates, beside a few KiB of
 *               tile counters.  The native commit's "Memory" section reports
 *               the same kind of reusable workspace, and pull request 1294's
 *               "Kernel design notes" a reusable per-chunk grad_logits buffer.
 * Either output pointer may be NULL.  The same buffer may serve both calls.
 * Returns FLP_ERR_INVALID_ARG for negative sizes, FLP_ERR_CUDA if the device
 * cannot be queried (FLP_ERR_UNSUPPORTED if it is not an sm_103 device).
 */
flp_status flp_workspace_query(int64_t M, int64_t H, int64_t V, int compute_entropy,
                               size_t* fwd_bytes, size_t* bwd_bytes);

/*
 * flp_workspace_query with the backward's wave size chosen by the caller:
 * bwd_bytes is what flp_backward needs to process the rows in waves of
 * `chunk_rows` rows (rounded up to a multiple of 128, at most M;
 * chunk_rows <= 0 selects the default of flp_workspace_query).  A smaller
 * wave trades speed for a smaller workspace; below 2048-row waves
 * flp_backward runs the vocabulary-split schedule instead when the same bytes
 * also hold its fp32 dX scratch (see flp_backward_ex).  Errors as
 * flp_workspace_query.
 */
flp_status flp_workspace_query_ex(int64_t M, int64_t H, int64_t V, int compute_entropy,
                                  int64_t chunk_rows, size_t* fwd_bytes, size_t* bwd_bytes);

/*
 * Forward: writes logprob[M], lse[M] and (when compute_entropy != 0)
 * entropy[M], all fp32 device arrays.  entropy must be NULL when
 * compute_entropy == 0 and non-NULL otherwise (the SkyRL page's "Overview":
 * compute_entropy gates the entropy buffers and kernel work).
 * Two kernels run on `stream`: the fused tcgen05 GEMM + online
 * max / sum-exp / target / entropy epilogue writing raw per-split partials to
 * the workspace, then the merge of those partials into the outputs.  If a
 * bounded wait of the first kernel runs out (FLP_ERR_TIMEOUT in the error
 * word), the merge writes NaN to every output row.
 */
flp_status flp_forward(const void* X, const void* W, const int64_t* targets, int64_t M,
                       int64_t H, int64_t V, int64_t ignore_index, float scale,
                       int compute_entropy, float* logprob, float* lse, float* entropy,
                       void* workspace, size_t workspace_bytes, void* stream);

/*
 * Backward: given the forward's lse (and entropy when compute_entropy != 0),
 * writes dX [M, H] (dtype dX_dtype, overwritten) and dW [V, H] (dtype
 * dW_dtype; overwritten, or added to when accumulate_dW != 0).  An FLP_F32 dW
 * accumulates in fp32 across waves.  An FLP_BF16 dW is written once, rounded
 * from the fp32 accumulator, so it needs the whole backward in one wave (a
 * workspace that holds all M rows of dZ) and no accumulate_dW; otherwise the
 * call returns FLP_ERR_UNSUPPORTED before launching anything.
 *   grad_logprob, grad_entropy : fp32 [M] upstream gradients of logprob and
 *       entropy; NULL means zero.  grad_entropy is ignored when
 *       compute_entropy == 0.  For a mean NLL loss over N valid rows pass
 *       grad_logprob = -1/N on every row.
 * Rows are processed in waves of as many rows as the workspace holds (at most
 * M, at least 128): each wave recomputes its logits tiles, writes bf16 dZ to
 * the workspace, and runs the dX and dW contractions; dW accumulates in fp32
 * across waves in a fixed order.  flp_backward picks the schedule
 * (FLP_BWD_AUTO of flp_backward_ex).
 */
flp_status flp_backward(const void* X, const void* W, const int64_t* targets, int64_t M,
                        int64_t H, int64_t V, int64_t ignore_index, float scale,
                        int compute_entropy, const float* lse, const float* entropy,
                        const float* grad_logprob, const float* grad_entropy, void* dX,
                        flp_dtype dX_dtype, void* dW, flp_dtype dW_dtype, int accumulate_dW,
                        void* workspace, size_t workspace_bytes, void* stream);

/*
 * How the backward's tiles are scheduled (the Liger-Kernel native commit,
 * "Implementation > Backward": persistent kernels over token waves).
 *   FLP_BWD_SPLIT : per wave, one launch of the wave's dZ tiles, then one
 *                   launch of its dX and dW tiles.  Waves may be any multiple
 *                   of 128 rows.
 *   FLP_BWD_FUSED : one persistent launch for every wave: dX and dW tiles
 *                   start as soon as the dZ tiles they read are stored (tile
 *                   counters in the workspace), most dW tiles run interleaved
 *                   with the dZ sweep while their dZ column is still in L2,
 *                   and a wave's last dW tiles overlap the next wave's dZ
 *                   tiles.  With more than one wave, waves are multiples of
 *                   256 rows.
 *   FLP_BWD_VSPLIT: all rows in one wave and the vocabulary in chunks of as
 *                   many columns as the workspace holds after an fp32 [M, H]
 *                   dX scratch: per chunk, one launch of its dZ tiles and one
 *                   of its dX and dW tiles.  dX accumulates over the chunks
 *                   in fp32 (in the scratch when dX is bf16, rounded once at
 *                   the end), and every dW tile is written once with K = all
 *                   rows, so a small workspace keeps long dW contractions and
 *                   a bf16 dW stays possible.  dW is bit-identical to a
 *                   one-wave run of the other schedules; dX differs from it
 *                   by the fp32 summation order over the chunks.
 *   FLP_BWD_AUTO  : the faster one on GB300: FLP_BWD_SPLIT when its waves
 *                   hold all rows or at least 2048 rows, else FLP_BWD_VSPLIT
 *                   when the workspace allows it (else FLP_BWD_SPLIT).  The
 *                   fused launch keeps 256 x 256 dZ and dW tiles (its
 *                   dependency counters count 256-column tiles) where the
 *                   split schedule runs 256 x 512 ones, and measured ~7%
 *                   slower per headline step; with the same tile shapes in
 *                   both schedules it was 0.6-2% slower at every shape
 *                   measured.
 * The split and fused schedules compute every output tile with the same
 * instructions in the same order: their results are bit-identical.
 */
typedef enum { FLP_BWD_AUTO = 0, FLP_BWD_SPLIT = 1, FLP_BWD_FUSED = 2, FLP_BWD_VSPLIT = 3 } flp_bwd_schedule;

/*
 * flp_backward with an explicit schedule.  FLP_BWD_FUSED returns
 * FLP_ERR_UNSUPPORTED when the workspace holds fewer than 256 rows of dZ but
 * not all M rows; other arguments and errors are those of flp_backward.
 */
flp_status flp_backward_ex(const void* X, const void* W, const int64_t* targets, int64_t M,
                           int64_t H, int64_t V, int64_t ignore_index, float scale,
                           int compute_entropy, const float* lse, const float* entropy,
                           const float* grad_logprob, const float* grad_entropy, void* dX,
                           flp_dtype dX_dtype, void* dW, flp_dtype dW_dtype, int accumulate_dW,
                           void* workspace, size_t workspace_bytes, flp_bwd_schedule schedule,
                           void* stream);

/*
 * The wave size, wave count and schedule (FLP_BWD_SPLIT, FLP_BWD_FUSED or
 * FLP_BWD_VSPLIT) that flp_backward_ex would use for this problem, workspace
 * size and requested schedule; for FLP_BWD_VSPLIT *waves counts vocabulary
 * chunks.  Host arithmetic only: touches no device.  Any output
 * pointer may be NULL.  Returns FLP_ERR_WORKSPACE / FLP_ERR_UNSUPPORTED
 * exactly when the backward call would.
 */
flp_status flp_backward_plan(int64_t M, int64_t H, int64_t V, size_t workspace_bytes,
                             flp_bwd_schedule schedule, int64_t* wave_rows, int64_t* waves,
                             flp_bwd_schedule* schedule_used);

/*
 * The backward's tile schedule, for inspection (a diagnostic; host arithmetic
 * only, touches no device): the units that flp_backward_ex would hand out, in
 * ticket order over its launches, for `pairs` resident CTA pairs.  Entry n is
 * units[5n .. 5n+4] = (launch, kind, wave, a, b), kind 0 = dZ tile (a = row
 * tile of the wave, b = vocabulary tile), 1 = dX tile (a = row tile, b =
 * hidden tile), 2 = dW tile (a = vocabulary tile, b = hidden tile), 3 = wide
 * dX tile (a = row tile, b = 512-column hidden tile: the hidden tiles 2b and
 * 2b + 1), 4 = wide dZ tile (a = row tile, b = its first vocabulary tile: the
 * vocabulary tiles b and b + 1; one whose second half lies past the launch's
 * vocabulary is listed as the dZ tile b, kind 0), 5 = wide dW tile (a =
 * vocabulary tile, b = 512-column hidden tile: the hidden tiles 2b and
 * 2b + 1); tiles are 256 x 256 except the wide ones.  At most `capacity` entries are written; *count receives the
 * total.  units may be NULL to query the count.
 */
flp_status flp_backward_schedule(int64_t M, int64_t H, int64_t V, size_t workspace_bytes,
                                 flp_bwd_schedule schedule, int pairs, int32_t* units,
                                 int64_t capacity, int64_t* count);

/*
 * Forward that allocates nothing and takes no workspace.  The pages have no
 * counterpart; it exists for callers that cannot call cudaMalloc and have no
 * workspace to hand: code running inside a host framework that owns every
 * device allocation and gives its plugins no allocator, or latency-critical
 * loops where the implicit device synchronisation of cudaMalloc/cudaFree is
 * not acceptable.  Arguments and outputs are those of flp_forward; the
 * per-split partials and the error word live instead in one file-scope
 * device array of FLP_STATIC_SCRATCH_BYTES (16 MiB) that every GPU which
 * loads this library holds until the process exits.
 *  - It takes the fastest vocabulary-split plan whose scratch fits that size
 *    (flp_forward's own plan when its fwd_bytes fit, with the same results
 *    bit for bit; otherwise fewer splits, whose merged results can differ from
 *    flp_forward's in the last bits).  Problems that do not fit even with one
 *    split are rejected with FLP_ERR_UNSUPPORTED before any launch.
 *  - The first call on a device looks up the array's device address on that
 *    device (cudaGetSymbolAddress, with the device current); make that first
 *    call before any stream capture.  No cudaMalloc, cudaFree or allocating
 *    library routine is ever called.
 *  - Every call, on any stream, shares the one array and it keeps the last
 *    call's contents (each call clears its error word first): calls that
 *    overlap on the GPU race and corrupt each other's results.
 *  - Out-of-range targets still give logprob = NaN; the error word of this
 *    array is not readable through flp_get_error.  If a bounded wait of the
 *    forward kernel ever runs out, the merge writes NaN to every output row,
 *    so a failed call cannot pass stale values from the array for results.
 */
#define FLP_STATIC_SCRATCH_BYTES (16u << 20)
flp_status flp_forward_noalloc(const void* X, const void* W, const int64_t* targets, int64_t M,
                               int64_t H, int64_t V, int64_t ignore_index, float scale,
                               int compute_entropy, float* logprob, float* lse, float* entropy,
                               void* stream);

/*
 * Loss heads on the forward's per-row log-probs (the chunked GRPO page,
 * "Chunked Triton GRPO loss": a loss on top of the lm_head's per-token
 * log-probs).  With N = the number of rows whose target is not ignore_index:
 *   FLP_LOSS_NLL_MEAN           loss = -(1/N) sum_i lp_i
 *   FLP_LOSS_NLL_SUM            loss = -sum_i lp_i  (token-sum reduction;
 *                               grad_logprob = -1 on every valid row)
 *   FLP_LOSS_CLIPPED_SURROGATE  r_i = exp(lp_i - old_i),
 *       loss = (1/N) sum_i [ -min(r_i A_i, clip(r_i, 1 - eps_low, 1 + eps_high) A_i)
 *                            + beta (exp(ref_i - lp_i) - (ref_i - lp_i) - 1) ]
 *       (token-level ratio, two-sided clip, k3 KL estimator against a
 *       reference policy when ref_logprob != NULL).
 * All arrays are fp32 [M] device arrays: old_logprob and advantage are
 * required for the clipped surrogate and ignored otherwise; per_token_loss
 * (the bracketed terms, 0 on ignored rows) and grad_logprob (d loss / d lp_i,
 * the upstream gradient to hand to flp_backward) may be NULL; loss is one
 * fp32 on the device.  One block with fixed-order fp64 reductions:
 * deterministic.  N = 0 gives loss 0 and zero gradients.
 */
typedef enum { FLP_LOSS_NLL_MEAN = 1, FLP_LOSS_CLIPPED_SURROGATE = 2, FLP_LOSS_NLL_SUM = 3 } flp_loss_kind;
flp_status flp_loss(const float* logprob, const int64_t* targets, int64_t M, int64_t ignore_index,
                    int kind, const float* old_logprob, const float* advantage,
                    const float* ref_logprob, float eps_low, float eps_high, float beta,
                    float* per_token_loss, float* grad_logprob, float* loss, void* stream);

/*
 * Clipped-surrogate policy loss over sequences (the chunked GRPO page: its
 * "Setup" runs loss_type="dapo" with importance_sampling_level="sequence" and
 * num_items_in_batch, its "Correctness" section covers the grpo / bnpo /
 * dr_grpo / dapo aggregations with token- and sequence-level ratios).  The
 * page names these options without defining them; this library reads them so:
 *   seq_offsets : int64 [num_seqs + 1] device array; rows [off[b], off[b+1])
 *                 form sequence b (ranges are clamped to [0, M); they must not
 *                 overlap).  NULL: one sequence of all M rows.  A row is a
 *                 token of the loss when its target is not ignore_index; n_b
 *                 counts the tokens of sequence b, N all of them.
 *   is_level    : FLP_IS_TOKEN     log r_t = lp_t - old_t
 *                 FLP_IS_SEQUENCE  log r_t = (1/n_b) sum_{u in b} (lp_u - old_u),
 *                                  shared by every token of b
 *   term_t      = -min(r_t A_t, clip(r_t, 1 - eps_low, 1 + eps_high) A_t)
 *                 + beta (exp(ref_t - lp_t) - (ref_t - lp_t) - 1)  (when ref_logprob != NULL)
 *   aggregation : FLP_AGG_TOKEN_MEAN     loss = (1/N) sum_t term_t            (bnpo)
 *                 FLP_AGG_SEQUENCE_MEAN  loss = (1/B) sum_b (1/max(n_b,1)) sum_{t in b} term_t (grpo)
 *                 FLP_AGG_SUM_OVER       loss = (1/D) sum_t term_t, D = normalizer when > 0
 *                                        (dapo: num_items_in_batch, the token count of the
 *                                        whole global batch; dr_grpo: B x the longest
 *                                        completion), else D = N
 * Outputs as flp_loss: per_token_loss (term_t, 0 on rows that are not
 * tokens) and grad_logprob (d loss / d lp_t, the upstream gradient for
 * flp_backward; with a sequence-level ratio it includes every term of the
 * sequence through log r_b) may be NULL; loss is one fp32 on the device.
 * old_logprob and advantage (per row: broadcast a per-sequence advantage) are
 * required.  One block, fp64 arithmetic, fixed-order reductions:
 * deterministic.  FLP_LOSS_CLIPPED_SURROGATE of flp_loss is the token-level
 * ratio with FLP_AGG_TOKEN_MEAN.
 */
typedef enum { FLP_IS_TOKEN = 0, FLP_IS_SEQUENCE = 1 } flp_is_level;
typedef enum { FLP_AGG_TOKEN_MEAN = 0, FLP_AGG_SEQUENCE_MEAN = 1, FLP_AGG_SUM_OVER = 2 } flp_loss_aggregation;
flp_status flp_policy_loss(const float* logprob, const int64_t* targets, int64_t M,
                           int64_t ignore_index, const int64_t* seq_offsets, int64_t num_seqs,
                           const float* old_logprob, const float* advantage,
                           const float* ref_logprob, float eps_low, float eps_high, float beta,
                           int is_level, int aggregation, double normalizer,
                           float* per_token_loss, float* grad_logprob, float* loss, void* stream);

/*
 * Synchronises `stream`, then reads and returns the workspace's error word
 * (FLP_OK, FLP_ERR_BAD_TARGET or FLP_ERR_TIMEOUT) written by the most recent
 * flp_forward / flp_backward that used this workspace.  Each of those calls
 * clears the word when it starts.  Returns FLP_ERR_CUDA if the copy fails.
 */
flp_status flp_get_error(const void* workspace, void* stream);

/*
 * Optional instrumentation for benchmarks and profiling.  After this call the
 * calling thread's flp_forward / flp_backward record events[2k] immediately
 * before and events[2k+1] immediately after kernel phase k, on the call's
 * stream:
 *   k = 0  forward tile kernel          k = 1  split merge
 *   k = 2  FLP_BWD_SPLIT: the first wave's dZ launch;
 *          FLP_BWD_FUSED: the one backward launch (every wave)
 *   k = 3  FLP_BWD_SPLIT: the first wave's dX and dW launch (not recorded
 *          by FLP_BWD_FUSED)
 *   k = 4  reserved (never recorded)
 * `events` holds `count` (<= 10) caller-created cudaEvent_t handles passed as
 * void*; NULL entries are skipped.  events == NULL or count == 0 turns the
 * instrumentation off.  The array is copied; the events stay caller-owned.
 * Returns FLP_ERR_INVALID_ARG when count is outside [0, 10].
 */
flp_status flp_set_phase_events(void* const* events, int count);

/*
 * Self-test of the kernels' bounded waits (a diagnostic; the pages have no
 * counterpart).  Runs the forward (tile kernel, then the split merge) on a
 * small internal problem (M = 256, H = 256, V = 512, all-zero inputs, targets
 * 0) laid out in `workspace` (caller-owned device memory of at least
 * FLP_SELFTEST_WORKSPACE_BYTES).  With stall_after >= 0 the TMA producers
 * stop after that many pipeline stages, so the MMA issuer waits for data that
 * never arrives: every wait gives up after wait_limit_ns, the kernel records
 * FLP_ERR_TIMEOUT in the error word, lets its copies and MMAs in flight
 * finish, frees its TMEM and returns; nothing faults and the context stays
 * usable.  The merge then finds the timeout bit and writes NaN to every
 * output.  With stall_after < 0 the same launches run normally (every row:
 * lse = entropy = log 512, logprob = -log 512).  The outputs, fp32 logprob,
 * lse and entropy of the 256 rows one after the other, are left in the
 * workspace at byte offset FLP_SELFTEST_OUTPUT_OFFSET.  Synchronises `stream`
 * and returns the error word (FLP_ERR_TIMEOUT, or FLP_OK), or an argument /
 * CUDA error.
 */
#define FLP_SELFTEST_WORKSPACE_BYTES (1u << 20)
#define FLP_SELFTEST_OUTPUT_OFFSET (768u << 10)
flp_status flp_selftest_wait_timeout(void* workspace, size_t workspace_bytes, int stall_after,
                                     int64_t wait_limit_ns, void* stream);

/*
 * Self-test of the fused backward schedule's dependency waits (a diagnostic;
 * the pages have no counterpart).  Runs one fused-schedule launch of the
 * backward kernel on a small internal all-zero problem (M = H = V = 256)
 * laid out in `workspace` (at least FLP_SELFTEST_WORKSPACE_BYTES).  With
 * broken != 0 the schedule holds only the dX tile, whose wait for its dZ tile
 * can never be met: the wait gives up after wait_limit_ns, the kernel records
 * FLP_ERR_TIMEOUT, winds down (bounded) and returns; nothing faults and the
 * context stays usable.  With broken == 0 the full schedule runs normally.
 * Synchronises `stream` and returns the error word (FLP_ERR_TIMEOUT or
 * FLP_OK), or an argument / CUDA error.
 */
flp_status flp_selftest_dependency_timeout(void* workspace, size_t workspace_bytes, int broken,
                                           int64_t wait_limit_ns, void* stream);

/*
 * The same self-test for the backward's dZ kernel (the split and
 * vocabulary-split schedules' dZ launch; a diagnostic, the pages have no
 * counterpart): one 256 x 512 dZ tile of a small internal all-zero problem
 * (M = 256, H = 256, V = 512) laid out in `workspace` (at least
 * FLP_SELFTEST_WORKSPACE_BYTES).  With stall_after >= 0 its TMA producers
 * stop after that many pipeline stages: the MMA issuer's wait gives up after
 * wait_limit_ns, the kernel records FLP_ERR_TIMEOUT, its epilogue warps stop
 * together (a vote before any store barrier), it winds down (bounded) and
 * returns; nothing faults and the context stays usable.  With
 * stall_after < 0 the tile runs normally.  Synchronises `stream` and returns
 * the error word (FLP_ERR_TIMEOUT or FLP_OK), or an argument / CUDA error.
 */
flp_status flp_selftest_dz_wait_timeout(void* workspace, size_t workspace_bytes, int stall_after,
                                        int64_t wait_limit_ns, void* stream);

/* ------------------------------------------------------------------------
 * Training-step operators beside the head: the norm that makes its hidden
 * states, 8-bit checkpoints of activations and their use in the backward
 * pass, and the balance loss of a mixture-of-experts router.  They follow the
 * conventions above (asynchronous on `stream`, caller-owned memory,
 * deterministic, argument errors returned before any launch) except that rows
 * may have a pitch (ld*, in elements, at least the width) and any width and
 * alignment: rows move as 16-byte vectors where base, pitch and width allow,
 * else as 4-byte words.  Every pointer is aligned to its elements.
 */

/*
 * Layer norm over the last dimension of X [M, H] (bf16 or fp32, dtype):
 *   mean = sum_j x_j / H, rstd = (sum_j (x_j - mean)^2 / H + eps)^(-1/2),
 *   y_j  = (x_j - mean) rstd weight_j + bias_j          (fp32, rounded once)
 * Y has X's type.  weight and bias ([H], param_dtype) may be NULL (1 and 0),
 * mean and rstd (fp32 [M]) may be NULL (not written).  With q and scale
 * non-NULL the call also writes the 8-bit checkpoint of X (flp_checkpoint_pack)
 * from the same read.  Y may be X itself.  H <= 16384, else
 * FLP_ERR_UNSUPPORTED.
 */
flp_status flp_layer_norm(const void* X, int64_t ldx, int dtype, const void* weight, const void* bias,
                          int param_dtype, int64_t M, int64_t H, float eps, void* Y, int64_t ldy,
                          float* mean, float* rstd, void* q, void* scale, void* stream);

/* Workspace bytes of flp_layer_norm_backward on the current device (0 for few rows). */
flp_status flp_layer_norm_workspace(int64_t M, int64_t H, size_t* bytes);

/*
 * Layer norm backward, with xh = (x - mean) rstd and g = dy weight:
 *   dx = rstd (g - sum(g) / H - xh sum(g xh) / H)    (the type of dY)
 *   dweight = sum over rows of dy xh,  dbias = sum over rows of dy   (fp32 [H])
 * The activations come as X (the type of dY) or as their checkpoint q, scale
 * (exactly one of the two); mean and rstd are the forward's.  dweight and
 * dbias may be NULL (with both NULL no workspace is needed).  M == 0 writes
 * zeros to them.  dX may be dY itself.
 */
flp_status flp_layer_norm_backward(const void* dY, int64_t lddy, const void* X, int64_t ldx, const void* q,
                                   const void* scale, int dtype, const void* weight, int param_dtype,
                                   const float* mean, const float* rstd, int64_t M, int64_t H, void* dX,
                                   int64_t lddx, float* dweight, float* dbias, void* workspace,
                                   size_t workspace_bytes, void* stream);

/*
 * 8-bit checkpoint of X [M, H].  Blocks are 32 consecutive columns of a row
 * (the last block of a row may be short).  With a the block's largest |x| and
 * E = floor(log2 a), its step is 2^max(E - 6, -126) and each element is kept as
 *   q = clamp(rint(x / step), -127, 127),        read back as q * step.
 *   q     : int8  [M, Hp], Hp = H rounded up to a multiple of 32, 16-byte
 *           aligned, zero in the columns past H
 *   scale : uint8 [M, Hp / 32], log2(step) + 127 (1..249)
 * The error is at most half a step (one step for fp32 values within half a
 * step of 2^(E+1), which are clamped).  A block with a NaN or an infinity gets
 * the byte 255 and reads back as NaN throughout, so that an overflow is not
 * lost.  Read back as bf16 or fp32 the values are exact.
 */
flp_status flp_checkpoint_pack(const void* X, int64_t ldx, int dtype, int64_t M, int64_t H, void* q,
                               void* scale, void* stream);
flp_status flp_checkpoint_unpack(const void* q, const void* scale, int64_t M, int64_t H, void* X,
                                 int64_t ldx, int dtype, void* stream);

/*
 * Weight gradient of a linear layer y = x W^T whose input x [M, K] was kept as
 * a checkpoint:  dW [N, K] (+)= dY^T x^,  dY bf16 [M, N], x^ the checkpoint's
 * values (exact in bf16), fp32 accumulation on the tensor cores.  dW is fp32
 * (added to when accumulate_dW != 0) or bf16 (overwritten; accumulating into
 * it is FLP_ERR_UNSUPPORTED), contiguous, 16-byte aligned.  M == 0 writes
 * zeros (or adds nothing).  The workspace's first word is the error word of
 * flp_get_error (FLP_ERR_TIMEOUT); after a timeout every tile of dW that was
 * not finished is NaN.  The workspace query takes dY for its
 * alignment only.
 */
flp_status flp_checkpoint_weight_grad_workspace(const void* dY, int64_t lddy, int64_t M, int64_t N,
                                                int64_t K, int dW_dtype, size_t* bytes);
flp_status flp_checkpoint_weight_grad(const void* dY, int64_t lddy, const void* q, const void* scale,
                                      int64_t M, int64_t N, int64_t K, void* dW, int dW_dtype,
                                      int accumulate_dW, void* workspace, size_t workspace_bytes,
                                      void* stream);

/*
 * Self-test of the contraction's bounded waits, like flp_selftest_wait_timeout
 * (a diagnostic): a weight gradient of M = 192, N = 136 and K = 520 (two tiles
 * of dW, one of 512 columns, written directly) or, with odd != 0, K = 521
 * (through partial tiles), all zeros, on one CTA pair in runs of one 64-row
 * block, laid out in `workspace` (at least FLP_SELFTEST_WEIGHT_GRAD_BYTES).
 * With stall_after >= 0 its TMA producers stop after that many blocks, of which
 * a tile has three.  The result, fp32 [N, K], is left at byte offset
 * FLP_SELFTEST_WEIGHT_GRAD_OUTPUT_OFFSET: zeros, or NaN where the stall kept a
 * tile from being finished (with odd, in every tile).  Synchronises `stream` and
 * returns the error word (FLP_ERR_TIMEOUT or FLP_OK), or an argument / CUDA error.
 */
#define FLP_SELFTEST_WEIGHT_GRAD_BYTES (3u << 20)
#define FLP_SELFTEST_WEIGHT_GRAD_OUTPUT_OFFSET (2u << 20)
flp_status flp_selftest_weight_grad_timeout(void* workspace, size_t workspace_bytes, int odd, int stall_after,
                                            int64_t wait_limit_ns, void* stream);

/*
 * Balance loss of a mixture-of-experts router over T tokens and E experts
 * (1 <= E <= 1024), the per-expert counts and the gradient by the logits:
 *   live row : mask[t] != 0 (mask NULL: every row) and some logit above -inf;
 *              N live rows, p_t = softmax(logits_t) on them
 *   chosen   : the top_k largest logits of a live row (equal logits: the lowest
 *              index first; -inf is never chosen, a row that holds a NaN or
 *              +inf chooses none), or experts[t, 0..top_k) when experts is
 *              non-NULL (values outside [0, E) are dropped slots)
 *   c_e      = times expert e is chosen, C = sum_e c_e
 *   loss     = coef E sum_e (c_e / C) (sum_t p_te / N)   (coef when the load is
 *              even; 0 when N or C is 0 and no live row holds a NaN or +inf)
 *   grad_te  = coef E / (N C) p_te (c_e - sum_f c_f p_tf), 0 on other rows
 * The counts are constants of the gradient.  logits: bf16 or fp32 [T, E] at
 * pitch ld; mask: bytes [T]; experts: int64 [T, top_k]; loss: one fp32; grad:
 * the logits' type, contiguous [T, E], or NULL; counts: int64 [E].  A NaN or
 * +inf in a live row makes the loss and that row's gradient NaN, whether or not
 * anything is chosen; what masked rows hold is not looked at.  Few rows need no workspace (the query says 0).
 */
flp_status flp_balance_loss_workspace(int64_t T, int64_t E, size_t* bytes);
flp_status flp_balance_loss(const void* logits, int64_t ld, int dtype, const uint8_t* mask,
                            const int64_t* experts, int64_t T, int64_t E, int64_t top_k, float coef,
                            float* loss, void* grad, int64_t* counts, void* workspace,
                            size_t workspace_bytes, void* stream);
/* The same with the gradient in the logits' type or in fp32 (grad_dtype): for a
 * gradient that is multiplied by an upstream one before it is rounded. */
flp_status flp_balance_loss_ex(const void* logits, int64_t ld, int dtype, const uint8_t* mask,
                               const int64_t* experts, int64_t T, int64_t E, int64_t top_k, float coef,
                               float* loss, void* grad, int grad_dtype, int64_t* counts, void* workspace,
                               size_t workspace_bytes, void* stream);

/*
 * Tokens sorted by expert.  T tokens choose k experts each; slot t k + j is
 * token t's j-th choice.  experts: int64 [T, k], values outside [0, E) are
 * dropped slots (1 <= E <= 1024, k <= 2^30, T k < 2^31).  A stable counting sort, dropped
 * slots last:
 *   rows    int32 [T, k]  the position of every slot
 *   slots   int32 [T k]   the slot at every position
 *   counts  int64 [E]     slots of each expert
 *   offsets int64 [E + 1] where each expert's positions begin; offsets[E] is the
 *                         number of slots that were not dropped
 * The same expert may be chosen more than once by a token.  Few slots need no
 * workspace (the query says 0).
 */
flp_status flp_expert_sort_workspace(int64_t T, int64_t k, int64_t E, size_t* bytes);
flp_status flp_expert_sort(const int64_t* experts, int64_t T, int64_t k, int64_t E, int32_t* rows, int32_t* slots,
                           int64_t* counts, int64_t* offsets, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Rows brought to the experts and back, by the sort's rows and its
 * total = &offsets[E] (on the device):
 *   gather             XS[rows[t, j]] = X[t]; positions from total on get zeros
 *   combine            Y[t] = sum_j weights[t, j] YS[rows[t, j]] over the positions
 *                      below total (fp32, in the order of j, rounded once; 0 if none)
 *   combine backward   dYS[rows[t, j]] = weights[t, j] dY[t], zeros from total on
 *                      dweights[t, j] = <dY[t], YS[rows[t, j]]>, 0 for dropped slots
 * X, Y, dY: [T, H]; XS, YS, dYS: [T k, H], bf16 or fp32 (dtype).  What rows of
 * YS from total on hold is not looked at.  weights: [T, k] in weight_dtype, or
 * NULL: 1 (combine without weights is the gradient of gather).  dweights: fp32,
 * or NULL (YS is then not read and may be NULL).  An entry of rows that is no
 * position is passed over.  Inputs and outputs must not overlap.
 */
flp_status flp_expert_gather(const void* X, int64_t ldx, int dtype, int64_t T, int64_t H, int64_t k,
                             const int32_t* rows, const int64_t* total, void* XS, int64_t ldxs, void* stream);
flp_status flp_expert_combine(const void* YS, int64_t ldys, int dtype, const void* weights, int weight_dtype,
                              int64_t T, int64_t H, int64_t k, const int32_t* rows, const int64_t* total, void* Y,
                              int64_t ldy, void* stream);
flp_status flp_expert_combine_backward(const void* dY, int64_t lddy, const void* YS, int64_t ldys, int dtype,
                                       const void* weights, int weight_dtype, int64_t T, int64_t H, int64_t k,
                                       const int32_t* rows, const int64_t* total, void* dYS, int64_t lddys,
                                       float* dweights, void* stream);

/*
 * Log-probabilities of given tokens from logits [M, V] in memory (bf16 or fp32,
 * row pitch ld): with z = scale * logits (scale > 0, finite),
 *   lse = log sum_j exp(z_j),   logprob = z_y - lse,
 *   entropy = lse - sum_j p_j z_j,   p_j = exp(z_j - lse)      (fp32 [M])
 * entropy may be NULL.  The `top` largest logits of each row (0 <= top <=
 * min(V, 32); equal ones by their column, lowest first) are written as
 * top_logprob [M, top] (fp32, z - lse) and top_index [M, top] (int64).  -inf is
 * never among them: where fewer are left, the value is -inf and the index -1.
 * An ignored row (target == ignore_index) has logprob = entropy = 0; its lse and
 * alternatives are still written.  Any other target outside [0, V) gives
 * logprob = NaN.  A row with a NaN or +inf gives NaN (and index -1) throughout;
 * a row with nothing above -inf gives lse = logprob = -inf and entropy 0.
 * No workspace is needed.
 */
flp_status flp_token_logprob(const void* logits, int64_t ld, int dtype, const int64_t* targets, int64_t M,
                             int64_t V, int64_t ignore_index, float scale, float* logprob, float* lse,
                             float* entropy, int64_t top, float* top_logprob, int64_t* top_index, void* stream);

/*
 * Its gradient by the logits, from the forward's lse and entropy:
 *   dlogits_j = scale [ g_lp (1[j = y] - p_j) - g_ent p_j (z_j - lse + entropy) ]
 * in the logits' type (dlogits may be logits itself).  grad_logprob and
 * grad_entropy (fp32 [M]) may be NULL: 0; grad_entropy needs entropy.  Ignored
 * rows and rows of lse = -inf get zeros; a target outside [0, V) has no 1[j = y].
 */
flp_status flp_token_logprob_backward(const void* logits, int64_t ld, int dtype, const int64_t* targets, int64_t M,
                                      int64_t V, int64_t ignore_index, float scale, const float* lse,
                                      const float* entropy, const float* grad_logprob, const float* grad_entropy,
                                      void* dlogits, int64_t lddl, void* stream);

/*
 * Linear layer with its epilogue, bf16 x [M, K], W [N, K] and y [M, N] (rows at
 * any pitch and alignment; rows of X or W that are not aligned to 16 bytes are
 * copied to the workspace first):
 *   v = x W^T + bias,   y = act(v) + residual
 * in fp32 up to one rounding (contractions above 131072 as fp32 sums of shorter runs;
 * those of more than 2^22 runs of 256 x 256 outputs are refused).  bias: [N], bf16 or
 * fp32 (bias_dtype), or NULL; residual: [M, N] bf16, or NULL (Y may be the residual
 * itself; the outputs overlap nothing else); pre: v rounded to bf16, for the backward
 * pass, or NULL.  Activations: relu, gelu (v Phi(v)),
 * gelu_tanh (v / 2 (1 + tanh(sqrt(2 / pi) (v + 0.044715 v^3)))), silu (v sigmoid(v)).
 * At v = -inf they are 0, 0 (the limit), NaN and NaN (the products).
 * The workspace query takes X and W for their alignment only and may say 0.  A
 * kernel's bounded wait that runs out leaves NaN in every tile of the outputs that
 * was not finished.
 */
typedef enum { FLP_ACT_NONE = 0, FLP_ACT_RELU = 1, FLP_ACT_GELU = 2, FLP_ACT_GELU_TANH = 3, FLP_ACT_SILU = 4 } flp_activation;
flp_status flp_linear_workspace(const void* X, int64_t ldx, const void* W, int64_t ldw, int64_t M, int64_t N, int64_t K,
                                size_t* bytes);
flp_status flp_linear(const void* X, int64_t ldx, const void* W, int64_t ldw, const void* bias, int bias_dtype,
                      int activation, const void* residual, int64_t ldr, int64_t M, int64_t N, int64_t K, void* Y,
                      int64_t ldy, void* pre, int64_t ldpre, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Its gradients, with d = dY act'(pre) (pre as the forward kept it; not read
 * without an activation; relu' is 1 for v > 0 and else 0, the others' slopes are 0 at
 * -inf and 1 at inf):
 *   dX = d W (bf16),   dW [N, K] = d^T X (fp32 or bf16, contiguous, 16-byte
 *   aligned),   dbias [N] = column sums of d (fp32)
 * d enters the two products rounded to bf16 (2^-8 of it; where that changes it, as the
 * sum of two bf16 numbers, 2^-16 of it, for an fp32 dW, and for both where M <= 64) and
 * dbias unrounded.  The _ex forms take the choice: d_terms 0 is this rule, 1 one number
 * in both products, 2 two numbers in both (twice the operations; M <= 2^29).
 * An infinite d makes its row of dX and of dW infinite as in the formulas; an infinite X
 * or W meets both numbers, and may leave NaN where the formula has an infinity.
 * Each output may be NULL: it is not computed, and X (for dW) or W (for dX) is not
 * read.  No output overlaps an input.  The residual's gradient is dY.  M == 0 writes zeros to dW and dbias.  The
 * workspace's first word is the error word of flp_get_error (FLP_ERR_TIMEOUT);
 * after a timeout what was not finished is NaN.
 */
flp_status flp_linear_backward_workspace(const void* dY, int64_t lddy, const void* X, int64_t ldx, const void* W, int64_t ldw,
                                         int activation, int want_dX, int want_dW, int want_dbias, int64_t M, int64_t N,
                                         int64_t K, int dW_dtype, size_t* bytes);
flp_status flp_linear_backward(const void* dY, int64_t lddy, const void* X, int64_t ldx, const void* W, int64_t ldw,
                               const void* pre, int64_t ldpre, int activation, int64_t M, int64_t N, int64_t K, void* dX,
                               int64_t lddx, void* dW, int dW_dtype, float* dbias, void* workspace, size_t workspace_bytes,
                               void* stream);
flp_status flp_linear_backward_workspace_ex(const void* dY, int64_t lddy, const void* X, int64_t ldx, const void* W, int64_t ldw,
                                            int activation, int d_terms, int want_dX, int want_dW, int want_dbias, int64_t M,
                                            int64_t N, int64_t K, int dW_dtype, size_t* bytes);
flp_status flp_linear_backward_ex(const void* dY, int64_t lddy, const void* X, int64_t ldx, const void* W, int64_t ldw,
                                  const void* pre, int64_t ldpre, int activation, int d_terms, int64_t M, int64_t N, int64_t K,
                                  void* dX, int64_t lddx, void* dW, int dW_dtype, float* dbias, void* workspace,
                                  size_t workspace_bytes, void* stream);

/*
 * Self-test of the product's bounded waits, like flp_selftest_wait_timeout (a
 * diagnostic): M = 192, N = 520, K = 192 (two tiles of three 64-deep blocks), all
 * zeros, on one CTA pair, laid out in `workspace` (at least
 * FLP_SELFTEST_LINEAR_BYTES); with form 1 through partial tiles of one block, with
 * form 2 in the tiles of few rows, with form 3 in those split over three CTAs of a
 * block each.  With stall_after >= 0 the TMA producers stop after that many blocks.  y, bf16
 * [M, N], is left at byte offset FLP_SELFTEST_LINEAR_OUTPUT_OFFSET: zeros, or NaN
 * where the stall kept a tile from being finished.  Synchronises `stream` and
 * returns the error word (FLP_ERR_TIMEOUT or FLP_OK), or an argument / CUDA error.
 */
#define FLP_SELFTEST_LINEAR_BYTES (4u << 20)
#define FLP_SELFTEST_LINEAR_OUTPUT_OFFSET (3u << 20)
flp_status flp_selftest_linear_timeout(void* workspace, size_t workspace_bytes, int form, int stall_after,
                                       int64_t wait_limit_ns, void* stream);

/* Static description of a status code. */
const char* flp_status_string(flp_status status);

/* Text of the last FLP_ERR_CUDA / FLP_ERR_UNSUPPORTED on the calling thread. */
const char* flp_last_error_message(void);

#ifdef __cplusplus
}
#endif

#endif /* FLP_H */
