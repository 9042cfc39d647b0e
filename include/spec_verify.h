/*
 * spec_verify.h - C ABI of the batched draft-verification library (sm_103a).
 *
 * The operation is speculative-decoding verification as described on the
 * AngelSpec / DFly pages (agifrontier tutorial, section "KL to end-to-end
 * TV loss"; abstract; section on verification as a shared batch-level pool):
 *
 *   p_k = softmax(z_T[b,k,:] / T),  q_k = softmax(z_D[b,k,:] / T)
 *   alpha_k = sum_v min(p_k(v), q_k(v)) = 1 - TV(p_k, q_k)
 *   c_m = prod_{k<=m} alpha_k,   E = sum_{m<K} c_m (expected accepted drafts)
 *   serial test at k = 0..d_b-1:  accept x_k iff u[b,k] * q_k(x_k) < p_k(x_k);
 *   the first rejection at n emits a draw from norm(max(0, p_n - q_n)),
 *   full acceptance emits a bonus draw from p_{d_b};
 *   T == 0: accept iff x_k == argmax z_T[b,k] (lowest index on ties); the
 *   emitted token is the target argmax at the first mismatch or at d_b.
 * Draws use the inverse CDF in vocabulary order: the smallest v whose
 * inclusive prefix mass is strictly above u[b,K] * (total mass).
 * The budget spends N verified positions on the N best prefix confidences
 * c[b,m] over the whole batch (order: c desc, m asc, b asc), which is
 * prefix-closed and yields a per-request depth d_b.
 *
 * Conventions for every entry point
 * - Pointers named *_logits, tokens, uniforms, depth, out_* and workspace
 *   are DEVICE pointers (cudaMalloc / torch CUDA memory) on the current
 *   device; tensors are dense row-major: target [B, K+1, V], draft [B, K, V],
 *   tokens [B, K] int32, uniforms [B, K+1] float32, outputs as stated.
 * - The caller owns every buffer.  The library allocates no device memory,
 *   keeps no per-call state, and never synchronises the stream except in
 *   spec_get_status.  Every call is asynchronous on `stream` (a cudaStream_t
 *   passed as void*, NULL = legacy default stream).
 * - Argument errors are returned synchronously (nothing is launched).
 *   Data errors found on the device (a draft token outside [0, V), a wait
 *   that ran out) are recorded in a status word inside the workspace and
 *   read with spec_get_status.
 * - The workspace (at least spec_workspace_bytes) holds the status word,
 *   per-row intermediate records and per-row argmax slots that every call
 *   leaves zeroed.  Its layout depends only on ws_bytes: zero-fill it
 *   (spec_workspace_init) before its first use and again whenever the same
 *   buffer is passed with a different ws_bytes.  Calls that share a
 *   workspace must be ordered on one stream.
 * - Launches on `stream`: at T == 0 without a budget one kernel (the argmax,
 *   with the serial cut fused in); otherwise the row kernel and a small kernel
 *   (the serial cut, or the budget and the cut) chained to it with
 *   programmatic dependent launch.
 * - Logits may contain -inf (probability 0); each row needs one finite
 *   value.  NaN / +inf give unspecified tokens (they are not scanned for).
 * - Limits: 1 <= V <= 262144 (fp32 logits at T > 0: V <= 131072),
 *   0 <= K <= 31, B >= 0 (B == 0 is a no-op), T >= 0 and finite.
 */
#ifndef SPEC_VERIFY_H
#define SPEC_VERIFY_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  SPEC_OK = 0,
  SPEC_ERR_INVALID_ARG = 1,     /* bad pointer, size, dtype, temperature */
  SPEC_ERR_UNSUPPORTED = 2,     /* shape outside the limits above */
  SPEC_ERR_CUDA = 3,            /* a launch or runtime call failed */
  SPEC_ERR_DEVICE_TIMEOUT = 4,  /* a bounded on-device wait ran out */
  SPEC_ERR_TOKEN_RANGE = 5,     /* a draft token id outside [0, V) */
  SPEC_ERR_WORKSPACE = 6,       /* workspace too small or misaligned */
  SPEC_ERR_PAGE_RANGE = 7       /* a page id outside the cache, or a position beyond the page table */
} spec_status_t;

/* SPEC_F16: rope and attention only. */
typedef enum { SPEC_F32 = 0, SPEC_BF16 = 1, SPEC_F16 = 2 } spec_dtype_t;

/* Library version (major*10000 + minor*100 + patch). */
int spec_version(void);

/* Static text for a status code. */
const char* spec_error_string(int status);

/* Bytes of workspace a call with these sizes needs (256-byte aligned start). */
size_t spec_workspace_bytes(int B, int K, int V, int dtype);

/* Zero-fill a workspace once before its first use (cudaMemsetAsync). */
spec_status_t spec_workspace_init(void* workspace, size_t ws_bytes, void* stream);

/*
 * Read and clear the device status word of a workspace.  Synchronises
 * `stream`.  *out_status receives SPEC_OK, SPEC_ERR_DEVICE_TIMEOUT,
 * SPEC_ERR_TOKEN_RANGE or SPEC_ERR_PAGE_RANGE (the first of them found, in
 * that priority).  After SPEC_ERR_DEVICE_TIMEOUT re-initialise the
 * workspace before reuse.
 */
spec_status_t spec_get_status(void* workspace, void* stream, int32_t* out_status);

/*
 * Verify an MTP chain (K = drafting depth).  Serial acceptance, first
 * rejection cut, residual / bonus draw (AngelSpec pages, "KL to end-to-end
 * TV loss": alpha = 1 - TV and the multiplicative, serial acceptance).
 *
 *   target_logits [B, K+1, V] dtype; row K is the bonus position.
 *   draft_logits  [B, K, V] dtype; may be NULL iff temperature == 0 and
 *                 out_alpha == NULL.
 *   tokens        [B, K] int32 drafted ids.
 *   uniforms      [B, K+1] float32 in [0, 1); u[b,k] tests position k,
 *                 u[b,K] drives the final draw.  Ignored at T == 0 (may be
 *                 NULL then).
 *   temperature   T > 0 stochastic, T == 0 greedy; negative or NaN ->
 *                 SPEC_ERR_INVALID_ARG.
 *   depth         [B] int32 in [0, K] (e.g. from spec_alloc_budget) or NULL
 *                 (= K): positions >= depth[b] are not tested and the bonus
 *                 is drawn at depth[b].  Values outside [0, K] are clamped.
 *   out_tokens    [B, K+1] int32: accepted drafts, then the emitted token,
 *                 then -1.
 *   out_accepted  [B] int32: number n_b of accepted drafts (emitted = n+1).
 *   out_alpha     [B, K] float32 or NULL (at T == 0: 1 if the argmaxes of
 *                 target and draft agree, else 0).
 */
spec_status_t spec_verify_chain(const void* target_logits, const void* draft_logits, int dtype,
                                const int32_t* tokens, const float* uniforms,
                                int B, int K, int V, float temperature,
                                const int32_t* depth,
                                int32_t* out_tokens, int32_t* out_accepted, float* out_alpha,
                                void* workspace, size_t ws_bytes, void* stream);

/*
 * Verify a DFly block (K = block size) with the same rule as the chain
 * (block drafts are accepted left to right, AngelSpec pages, DFly section),
 * plus the block statistics and, optionally, the batch-level budget:
 *
 *   out_cum_alpha    [B, K] float32 prod_{k<=m} alpha_k, or NULL.
 *   out_expected_len [B] float32 sum_m prod_{k<=m} alpha_k, or NULL
 *                    (the L_e2e summand of the "KL to end-to-end TV loss"
 *                    section).
 *   budget_N         < 0: no budget (depth as in spec_verify_chain);
 *                    >= 0: spend N verified positions over the batch on the
 *                    best prefix confidences (the D-cut shared pool, section
 *                    on verification as a shared batch-level resource); the
 *                    depth argument must then be NULL.  The logits are read
 *                    once: alpha of every position, the budget and the
 *                    decisions come from that one pass.
 *   out_depth        [B] int32 chosen depth d_b, or NULL.
 * B * K <= 8192 when budget_N >= 0.  draft_logits is required when
 * budget_N >= 0 (alpha needs it, also at T == 0).
 */
spec_status_t spec_verify_block(const void* target_logits, const void* draft_logits, int dtype,
                                const int32_t* tokens, const float* uniforms,
                                int B, int K, int V, float temperature,
                                const int32_t* depth, int budget_N,
                                int32_t* out_tokens, int32_t* out_accepted, float* out_alpha,
                                float* out_cum_alpha, float* out_expected_len, int32_t* out_depth,
                                void* workspace, size_t ws_bytes, void* stream);

/*
 * Overlap statistics only (no decisions): alpha_k for k < K, the prefix
 * confidences and the expected accepted length (AngelSpec pages, "KL to
 * end-to-end TV loss", inline formula and L_e2e summand).  Reads target
 * rows 0..K-1 of the [B, K+1, V] tensor and the [B, K, V] draft tensor.
 * out_alpha [B, K] required; out_cum_alpha [B, K] and out_expected_len [B]
 * may be NULL.  T == 0 gives the one-hot limit.
 */
spec_status_t spec_overlap_alpha(const void* target_logits, const void* draft_logits, int dtype,
                                 int B, int K, int V, float temperature,
                                 float* out_alpha, float* out_cum_alpha, float* out_expected_len,
                                 void* workspace, size_t ws_bytes, void* stream);

/*
 * Batch-level verification budget (AngelSpec abstract and the section on
 * verification as a shared batch-level resource): alpha [B, K] (device,
 * float32; clamped to [0, 1], NaN read as 0) -> prefix confidences
 * c[b,m] = prod_{k<=m} alpha[b,k]; the first min(N, B*K) keys in the order
 * (c desc, m asc, b asc) are selected; out_depth[b] = number selected in
 * row b (prefix-closed).  out_conf [B, K] may be NULL.  N >= 0.
 * B * K <= 8192.  Needs no workspace contents beyond its status word.
 */
spec_status_t spec_alloc_budget(const float* alpha, int B, int K, int budget_N,
                                int32_t* out_depth, float* out_conf,
                                void* workspace, size_t ws_bytes, void* stream);

/*
 * The budget with N chosen online (AngelSpec, section on verification as a
 * shared pool: verification is spent where it pays against a profiled cost
 * of verifying more positions).  With the keys and selection of
 * spec_alloc_budget and S(N) the sum of the N largest prefix confidences,
 * N = the first N in 0 .. B*K maximising
 *     (B + S(N)) / cost(B + N),
 * B + N being the positions the batch verifies (every request verifies its
 * first emitted position).  cost is the table (cost_n [n_cost] strictly
 * increasing, cost_t [n_cost]; device, float32) interpolated piecewise-
 * linearly and held constant beyond its ends.  1 <= n_cost <= 64.
 * out_N (device int32, nullable) receives N; out_depth and out_conf as in
 * spec_alloc_budget.  B * K <= 8192.
 */
spec_status_t spec_alloc_budget_adaptive(const float* alpha, int B, int K,
                                         const float* cost_n, const float* cost_t, int n_cost,
                                         int32_t* out_N, int32_t* out_depth, float* out_conf,
                                         void* workspace, size_t ws_bytes, void* stream);

/*
 * The budget chosen from the draft alone, before the target runs (AngelSpec,
 * section on verification as a shared pool: the budget is decided from the
 * draft model's output distribution).  The confidence of drafted position
 * (b, k) is q_k(x_k) = softmax(draft_logits[b, k] / T)[tokens[b, k]] (at
 * T == 0 the one-hot [tokens[b, k] == argmax], lowest index on ties; 0 for a
 * token outside [0, V)), and the keys are its prefix products
 * c[b, m] = prod_{k<=m} q_k(x_k), selected as in spec_alloc_budget: with
 * n_cost == 0 the first min(budget_N, B*K) keys (budget_N >= 0), with
 * n_cost > 0 the N of spec_alloc_budget_adaptive (budget_N ignored).
 *   draft_logits  device [B, K, V], dtype SPEC_BF16 or SPEC_F32; one pass
 *   tokens        device int32 [B, K]
 *   out_N         device int32 or NULL: the N spent
 *   out_depth     device int32 [B]: per-request verification depth d_b
 *   out_conf      device float32 [B, K] or NULL: the prefix confidences
 * The caller then runs the target on the selected depths and verifies with
 * spec_verify_chain / spec_verify_block and `depth`.  B * K <= 8192.
 * Workspace as for spec_verify_block (spec_workspace_bytes(B, K, V, dtype)).
 */
spec_status_t spec_draft_budget(const void* draft_logits, int dtype, const int32_t* tokens,
                                int B, int K, int V, float temperature, int budget_N,
                                const float* cost_n, const float* cost_t, int n_cost,
                                int32_t* out_N, int32_t* out_depth, float* out_conf,
                                void* workspace, size_t ws_bytes, void* stream);

/*
 * Greedy (T == 0) chain verification that allocates nothing and needs no
 * workspace.  The pages have no counterpart: this entry point exists for
 * callers that cannot give the library device memory -- serving engines that
 * reserve all device memory up front in their own pool and expose no
 * allocator, and hosts that forbid cudaMalloc / cudaFree after start-up
 * because those calls can synchronise the whole device.
 *
 * Same result as spec_verify_chain at temperature 0 (tokens, accepted
 * counts, one-hot alpha when out_alpha is given; draft_logits needed only
 * then).  Its scratch (status word, argmax slots, request counters) is one
 * fixed device array of 80.25 KiB inside the library, held by every GPU that
 * loads it until the process exits:
 * - B * (K + 1) <= SPEC_STATIC_MAX_ROWS (4096), else SPEC_ERR_UNSUPPORTED;
 * - every call looks up the array's device address in the current device's
 *   context (cudaGetSymbolAddress); the first call on a device may load the
 *   module, so make it before any stream capture;
 * - every call clears the parts it uses (cudaMemsetAsync) and shares the one
 *   array, so calls that overlap on the GPU (other streams, other threads)
 *   race: order them on one stream;
 * - out_status (device int32, nullable) receives the raw status bits of the
 *   call: 1 = a bounded wait ran out, 2 = a draft token outside [0, V).
 * It calls no cudaMalloc, cudaFree or allocating library routine.
 */
#define SPEC_STATIC_MAX_ROWS 4096
spec_status_t spec_verify_chain_greedy_static(const void* target_logits, const void* draft_logits, int dtype,
                                              const int32_t* tokens, int B, int K, int V,
                                              const int32_t* depth, int32_t* out_tokens,
                                              int32_t* out_accepted, float* out_alpha,
                                              int32_t* out_status, void* stream);

/*
 * Test and tuning knobs of one call (no process-wide settings exist).  A
 * zero-filled struct means the defaults everywhere.
 *   wait_limit_us   0: default wall-time limit of every bounded on-device wait
 *                   (200 ms, read from the GPU's global timer); > 0: that
 *                   limit; < 0: every such wait gives up at once, which sets
 *                   SPEC_ERR_DEVICE_TIMEOUT in the status word (the kernel
 *                   then waits once more, up to 100 ms, so its copies and
 *                   cluster exchanges still complete before it returns).
 *   cluster         T > 0: CTAs per row of the sampling kernel (1, 2, 4, 8 or
 *                   16; a CTA's slice of a row must fit 6 items of 16 KB,
 *                   else SPEC_ERR_UNSUPPORTED); 0: chosen per call shape.
 *   greedy_variant  T == 0: bit 1 runs the cut in its own kernel instead of
 *                   fusing it into the argmax kernel; bit 2 launches every
 *                   resident CTA slot with the tiles spread evenly.
 *   split_event     a cudaEvent_t (as void*) or NULL: recorded on the stream
 *                   between the row kernel and the kernel chained after it
 *                   (which is then launched without programmatic dependent
 *                   launch), so a caller can time the two apart.
 *   plan_out        host int32[8] or NULL: receives the launched plan,
 *                   sampling kernel {threads, cluster, clusters launched, max
 *                   co-resident clusters, slice, items per slice, dynamic
 *                   shared memory bytes, flags};
 *                   argmax kernel {threads, 1, grid, resident CTAs, tile, 0,
 *                   0, -1}.
 */
typedef struct spec_tuning {
  long long wait_limit_us;
  int cluster;
  int greedy_variant;
  int32_t* plan_out;
  void* split_event;
} spec_tuning_t;

/*
 * spec_verify_block with per-call knobs (tuning may be NULL = defaults).
 * stats_only != 0 computes what spec_overlap_alpha computes (tokens,
 * uniforms, depth, budget_N, out_tokens, out_accepted and out_depth are then
 * ignored).  Same argument meaning, ownership and errors as those calls;
 * SPEC_ERR_INVALID_ARG for a cluster size that is not a power of two in
 * [1, 16].
 */
spec_status_t spec_verify_tuned(const void* target_logits, const void* draft_logits, int dtype,
                                const int32_t* tokens, const float* uniforms,
                                int B, int K, int V, float temperature,
                                const int32_t* depth, int budget_N, int stats_only,
                                int32_t* out_tokens, int32_t* out_accepted, float* out_alpha,
                                float* out_cum_alpha, float* out_expected_len, int32_t* out_depth,
                                void* workspace, size_t ws_bytes, void* stream,
                                const spec_tuning_t* tuning);

/* ------------------------------------------------------------------------
 * The operators around a verification: what produces the logits it reads and
 * the tokens it tests.  One speculative step is
 *   spec_sample_tokens  (the draft's tokens and their truncated logits)
 *   spec_rope_append    (positions of the K + 1 new tokens, cache write)
 *   spec_chunk_attention (the new tokens over the cache)
 *   spec_sample_tokens with out_filtered (the target's truncated logits)
 *   spec_verify_chain / spec_verify_block.
 * A rejected draft needs no undoing: the next step's kv_lens are shorter and
 * its tokens overwrite the slots.
 */

/*
 * A batch of requests over a paged cache.  New token n of request b
 * (cu_q[b] <= n < cu_q[b+1]) sits at position kv_lens[b] - (cu_q[b+1] - n)
 * of its request, whose token t is in page page_table[b][t / page_size],
 * slot t % page_size.  Device pointers; strides in elements, multiples of 16
 * bytes, as are the bases of k and v; a head's `dim` values are contiguous
 * (both [pages, page_size, heads, dim] and [pages, heads, page_size, dim]
 * are described by their strides).  Lengths are read on the device only.
 * kv_lens[b] counts the new tokens; 0 (an idle slot) and less than the
 * number of new tokens are allowed: the tokens before position 0 see
 * nothing and are not stored.  Positions are counted from kv_lens[b] also
 * where it is beyond table_width * page_size: the tokens that the table has no
 * page for are neither stored nor seen, and SPEC_ERR_PAGE_RANGE is set.  Page
 * ids are looked at only where a token is read or written; one outside
 * [0, pages) reads as zeros, is not written, and sets SPEC_ERR_PAGE_RANGE in
 * the status word.
 */
typedef struct spec_paged_batch {
  void* k;
  void* v;
  long long k_page, k_token, k_head;
  long long v_page, v_token, v_head;
  int pages, page_size, kv_heads, dim;
  const int32_t* page_table;     /* [batch, table_width], rows table_stride apart */
  long long table_stride;
  int table_width;
  int batch;
  const int32_t* kv_lens;        /* [batch] */
  const int32_t* cu_q;           /* [batch + 1], from 0, not decreasing */
  int tokens;                    /* new tokens: cu_q[batch] */
} spec_paged_batch_t;

/*
 * Workspace of spec_chunk_attention (256-byte aligned; status word first, so
 * spec_workspace_init and spec_get_status apply; nothing else in it outlives
 * a call).  Depends on the current device; 0 for sizes that are refused.
 */
size_t spec_attention_workspace_bytes(int dtype, int q_heads, int kv_heads, int dim, int max_q);

/*
 * Attention of the new tokens over the cache:
 *   out[n, h] = sum_t softmax_t(scale q[n, h] . k[t, g]) v[t, g],
 *   lse[n, h] = ln sum_t exp(scale q[n, h] . k[t, g]),  g = h / (q_heads / kv_heads)
 * over the keys t < kv_lens[b] with, for causal != 0, t <= position of n and,
 * for window > 0, t > position of n - window.  A row that sees no key gives
 * out = 0, lse = -inf.  Keys and values at or beyond kv_lens[b] are never
 * used (they may be anything); those before it must be finite, except in
 * pages that lie wholly behind the window of all the request's new tokens:
 * those are not looked at, nor are their ids.
 *   q         [tokens, q_heads, dim] with strides (multiples of 16 bytes)
 *   dtype     SPEC_BF16 or SPEC_F16, of q, k, v and out
 *   max_q     an upper bound of the new tokens per request (chooses the
 *             kernel; a wrong one costs speed, not results)
 *   out       [tokens, q_heads, dim] contiguous, 16-byte aligned
 *   out_lse   [tokens, q_heads] float32 or NULL
 * dim a multiple of 8, at most 256; q_heads a multiple of kv_heads.
 * Rows of tokens that no request has stay unwritten.  Results do not depend
 * on timing.  Two launches, the second chained by programmatic dependent
 * launch; threads may share a workspace whose calls go to one stream.  Waits inside the kernel are bounded (2 s); one that runs out sets
 * SPEC_ERR_DEVICE_TIMEOUT in the status word, and the outputs are then
 * unspecified.
 */
spec_status_t spec_chunk_attention(const void* q, long long q_token, long long q_head, int dtype, int q_heads,
                                   const spec_paged_batch_t* batch, int max_q, float scale, int causal, int window,
                                   void* out, float* out_lse, void* workspace, size_t ws_bytes, void* stream);

/*
 * spec_chunk_attention with tuning->wait_limit_us for the waits inside the
 * kernel (0: 2 s; < 0: the first wait gives up at once, and those that wait
 * for what it would have brought); the other knobs are the verification's and
 * are not read.  tuning may be NULL.  After a wait that ran
 * out the outputs are unspecified, and nothing else is written.
 */
spec_status_t spec_chunk_attention_tuned(const void* q, long long q_token, long long q_head, int dtype, int q_heads,
                                         const spec_paged_batch_t* batch, int max_q, float scale, int causal, int window,
                                         void* out, float* out_lse, void* workspace, size_t ws_bytes, void* stream,
                                         const spec_tuning_t* tuning);

/* New tokens of spec_rope_append; strides in elements, values of a head contiguous. */
typedef struct spec_rope_tensors {
  const void* q;        /* [tokens, q_heads, dim] */
  const void* k;        /* [tokens, kv_heads, dim] */
  const void* v;        /* [tokens, kv_heads, dim]; unused without a cache */
  void* q_out;          /* rotated queries; may be q */
  void* k_out;          /* rotated keys, or NULL (they go to the cache); may be k */
  long long q_token, q_head, k_token, k_head, v_token, v_head;
  long long q_out_token, q_out_head, k_out_token, k_out_head;
} spec_rope_tensors_t;

/*
 * Rotary positions: of the first rotary_dim values of every head of q and k,
 * pairs (x, y) = (j, j + rotary_dim/2), or (2j, 2j+1) if interleaved, become
 *   factor (x cos a - y sin a), factor (y cos a + x sin a),
 *   a = 2 pi position freq[j] / 2^64;
 * the values behind them are copied.  Rotated keys and the values v go to the
 * cache's slots (batch->k != NULL) and the rotated keys to k_out (if given).
 *   freq      device uint64 [rotary_dim / 2]: turns a position x 2^64
 *   dtype     SPEC_F32, SPEC_BF16 or SPEC_F16, of every tensor
 *   workspace as spec_chunk_attention's (status word only); may be NULL
 *             without a cache
 * dim at most 1024.  Rows of q_out and k_out of tokens that no request has
 * stay unwritten.  q_out and k_out overlap no input but q and k themselves,
 * with the same strides.  One launch.
 */
spec_status_t spec_rope_append(const spec_rope_tensors_t* t, int dtype, int q_heads, const spec_paged_batch_t* batch,
                               const unsigned long long* freq, int rotary_dim, float factor, int interleaved,
                               void* workspace, void* stream);

/* Sampling settings: a scalar each, or a device array of one per row where its pointer is not NULL. */
typedef struct spec_sampling {
  float temperature;             /* 0: greedy (a negative one is refused; in an array <= 0 is greedy) */
  int top_k;                     /* <= 0: all */
  float top_p;                   /* >= 1: all */
  float min_p;                   /* <= 0: all */
  const float* temperature_rows;
  const int32_t* top_k_rows;
  const float* top_p_rows;
  const float* min_p_rows;
} spec_sampling_t;

/*
 * Sampling from given uniforms.  A row's tokens are ordered by (logit
 * descending, index ascending); w = exp((z - max) / temperature).  Kept are
 * the first n = min(n_k, n_p, n_m), at least 1, of that order:
 *   n_k  top_k;
 *   n_p  the shortest prefix whose weight is >= top_p x the weight of the
 *        first n_k;
 *   n_m  the tokens with w >= min_p.
 * The token drawn is the first whose inclusive prefix weight is strictly
 * above uniforms[r] x the weight of the kept ones.  Temperature 0 (in an
 * array <= 0 or NaN) keeps the first token alone.
 *   logits       [rows, V] SPEC_BF16 or SPEC_F32, rows row_stride apart
 *   uniforms     [rows] float32 in [0, 1) (clamped to it)
 *   out_tokens   [rows] int32; -1 for a row without a logit above -inf
 *   out_probs    [rows] float32 or NULL: the drawn token's probability among
 *                the kept ones (0 for such a row)
 *   out_kept     [rows] int32 or NULL: n (0 for such a row)
 *   out_filtered [rows, V] of the logits' type, rows filtered_stride apart,
 *                or NULL: the kept tokens' logits, -inf elsewhere (what the
 *                verification calls take as the truncated distribution, at
 *                their one temperature for the batch); must not overlap
 *                logits
 * NaN logits count as -inf.  Weights are in units of 2^-44 of the largest:
 * nearer ones than that are equal, min_p's too, and a probability is exact to
 * 2^-45 / (weight of the kept ones) or fp32's rounding.  Their sums are exact
 * integers, so results do not depend on timing.  V <= 262144.  One launch, no
 * workspace.
 */
spec_status_t spec_sample_tokens(const void* logits, long long row_stride, int dtype, int rows, int V,
                                 const float* uniforms, const spec_sampling_t* how, int32_t* out_tokens,
                                 float* out_probs, int32_t* out_kept, void* out_filtered, long long filtered_stride,
                                 void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_VERIFY_H */
