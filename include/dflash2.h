/*
 * dflash2.h -- C ABI of the DFlash 2 draft-selection + verify path on one GPU.
 *
 * The DFlash 2 proposer keeps the 16 best candidates of every drafted
 * position, scores adjacent candidate pairs with a low-rank bilinear term
 * gated by the drafter's hidden state, walks those scores once to pick the
 * proposed path, and the verify accepts drafted tokens with probability
 * min(1, p/q) and resamples a rejected one from max(0, p - q).  Sources:
 *   [P] "qwen3/dflash: DFlash 2 proposer -- top-16 path selector + two-tap
 *       dynamic convolution" (pegainfer issue 930): "What upstream shipped"
 *       items 1-2, "Proposal" phases 1-3.
 *   [F] FreeToken PR 857 (DFlash 2 next to MTP): "Details" (Runtime, Sampled
 *       verify, Refused at startup), "Tests added or changed", "Known gaps".
 *
 * Conventions shared by every entry point
 *   - Tensor arguments are DEVICE pointers owned by the caller, row-major and
 *     16-byte aligned.  Nothing here allocates, frees or synchronises: each
 *     call enqueues its kernels on `stream` and returns.
 *   - A call returns DFLASH2_ERR_INVALID_ARG before launching anything when an
 *     argument is out of range (see each call); DFLASH2_ERR_CUDA when a launch
 *     fails (the CUDA error is left for cudaGetLastError).
 *   - Per-request data problems never abort a batch: they are reported per
 *     request in `status` (DFLASH2_ST_*) or as -1 / NaN outputs.
 *   - Workspaces (`ws`) are caller-provided device buffers of at least the
 *     size returned by the matching *_workspace_bytes function.  They must be
 *     zero-filled once before first use.  A call needs zeros only where it
 *     counts (its tickets and marks) and leaves zeros there; behind them it
 *     leaves its scratch.  So a workspace is for calls of one kind: the scans
 *     and the fused LM head (dflash2_topk16, _shard, dflash2_verify,
 *     dflash2_lmhead_topk16) keep one workspace per entry point and set of
 *     sizes (rows, V, or B and K), and dflash2_paged_attn and dflash2_kv_evict
 *     may share one, for calls of any sizes that it is large enough for.
 *     Zero-fill a workspace before it goes to another kind of call.  After a call that returned DFLASH2_ERR_CUDA, or after
 *     dflash2_device_error reported a nonzero code (a kernel gave up on a
 *     bounded wait), zero-fill the workspaces of the calls involved again
 *     before reusing them.  Two calls that share a workspace must not run
 *     concurrently.
 *   - The first call on a device performs one-time set-up (device attributes,
 *     kernel attributes); make it before any stream capture.  Later calls are
 *     capturable into CUDA graphs.
 *   - Ties in logits are broken by the lower token id everywhere.
 */
#ifndef DFLASH2_H
#define DFLASH2_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t; NULL is the legacy default stream. */
typedef struct CUstream_st *dflash2_stream;

typedef enum {
    DFLASH2_OK = 0,
    DFLASH2_ERR_INVALID_ARG = 1,
    DFLASH2_ERR_UNSUPPORTED = 2,
    DFLASH2_ERR_CUDA = 3,
    DFLASH2_ERR_WORKSPACE = 4
} dflash2_status;

typedef enum { DFLASH2_F32 = 0, DFLASH2_BF16 = 1 } dflash2_dtype;

/* Per-request verify status. */
enum {
    DFLASH2_ST_OK = 0,
    DFLASH2_ST_NAN = 1,         /* NaN or +Inf (or no value above -Inf) in a target row; NaN, Inf or
                                   a negative value in a q row */
    DFLASH2_ST_BAD_Q = 2,       /* a q row does not sum to 1 within 1e-3, or a drafted token is not
                                   the candidate at its slot */
    DFLASH2_ST_BAD_PARAMS = 3,  /* temperature < 0 or not finite, top_k < 0, top_p outside (0, 1] */
    DFLASH2_ST_UNSUPPORTED = 4  /* kept for the ABI: no parameters produce it any more */
};

#define DFLASH2_NC 16        /* candidates per draft position ([P] item 1) */
#define DFLASH2_MAX_K 15     /* drafted positions: [F] Details refuses k outside 1 .. block_size - 1; the pages
                                set no bound on block_size, and the cap of 15 (block_size <= 16) is this
                                library's own limit, not a number the pages print */
#define DFLASH2_MAX_TOPK 64  /* top_k up to this is taken from the row's best-key list in one pass;
                                larger top_k, or top_p with top_k off, need further passes */

/*
 * Sampling parameters of one request, applied to draft and target alike in
 * the order temperature -> top_k -> renormalise -> top_p -> renormalise
 * ([F] "Speed": temperature 1.0, top_p 0.95, top_k 20 on both sides).
 * temperature == 0 is greedy.  top_k == 0 (or >= V) and top_p == 1 switch the
 * filters off.  Every combination is supported.  With top_k <= 64 the row's
 * best-key list settles the filter in one pass; with top_k above 64, or top_p
 * with top_k off, the kept prefix may reach further and the cut is found by
 * passes over the row (dflash2_topk16, dflash2_verify).  The fused LM head
 * and the vocabulary-sharded merge take only rows settled by 16 or 64 best
 * tokens and give the others -1 / NaN.
 */
typedef struct {
    float temperature;
    int32_t top_k;
    float top_p;
} dflash2_sampling;

/*
 * dflash2_topk16 -- [P] item 1 "keep top-16 candidates per position"; [F]
 * Runtime "the target LM head gives 16 candidates per slot".
 *
 * logits   [rows, ld] of dt (row stride ld elements, ld >= V, ld * elem
 *          size a multiple of 16 bytes); the first V entries of a row count.
 * params   device [ceil(rows / rows_per_param)] or NULL (all greedy); row r
 *          uses params[r / rows_per_param].
 * cand_idx [rows, 16] int32: the 16 best tokens, best first.
 * cand_U   [rows, 16] f32: log-probability of each candidate under the
 *          drafter's distribution: greedy rows log softmax(z), sampled rows
 *          log of the filtered softmax(z / T), -inf for a candidate the
 *          filter drops.
 * lse      [rows] f32: the log normaliser on the z / T' scale (T' = 1 for
 *          greedy rows), so that kept candidates have U = z / T' - lse.
 * A row holding a NaN or +Inf, or nothing above -Inf, or with invalid
 * parameters, gets cand_idx -1, U NaN and lse NaN.  Every filter is
 * supported: a row whose kept prefix reaches past its 64 best tokens (top_k
 * above 64, or top_p with top_k off) is finished with further passes over
 * the row (a radix select of the cut by count and by mass), in the same
 * kernel: the CTA that completes such a row finishes it once it has
 * streamed its share of the rows.
 * ws: dflash2_topk16_workspace_bytes(rows) bytes (the kernel splits long rows
 *   over several CTAs and combines the parts there, and marks there the rows
 *   a CTA finishes after its stream).
 * Errors: INVALID_ARG if a pointer is NULL or misaligned, rows < 0, V < 16,
 * V >= 2^31, ld < V, ld * elem size not a multiple of 16, rows_per_param < 1;
 * WORKSPACE if ws_bytes is too small.
 */
size_t dflash2_topk16_workspace_bytes(int64_t rows);
dflash2_status dflash2_topk16(const void *logits, dflash2_dtype dt, int64_t rows, int64_t V,
                              int64_t ld, const dflash2_sampling *params, int64_t rows_per_param,
                              int32_t *cand_idx, float *cand_U, float *lse, void *ws,
                              size_t ws_bytes, dflash2_stream stream);

/*
 * dflash2_topk16_noalloc -- no counterpart on the pages: an addition of this
 * library.  The same computation, arguments and argument errors as
 * dflash2_topk16, without the workspace, for callers that cannot give this
 * library device memory: a plugin, or an engine whose memory pool owns all
 * device memory and hands no scratch to the code it calls, or code that may
 * not call an allocator at the point where the drafter's rows are reduced.
 * The scratch (one ticket and one mark per row, and the partial records of
 * rows that the kernel splits over several CTAs) is a fixed array in the
 * library's own device memory, sized for
 * DFLASH2_TOPK16_NOALLOC_MAX_ROWS rows (about 1.2 MB),
 * held by every GPU that loads the library until the process exits.
 *   - rows > DFLASH2_TOPK16_NOALLOC_MAX_ROWS returns DFLASH2_ERR_WORKSPACE and
 *     launches nothing.
 *   - Nothing is allocated.  The tickets must start at zero: each call clears
 *     those of its rows (cudaMemsetAsync on `stream`) before the kernel.  The
 *     partial records are written before they are read.
 *   - The first call on a device looks up the array's device address (once,
 *     with that device current); make that first call before any stream
 *     capture.
 *   - All calls share the one array: calls that overlap on the GPU (on
 *     different streams, or from different threads) race on it and their
 *     outputs are undefined.  Issue them on one stream.
 */
#define DFLASH2_TOPK16_NOALLOC_MAX_ROWS 16384
dflash2_status dflash2_topk16_noalloc(const void *logits, dflash2_dtype dt, int64_t rows, int64_t V,
                                      int64_t ld, const dflash2_sampling *params, int64_t rows_per_param,
                                      int32_t *cand_idx, float *cand_U, float *lse, dflash2_stream stream);

/*
 * Vocabulary-sharded top-16 -- no counterpart on the pages, which run the
 * drafter with --tp 1 ([F] Known gaps): an addition of this library for an
 * LM head split over GPUs by vocabulary.  Each GPU reduces its slice of the
 * vocabulary to a partial (dflash2_topk16_shard); the partials of all slices
 * are exchanged once (an all-gather of DFLASH2_SHARD_LIST * 8 + 8 bytes per
 * row and slice, done by the caller); dflash2_topk16_merge then gives the
 * outputs dflash2_topk16 gives for the whole row, with the same sampling
 * parameters (top_k and top_p refer to the whole vocabulary V_total).
 *
 * dflash2_topk16_shard: logits [rows, ld] of dt hold tokens id_offset ..
 *   id_offset + V_shard - 1 of each row (V_shard >= 16).  Outputs:
 *   part_idx [rows, DFLASH2_SHARD_LIST] int32: the slice's best tokens in
 *     rank order as global ids, as many as the row needs (16; max(16, top_k)
 *     for a top_k-filtered row), -1 after;
 *   part_z [rows, DFLASH2_SHARD_LIST] f32: their logits, -inf after;
 *   part_m [rows] f32: the slice's largest logit;
 *   part_s [rows] f32: the sum over the slice of exp((z - part_m) / T'), T'
 *     the temperature (1 for greedy rows); 0 for filtered rows.
 *   A row with a NaN or +Inf in the slice, invalid parameters, or a filter
 *   that needs the whole row (top_k above 64, or top_p with top_k off), gets
 *   -1 ids and NaN m and s.  A slice of masked tokens (all
 *   -inf) is not an error: m = -inf, s = 0.
 *   ws: dflash2_topk16_workspace_bytes(rows).  Errors: those of dflash2_topk16
 *   (with V_shard as V), and INVALID_ARG for id_offset < 0 or
 *   id_offset + V_shard > V_total.
 *
 * dflash2_topk16_merge: the partials of the S slices laid out [S, rows, ...]
 *   (slice s at s * rows * DFLASH2_SHARD_LIST and s * rows); params and
 *   rows_per_param as for dflash2_topk16.  Outputs cand_idx, cand_U, lse as
 *   dflash2_topk16's for the whole rows (lse and U equal up to fp32 rounding:
 *   the log normaliser is summed per slice).  A row with a NaN partial or no
 *   finite largest logit gets -1 / NaN.  Errors: INVALID_ARG for S outside
 *   1..DFLASH2_MAX_SHARDS, rows < 0, V_total < 16, NULL pointers.
 */
#define DFLASH2_SHARD_LIST 64
#define DFLASH2_MAX_SHARDS 1024
dflash2_status dflash2_topk16_shard(const void *logits, dflash2_dtype dt, int64_t rows, int64_t V_shard, int64_t ld,
                                    int64_t id_offset, int64_t V_total, const dflash2_sampling *params,
                                    int64_t rows_per_param, int32_t *part_idx, float *part_z, float *part_m,
                                    float *part_s, void *ws, size_t ws_bytes, dflash2_stream stream);
dflash2_status dflash2_topk16_merge(int32_t S, int64_t rows, const int32_t *part_idx, const float *part_z,
                                    const float *part_m, const float *part_s, int64_t V_total,
                                    const dflash2_sampling *params, int64_t rows_per_param, int32_t *cand_idx,
                                    float *cand_U, float *lse, dflash2_stream stream);

/*
 * dflash2_lmhead_topk16 -- the drafter's LM head fused with dflash2_topk16:
 * [P] "What upstream shipped" item 1 (keep the top-16 candidates of each
 * drafted position) and [F] Runtime (16 candidates per slot from the LM
 * head), with the logits z = h . W^T never written to memory.  The GEMM runs
 * on the tensor cores (bf16 inputs, fp32 accumulation); the candidates, U
 * and lse are those of dflash2_topk16 on the fp32 logits.
 *
 * h [rows, hidden] bf16 and W [V, hidden] bf16, row-major (W is the LM head's
 * weight, one row per token).  hidden a multiple of 64.  params and
 * rows_per_param as for dflash2_topk16.  Rows that would need more than 16
 * candidates (a top_k filter above 16) or the whole row (top_p with top_k
 * off) get -1 / NaN.
 * ws: dflash2_lmhead_topk16_workspace_bytes(rows, V) bytes, for the current
 *   device (the per-row partials of each CTA's vocabulary range, combined by
 *   dflash2_topk16_merge on the same stream).
 * Errors: INVALID_ARG for NULL or misaligned pointers, rows < 0, hidden not a
 * positive multiple of 64, V < 16 or V >= 2^31, rows_per_param < 1;
 * WORKSPACE if ws_bytes is too small.
 */
size_t dflash2_lmhead_topk16_workspace_bytes(int64_t rows, int64_t V);
dflash2_status dflash2_lmhead_topk16(const void *h, const void *W, int64_t rows, int64_t hidden, int64_t V,
                                     const dflash2_sampling *params, int64_t rows_per_param, int32_t *cand_idx,
                                     float *cand_U, float *lse, void *ws, size_t ws_bytes, dflash2_stream stream);

/*
 * dflash2_ctx_gate -- [P] item 1 "context gate" of the bilinear selector,
 * taken as gate = sigmoid(W_g h) with no bias.
 *
 * h     [n, hidden] of dt;  Wg [D, hidden] of dt;  gate [n, D] f32.
 * bf16 runs on the tensor cores (fp32 accumulation); f32 on the CUDA cores.
 * The bf16 grid may start while the previous kernel in the stream still
 * runs, once that kernel allows it (programmatic dependent launch; of this
 * library's kernels, the row scans allow it at their start), so that it
 * overlaps dflash2_topk16's tail: h and Wg must not be written by the
 * kernel just before it.  It completes only after that kernel does.
 * Errors: INVALID_ARG if a pointer is NULL or misaligned, n < 0, D not in
 * {16, 32, ..., 512} (a power of two), hidden < 1, or (bf16) hidden not a
 * multiple of 64.
 */
dflash2_status dflash2_ctx_gate(const void *h, dflash2_dtype dt, int64_t n, int64_t hidden,
                                const void *Wg, int32_t D, float *gate, dflash2_stream stream);

/*
 * dflash2_pair_score_walk -- [P] item 1 (S_t(a,b) = U_t(b) + <A(a) * H(h_t),
 * B(b)>, one greedy or sampled walk over the precomputed scores) and
 * "Proposal" phase 1 (block_size x 16 preds x 16 cands x 256 dims, a
 * <= block_size-step argmax walk); [F] Runtime (sampled from q, argmax when
 * greedy).
 *
 * cand_idx [B, K, 16] int32, cand_U [B, K, 16] f32 (from dflash2_topk16).
 * last_tok [B] int32: the last verified token, the only predecessor at t = 0.
 * A, Bt    [V, D] of tdt: the two token-embedding tables.
 * gate     [B, K, D] f32 (from dflash2_ctx_gate).
 * params   [B] or NULL (all greedy); only temperature is read (0 = greedy).
 * u_walk   [B, K] f32 uniforms in [0, 1); may be NULL when params is NULL.
 * Outputs: path_tok [B, K] int32, path_slot [B, K] int32 (index into the
 *   candidates), q_sel [B, K, 16] f32 (the walk's distribution at each step;
 *   one-hot when greedy), scores [B, K, 16, 16] f32: scores[b,t,i,j] pairs
 *   predecessor i with candidate j; at t = 0 row 0 is the last verified
 *   token and rows 1..15 are -inf.
 * Greedy steps take the first slot with the largest score; sampled steps
 * take the first slot whose cumulative q exceeds u_walk.  A step whose row
 * holds a NaN, or only -inf, ends the walk: that step and the rest get
 * token -1, slot -1 and NaN q.  Ids outside [0, V) give NaN scores.
 * No workspace: one thread-block cluster of K CTAs per request keeps the
 *   request's state in its shared memory.
 * Errors: INVALID_ARG for NULL/misaligned pointers, B < 0, K outside 1..15,
 * D not a power of two in 16..1024, V < 16, u_walk NULL with params set;
 * UNSUPPORTED for B > 65535, or when a cluster of K CTAs with the shared
 * memory that D needs cannot be resident on this GPU (clusters above 8 CTAs
 * must fit in one GPC; the answer is cached per device, K and D).
 */
dflash2_status dflash2_pair_score_walk(int64_t B, int32_t K, const int32_t *cand_idx,
                                       const float *cand_U, const int32_t *last_tok,
                                       const void *A, const void *Bt, dflash2_dtype tdt, int64_t V,
                                       int32_t D, const float *gate,
                                       const dflash2_sampling *params, const float *u_walk,
                                       int32_t *path_tok, int32_t *path_slot, float *q_sel,
                                       float *scores, dflash2_stream stream);

/*
 * dflash2_verify -- [F] Sampled verify (accept with min(1, p/q); on a reject
 * resample from max(0, p - q); all-greedy batches keep the prefix match);
 * [P] "Proposal" phase 3; [F] "Tests added or changed" (trusted, NaN,
 * wrong-total and greedy rows).
 *
 * tlogits [B, K+1, ld] of dt: target logits of the K drafted positions and
 *   the bonus position, row (b, t) at (b * (K+1) + t) * ld.
 * path_tok, path_slot [B, K]; cand_idx, q_sel [B, K, 16] (from the walk).
 * params [B] or NULL (all greedy).  u_acc [B, K], u_res [B, K+1] f32
 *   uniforms in [0, 1); may be NULL when params is NULL.
 * flags: DFLASH2_VERIFY_TRUST_Q skips the q-total check.
 * Per request b: p_t is the target distribution of row t (greedy: all mass
 *   on the argmax).  Greedy requests accept while the drafted token is the
 *   argmax and then emit the argmax.  Sampled requests accept position t iff
 *   u_acc[t] * q < p at the drafted token; on a reject they draw from
 *   max(0, p - q) (normalised; from p when its total is <= 1e-12) by inverse
 *   CDF over ascending token ids with u_res[t]; after K accepts they draw the
 *   bonus token from p_K with u_res[K].  Every filter is supported: when
 *   p's support reaches past the row's 64 best tokens (no filter, top_p with
 *   top_k off, top_k above 64), the cut is found by further passes over the
 *   row and the residual and bonus draws walk the whole row in token-id order,
 *   in the same kernel, by the CTA that completes the row once it has
 *   streamed its share of the rows.
 * Outputs: accept_len [B] in 0..K; out_tok [B, K+1]: the accepted tokens,
 *   then the corrected or bonus token, then -1; status [B] (DFLASH2_ST_*).
 *   A request with status != 0 commits nothing (accept_len 0, all -1).
 * ws: dflash2_verify_workspace_bytes(B, K).
 * Errors: INVALID_ARG as for dflash2_topk16 plus K outside 1..15 and NULL
 * uniforms with params set.
 */
#define DFLASH2_VERIFY_TRUST_Q 1u
size_t dflash2_verify_workspace_bytes(int64_t B, int32_t K);
dflash2_status dflash2_verify(const void *tlogits, dflash2_dtype dt, int64_t B, int32_t K,
                              int64_t V, int64_t ld, const int32_t *path_tok,
                              const int32_t *cand_idx, const float *q_sel,
                              const int32_t *path_slot, const dflash2_sampling *params,
                              const float *u_acc, const float *u_res, uint32_t flags,
                              int32_t *accept_len, int32_t *out_tok, int32_t *status, void *ws,
                              size_t ws_bytes, dflash2_stream stream);

/*
 * dflash2_conv2tap -- [P] item 2: Conv(x)_t = k_{t,0} * x_t + k_{t,1} * x_{t-1},
 * the first position tapping the last verified token's hidden state; [F]
 * Refused at startup (conv_group_size divides the hidden size).
 *
 * x [B, T, H], k0 and k1 [B, T, H / group_size], x_prev [B, H], y [B, T, H],
 * all of dt.  With group_size G, channel c uses tap c / G.  bf16 outputs are
 * the exact value rounded once to bf16 (nearest, ties to even); f32 outputs
 * use one fused multiply-add.
 * Errors: INVALID_ARG for NULL/misaligned pointers, B < 0, T < 1, H < 1,
 * group_size < 1 or not dividing H.
 */
dflash2_status dflash2_conv2tap(const void *x, const void *k0, const void *k1, const void *x_prev,
                                dflash2_dtype dt, int64_t B, int32_t T, int64_t H,
                                int32_t group_size, void *y, dflash2_stream stream);

/*
 * dflash2_dynconv2tap -- [P] item 2 with the taps made from the input: the
 * pages name the conv "dynamic" and give its group size ([F] Refused at
 * startup: conv_group_size divides the hidden size), not how the taps are
 * made.  The reading is dynamic convolution as published (Wu et al., "Pay
 * Less Attention with Lightweight and Dynamic Convolutions", 2019): the
 * taps of position t are a linear map of x_t, normalised by a softmax over
 * the kernel's width and shared by the group_size channels of a group.  For
 * two taps that softmax is (s, 1 - s) with s = sigmoid(a0 - a1), so the map
 * enters through its difference Wd:
 *   taps[b, t, g] = k0 = sigmoid(Wd[g] . x[b, t]),  k1 = 1 - k0,
 *   y[b, t, c] = k0 x[b, t, c] + k1 x[b, t-1, c]   (x_prev at t = 0, g = c / group_size).
 *
 * x [B, T, H], x_prev [B, H], Wd [H / group_size, H], y [B, T, H], all of dt;
 * taps [B, T, H / group_size] f32 (an output).  bf16: the taps on the tensor
 * cores (fp32 accumulation) as dflash2_ctx_gate computes its gate; y is
 * fma(k0, x_t, k1 x_{t-1}) in fp32 rounded once to bf16 (within one bf16 ulp
 * of the exact value).  f32: CUDA cores, y by one fused multiply-add.
 * Not built: fusing the conv with the drafter sublayer's norm and residual
 * (the pages give no form for them).
 * Errors: INVALID_ARG for NULL/misaligned pointers (x, Wd, taps 16-byte
 * aligned), B < 0, T < 1, H < 1, group_size < 1 or not dividing H;
 * UNSUPPORTED for bf16 unless H is a multiple of 64 and H / group_size a
 * power of two in 16..512.
 */
dflash2_status dflash2_dynconv2tap(const void *x, const void *x_prev, const void *Wd, dflash2_dtype dt,
                                   int64_t B, int32_t T, int64_t H, int32_t group_size, float *taps, void *y,
                                   dflash2_stream stream);

/*
 * ------------------------------------------------- the paged cache path ----
 *
 * The attention that the drafter and the target run around this library's
 * selection and verify, on a paged key-value cache: dflash2_rope_append puts
 * a block's new keys and values into the cache, dflash2_paged_attn lets the
 * block's queries attend to it, dflash2_kv_evict keeps a cache within a
 * budget.  No counterpart on the pages beyond the shapes: blocks of K + 1
 * tokens per request, causal in a verify and seen both ways in a drafter's
 * block ([P] "What upstream shipped"), a drafter's cache bounded by a window
 * of 2048 positions ([F] Details).  Additions of this library.
 *
 * The cache is a pool of pages.  Slot s of request b lies in page
 * page_table[b, s / page_size] at offset s % page_size; slots 0 .. n - 1 are
 * in use.  Element (page, head, offset, c) of k and of v is at
 *   page * page_stride + head * head_stride + offset * slot_stride + c
 * (in elements), so both [num_pages, Hkv, page_size, d] and
 * [num_pages, page_size, Hkv, d] pools are taken.  Optional side arrays, both
 * contiguous [num_pages, Hkv, page_size]: `weight`, the attention weight each
 * cached key has received so far, and `pos`, the position of the key in its
 * sequence (after an eviction a slot's number no longer is; without the array
 * slot s holds position s).  A page may belong to several requests as long as
 * no call writes to it (append, weights, evict).
 *
 * Page table entries outside [0, num_pages) and tables that are too short
 * never lead to an access outside the pool: see each call.
 *
 * Common errors of the three calls: INVALID_ARG for a NULL cache, k, v or
 * page_table; num_pages, Hkv, page_size, d or max_pages < 1; k, v, the
 * strides or d * elem size not multiples of 16 bytes; slot_stride < d,
 * head_stride or page_stride < 0; side arrays, page_table or per-request
 * arrays not 4-byte aligned; B or T < 0.  B = 0 is an empty batch: nothing is
 * launched, and page_table may be NULL and max_pages 0.
 */
typedef struct {
    void *k;              /* device, of dt */
    void *v;              /* device, of dt, laid out as k */
    float *weight;        /* device [num_pages, Hkv, page_size] or NULL */
    int32_t *pos;         /* device [num_pages, Hkv, page_size] or NULL */
    int64_t num_pages;
    int64_t page_stride;  /* elements */
    int64_t head_stride;
    int64_t slot_stride;
    int32_t Hkv;
    int32_t page_size;
    int32_t d;            /* head dimension */
    dflash2_dtype dt;
} dflash2_kv_cache;

/*
 * dflash2_rope_append -- rotary positions on one or several axes, and the
 * append to the cache, in one pass over a block's new tokens.
 *
 * For new token t < q_len[b] of request b, with x the query or key head:
 *   y = x / sqrt(mean(x^2) + eps) * w       (q_norm / k_norm given; else y = x)
 *   (y_i, y_j) -> (y_i cos - y_j sin, y_j cos + y_i sin)   for each pair of
 * the first rot entries: pair p is (p, p + rot / 2), or (2p, 2p + 1) with
 * interleaved != 0; the others stay.  cos and sin come from row
 * pos_ids[pair_axis[p], b, t] of the table, columns p and rot / 2 + p (the
 * table is made once, in as many bits as the caller likes, so a position of
 * any size is exact).  All arithmetic in fp32, one rounding to dt at the end.
 * Rotated queries go to q_out, keys and values to slot kv_len[b] + t, the
 * slot's weight is set to 0 and its position to seq_pos[b] + t.
 *
 * q [B, T, Hq, d], k and v [B, T, Hkv, d] of the cache's dt; heads contiguous,
 *   q_stride, k_stride, v_stride elements from one token to the next (slices
 *   of one fused projection are taken as they are).
 * kv_len [B]: slots in use before the call.  q_len [B] or NULL (all T);
 *   clamped to 0 .. T; queries of tokens t >= q_len[b] come out 0 and their
 *   keys are not stored.  seq_pos [B] or NULL (kv_len).
 * cos_sin [n_pos, rot] f32.  pos_ids [axes, B, T].  pair_axis [rot / 2] or
 *   NULL (axis 0); values above axes - 1 count as axes - 1.
 * q_norm, k_norm [d] of dt, or NULL.
 * q_out [B, T, Hq, d], contiguous; may be q itself where q is contiguous
 *   (q_stride = Hq * d), and must not overlap q, k or v otherwise.
 * kv_len_out [B] or NULL: kv_len + q_len; must not overlap kv_len, q_len or
 *   seq_pos.  With T = 0 it is kv_len, and nothing else is read or written.
 * A token whose position id is outside [0, n_pos) gets NaN in the rotated
 * entries of its query and key.  A token whose slot has no valid page (past
 * the table, or a page id out of range) is not stored and its query comes
 * out NaN.
 * Errors: the common ones; INVALID_ARG for NULL q, k, v, q_out, kv_len,
 * cos_sin or pos_ids; kv_len_out the same as kv_len, q_len or seq_pos; q_out the
 * same as k, v or a q of several tokens that is not contiguous; Hq < 1,
 * rot odd, < 2 or > d, axes < 1, n_pos < 1, strides below the width of a
 * token's heads or not multiples of 16 bytes; dt not F32 or BF16.
 * UNSUPPORTED for d > 1024, B * T >= 2^31 or Hq + 2 Hkv >= 2^31.
 */
dflash2_status dflash2_rope_append(const dflash2_kv_cache *cache, const int32_t *page_table, int32_t max_pages,
                                   const int32_t *kv_len, const int32_t *q_len, const int32_t *seq_pos,
                                   const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride,
                                   int64_t v_stride, int64_t B, int32_t T, int32_t Hq, const float *cos_sin,
                                   int64_t n_pos, int32_t rot, const int32_t *pos_ids, int32_t axes,
                                   const uint8_t *pair_axis, int32_t interleaved, const void *q_norm,
                                   const void *k_norm, float eps, void *q_out, int32_t *kv_len_out,
                                   dflash2_stream stream);

/*
 * dflash2_paged_attn -- attention of a block of T new tokens per request over
 * the request's paged cache (the new tokens' own slots are in it).
 *
 * Query head h of token t reads the cached head h / (Hq / Hkv).  It sees slot
 * s < kv_len[b] at position P(s) (the cache's `pos`, or s) if
 *   P(s) <= seq_pos[b] + t            (with DFLASH2_ATTN_CAUSAL), and
 *   P(s) >  seq_pos[b] + t - window   (with window > 0).
 * Over the slots it sees, with x_s = scale * <q, k_s>:
 *   lse = log sum_s exp(x_s),  p_s = exp(x_s - lse),  out = sum_s p_s v_s.
 * With DFLASH2_ATTN_WEIGHTS every cached key's `weight` grows by the sum of
 * its p_s over the block's tokens and the query heads that share it: all
 * tokens t < q_len[b], also those that a verify rejects afterwards.
 * A row that sees nothing (or sees only x_s = -inf) gets out 0, lse -inf and
 * adds no weight; tokens t >= q_len[b] are such rows.  What lies in slots
 * that a row does not see (NaN and Inf too) does not touch it.
 *
 * q, out [B, T, Hq, d] of dt, contiguous, not overlapping; lse [B, T, Hq] f32
 *   (may be NULL without DFLASH2_ATTN_WEIGHTS).
 * kv_len [B]: slots in use, the new tokens among them; clamped to what the
 *   table can hold.  q_len [B] or NULL (all T).  seq_pos [B]: the position
 *   of the block's first token, or NULL (kv_len - q_len).
 * Slots whose page id is out of range are seen by no row.
 * Scores, softmax statistics and sums are fp32.  On the tensor cores (bf16, d
 * 64, 128 or 256, pages of a multiple of 8 slots) exp(x_s - m), m near the
 * row's maximum, is rounded to bf16 once where it multiplies the values, so
 * out is within 2^-8 sum_s p_s |v_s| of the definition before its own rounding
 * to bf16; the other kernels (f32, other d and pages) keep it in fp32.  A
 * weight is added as exp(x_s - lse) with the fp32 lse, so it is off by a
 * factor of up to exp(2^-23 |lse|).  The cache's length is split over the GPU
 * and the parts are joined in a fixed order: the same call gives the same bits.
 * ws: dflash2_paged_attn_workspace_bytes(B, T, Hq, Hkv, d, dt) bytes, the first
 *   4096 zero at the start and left zero.
 * Errors: the common ones; INVALID_ARG for NULL q, out or kv_len, out the same
 * as q, lse or the cache's weight NULL with DFLASH2_ATTN_WEIGHTS, Hq not a
 * positive multiple of Hkv, scale not finite, window < 0, unknown flags;
 * WORKSPACE if ws is too small; UNSUPPORTED for d > 256, Hq / Hkv > 128,
 * Hq >= 2^24, num_pages >= 2^31, max_pages * page_size >= 2^31 - 256 or
 * B * Hkv * T * (max_pages * page_size / 32 + 5) >= 2^31.
 */
enum { DFLASH2_ATTN_CAUSAL = 1, DFLASH2_ATTN_WEIGHTS = 2 };
size_t dflash2_paged_attn_workspace_bytes(int64_t B, int32_t T, int32_t Hq, int32_t Hkv, int32_t d,
                                          dflash2_dtype dt);
dflash2_status dflash2_paged_attn(const dflash2_kv_cache *cache, const int32_t *page_table, int32_t max_pages,
                                  const int32_t *kv_len, const int32_t *q_len, const int32_t *seq_pos, const void *q,
                                  int64_t B, int32_t T, int32_t Hq, float scale, int32_t window, uint32_t flags,
                                  void *out, float *lse, void *ws, size_t ws_bytes, dflash2_stream stream);

/*
 * dflash2_kv_evict -- eviction by accumulated attention weight.
 *
 * A request with n = kv_len[b] <= budget slots is left alone.  Of any other,
 * every head keeps `budget` of its n slots on its own: first those at
 * positions >= seq_len[b] - recent or < sink, then the others in the order of
 * their weight, largest first (NaN counts as the smallest; equal weights: the
 * lower slot first).
 * Kept slots below `budget` stay where they are; kept slots from `budget` on
 * move, in order, to the evicted slots below `budget`, in order, with their
 * key, value, weight and position.  So the least is moved, and slots are in
 * no order of position afterwards (`pos` says which is which).  Slots from
 * `budget` on keep what was in them; the caller may release their pages.
 *
 * kv_len [B]: slots in use (clamped to what the table holds).  seq_len [B]:
 *   the length of the sequence (the newest key's position + 1), or NULL
 *   (kv_len).  kv_len_out [B]: min(kv_len, budget); may be kv_len or seq_len
 *   itself, and must not overlap them otherwise.
 * A slot whose page id is out of range is never kept before another one and
 * never copied.
 * If more than `budget` slots are protected, the lower slots stay.
 * ws: dflash2_kv_evict_workspace_bytes(B, Hkv, max_pages * page_size, budget)
 *   bytes, of which no zeros are needed; the first 4096 are not touched.
 * Errors: the common ones; INVALID_ARG for the cache's weight or pos NULL,
 * NULL kv_len or kv_len_out, budget < 1, recent < 0 or sink < 0; WORKSPACE;
 * UNSUPPORTED for max_pages * page_size >= 2^31 - 2048 or B * Hkv >= 2^31.
 */
size_t dflash2_kv_evict_workspace_bytes(int64_t B, int32_t Hkv, int64_t capacity, int32_t budget);
dflash2_status dflash2_kv_evict(const dflash2_kv_cache *cache, const int32_t *page_table, int32_t max_pages,
                                const int32_t *kv_len, const int32_t *seq_len, int64_t B, int32_t budget,
                                int32_t recent, int32_t sink, int32_t *kv_len_out, void *ws, size_t ws_bytes,
                                dflash2_stream stream);

/* Human-readable name of a status code (static string). */
const char *dflash2_status_string(dflash2_status s);

/*
 * Weights held in 4 bits -- [R] and [F] run this path for targets and drafters
 * with 4-bit weights; the pages give no kernel.  An addition of this library.
 *
 * A record stands for a matrix W [N, K].  Each row is cut into groups of
 * `group` neighbours (the last one may be short), and
 *   W[n, k] = (code[n, k] - zero[n, k / group]) * scale[n, k / group].
 * codes  [N, code_stride] bytes, two codes of 0..15 to a byte, the even k in
 *        the low half.  code_stride is a multiple of 16 and at least
 *        16 * ceil(K / 32); what the codes behind K hold does not matter.
 * scale  [N, side_stride] of side_dt, side_stride >= ceil(K / group).
 * zero   the same as scale, or NULL: 8 everywhere.
 * Rows may lie further apart than they are long, so that some rows, or some
 * columns from a multiple of `group` and 32 on, of a larger matrix are a
 * record too.  The record is read on the host by each call; it holds device
 * pointers (codes 16-byte aligned, scale and zero aligned to their type).
 */
typedef struct {
    void *codes;
    void *scale;
    void *zero;
    int64_t N;
    int64_t K;
    int64_t code_stride;
    int64_t side_stride;
    int32_t group; /* 32, 64 or 128 */
    dflash2_dtype side_dt;
} dflash2_weight4;

/*
 * dflash2_quant4 -- codes, scales and (where the record has room for them)
 * zero points of W [N, ld] (dt; row stride ld elements), nearest codes.  In
 * f32, every step rounded to nearest even:
 *   without zero points  scale = max|w| / 7;  code = w / scale + 8
 *   with zero points     scale = max(w, 0) / 15 - min(w, 0) / 15;
 *                        zero = -min(w, 0) / scale;  code = w / scale + zero
 * with scale rounded to side_dt before it divides, the quotients rounded to
 * whole numbers, zero and code held within 0..15, and a scale of 0 dividing
 * as 1.  A group with a NaN or an infinity gets scale NaN (codes and zero 8).
 * The codes behind K, up to a multiple of 32, are 8.
 *
 * dflash2_dequant4 -- out [N, ld] (dt): what the record stands for, in f32
 * and rounded once.
 *
 * Errors: INVALID_ARG for a NULL or misaligned pointer (W and out: aligned to
 * their type), N < 0 or above 2^31 - 1, K < 1 or above 2^31 - 129, a group
 * other than 32, 64, 128, strides that are too small or (code_stride) no multiple of 16, ld < K;
 * UNSUPPORTED for matrices of 2^36 entries and more, counted in whole groups.
 */
dflash2_status dflash2_quant4(const void *W, dflash2_dtype dt, int64_t ld, const dflash2_weight4 *w,
                              dflash2_stream stream);
dflash2_status dflash2_dequant4(const dflash2_weight4 *w, void *out, dflash2_dtype dt, int64_t ld,
                                dflash2_stream stream);

/*
 * dflash2_linear4 -- y = x . W^T with 4-bit weights: the LM head or a
 * projection of one decoded token, of a verify block, or of many.
 *
 * x [rows, x_stride] (dt), the first K entries of a row count.
 * y [rows, y_stride] (y_dt): the first N entries of a row are written.
 *   y_dt is dt, or f32.  A row of x that holds a NaN or an infinity gives a
 *   row of NaN.
 *   Sums are f32 sums of exact products of codes and of zero points with x,
 *   rounded once to y_dt, for any number of rows;
 *   entries of x below 2^-130 of their row's largest (f32: 2^-110) and scales
 *   below 2^-100 lose bits, and (code + |zero|) * |scale| * K from 2^132 on
 *   may overflow where y does not.
 * ws: dflash2_linear4_workspace_bytes(dt, rows, N, K) bytes, which is 0 for
 *   few rows (ws may then be NULL).  It needs no zeros and is left with
 *   scratch.
 * Errors: INVALID_ARG for a NULL or misaligned pointer (x and y: aligned to
 * their type), rows < 0, x_stride < K, y_stride < N, f32 x with bf16 y, or a
 * record that dflash2_dequant4 refuses; UNSUPPORTED for K above 2^17, rows
 * above 2^19, rows above 2^15 with K above 2^13 where no workspace is taken,
 * and some products with N K rows above 2^54; WORKSPACE if ws_bytes is too
 * small.
 *
 * dflash2_linear4_rounded -- the same, where the weights of a call with bf16
 * x, results and scales that takes a workspace may be rounded to bf16 (code - zero, then
 * its product with the scale): faster for many rows, and most of all for
 * small groups.  Its results are off by the weights' rounding besides their
 * own, so a row's are not those that it has in a call of few rows.  A weight
 * row with a scale outside 2^-80 .. 2^30 (and not 0) or a zero point above
 * 2^40 gives NaN in such a call; entries of x below 2^-80 of their row's
 * largest lose bits.  Every other call is dflash2_linear4.
 */
size_t dflash2_linear4_workspace_bytes(dflash2_dtype dt, int64_t rows, int64_t N, int64_t K);
dflash2_status dflash2_linear4(const void *x, dflash2_dtype dt, int64_t rows, int64_t x_stride,
                               const dflash2_weight4 *w, void *y, dflash2_dtype y_dt, int64_t y_stride, void *ws,
                               size_t ws_bytes, dflash2_stream stream);
dflash2_status dflash2_linear4_rounded(const void *x, dflash2_dtype dt, int64_t rows, int64_t x_stride,
                                       const dflash2_weight4 *w, void *y, dflash2_dtype y_dt, int64_t y_stride,
                                       void *ws, size_t ws_bytes, dflash2_stream stream);

/*
 * dflash2_sample -- one token per row of logits from a given uniform: what a
 * request decodes without a draft (its first token, or every token when it
 * runs without a drafter).  [F] Speed gives the filters' values; min_p and
 * this entry point are additions of this library.
 *
 * logits [rows, ld] of dt as for dflash2_topk16 (V >= 1).
 * params [ceil(rows / rows_per_param)] or NULL (all greedy), min_p the same
 *   or NULL (0, off); row r uses entry r / rows_per_param.
 * u      [rows] f32 uniforms in [0, 1).
 * Tokens are ranked by logit, ties by the lower id, with the masses
 * w = exp((z - max) / T).  top_k keeps the first top_k; top_p the shortest
 * prefix of those whose mass reaches top_p of theirs; min_p those with w >=
 * min_p (the best one's w is 1).  The row draws the first kept token, in
 * rank order, whose running mass exceeds u times the kept mass, else the
 * last one with any mass.  Greedy rows take the first token.
 * token [rows] int32; prob [rows] f32: the drawn token's share of the kept
 *   mass (1 for greedy rows).
 * Masses are summed as whole numbers of 2^-44 (of 2^-(63 - ceil(log2(V + 1)))
 *   for V of 2^19 and more), so a row's token depends neither on the other rows nor on
 *   how the row is split.
 * A temperature between 0 and 2^-127 counts as 2^-127.
 * A row with a NaN or +Inf, nothing above -Inf, a NaN uniform or invalid
 * parameters (as DFLASH2_ST_BAD_PARAMS; min_p outside [0, 1]) gets token -1 and
 * prob NaN.  f32 logits further below the largest than f32 reaches have no mass.
 * Errors: INVALID_ARG for a NULL or misaligned pointer (logits: 16 bytes; the
 * others: 4), rows < 0, V < 1 or V >= 2^31, ld < V, ld * elem size not a
 * multiple of 16, rows_per_param < 1; UNSUPPORTED for 2^28 rows and more.
 */
dflash2_status dflash2_sample(const void *logits, dflash2_dtype dt, int64_t rows, int64_t V, int64_t ld,
                              const dflash2_sampling *params, const float *min_p, int64_t rows_per_param,
                              const float *u, int32_t *token, float *prob, dflash2_stream stream);

/*
 * Error word of the library's kernels on the current device: nonzero after a
 * kernel gave up on a bounded wait (it then wrote -1 / NaN outputs instead of
 * hanging, dflash2_rope_append NaN to the cached keys and values and
 * dflash2_paged_attn to the weights too, dflash2_linear4 NaN to
 * the outputs; the word then holds
 * DFLASH2_DEVERR_WAIT_TIMEOUT).  Synchronises the device.  clear != 0 resets
 * the word.
 */
#define DFLASH2_DEVERR_WAIT_TIMEOUT 1u
dflash2_status dflash2_device_error(uint32_t *code, int clear);

/*
 * dflash2_test_hold -- no counterpart on the pages: a test hook of this
 * library, for exercising the bounded waits without a GPU fault.  With `flag`
 * set (a 4-byte aligned device word), every streaming warp of every
 * dflash2_topk16 / dflash2_topk16_noalloc / dflash2_verify kernel launched
 * afterwards by this process first waits until *flag is nonzero, giving up
 * after max_cycles SM clock cycles (1 .. 2^32).  A warp that gives up issues
 * no copy, sets the device error word (DFLASH2_DEVERR_WAIT_TIMEOUT) and goes
 * through its rows as after any time-out: their outputs are -1 / NaN, and a
 * verify request that reads such a row gets status DFLASH2_ST_NAN.  The same
 * holds for the warps of dflash2_paged_attn's tensor-core kernels that copy
 * the values (with DFLASH2_ATTN_WEIGHTS, the keys of the weights' pass
 * instead), of dflash2_rope_append's kernel for long blocks and of the one of
 * dflash2_linear4's for many rows that copies x: they give up as after any
 * time-out.  flag NULL switches the hook off.  Kernels already
 * launched or captured keep the setting they were launched with.
 * Errors: INVALID_ARG for a misaligned flag or max_cycles out of range.
 */
dflash2_status dflash2_test_hold(const uint32_t *flag, int64_t max_cycles);

#ifdef __cplusplus
}
#endif

#endif /* DFLASH2_H */
