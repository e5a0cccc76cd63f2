/*
 * blink.h -- C ABI of the GB300 (sm_103a) library for the shared-prefix one-pass decision path.
 *
 * Many questions share one prefix (a system prompt plus the evidence).  The prefix KV is held
 * once in a contiguous arena; each question runs only its tail, which attends to the prefix
 * without a mask and to its own tail causally.  The answer is read from the next-token
 * distribution restricted to the offered option labels: the last-token hidden state against
 * the unembedding rows of those labels, then a temperature softmax.  No tokens are generated.
 *
 * Sources (the pages this library restates):
 *   blink.py   -- the "blink-4b" serving module: `_batches`, `_padded`, `_forward`,
 *                 `_forward_shared`, `_read`, `_read_batched`, `softmax`, the limits
 *                 MAX_OPTIONS / MAX_QUESTIONS / MAX_INPUT_TOKENS / TOKEN_BUDGET and the
 *                 PREFIX_CACHE note;
 *   engine.py  -- "simit" backends/mot: the contiguous KV arena and its varlen attention
 *                 metadata (cu_seqlens, per-request region start, keys used).
 *
 * Conventions for every entry point:
 *   - Pointers named d_* and all tensor pointers are DEVICE pointers; h_* are HOST pointers
 *     (pinned memory for asynchronous copies).  The caller owns every buffer; the library
 *     allocates nothing and keeps no state between calls.
 *   - bf16 tensors are passed as `blink_bf16` (16-bit storage of bfloat16 values), row-major.
 *   - Calls are asynchronous on `stream` unless a host output is requested, in which case the
 *     call synchronises the stream before returning.
 *   - Any host thread may call, several at once with a workspace each (but see the readout that allocates nothing).
 *   - Arguments are checked on the host first (BLINK_INVALID_ARG / BLINK_OUT_OF_RANGE, nothing
 *     launched).  Problems only visible on the device (a bad length or label id inside a
 *     device array, a bounded wait that ran out) are latched in a device error word, read back
 *     by the host-output path or by blink_read_device_status().  No kernel traps.
 */
#ifndef BLINK_H
#define BLINK_H

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef uint16_t blink_bf16;
typedef int32_t blink_status;

#define BLINK_OK 0
#define BLINK_INVALID_ARG 1          /* malformed argument (null pointer, bad shape, T <= 0 ...) */
#define BLINK_OUT_OF_RANGE 2         /* a limit of the pages is exceeded (options, questions, context) */
#define BLINK_WORKSPACE_TOO_SMALL 3  /* ws_bytes below what the *_workspace() query returned */
#define BLINK_CUDA_ERROR 4           /* a CUDA runtime call failed; cudaGetLastError() has the detail */
#define BLINK_DEVICE_FLAG 5          /* a device-side check failed (bad length, label id, CSR offsets) */
#define BLINK_DEVICE_TIMEOUT 6       /* a bounded wait inside a kernel ran out; outputs are invalid */

/* Limits from blink.py: MAX_OPTIONS, MAX_QUESTIONS, MAX_INPUT_TOKENS.  The planner also takes
 * up to 64 requests of 512 questions at once (blink.py `Batcher.MAX_REQUESTS` packs every
 * question of every request into the same forwards). */
#define BLINK_MAX_OPTIONS 255
#define BLINK_MAX_QUESTIONS 512
#define BLINK_MAX_INPUT_TOKENS 131072
#define BLINK_MAX_PLAN_SEQUENCES 32768

/* A short English description of a status code (a static string). */
const char *blink_status_string(blink_status s);

/* Reads (and, if `clear` != 0, resets) the device error word at the start of a workspace
 * passed to blink_prefix_tail_attention or blink_label_readout.  Synchronises `stream`.
 * Returns BLINK_OK, BLINK_DEVICE_FLAG or BLINK_DEVICE_TIMEOUT (or BLINK_CUDA_ERROR). */
blink_status blink_read_device_status(void *d_ws, int32_t clear, cudaStream_t stream);

/* Self-test of the failure path every kernel relies on (no counterpart on the pages): one
 * thread waits, with the library's bounded wait, on a barrier that nothing arrives at; after
 * limit_us microseconds (1..1000000) the wait gives up and latches BLINK_DEVICE_TIMEOUT in the
 * workspace's error word, exactly as a kernel whose copy or peer never arrived would.  A warp then
 * waits together on it, half of its lanes for a phase that is complete: all have to give up.  Returns
 * the status (BLINK_DEVICE_TIMEOUT when both work), after clearing the word.  Nothing
 * faults or traps and the context stays usable.  d_ws: a workspace of at least 256 bytes.
 * Synchronises `stream`. */
blink_status blink_selftest_wait_timeout(uint32_t limit_us, void *d_ws, size_t ws_bytes, cudaStream_t stream);

/* ------------------------------------------------------------------------------------------
 * Pack plan -- blink.py `_batches` (token-budget packing, shortest first, a forward closes when
 * (longest x count) would pass the padded-token budget or at the row cap; a sequence longer
 * than the budget runs alone) and `_padded` (right padding to each forward's longest).
 *
 * d_lengths [n]        sequence lengths (tails, or whole prompts on the plain path), 1..131072
 * n                    1..BLINK_MAX_PLAN_SEQUENCES
 * budget               padded tokens per forward (blink.py TOKEN_BUDGET = 32768), >= 1
 * max_rows             row cap per forward, 0 = none (blink.py caps rows on the prefix path)
 * Outputs (device, int32; slot s = the s-th sequence in the stable ascending length order):
 *   d_order [n]            sequence index held by slot s
 *   d_slot_of [n]          the inverse: slot holding sequence i (d_slot_of[d_order[s]] == s)
 *   d_fwd_of_slot [n]      forward of slot s
 *   d_fwd_slot_start [n+1] first slot of forward f for f <= n_forwards; n beyond
 *   d_fwd_width [n]        padded width (longest length) of forward f; 0 beyond n_forwards
 *   d_cu_seqlens [n+1]     varlen token offsets of the slots (cu[0] = 0)
 *   d_last_varlen [n]      last token of slot s in the varlen packing: cu[s+1] - 1
 *   d_last_padded [n]      last token of slot s in its forward's padded [rows, width] batch:
 *                          row * width + len - 1
 *   d_n_forwards [1]       number of forwards, or -1 if a length was outside 1..131072
 *   h_n_forwards           optional (may be NULL): the same count copied to pinned host memory;
 *                          when given, the call synchronises the stream.
 * Errors: BLINK_INVALID_ARG (null output, budget < 1, max_rows < 0), BLINK_OUT_OF_RANGE (n),
 * BLINK_DEVICE_FLAG (only with h_n_forwards: a length out of range), BLINK_CUDA_ERROR.
 * Up to 2048 lengths the whole plan is one thread block.  Above that, the stable sort runs over
 * the whole GPU first (blocks sort runs of 1024 keys, then merge rounds), with d_fwd_of_slot and
 * d_last_padded as its two ping-pong buffers; the one-block plan kernel reads the sorted keys
 * before it writes those outputs.  So the planner needs no workspace of its own:
 * blink_pack_plan_workspace() returns 0 for every n.
 * ------------------------------------------------------------------------------------------ */
size_t blink_pack_plan_workspace(int32_t n);

blink_status blink_pack_plan(const int32_t *d_lengths, int32_t n, int32_t budget, int32_t max_rows,
                             int32_t *d_order, int32_t *d_slot_of, int32_t *d_fwd_of_slot, int32_t *d_fwd_slot_start,
                             int32_t *d_fwd_width, int32_t *d_cu_seqlens, int32_t *d_last_varlen,
                             int32_t *d_last_padded, int32_t *d_n_forwards, int32_t *h_n_forwards,
                             cudaStream_t stream);

/* ------------------------------------------------------------------------------------------
 * Shared-prefix length -- blink.py `_shared_prefix_len`: the number of leading tokens common to
 * every sequence, leaving each sequence at least one token of its own (its answer position is
 * computed in the per-question pass); 0 for fewer than two sequences.  blink.py `_forward` takes
 * the shared path only when this is at least PREFIX_MIN_TOKENS (256), a host decision.
 *
 * d_tokens, n_tokens  int32 token ids of all sequences back to back (n_tokens of them); sequence i
 *                     at d_tokens + (d_cu[i] - d_cu[0]) with length d_cu[i+1] - d_cu[i] (>= 1)
 * d_cu [n+1], n       1..BLINK_MAX_PLAN_SEQUENCES sequences
 * d_len [1]           output (device); h_len optional pinned host copy (the call then synchronises)
 * d_ws, ws_bytes      workspace of blink_shared_prefix_len_workspace() bytes (error word)
 * A length below 1 or a sequence past n_tokens latches BLINK_DEVICE_FLAG.
 * ------------------------------------------------------------------------------------------ */
size_t blink_shared_prefix_len_workspace(void);

blink_status blink_shared_prefix_len(const int32_t *d_tokens, int64_t n_tokens, const int32_t *d_cu, int32_t n,
                                     int32_t *d_len, int32_t *h_len, void *d_ws, size_t ws_bytes, cudaStream_t stream);

/* ------------------------------------------------------------------------------------------
 * KV rows into the arena -- simit engine.py: one contiguous KV arena with a region per request
 * (`KVArena`, `arena.copy`): the prefix's K/V, computed once, are written into its region, and a
 * cached prefix region can be copied into another request's region.
 *
 * Copies n_rows token rows of row_elems (= Hkv * d, a multiple of 8) bf16 values, for K and V,
 * from k_src / v_src (rows src_row_stride elements apart) to arena rows
 * [dst_slot, dst_slot + n_rows) (rows arena_row_stride elements apart, arena_slots rows in all).
 * Source and destination must not overlap.  Asynchronous on `stream`.
 * Errors: BLINK_INVALID_ARG (null, alignment, strides), BLINK_OUT_OF_RANGE (rows past the arena).
 * ------------------------------------------------------------------------------------------ */
blink_status blink_kv_to_arena(const blink_bf16 *k_src, const blink_bf16 *v_src, int64_t src_row_stride,
                               int64_t n_rows, int32_t row_elems, blink_bf16 *k_arena, blink_bf16 *v_arena,
                               int64_t arena_row_stride, int64_t arena_slots, int64_t dst_slot, cudaStream_t stream);

/* ------------------------------------------------------------------------------------------
 * Prefix-tail attention -- blink.py PREFIX_CACHE note and `_forward_shared` (the prefix is
 * encoded once; every tail runs against it: same tokens, same positions, only the
 * floating-point order differs), with the arena layout of simit engine.py.
 *
 * For question b, query head h (kv head h / (Hq/Hkv)) and tail row i:
 *   O = softmax(scale * q . [K_pre ; K_tail_b[0..i]]^T) [V_pre ; V_tail_b[0..i]]
 * i.e. every prefix key without a mask and the question's own tail causally.  The prefix part
 * and the tail part are merged by log-sum-exp.
 *
 * q      [rows, Hq, d]   bf16; question b's tail at rows start_b .. start_b + len_b - 1
 * k_pre  [P, Hkv, d]     bf16; position p's keys at k_pre + p * pre_row_stride (elements), so
 * v_pre                  the prefix may be a region of a wider KV arena; pre_row_stride >= Hkv*d
 *                        and a multiple of 8; 16-byte aligned base.  Unused when P == 0.
 * k_tail, v_tail [rows, Hkv, d] bf16, same rows as q
 * d_cu_seqlens [B+1]     len_b = cu[b+1] - cu[b]; in the varlen layout (d_seq_start == NULL)
 *                        start_b = cu[b] - cu[0], so a slice of a larger cu array can be passed
 *                        together with pointers offset by cu[0] rows
 * d_seq_start [B]        right-padded layout: start_b, strictly increasing, rows not shared;
 *                        rows owned by no question get O = 0 and LSE = -inf
 * B                      1..BLINK_MAX_PLAN_SEQUENCES questions
 * rows                   token rows of q / k_tail / v_tail / out (>= 1)
 * P                      prefix length, 0 (plain causal path) .. 131072
 * max_tail               upper bound of len_b, checked on the device; P and max_tail are each at
 *                        most 131072 (blink.py MAX_INPUT_TOKENS bounds one rendered prompt; the
 *                        largest request keeps a full 131072-token prefix plus its tails)
 * Hq, Hkv, d             Hq % Hkv == 0, Hq/Hkv <= 128, d in {64, 128}
 * scale                  softmax scale; <= 0 selects 1/sqrt(d)
 * out   [rows, Hq, d]    bf16 (round to nearest even)
 * lse   [Hq, rows]       optional (may be NULL): fp32 natural-log log-sum-exp of each row
 * d_ws, ws_bytes         workspace of at least blink_attention_workspace(...) bytes, zero-filled
 *                        before its first use; the first word is the device error word
 * Prefix chunks (one request with a prefix; the work units are (row pair, kv head)): when a
 * launch-time model predicts a clear gain, units run their prefix in chunks of key tiles on
 * separate blocks whose partial outputs are merged by LSE in a second kernel (the merge of the
 * prefix and tail parts, applied again), launched as the attention launch's programmatic
 * dependent on `stream`.  Either every unit is cut (a small grid, e.g. a few questions against
 * a long prefix: chunks of at least 4 tiles), or whole waves of units run unsplit and only the
 * units of the last, partial wave are cut, into chunks that run, in the same launch, on the SMs
 * the whole units free first.  The last chunk of a unit, which also runs its tail tiles, takes
 * fewer prefix tiles.  blink_attention_workspace then includes room for the fp32 partials (it
 * sizes them for the current device); with a smaller workspace the call runs unsplit.  Results
 * agree with the unsplit path within the rounding of the merge.
 * Errors: BLINK_INVALID_ARG, BLINK_OUT_OF_RANGE, BLINK_WORKSPACE_TOO_SMALL, BLINK_CUDA_ERROR;
 * device-side: BLINK_DEVICE_FLAG (a length outside 1..max_tail or past `rows`),
 * BLINK_DEVICE_TIMEOUT.
 * ------------------------------------------------------------------------------------------ */
size_t blink_attention_workspace(int32_t rows, int32_t B, int32_t P, int32_t Hq, int32_t Hkv, int32_t d);

/* The prefix-chunk plan blink_prefix_tail_attention uses for one request of `rows` tail rows
 * against a prefix of P tokens, on a GPU with `sms` SMs, when the workspace has room for it (no
 * device call: for inspection and tests).  Units are (row pair, kv head): with g = Hq / Hkv and
 * 128 / g tokens per 128-row tile, ceil(ceil(rows / (128 / g)) / 2) * Hkv of them.
 * *whole_units  units [0, *whole_units) run whole (all units when nothing is cut)
 * *chunks       chunks each remaining unit is cut into (1: nothing is cut)
 * *chunk_tiles  prefix key tiles (128 keys each) of chunks 0 .. chunks-2; the last chunk takes the
 *               remaining 0 .. *chunk_tiles tiles and the unit's tail tiles (with *chunks = 1:
 *               the whole prefix in tiles)
 * Errors: BLINK_INVALID_ARG (a null output, sms < 1, or a shape the attention call rejects). */
blink_status blink_attention_split_plan(int32_t rows, int32_t P, int32_t Hq, int32_t Hkv, int32_t d, int32_t sms,
                                        int64_t *whole_units, int32_t *chunks, int32_t *chunk_tiles);

blink_status blink_prefix_tail_attention(const blink_bf16 *q, const blink_bf16 *k_pre, const blink_bf16 *v_pre,
                                         int64_t pre_row_stride, const blink_bf16 *k_tail,
                                         const blink_bf16 *v_tail, const int32_t *d_cu_seqlens,
                                         const int32_t *d_seq_start, int32_t B, int32_t rows, int32_t P,
                                         int32_t max_tail, int32_t Hq, int32_t Hkv, int32_t d, float scale,
                                         blink_bf16 *out, float *lse, void *d_ws, size_t ws_bytes,
                                         cudaStream_t stream);

/* ------------------------------------------------------------------------------------------
 * Prefix-tail attention over several requests in one launch -- blink.py `logits_many` /
 * `Batcher` (every question of up to 64 requests packed into the same forwards, each request's
 * rows taken only from its own prompts) with simit engine.py's arena (one arena, a region per
 * request).  Request r owns the tail rows [h_req_rows[r], h_req_rows[r+1]) (whole questions
 * only) and attends to its own prefix of h_req_prefix_len[r] tokens at arena slots
 * [h_req_prefix_start[r], + h_req_prefix_len[r]).  Per row the result is exactly that of
 * blink_prefix_tail_attention with the request's prefix.
 *
 * k_arena, v_arena  [arena_slots, Hkv, d] bf16 rows arena_row_stride elements apart
 * n_req             1..64
 * h_req_rows        host [n_req+1], h_req_rows[0] = 0, non-decreasing, h_req_rows[n_req] = rows
 * h_req_prefix_*    host [n_req]; a request with prefix length 0 runs the plain causal path
 * Other arguments and errors as blink_prefix_tail_attention; a question that starts before its
 * request's first row latches BLINK_DEVICE_FLAG.
 * ------------------------------------------------------------------------------------------ */
blink_status blink_prefix_tail_attention_multi(const blink_bf16 *q, const blink_bf16 *k_arena, const blink_bf16 *v_arena,
                                               int64_t arena_row_stride, int64_t arena_slots, const blink_bf16 *k_tail,
                                               const blink_bf16 *v_tail, const int32_t *d_cu_seqlens,
                                               const int32_t *d_seq_start, int32_t B, int32_t rows, int32_t n_req,
                                               const int32_t *h_req_rows, const int32_t *h_req_prefix_start,
                                               const int32_t *h_req_prefix_len, int32_t max_tail, int32_t Hq,
                                               int32_t Hkv, int32_t d, float scale, blink_bf16 *out, float *lse,
                                               void *d_ws, size_t ws_bytes, cudaStream_t stream);

/* ------------------------------------------------------------------------------------------
 * Label readout -- blink.py `_read` / `_read_batched` (the last hidden state of each question
 * against the lm_head rows of its offered labels only, in FP32), `softmax` (z / T, minus the
 * max, exp, normalise), `decide` (the temperature must be positive) and, optionally,
 * `answer_for` (the typed answer per question).
 *
 * hidden [hidden_rows, H] bf16, row r at hidden + r * hidden_row_stride (elements; multiple of 8)
 * d_last_idx              hidden row of each last token (0 <= idx < hidden_rows): indexed by
 *                         question (d_slot_of == NULL) or by slot (question b reads
 *                         d_last_idx[d_slot_of[b]]), so the plan's d_last_varlen / d_slot_of
 *                         can be passed straight through
 * unembed [V, H]          bf16 row-major; H a multiple of 8, 16-byte aligned
 * d_label_off [B+1], d_label_ids [sum_k]  CSR, request order: question b offers
 *                         label_ids[off[b] .. off[b+1]), 1..255 labels each, ids in [0, V)
 * temperature             > 0 and finite
 * d_probs [sum_k]         fp32 output probabilities (CSR like the ids)
 * h_probs                 optional pinned host copy of d_probs; when given the call copies once
 *                         and synchronises the stream, and reports device-side errors
 * d_logits [sum_k]        optional fp32 raw logits (before the temperature)
 * d_qtype [B], d_answers [B][3], h_answers   optional, together: blink.py `answer_for` on the device.
 *                         d_qtype[b] is 0 (choice), 1 (noul: first label = "yes") or 2 (score:
 *                         label i = level i); d_answers[b] = {index, confidence, value} as fp32:
 *                         the chosen label (first of equal probabilities), for a choice
 *                         (p_best - 1/K)/(1 - 1/K) and p_best, for a score the same confidence
 *                         clamped to [0, 1] and the expected level sum_i i p_i, for a noul NaN and
 *                         p_yes (probabilities renormalised first).  h_answers (pinned) receives a
 *                         copy in the same synchronising host transfer as h_probs.
 * d_ws, ws_bytes          workspace of blink_label_readout_workspace(B) bytes, zero-filled before
 *                         its first use; the call leaves its counters at zero
 * A label id outside [0, V) makes that question's probabilities NaN and latches
 * BLINK_DEVICE_FLAG; so do malformed offsets (then no probability is written).
 * ------------------------------------------------------------------------------------------ */
size_t blink_label_readout_workspace(int32_t B);

blink_status blink_label_readout(const blink_bf16 *hidden, int64_t hidden_row_stride, int32_t hidden_rows,
                                 const int32_t *d_last_idx, const int32_t *d_slot_of, const blink_bf16 *unembed,
                                 int32_t V, int32_t H,
                                 const int32_t *d_label_off, const int32_t *d_label_ids, int32_t B,
                                 int32_t sum_k, float temperature, float *d_probs, float *h_probs,
                                 float *d_logits, const int32_t *d_qtype, float *d_answers, float *h_answers,
                                 void *d_ws, size_t ws_bytes, cudaStream_t stream);

/* ------------------------------------------------------------------------------------------
 * Log-space readout over several option orders -- the ruling engine (engine.py `_score_plain`,
 * `_prior`, `answer`): each question is scored in passes, one per order of its options; per
 * pass the answer codes' logits z (from blink_label_readout's d_logits) give
 *   lp_j = z_j - logsumexp(z) - prior_K[j]          (position j of the pass)
 * and option i's raw score is the mean of lp over the passes, taken at the position each pass
 * showed option i in.  Then p = softmax(raw / T) and, optionally, the typed answer (as in
 * blink_label_readout).
 *
 * d_logits [..]          pass p's K logits at d_logits[d_pass_off[p] .. d_pass_off[p+1])
 * d_key_of_pos [..]      same layout: the option index (0..K-1) pass p shows at each position;
 *                        each pass's entries must be a permutation of 0..K-1
 * n_pass, d_pass_off [n_pass+1]
 * d_question_pass [B+1]  question q's passes are [d_question_pass[q], d_question_pass[q+1]) (>= 1)
 * d_raw_off [B+1], sum_k question q's options at [d_raw_off[q], d_raw_off[q+1]) of d_raw/d_probs;
 *                        every pass of q has that many positions (1..255)
 * d_prior                optional [255][255] fp32: row K-1 holds the content-free log-probability
 *                        of each position for K options (NULL: no prior subtracted)
 * temperature            > 0 and finite
 * d_raw [sum_k]          optional output: the mean debiased log-probabilities
 * d_probs [sum_k]        output: softmax(raw / T); h_probs optional pinned copy
 * d_qtype, d_answers, h_answers  optional typed answers, as for blink_label_readout
 * d_ws, ws_bytes         blink_rotation_debias_workspace() bytes (error word)
 * A malformed table (a pass of the wrong size, an option index out of range) latches
 * BLINK_DEVICE_FLAG and makes that question's probabilities NaN.
 * ------------------------------------------------------------------------------------------ */
size_t blink_rotation_debias_workspace(void);

blink_status blink_rotation_debias(const float *d_logits, const int32_t *d_pass_off, const int32_t *d_key_of_pos,
                                   int32_t n_pass, const int32_t *d_question_pass, const int32_t *d_raw_off, int32_t B,
                                   int32_t sum_k, const float *d_prior, float temperature, float *d_raw,
                                   float *d_probs, float *h_probs, const int32_t *d_qtype, float *d_answers,
                                   float *h_answers, void *d_ws, size_t ws_bytes, cudaStream_t stream);

/* ------------------------------------------------------------------------------------------
 * Label readout that allocates nothing.  The pages have no counterpart: this entry point is an
 * addition of this library for callers that cannot hand it a workspace.
 *
 * Who needs it: code embedded in a host that gives it only its input and output buffers and
 * owns every other byte of device memory (a serving runtime with a fixed memory plan made at
 * start-up), and latency-critical loops that must never call cudaMalloc, which may synchronise
 * the whole device.  Such callers cannot provide the `d_ws` that blink_label_readout needs.
 *
 * Arguments and results are those of blink_label_readout without d_ws / ws_bytes and without the
 * answer outputs.  The scratch
 * (an error word and one ticket per question) is a static device array of
 * 256 + 4 * BLINK_STATIC_SCRATCH_QUESTIONS bytes (128.25 KiB) that every GPU which loads this
 * library keeps until the process exits.
 *   - B above BLINK_STATIC_SCRATCH_QUESTIONS returns BLINK_OUT_OF_RANGE; nothing is launched.
 *   - The first call on a device looks up the array's device address with that device current
 *     (cudaGetSymbolAddress); make that first call before any stream capture on the device.  The
 *     address is kept per device and context: after a device reset (a new context, so a new copy
 *     of the array) the next call looks it up again, and that call too should come before any
 *     capture.
 *   - From 8192 labels on, the softmaxes run in a second launch (as in blink_label_readout), so
 *     only the error word is used; below that, one ticket per question as well.
 *   - Every call first clears the array's error word and tickets on `stream`.  All calls share
 *     the one array, which keeps the last call's contents: calls whose work can overlap on the
 *     GPU (different streams with no ordering between them) race, and must not be made.
 *   - Device-side errors are reported only through the host-output path (h_probs != NULL).
 *   - No cudaMalloc, cudaFree or other allocating routine is called.
 * ------------------------------------------------------------------------------------------ */
#define BLINK_STATIC_SCRATCH_QUESTIONS 32768

blink_status blink_label_readout_noalloc(const blink_bf16 *hidden, int64_t hidden_row_stride, int32_t hidden_rows,
                                         const int32_t *d_last_idx, const int32_t *d_slot_of,
                                         const blink_bf16 *unembed, int32_t V, int32_t H, const int32_t *d_label_off,
                                         const int32_t *d_label_ids, int32_t B, int32_t sum_k, float temperature,
                                         float *d_probs, float *h_probs, float *d_logits, cudaStream_t stream);

/* ------------------------------------------------------------------------------------------
 * Attention weight received by each prefix key -- the quantity a cache is evicted by.  The pages
 * evict whole cached prefixes; this call and the next are additions of this library for callers
 * that shorten a cached prefix instead (long documents held for many questions).
 *
 * For kv head h and prefix position p:
 *   w[h][p] = decay * prev[h][p] + sum over rows i and the g = Hq / Hkv query heads j of the group
 *             of exp(scale * q[i][h g + j] . k_pre[p][h] - lse[h g + j][i])
 * i.e. the softmax weights blink_prefix_tail_attention gave that key, summed over the rows and the
 * query heads that share it, when lse is that call's output.  A row whose lse is -inf (a row owned
 * by no question) adds nothing, whatever its q or the keys hold; a NaN in any other row or its lse makes
 * the weights of that kv head NaN, a NaN or an infinity in a key what the formula gives for that key
 * alone.  lse must not be smaller than the scores it normalises by more than
 * 80 (an attention's own lse never is).
 *
 * q       [rows, Hq, d] bf16, rows in 1..2^30 (one row: a single decoded token)
 * k_pre   [P, Hkv, d]   bf16 rows pre_row_stride elements apart, as for the attention; P in 1..131072
 * lse     fp32 natural-log log-sum-exp, head h at lse + h * lse_stride (lse_stride >= rows), so the
 *         rows of one request can be passed as a slice of a larger launch
 * scale   softmax scale; <= 0 selects 1/sqrt(d).  d in {64, 128}, Hq/Hkv <= 128
 * decay   finite, >= 0; 0: d_prev is not read and may be NULL
 * d_prev  fp32, head h at d_prev + h * prev_stride (stride >= P); may be d_weights itself with the
 *         same stride (accumulation in place), otherwise the two must not overlap
 * d_weights  fp32 output, head h at d_weights + h * w_stride (stride >= P)
 * d_ws    workspace of blink_prefix_key_weights_workspace(...) bytes, 16-byte aligned, its first 256
 *         zero-filled before its first use; not shared by calls that may run at the same time
 * The sum's order is fixed by the shapes and the GPU: repeated calls give the same bits.
 * Errors: BLINK_INVALID_ARG, BLINK_OUT_OF_RANGE, BLINK_WORKSPACE_TOO_SMALL, BLINK_CUDA_ERROR;
 * device-side: BLINK_DEVICE_TIMEOUT.
 * ------------------------------------------------------------------------------------------ */
size_t blink_prefix_key_weights_workspace(int32_t rows, int32_t P, int32_t Hq, int32_t Hkv, int32_t d);

blink_status blink_prefix_key_weights(const blink_bf16 *q, const blink_bf16 *k_pre, int64_t pre_row_stride,
                                      const float *lse, int64_t lse_stride, int32_t rows, int32_t P, int32_t Hq,
                                      int32_t Hkv, int32_t d, float scale, float decay, const float *d_prev,
                                      int64_t prev_stride, float *d_weights, int64_t w_stride, void *d_ws,
                                      size_t ws_bytes, cudaStream_t stream);

/* ------------------------------------------------------------------------------------------
 * Eviction of a cached prefix's lightest keys -- every kv head keeps `keep` of its P keys and its
 * arena region is compacted to slots [0, keep).  Keys carry their positions (they are stored after
 * the rotation), so the attention reads the kept ones in any order: pass P = keep to it.
 *
 * Order of a head's keys: protected keys first (position < sink or >= recent_from), then larger
 * weight first (a NaN weight counts as the smallest), then lower slot first; the first `keep` are
 * kept.  A kept key in a slot below `keep` stays there; the other slots below `keep` receive the kept
 * keys of the slots at `keep` and above, both in ascending slot order.  So at most min(keep, P - keep)
 * keys per head move when the region is compacted in place.
 *
 * d_weights   fp32, head h's P weights at d_weights + h * w_stride
 * d_pos       int32, original position of the key in each slot, head h at d_pos + h * pos_stride;
 *             NULL: slot s holds position s (a region that was never evicted)
 * P, keep     1 <= keep <= P <= 131072
 * sink        >= 0; recent_from >= 0 (INT32_MAX protects no recent position)
 * k, v        [P, Hkv, d] bf16 rows row_stride elements apart (d a multiple of 8, at most 1024;
 *             16-byte aligned; strides multiples of 8)
 * k_dst, v_dst  where the kept keys go, rows dst_row_stride elements apart: k and v themselves with
 *             the same stride (in place), or memory that overlaps neither k nor v
 * d_slots     [Hkv][keep] int32 output: the slot each kept key came from
 * d_weights_dst, d_pos_dst  optional outputs [Hkv][keep] (row strides wd_stride, pd_stride): weights
 *             and positions of the kept keys; each may be its input itself with the same stride, or
 *             memory that overlaps neither input
 * d_ws        workspace of blink_kv_evict_workspace(...) bytes, 16-byte aligned; not shared by calls that
 *             may run at the same time (its error word is never set: nothing on the device can fail here)
 * Errors: BLINK_INVALID_ARG (null, alignment, strides, overlap), BLINK_OUT_OF_RANGE (P, keep, Hkv, d),
 * BLINK_WORKSPACE_TOO_SMALL, BLINK_CUDA_ERROR.
 * ------------------------------------------------------------------------------------------ */
size_t blink_kv_evict_workspace(int32_t P, int32_t keep, int32_t Hkv);

blink_status blink_kv_evict(const float *d_weights, int64_t w_stride, const int32_t *d_pos, int64_t pos_stride,
                            int32_t P, int32_t keep, int32_t sink, int32_t recent_from, int32_t Hkv, int32_t d,
                            const blink_bf16 *k, const blink_bf16 *v, int64_t row_stride, blink_bf16 *k_dst,
                            blink_bf16 *v_dst, int64_t dst_row_stride, int32_t *d_slots, float *d_weights_dst,
                            int64_t wd_stride, int32_t *d_pos_dst, int64_t pd_stride, void *d_ws, size_t ws_bytes,
                            cudaStream_t stream);

/* ------------------------------------------------------------------------------------------
 * Log probabilities over the whole vocabulary -- the label readout's next-token distribution
 * without the restriction to the offered labels: how likely a given token is, how uncertain the
 * model is, and which tokens it prefers (so also how much of the distribution the labels hold).
 *
 * For row r: z = hidden[idx[r]] . unembed^T / temperature (FP32 accumulation; the logits are never
 * written to memory), lse = logsumexp(z), and
 *   d_logprob[r] = z[d_targets[r]] - lse      d_entropy[r] = lse - sum softmax(z) z  (nats)
 *   d_lse[r] = lse      d_top_ids[r][j], d_top_logprobs[r][j]: the j-th largest z - lse, equal
 *   logits by ascending token id
 *
 * hidden [hidden_rows, H] bf16, row r at hidden + r * hidden_row_stride (multiple of 8 elements)
 * d_row_idx  int32 [n] hidden rows (in any order, repeats allowed); NULL: row r of hidden (n <= hidden_rows)
 * unembed [V, H] bf16 row-major; H a multiple of 8, 16-byte aligned; H in 8..32768, V in 1..2^24
 * n          1..131072 rows (one row: a single decoded token)
 * d_targets  int32 [n]; -1: the row has no target (its log probability is NaN).  NULL without d_logprob
 * temperature  > 0, finite, and not so small that log2(e) / temperature is not (4.3e-39); logits divided by it
 *            have to stay within 1e38
 * top        0..BLINK_MAX_TOP_TOKENS alternatives per row, at most V
 * Outputs: each may be NULL, not all; d_top_ids and d_top_logprobs [n][top] together, when top > 0
 * d_ws       workspace of blink_token_logprobs_workspace(...) bytes (of the current device; one for n rows
 *            serves calls of fewer), 16-byte aligned,
 *            its first 256 zero-filled before its first use; not shared by calls that may run at the same time
 * A row index outside [0, hidden_rows) latches BLINK_DEVICE_FLAG and makes the row's outputs NaN and
 * -1; a target outside [-1, V) latches it and makes that log probability NaN.  A row with a NaN logit
 * gets NaN (ids: those of its other logits, then -1); logits must not be infinite.
 * Errors: BLINK_INVALID_ARG, BLINK_OUT_OF_RANGE, BLINK_WORKSPACE_TOO_SMALL, BLINK_CUDA_ERROR;
 * device-side: BLINK_DEVICE_FLAG, BLINK_DEVICE_TIMEOUT.
 * ------------------------------------------------------------------------------------------ */
#define BLINK_MAX_TOP_TOKENS 32

size_t blink_token_logprobs_workspace(int32_t n, int32_t H, int32_t V, int32_t top);

/* The workspace of a call on a GPU with `sms` SMs (host computation only): *ws_bytes is what the query above gives
 * there, which is never less for more rows, and *used the most that a launch of the call lays out. */
blink_status blink_token_logprobs_workspace_plan(int32_t n, int32_t H, int32_t V, int32_t top, int32_t sms,
                                                 size_t *ws_bytes, size_t *used);

blink_status blink_token_logprobs(const blink_bf16 *hidden, int64_t hidden_row_stride, int32_t hidden_rows,
                                  const int32_t *d_row_idx, const blink_bf16 *unembed, int32_t V, int32_t H,
                                  const int32_t *d_targets, int32_t n, float temperature, int32_t top,
                                  float *d_logprob, float *d_entropy, float *d_lse, int32_t *d_top_ids,
                                  float *d_top_logprobs, void *d_ws, size_t ws_bytes, cudaStream_t stream);

/* ------------------------------------------------------------------------------------------
 * Rotary positions -- the step before the path, whose calls take rotated queries and keys: pair i
 * of each head turns by position * theta_i, theta_i = base^(-2 i / rot).
 *
 * blink_rope_table computes the frequencies on the host, once per model: h_turns [rot/2] gets
 * theta_i / (2 pi) as a fraction of a turn times 2^64 (copy it to the device for the calls below), and
 * *h_amplitude the factor of the rotated values that belongs to the scaling (1 but for BY_DIM).
 *   rot        even, 2..BLINK_MAX_ROPE_DIM: values of a head that turn
 *   base       > 1
 *   scaling    for contexts longer than the model was trained on (`original` tokens), by `factor` >= 1:
 *     PLAIN      theta_i as above (the other arguments are not read)
 *     LINEAR     theta_i / factor
 *     BASE       base * factor^(rot / (rot - 2)) in place of base (rot >= 4)
 *     BY_DIM     pairs below lo keep theta_i, pairs from hi on get theta_i / factor, a linear ramp over i
 *                between: lo = floor(i(high)), hi = ceil(i(low)), where pair i(n) = rot ln(original /
 *                (2 pi n)) / (2 ln base) turns n times over the original context (lo >= 0, hi <= rot - 1);
 *                the amplitude is 0.1 ln(factor) + 1
 *     BY_TURNS   with n_i = original theta_i / (2 pi) turns over the original context, the share
 *                (n_i - low) / (high - low), clipped to 0..1, of theta_i and the rest of theta_i / factor
 *   low, high  0 < low < high, in turns over the original context (BY_DIM, BY_TURNS)
 *
 * blink_rope turns the first `rot` values of every head of q and, if given, k, and copies the others:
 * (y0, y1) = amplitude (x0 cos - x1 sin, x0 sin + x1 cos), in 32 bits, rounded once.
 *   q [rows, Hq, d], k [rows, Hkv, d]  bf16, heads d apart, rows *_stride elements apart (slices of one
 *               projection's rows are fine); k NULL: q alone.  Any alignment of 2 bytes; fastest where
 *               addresses, strides, d and (halves) rot/2 are multiples of 8 values
 *   d_positions [rows]   any int32 values (negative ones turn back)
 *   d           2..BLINK_MAX_ROPE_DIM;  rows 0..2^30 (0: nothing is done)
 *   interleaved 0: pair i is values (i, i + rot/2); 1: values (2 i, 2 i + 1)
 *   q_out, k_out  as q and k: the same memory with the same stride (in place), or memory that overlaps
 *               neither input nor the other output
 * Errors: BLINK_INVALID_ARG, BLINK_OUT_OF_RANGE, BLINK_CUDA_ERROR.
 * ------------------------------------------------------------------------------------------ */
#define BLINK_MAX_ROPE_DIM 512
#define BLINK_ROPE_PLAIN 0
#define BLINK_ROPE_LINEAR 1
#define BLINK_ROPE_BASE 2
#define BLINK_ROPE_BY_DIM 3
#define BLINK_ROPE_BY_TURNS 4

blink_status blink_rope_table(int32_t rot, double base, int32_t scaling, double factor, int32_t original, double low,
                              double high, uint64_t *h_turns, float *h_amplitude);

blink_status blink_rope(const blink_bf16 *q, int64_t q_stride, const blink_bf16 *k, int64_t k_stride,
                        const int32_t *d_positions, int32_t rows, int32_t Hq, int32_t Hkv, int32_t d, int32_t rot,
                        const uint64_t *d_turns, float amplitude, int32_t interleaved, blink_bf16 *q_out,
                        int64_t q_out_stride, blink_bf16 *k_out, int64_t k_out_stride, cudaStream_t stream);

/* ------------------------------------------------------------------------------------------
 * The 8-bit paged cache -- half the bytes of the arena, in pages that sequences take as they grow and
 * requests with a common prefix share.  The caller owns it:
 *
 * k_codes, v_codes  pages of `page_tokens` (16, 32, 64 or 128) tokens, [Hkv][page_tokens][d] e4m3 codes
 *                   each, page_stride bytes apart (>= Hkv * page_tokens * d, a multiple of 16; 16-byte
 *                   aligned), d in {64, 128}, Hkv 1..BLINK_MAX_PAGED_HEADS
 * k_scale, v_scale  [Hkv] e8m0 scales each (a byte b stands for 2^(b - 127)), scale_stride bytes apart:
 *                   a value is its code times the scale of its page and head.  e is read as the nearest in
 *                   BLINK_PAGED_SCALE_MIN..MAX, which the calls write (a page of zeros is zeros)
 * d_page_table      int32, sequence s's pages at d_page_table + s * table_stride, table_width of them:
 *                   token p lies in slot p % page_tokens of page p / page_tokens
 *
 * blink_paged_append writes the next tokens of S sequences and turns their keys on the way.  With m the
 * largest finite magnitude of the tokens that a page gets for a head, the scale is the smallest 2^e with
 * m <= 448 * 2^e, e in BLINK_PAGED_SCALE_MIN..MAX (m of the keys turned in 32 bits); a code is value / scale rounded to the
 * nearest (ties to even) and at most 448, an infinity too, a NaN stays one.  Turned keys' codes are those of the exact rotation,
 * but those of a page and head among whose new keys is an infinity, which are of the 32-bit one.  A page that holds tokens of the sequence already (start is
 * not a multiple of page_tokens) keeps its scale if that is larger; if the scale grows, its tokens' codes
 * are rounded again, which changes only those that become subnormal.  Slots that get no token keep
 * their codes.
 * k [n, Hkv, d], v  bf16, rows *_stride elements apart (multiples of 8, 16-byte aligned); keys not yet rotated; n 0:
 *                   nothing is done or checked on the device
 * d_cu_new [S+1]    sequence s's tokens are rows cu[s] - cu[0] .. of k and v (none is fine)
 * d_start [S]       tokens that the sequence holds; its new ones follow them
 * S, max_new        1..BLINK_MAX_PLAN_SEQUENCES; upper bound of the new tokens of a sequence, checked on the
 *                   device (at most 131072)
 * d_positions [n]   positions of the rows, or NULL: start + 0, 1, ...
 * d_turns, rot, amplitude, interleaved  as for blink_rope; rot 0: the keys are rotated already
 * d_ws              blink_paged_append_workspace() bytes: the error word
 * A page that two sequences share must not be written (sharers append to pages of their own).  A bad length,
 * a page index outside [0, n_pages) or past table_width latches BLINK_DEVICE_FLAG; those pages are not written.
 * Where d_cu_new falls, which of the other sequences are written is open.
 * Errors: BLINK_INVALID_ARG, BLINK_OUT_OF_RANGE, BLINK_WORKSPACE_TOO_SMALL, BLINK_CUDA_ERROR.
 * ------------------------------------------------------------------------------------------ */
#define BLINK_MAX_PAGED_HEADS 1024
#define BLINK_MAX_PAGED_TOKENS 64
#define BLINK_PAGED_SCALE_MIN (-48)
#define BLINK_PAGED_SCALE_MAX 32

size_t blink_paged_append_workspace(void);

blink_status blink_paged_append(const blink_bf16 *k, int64_t k_stride, const blink_bf16 *v, int64_t v_stride, int32_t n,
                                int32_t Hkv, int32_t d, uint8_t *k_codes, uint8_t *v_codes, uint8_t *k_scale,
                                uint8_t *v_scale, int64_t page_stride, int64_t scale_stride, int32_t n_pages,
                                int32_t page_tokens, const int32_t *d_page_table, int64_t table_stride,
                                int32_t table_width, const int32_t *d_cu_new, const int32_t *d_start, int32_t S,
                                int32_t max_new, const int32_t *d_positions, const uint64_t *d_turns, int32_t rot,
                                float amplitude, int32_t interleaved, void *d_ws, size_t ws_bytes, cudaStream_t stream);

/* ------------------------------------------------------------------------------------------
 * Attention of each sequence's last tokens over its pages -- the single-token form (T = 1), or a few
 * tokens at once (a draft to verify).  The tokens' own keys and values are in the pages already.
 *
 * For sequence s with len cached tokens, token t of T, query head h (kv head h / (Hq/Hkv)):
 *   out = softmax(scale * q . K[0 .. len - T + t]^T) V[0 .. len - T + t]
 * q, out [S, T, Hq, d] bf16; lse [Hq, S * T] optional (may be NULL), fp32 natural log
 * d_len [S]      cached tokens, on the device, so that a captured graph follows a growing cache; a token
 *                that sees no key (len < T - t) gets zeros and -inf
 * max_len        upper bound of d_len (0..131072), which decides how the work is cut
 * S, T           1..BLINK_MAX_PLAN_SEQUENCES, 1..BLINK_MAX_PAGED_TOKENS; Hq/Hkv <= 128, and
 *                Hkv * ceil(T Hq/Hkv / 16) <= 65535
 * scale          softmax scale; <= 0 selects 1/sqrt(d)
 * d_ws           blink_paged_token_attention_workspace(...) bytes (of the current device), 16-byte aligned, its first
 *                256 zero-filled before its first use; not shared by calls that may run at the same time
 * Scores are exact products of the 8-bit values in 32-bit sums; weights enter the second product in fp16.
 * Keys that a token does not see have no influence, whatever their slots hold.  The same call gives the same bits.
 * A length outside 0..max_len or past the table is cut to that, a page index outside [0, n_pages) counts as
 * absent; both latch BLINK_DEVICE_FLAG.
 * Errors: BLINK_INVALID_ARG, BLINK_OUT_OF_RANGE, BLINK_WORKSPACE_TOO_SMALL, BLINK_CUDA_ERROR.
 * ------------------------------------------------------------------------------------------ */
size_t blink_paged_token_attention_workspace(int32_t S, int32_t T, int32_t max_len, int32_t Hq, int32_t Hkv, int32_t d);

blink_status blink_paged_token_attention(const blink_bf16 *q, const uint8_t *k_codes, const uint8_t *v_codes,
                                         const uint8_t *k_scale, const uint8_t *v_scale, int64_t page_stride,
                                         int64_t scale_stride, int32_t n_pages, int32_t page_tokens,
                                         const int32_t *d_page_table, int64_t table_stride, int32_t table_width,
                                         const int32_t *d_len, int32_t S, int32_t T, int32_t max_len, int32_t Hq,
                                         int32_t Hkv, int32_t d, float scale, blink_bf16 *out, float *lse, void *d_ws,
                                         size_t ws_bytes, cudaStream_t stream);

/* ------------------------------------------------------------------------------------------
 * Prefix-tail attention with the prefixes in pages -- blink_prefix_tail_attention (one request) and
 * blink_prefix_tail_attention_multi (several) for a prefix held in 8 bits.  Request r owns the tail rows
 * [h_req_rows[r], h_req_rows[r+1]) (whole questions) and attends to the first h_prefix_len[r] tokens of row r
 * of the page table; tails are bf16, as there.  Requests may share pages.
 *
 * h_req_rows [n_req+1], h_prefix_len [n_req]  host arrays; lengths 0..131072, n_req 1..64
 * d_ws   blink_paged_prefix_tail_workspace(...) bytes (of the current device), 32-byte aligned, its first 256
 *        zero-filled before its first use; not shared by calls that may run at the same time; one serves the
 *        caches of all layers
 * Where no request has more than 64 rows times Hq/Hkv the pages are read as they are (weights enter the second
 * product in fp16, a question's own keys in 32 bits); otherwise the workspace holds the prefixes as bf16 rows,
 * exactly, and the result is that of the calls named.
 * Other arguments as there.  A page index outside [0, n_pages) latches BLINK_DEVICE_FLAG; its keys and values are zeros
 * either way (they score 0 and have that weight).
 * Errors: BLINK_INVALID_ARG, BLINK_OUT_OF_RANGE, BLINK_WORKSPACE_TOO_SMALL, BLINK_CUDA_ERROR; device-side:
 * BLINK_DEVICE_FLAG, BLINK_DEVICE_TIMEOUT.
 * ------------------------------------------------------------------------------------------ */
size_t blink_paged_prefix_tail_workspace(const int32_t *h_req_rows, const int32_t *h_prefix_len, int32_t n_req, int32_t B,
                                         int32_t Hq, int32_t Hkv, int32_t d);

blink_status blink_paged_prefix_tail_attention(const blink_bf16 *q, const uint8_t *k_codes, const uint8_t *v_codes,
                                               const uint8_t *k_scale, const uint8_t *v_scale, int64_t page_stride,
                                               int64_t scale_stride, int32_t n_pages, int32_t page_tokens,
                                               const int32_t *d_page_table, int64_t table_stride, int32_t table_width,
                                               const blink_bf16 *k_tail, const blink_bf16 *v_tail,
                                               const int32_t *d_cu_seqlens, const int32_t *d_seq_start, int32_t B,
                                               int32_t rows, int32_t n_req, const int32_t *h_req_rows,
                                               const int32_t *h_prefix_len, int32_t max_tail, int32_t Hq, int32_t Hkv,
                                               int32_t d, float scale, blink_bf16 *out, float *lse, void *d_ws,
                                               size_t ws_bytes, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* BLINK_H */
