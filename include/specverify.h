/*
 * specverify -- the verify step of speculative sampling on AMD Instinct
 * MI355X (gfx950), as a C ABI.
 *
 * The operation (cited by page title and section):
 *   "CS3602_FINAL_SpeDec", section 2 (perplexity test) and its proof: p is
 *   the target distribution, q the draft distribution; a guess x ~ q is
 *   accepted with probability min(1, p(x)/q(x)); at the first rejection the
 *   token is drawn from the residual p' = norm(max(0, p - q)), whose
 *   normaliser is 1 - beta with beta = sum_x min(p(x), q(x)); this makes the
 *   emitted token exactly p-distributed.
 *   "Text Generation via Speculative Sampling, KV Caching, and OpenVINO",
 *   section "Prepare speculative sampling", steps 3 and 4: one uniform draw per
 *   draft position, stop at the first rejection, and draw one extra token from
 *   the last target position when every guess was accepted; section "Prepare
 *   autoregressive sampling": softmax over the vocabulary, argmax decode
 *   (the greedy mode here).  spec_draft_sample draws the guesses themselves
 *   (step 1 of "Prepare speculative sampling", sampling in place of the
 *   argmax), and spec_token_likelihood scores given tokens under the
 *   speculative step (the perplexity check of "CS3602_FINAL_SpeDec").
 *
 * Conventions shared by the calls
 *   Batch layout (packed, ragged).  Sequence b has K_b >= 0 draft tokens.
 *   With cu_draft == NULL every K_b equals shape->max_draft; otherwise
 *   cu_draft is a DEVICE array of B+1 int32 prefix sums (cu_draft[0] = 0,
 *   cu_draft[b+1] - cu_draft[b] = K_b, cu_draft[B] = shape->total_draft).
 *   Target rows: sequence b owns rows cu_draft[b] + b + k for k = 0..K_b
 *   (K_b + 1 rows; row K_b is the extra-token position).  Draft rows:
 *   cu_draft[b] + k for k = 0..K_b-1.  draft_ids[cu_draft[b] + k] is the
 *   guess at position k.  Each row holds `vocab` logits, row-major, with
 *   row_stride elements between row starts.
 *
 *   Output tokens: out_tokens[cu_draft[b] + b + j] for j = 0..K_b holds the
 *   accepted guesses x_0..x_{n-1}, then the new token at j = n, then -1.
 *   out_num_accepted[b] = n (0 <= n <= K_b), or -1 when the sequence's
 *   cu_draft entries or draft ids are out of range (then its token slots are
 *   left untouched).
 *
 *   Memory.  Every pointer is device memory owned by the caller.  The
 *   library allocates nothing and keeps no state between calls; it reads
 *   the inputs, overwrites the outputs and uses `workspace` as scratch.
 *   Vectorised reads may touch bytes outside a row that share its 16-byte
 *   aligned blocks (never outside those blocks); the values read there are
 *   discarded.  Logit pointers must be aligned to their element size.
 *
 *   Execution.  Asynchronous on `stream` (NULL = the null stream); no host
 *   synchronisation inside the call.  Concurrent calls are safe when they
 *   use different workspaces and outputs.  Results are a pure function of
 *   (inputs, temperature, top_k, seed, offset): bit-identical across runs.
 *
 *   Workspace.  Call once with workspace == NULL: *workspace_bytes receives
 *   the size needed for this shape and mode and nothing is launched.  Then
 *   call with a device buffer of at least that many bytes (256-byte aligned).
 *
 *   Errors.  Argument checks are synchronous and happen before any launch:
 *   SV_ERR_INVALID_ARGUMENT (null or misaligned pointer, B < 1, V < 1,
 *   K < 0, total_draft inconsistent with B*K when cu_draft is NULL, stride
 *   < V, temperature not finite and > 0, or so small that log2(e) / T
 *   overflows fp32 (T below about 4.2e-39), top_k < 0 or > V),
 *   SV_ERR_UNSUPPORTED (V > SV_MAX_VOCAB, max_draft > SV_MAX_DRAFT),
 *   SV_ERR_WORKSPACE_TOO_SMALL, SV_ERR_HIP (a launch failed).  Data
 *   preconditions are the caller's: logits finite or -inf with at least one
 *   finite logit in each row's kept set, and |logit| * log2(e) / T finite in
 *   fp32; cu_draft monotone.  The kernels
 *   never read out of bounds when they are violated: a bad sequence reports
 *   num_accepted = -1.
 */
#ifndef SPECVERIFY_H
#define SPECVERIFY_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#if defined(SPECVERIFY_BUILDING)
#define SV_API __attribute__((visibility("default")))
#else
#define SV_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

#define SV_MAX_VOCAB (1 << 20)
#define SV_MAX_DRAFT 128

typedef enum {
    SV_OK = 0,
    SV_ERR_INVALID_ARGUMENT = 1,
    SV_ERR_UNSUPPORTED = 2,
    SV_ERR_WORKSPACE_TOO_SMALL = 3,
    SV_ERR_HIP = 4
} sv_status_t;

/* Logit element types.  Every type is widened exactly to fp32 on load and no
 * probability is ever formed in 16 bits ("CS3602_FINAL_SpeDec", problem
 * analysis, item 1: fp16 probabilities underflow).  SV_DTYPE_F16 is IEEE
 * binary16, the precision the pages' models ran in. */
typedef enum { SV_DTYPE_F32 = 0, SV_DTYPE_BF16 = 1, SV_DTYPE_F16 = 2 } sv_dtype_t;

typedef struct {
    int32_t batch;             /* B >= 1                                          */
    int32_t max_draft;         /* K, or the largest K_b when cu_draft != NULL     */
    int32_t total_draft;       /* sum_b K_b; must be B*K when cu_draft == NULL    */
    int32_t vocab;             /* V >= 1                                          */
    sv_dtype_t dtype;          /* element type of both logit tensors              */
    int64_t target_row_stride; /* elements between target rows, >= V             */
    int64_t draft_row_stride;  /* elements between draft rows, >= V              */
    const int32_t* cu_draft;   /* device [B+1] prefix sums of K_b, or NULL        */
} sv_shape_t;

/*
 * Speculative sampling verify.
 *   p_k = softmax(target row k / T) and q_k = softmax(draft row k / T), each
 *   restricted to its own top-k kept set when top_k > 0 (every id whose raw
 *   logit is >= the top_k-th largest, ties kept; top_k = 0 or V keeps all),
 *   then, when top_p < 1, to its own top-p nucleus: every id whose logit is
 *   >= tau_p, the largest logit value t for which the probability of
 *   {v : l_v >= t} reaches top_p (ties kept), renormalised.  Top-K and
 *   Top-P are the two filters the sampling helpers of "CS3602_FINAL_SpeDec"
 *   name (its module list; problem analysis, item 2).
 *   Position k accepts iff u_k < min(1, p_k(x_k) / q_k(x_k)) (q = 0 accepts
 *   iff p > 0), u_k = U(b, k, 0).  n = the first rejected position, or K_b.
 *   If n < K_b the new token is the first id (ascending) whose running sum
 *   of max(0, p_n - q_n) exceeds U(b, n, 1) times its total; otherwise it is
 *   the inverse-CDF draw of p_{K_b} with U(b, K_b, 2).
 *   U(b, pos, purpose) = (w >> 8) * 2^-24 where w is word 0 of
 *   Philox4x32-10 (Salmon et al., SC'11) with key (seed lo32, seed hi32)
 *   and counter (b, pos, purpose, offset).
 * Arguments
 *   target_logits [rows_t, stride] and draft_logits [rows_d, stride] in
 *   shape->dtype; draft_ids int32 [total_draft] in [0, V).
 *   temperature > 0, finite, and >= about 4.2e-39 (log2(e) / T must be a
 *   finite fp32).  top_k in [0, V].  top_p in (0, 1]; 1 is
 *   off.  top-p over full rows costs several extra reads of each row (a
 *   mass-weighted radix select); after top-k it works on the kept lists.
 *   out_tokens int32 [total_draft + B]; out_num_accepted int32 [B];
 *   out_probs (nullable) float [total_draft][2] = p_k(x_k), q_k(x_k) for
 *   every draft position; out_residual_mass (nullable) float [B] = the
 *   residual total sum_v max(0, p_n - q_n) = 1 - beta_n (0 if all accepted).
 */
SV_API sv_status_t spec_verify_sample(const sv_shape_t* shape,
                               const void* target_logits,
                               const void* draft_logits,
                               const int32_t* draft_ids,
                               float temperature,
                               int32_t top_k,
                               float top_p,
                               uint64_t seed,
                               uint32_t offset,
                               int32_t* out_tokens,
                               int32_t* out_num_accepted,
                               float* out_probs,
                               float* out_residual_mass,
                               void* workspace,
                               size_t* workspace_bytes,
                               hipStream_t stream);

/*
 * spec_verify_sample for callers that cannot allocate device memory (code
 * under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc): the same call, results and errors, with no workspace
 * argument.  Its scratch is one file-scope device array of
 * SV_NOALLOC_SCRATCH_BYTES that each GPU the library runs on holds until
 * the process ends; its address is taken once per device, on the first call
 * made with that device current.  The call allocates nothing.
 *   A shape and mode whose workspace (the size spec_verify_sample's query
 *   reports) exceeds SV_NOALLOC_SCRATCH_BYTES is rejected with
 *   SV_ERR_WORKSPACE_TOO_SMALL before anything is launched.
 *   Every call on one GPU shares that GPU's array and leaves the last call's
 *   contents in it (no call relies on them: every call writes what it
 *   reads).  Calls that overlap in time on one GPU race, on any streams:
 *   serialise them, or use spec_verify_sample with separate workspaces.
 */
#define SV_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)

SV_API sv_status_t spec_verify_sample_noalloc(const sv_shape_t* shape,
                               const void* target_logits,
                               const void* draft_logits,
                               const int32_t* draft_ids,
                               float temperature,
                               int32_t top_k,
                               float top_p,
                               uint64_t seed,
                               uint32_t offset,
                               int32_t* out_tokens,
                               int32_t* out_num_accepted,
                               float* out_probs,
                               float* out_residual_mass,
                               hipStream_t stream);

/*
 * Verify with argmax draws, the variant the OpenVINO page implements
 * ("Text Generation via Speculative Sampling, KV Caching, and OpenVINO",
 * "Prepare speculative sampling", steps 3 and 4): the same probabilistic
 * acceptance test as spec_verify_sample (same uniforms U(b, k, 0)), but the
 * new token is the argmax (lowest id among equal maxima) of
 * max(0, p_n - q_n) at the first rejection n < K_b -- of p_n when that
 * residual has no positive entry -- and the argmax of p_{K_b} when every
 * guess is accepted.  Arguments, outputs and errors as for
 * spec_verify_sample; out_residual_mass is the residual's total as there.
 */
SV_API sv_status_t spec_verify_argmax(const sv_shape_t* shape,
                               const void* target_logits,
                               const void* draft_logits,
                               const int32_t* draft_ids,
                               float temperature,
                               int32_t top_k,
                               float top_p,
                               uint64_t seed,
                               uint32_t offset,
                               int32_t* out_tokens,
                               int32_t* out_num_accepted,
                               float* out_probs,
                               float* out_residual_mass,
                               void* workspace,
                               size_t* workspace_bytes,
                               hipStream_t stream);

/*
 * Greedy argmax-compare verify (the argmax rule of the autoregressive decode
 * on the OpenVINO page).  a_k = the lowest index among the maxima of target
 * row k; n = the first k < K_b with draft_ids[k] != a_k, or K_b; the tokens
 * are x_0..x_{n-1}, a_n, then -1.  Temperature and top-k do not change an
 * argmax, so they are not arguments.  Draft logits are not read.
 * Arguments as in spec_verify_sample; shape->draft_row_stride is ignored.
 */
SV_API sv_status_t spec_verify_greedy(const sv_shape_t* shape,
                               const void* target_logits,
                               const int32_t* draft_ids,
                               int32_t* out_tokens,
                               int32_t* out_num_accepted,
                               void* workspace,
                               size_t* workspace_bytes,
                               hipStream_t stream);

/*
 * Draft-side sampling, the step before verify: every guess x(b, k) ~ q_k.
 * The draft model proposes its K guesses one position at a time ("Text
 * Generation via Speculative Sampling, KV Caching, and OpenVINO", section
 * "Prepare speculative sampling", step 1, which takes the argmax); the
 * acceptance proof of "CS3602_FINAL_SpeDec", section 2, assumes each guess
 * is drawn from q, and that page's sampling helpers filter by top-K.
 *   q_k = softmax(draft row k / T) over its top-k kept set and top-p
 *   nucleus, exactly as in spec_verify_sample; x(b, k) = the first id (ascending) whose running sum
 *   of q_k exceeds U(b, k, 3), with U as in spec_verify_sample.
 * Arguments
 *   shape as for spec_verify_sample; target_row_stride is ignored.
 *   draft_logits [total_draft, draft_row_stride] in shape->dtype.
 *   temperature > 0 and finite; top_k in [0, V]; top_p in (0, 1].
 *   out_ids int32 [total_draft]: x(b, k) at cu_draft[b] + k.  A sequence
 *   whose cu_draft entries are out of range leaves its slots untouched; a
 *   row with no finite logit in its kept set yields -1.
 * Memory, execution, workspace and errors as for spec_verify_sample.
 */
SV_API sv_status_t spec_draft_sample(const sv_shape_t* shape,
                              const void* draft_logits,
                              float temperature,
                              int32_t top_k,
                              float top_p,
                              uint64_t seed,
                              uint32_t offset,
                              int32_t* out_ids,
                              void* workspace,
                              size_t* workspace_bytes,
                              hipStream_t stream);

/*
 * Per-token speculative likelihood, the quantity behind the perplexity
 * check of "CS3602_FINAL_SpeDec" (section 2's proof, used by that report's
 * problem analysis, item 1, to score speculative output without summing
 * over the vocabulary).  For position (b, k), k < K_b, with p = the target
 * row's and q = the draft row's softmax at temperature T (each over its
 * top-k kept set and top-p nucleus, exactly as in spec_verify_sample) and
 * y = tokens[r]:
 *   accept part  P(guess accepted, x = y) = q(y) min(1, p(y)/q(y)) = min(p(y), q(y))
 *   reject part  P(guess rejected, x = y) = (1 - beta) p'(y)       = p(y) - min(p(y), q(y))
 *   beta         = sum_v min(p(v), q(v))   (the position's acceptance mass)
 *   nll[b]       = -sum_k log(accept part + reject part)
 * The two parts add to p(y): one speculative step emits y with the target's
 * probability.
 * Arguments
 *   shape: batch, vocab, dtype, strides and cu_draft as for
 *   spec_verify_sample, but position (b, k) is row r = cu_draft[b] + k of
 *   BOTH tensors (total_draft rows each; max_draft, the largest K_b, has no
 *   upper limit here).
 *   target_logits [total_draft, target_row_stride], draft_logits
 *   [total_draft, draft_row_stride] in shape->dtype; tokens int32
 *   [total_draft].  temperature > 0 and finite; top_k in [0, V]; top_p in
 *   (0, 1].
 *   out_terms (nullable) float [total_draft][2] = accept part, reject part;
 *   out_beta (nullable) float [total_draft]; out_nll (nullable) double [B].
 *   At least one output must be non-NULL.  beta over full rows costs a
 *   second read of both rows; leave out_beta NULL when it is not needed.
 *   A token outside [0, V), or a row with no finite logit in its kept set,
 *   gives NaN parts (and NaN beta for such a row); p(y) = 0 gives an infinite
 *   nll.  A sequence whose cu_draft entries are out of range gets nll = NaN
 *   and leaves its other slots untouched.
 * Memory, execution, workspace and errors as for spec_verify_sample.
 */
SV_API sv_status_t spec_token_likelihood(const sv_shape_t* shape,
                              const void* target_logits,
                              const void* draft_logits,
                              const int32_t* tokens,
                              float temperature,
                              int32_t top_k,
                              float top_p,
                              float* out_terms,
                              float* out_beta,
                              double* out_nll,
                              void* workspace,
                              size_t* workspace_bytes,
                              hipStream_t stream);

/*
 * Beam search's selection, the counterpart of spec_draft_sample for callers
 * that follow the best continuations instead of drawing one ("Text Generation
 * via Speculative Sampling, KV Caching, and OpenVINO", section "Prepare
 * autoregressive sampling", decodes by the argmax, the selection of one beam).
 * A group (one request) has `beams` hypotheses; row g * beams + w of `logits`
 * holds beam w's next-token logits.  Candidate (w, v) extends beam w by token
 * v and scores
 *     s(w, v) = scores[w] + logits[w, v] / T - log sum_u exp(logits[w, u] / T).
 * The num_select candidates of largest s are written in falling order, equal
 * scores in rising order of w * vocab + v.  The order is that of the scores in
 * fp64, formed as (scores[w] - log S_w) + (l - m_w) / T with m_w the row's
 * largest logit and S_w = sum_u exp((l_u - m_w) / T).
 *   A finished beam (finished[row] != 0) has one candidate, pad_token at its
 *   own score; its logits are not read.  A beam whose score is not finite (a
 *   place not yet in use has -inf) and a row with no finite logit, or with a
 *   NaN or +inf logit, have none.  A logit of -inf is no candidate.
 * Arguments
 *   logits [groups * beams, row_stride] in shape->dtype; scores float
 *   [groups * beams]; finished (nullable) one byte [groups * beams].
 *   temperature as for spec_verify_sample; pad_token in [0, vocab).
 *   out_scores float, out_tokens int32 and out_parents int32
 *   [groups * num_select]: the candidate's score, its token, and the beam it
 *   extends (0 .. beams - 1, within its group).  Places that no candidate
 *   fills hold -inf, -1, -1.  Logits may be any finite value: a candidate whose
 *   score lies below fp32's range (a masked token at the type's lowest value
 *   and T < 1) keeps its place, with -inf for its score.
 *   1 <= beams <= SV_MAX_BEAMS, 1 <= num_select <= SV_MAX_SELECT.
 * out_scores may be `scores` itself when num_select == beams; other overlaps of
 * outputs with inputs are not allowed.  Memory, execution, workspace and errors
 * as for spec_verify_sample; SV_ERR_UNSUPPORTED also for more than 2^32 threads.
 */
#define SV_MAX_BEAMS 64
#define SV_MAX_SELECT 128

typedef struct {
    int32_t groups;     /* G >= 1                                 */
    int32_t beams;      /* W: hypotheses per group                */
    int32_t vocab;      /* V >= 1                                 */
    int32_t num_select; /* candidates to keep per group           */
    sv_dtype_t dtype;   /* element type of the logits             */
    int64_t row_stride; /* elements between logit rows, >= V      */
} sv_beam_shape_t;

SV_API sv_status_t spec_beam_select(const sv_beam_shape_t* shape,
                              const void* logits,
                              const float* scores,
                              const uint8_t* finished,
                              float temperature,
                              int32_t pad_token,
                              float* out_scores,
                              int32_t* out_tokens,
                              int32_t* out_parents,
                              void* workspace,
                              size_t* workspace_bytes,
                              hipStream_t stream);

/*
 * Reorder of beam states, in place, the step after a selection: place w of
 * group g takes the state of beam parents[g * beams + w] of the same group.
 * A state is a cache of keys or values, a token history or anything else that
 * is indexed by beam; its bytes are moved as they are.  The tensor is
 *     states[slab][g * beams + w][head][position][0 .. row_bytes)
 * with any strides whose places are distinct.  A cache [layers, batch,
 * positions, heads * dim] has heads = 1 and one slab per layer (keys and
 * values in one allocation: two); [layers, batch, heads, positions, dim] has
 * its heads; a state with no position has positions = 1.
 *   Only positions below the parent's length move: place w receives positions
 *   0 .. lengths[g * beams + parent] - 1 and keeps its others.  lengths
 *   (nullable: every beam holds all positions) is read, not reordered.
 *   A parent outside [0, beams), as spec_beam_select's -1, and a parent equal
 *   to w leave the place as it was.  A length below 0 counts as 0, one above
 *   `positions` as `positions`.
 * Arguments
 *   states: device memory, read and written; parents int32 [groups * beams];
 *   lengths int32 [groups * beams] or NULL, neither of them among the states'
 *   bytes.  Strides are in bytes.
 * Errors: SV_ERR_INVALID_ARGUMENT (null or misaligned pointer, a count < 1,
 * positions, row_bytes or a stride < 0, places that overlap, parents or lengths
 * between the states' first and last byte),
 * SV_ERR_UNSUPPORTED (beams > SV_MAX_BEAMS, one slab and head of a beam of
 * more than 2^31 - 1 pieces, a piece being 16, 4, 2 or 1 bytes as the
 * alignment of states, row_bytes and the strides allows, or more than 2^32
 * threads of one or two pieces), SV_ERR_HIP.  Execution as for
 * spec_verify_sample; no workspace.
 */
typedef struct {
    int32_t slabs;           /* >= 1: layers, or layers * 2                  */
    int32_t groups;          /* G >= 1                                       */
    int32_t beams;           /* W: places per group                          */
    int32_t heads;           /* >= 1                                         */
    int32_t positions;       /* >= 0                                         */
    int64_t row_bytes;       /* contiguous bytes per position (and head)     */
    int64_t slab_stride;     /* bytes                                        */
    int64_t beam_stride;     /* bytes; beam w of group g is row g * W + w     */
    int64_t head_stride;     /* bytes                                        */
    int64_t position_stride; /* bytes                                        */
} sv_state_shape_t;

SV_API sv_status_t spec_state_reorder(const sv_state_shape_t* shape,
                                void* states,
                                const int32_t* parents,
                                const int32_t* lengths,
                                hipStream_t stream);

/*
 * Attention of a batch whose sequences share long prefixes: the beams of a
 * request, several samples of one prompt, or requests under one system prompt,
 * at a decode step or in the scoring pass that a verify judges ("Text
 * Generation via Speculative Sampling, KV Caching, and OpenVINO", its KV
 * caching, with the prompt's cache held and read once per group).
 *   The batch is that of spec_verify_sample: sequence b has K_b + 1 query rows
 *   (K_b = 0: a plain decode step), row cu_draft[b] + b + k for k = 0..K_b.
 *   Group g holds sequences cu_groups[g] .. cu_groups[g+1] - 1 (cu_groups[0] = 0,
 *   cu_groups[G] = batch; NULL: batch / groups each) and one prefix of prefix_lengths[g] positions; b's
 *   own cache holds suffix_lengths[b] positions, the keys and values of its
 *   K_b + 1 newest rows last.  Row k sees the whole prefix and the suffix
 *   positions j with j <= suffix_lengths[b] - 1 - K_b + k:
 *     a_j = scale * q . k_j,  lse = log sum_j exp(a_j),  out = sum_j exp(a_j - lse) v_j,
 *   where query head h reads key/value head h / (q_heads / kv_heads).  A row
 *   that sees nothing gets zeros and lse = -inf.
 *   Lengths below 0 count as 0, above max_prefix / max_suffix as that; NULL
 *   lengths are max_prefix / max_suffix.  Positions behind a length are not read.
 * Arguments
 *   q and out [total_draft + batch][q_heads][head_dim]; a cache is
 *   data[group or sequence][position][head][head_dim], all of shape->dtype,
 *   strides in elements, the last dimension contiguous.  prefix_k and
 *   prefix_v may be NULL when max_prefix is 0, the suffix's when max_suffix is.
 *   q and the caches lie on 16-byte places (pointers, and strides of a
 *   multiple of 8 elements), out on 8-byte ones.
 *   out_lse (nullable) float [total_draft + batch][q_heads].
 *   scale > 0 and finite (usually 1 / sqrt(head_dim)).
 *   dtype SV_DTYPE_BF16 or SV_DTYPE_F16; head_dim 64, 128 or 256.
 *   Sums, softmax statistics and scores are fp32; the softmax weights are
 *   rounded to dtype for the product with v.
 * Errors as for spec_verify_sample; SV_ERR_INVALID_ARGUMENT also for q_heads
 * no multiple of kv_heads and for rows of out that overlap; SV_ERR_UNSUPPORTED
 * also for fp32, another head_dim, more than 2^30 positions, positions more
 * than 32 MB apart, strides whose extents 64 bits do not count, or more than
 * 2^32 threads.  A query, key or value that is
 * not finite reaches only the rows that see it, where a NaN gives NaN (a value
 * in its column alone) and an infinite value itself, or NaN under a weight that
 * dtype rounds to 0.  Data preconditions: cu_draft and cu_groups prefix
 * sums, no K_b above max_draft, no group above max_group.  Where they are
 * violated, out holds unspecified values and nothing out of bounds is read or
 * written.  out may be q itself; it may not overlap the inputs otherwise.
 */
typedef struct {
    const void* data;
    int64_t batch_stride;    /* elements between groups (prefix) or sequences (suffix) */
    int64_t position_stride; /* elements */
    int64_t head_stride;     /* elements */
} sv_cache_t;

typedef struct {
    int32_t groups;          /* G >= 1                                              */
    int32_t batch;           /* B >= 1 sequences                                    */
    int32_t max_group;       /* the largest group's sequences (read with cu_groups) */
    int32_t max_draft;       /* K, or the largest K_b when cu_draft != NULL         */
    int32_t total_draft;     /* sum_b K_b; must be B*K when cu_draft == NULL        */
    int32_t q_heads;
    int32_t kv_heads;
    int32_t head_dim;
    int32_t max_prefix;      /* positions a prefix cache holds                      */
    int32_t max_suffix;      /* positions a suffix cache holds                      */
    sv_dtype_t dtype;
    int64_t q_row_stride, q_head_stride;
    int64_t out_row_stride, out_head_stride;
    const int32_t* cu_draft;       /* device [B+1], or NULL */
    const int32_t* cu_groups;      /* device [G+1], or NULL */
    const int32_t* prefix_lengths; /* device [G], or NULL   */
    const int32_t* suffix_lengths; /* device [B], or NULL   */
} sv_attention_shape_t;

SV_API sv_status_t spec_prefix_attention(const sv_attention_shape_t* shape,
                                   const void* q,
                                   const sv_cache_t* prefix_k,
                                   const sv_cache_t* prefix_v,
                                   const sv_cache_t* suffix_k,
                                   const sv_cache_t* suffix_v,
                                   float scale,
                                   void* out,
                                   float* out_lse,
                                   void* workspace,
                                   size_t* workspace_bytes,
                                   hipStream_t stream);

/*
 * Verify of trees of guesses.  The guesses of a sequence may branch: guess j
 * extends row parents[cu_draft[b] + j] of its sequence, 0 <= parent <= j, where row
 * 0 is the newest token accepted before and row j + 1 is guess j's own, so a parent
 * comes before its guesses.  parents (device int32 [total_draft]) NULL is the chain
 * (parent j).  Rows are laid out as in spec_verify_sample; the row after a guess
 * scores what follows it.
 *   In this and the calls below cu_draft[B] may be less than total_draft (a step of fixed
 * size that holds fewer guesses): rows and slots behind the last sequence's are left as
 * they were.
 *   Every row r has its own token y_r.  From row 0 on, the first guess (lowest j)
 * that extends the row and equals y of the row is accepted and its row is next; at
 * a row without one the walk ends, and y of that row is the new token.
 *   spec_verify_tree_greedy: y_r is the lowest index among the maxima of row r (on a
 * chain this is spec_verify_greedy).
 *   spec_verify_tree_sample: y_r is the inverse-CDF draw from the row's softmax at
 * temperature T over its top-k kept set and top-p nucleus, as in
 * spec_verify_sample, with U(b, r, 4).  Each token that the call emits is thereby
 * drawn from the target's distribution behind the tokens before it, however the
 * tree was made ("CS3602_FINAL_SpeDec", section 2, asks that of a speculative
 * step; a chain of guesses x ~ q may use spec_verify_sample's test instead, which accepts more).  A row with no finite logit in its kept set has the token
 * -1, which no guess equals.
 * Outputs: out_tokens and out_num_accepted as for spec_verify_sample, the accepted
 *   guesses in the order of the path; out_path (nullable) int32 [total_draft + B]:
 *   slot cu_draft[b] + b + i holds the row of the i-th accepted guess, 0 at i = 0,
 *   -1 behind the n-th.  A sequence whose cu_draft entries, draft ids or parents are
 *   out of range reports num_accepted = -1 and leaves its other slots untouched.
 * draft_row_stride is ignored.  Memory, execution, workspace and errors as for
 * spec_verify_sample.
 */
SV_API sv_status_t spec_verify_tree_greedy(const sv_shape_t* shape,
                               const void* target_logits,
                               const int32_t* draft_ids,
                               const int32_t* parents,
                               int32_t* out_tokens,
                               int32_t* out_num_accepted,
                               int32_t* out_path,
                               void* workspace,
                               size_t* workspace_bytes,
                               hipStream_t stream);

SV_API sv_status_t spec_verify_tree_sample(const sv_shape_t* shape,
                               const void* target_logits,
                               const int32_t* draft_ids,
                               const int32_t* parents,
                               float temperature,
                               int32_t top_k,
                               float top_p,
                               uint64_t seed,
                               uint32_t offset,
                               int32_t* out_tokens,
                               int32_t* out_num_accepted,
                               int32_t* out_path,
                               void* workspace,
                               size_t* workspace_bytes,
                               hipStream_t stream);

/*
 * Edits of logits before a verify, a draft's draw or a selection: penalties for
 * tokens already written, biases and grammar masks.  The rows are those of
 * spec_verify_sample's target (row cu_draft[b] + b + k, k = 0 .. K_b; K = 0: one row
 * per sequence, as a plain step or a draft model's step has).
 *   Of a token v in row k of sequence b: seen(v) if it is among the first lengths[b] tokens
 * of tokens[b], or a guess on the row's way up (the guesses that rows 1 .. k of
 * a chain, or of the tree given by parents, have put behind the newest token, the
 * row's own included); n(v) how often it is among tokens[b][prompt_lengths[b] ..] up to the length and those guesses.
 *     x = l > 0 ? l / repetition[b] : l * repetition[b]      if seen(v)
 *     x = x - frequency[b] * n(v) - presence[b]              if n(v) > 0
 *     x = x + bias(v)                                        if v has one
 *     x = -inf                                               if the row's mask lacks v
 * in this order, in fp32, rounded to dtype once (as to any other value: a
 * result beyond the type's range becomes infinite).  Elements that none of this
 * concerns keep their bits.
 *   bias: entries cu_bias[b] .. cu_bias[b+1] - 1 of bias_ids and bias_values; of an id given twice the last
 * entry counts.  Tokens, guesses and bias ids outside [0, vocab) are ignored, and a parent
 * outside [0, j] counts as 0.  Lengths below 0 count as 0, above max_tokens as that.
 * A sequence with repetition 1, presence 0 and frequency 0 has no penalties.  A sequence whose cu_draft entries
 * are out of range has its rows left as they were.
 *   masks: row m allows v where bit v % 32 of masks[m * mask_stride + v / 32] is
 * set.  Row r of the logits goes by mask mask_rows[r], or r where mask_rows is
 * NULL; an index outside [0, num_masks), as -1, is no mask.
 * Arguments
 *   logits and out [total_draft + batch, stride] in shape->dtype; out may be logits itself (with the same
 *   stride), otherwise they lie apart and every element of the vocabulary is
 *   written.  In place only what changes is written.  NULL in sv_adjust_t: tokens
 *   none, lengths max_tokens, prompt_lengths 0, repetition 1, presence and frequency 0,
 *   cu_bias all entries for every sequence, masks none; draft_ids NULL: no guess
 *   counts.  out overlaps no other input.  repetition > 0.
 * Errors: SV_ERR_INVALID_ARGUMENT (null or misaligned pointer, counts or strides as in spec_verify_sample,
 * token_stride < max_tokens, a mask_stride or num_masks too small, logits and out that
 * overlap), SV_ERR_UNSUPPORTED (limits as in spec_verify_sample, 2^30 or more
 * tokens of a sequence, more than 2^32 threads), SV_ERR_HIP.  Execution as for
 * spec_verify_sample; no workspace.
 */
typedef struct {
    int32_t batch;             /* B >= 1                                      */
    int32_t max_draft;         /* K, or the largest K_b when cu_draft != NULL */
    int32_t total_draft;       /* sum_b K_b                                   */
    int32_t vocab;             /* V >= 1                                      */
    sv_dtype_t dtype;          /* element type of logits and out              */
    int64_t row_stride;        /* elements between rows of logits, >= V       */
    int64_t out_row_stride;    /* elements between rows of out, >= V          */
    const int32_t* cu_draft;   /* device [B+1], or NULL                       */
    const int32_t* draft_ids;  /* device [total_draft], or NULL               */
    const int32_t* parents;    /* device [total_draft], or NULL: chains       */
} sv_adjust_shape_t;

typedef struct {
    const int32_t* tokens;         /* device [B][max_tokens], or NULL      */
    int64_t token_stride;          /* entries between its rows             */
    int32_t max_tokens;
    int32_t total_bias;            /* entries of bias_ids and bias_values  */
    const int32_t* lengths;        /* device [B], or NULL                  */
    const int32_t* prompt_lengths; /* device [B], or NULL                  */
    const float* repetition;       /* device [B], or NULL                  */
    const float* presence;         /* device [B], or NULL                  */
    const float* frequency;        /* device [B], or NULL                  */
    const int32_t* bias_ids;       /* device [total_bias], or NULL         */
    const float* bias_values;      /* device [total_bias], or NULL         */
    const int32_t* cu_bias;        /* device [B+1], or NULL                */
    const uint32_t* masks;         /* device [num_masks][mask_stride], or NULL */
    int64_t mask_stride;           /* words between masks, >= (V + 31) / 32 */
    int32_t num_masks;
    const int32_t* mask_rows;      /* device [total_draft + B], or NULL    */
} sv_adjust_t;

SV_API sv_status_t spec_adjust_logits(const sv_adjust_shape_t* shape,
                               const sv_adjust_t* adjust,
                               const void* logits,
                               void* out,
                               hipStream_t stream);

/*
 * Attention of the newest rows of every sequence over its cache in pages: a plain
 * decode step (K_b = 0), the scoring rows of a chain of guesses, or a tree of them.
 *   The rows are those of spec_verify_sample's target: sequence b has K_b + 1, row
 * cu_draft[b] + b + k. Its cache holds lengths[b] positions, the keys and values
 * of those rows last: row k's own is position lengths[b] - 1 - K_b + k.  Position p
 * lies in page page_table[b][p / page_size], at p % page_size.  Row k sees every
 * position before row 0's, its own, and those of the rows on its way up
 * (parents as for spec_verify_tree_greedy; a parent out of range counts as 0;
 * NULL: chains, where row k sees rows 0 .. k):
 *     a_j = scale * q . k_j,  lse = log sum_j exp(a_j),  out = sum_j exp(a_j - lse) v_j,
 * where query head h reads key/value head h / (q_heads / kv_heads).  Positions in
 * a page outside [0, pages) are not seen.  A row that sees nothing gets zeros and
 * lse = -inf.  Lengths below 0 count as 0, above max_pages * page_size as that;
 * NULL lengths are that.  Positions behind a length are not seen; where they
 * share a page with others they may be read.
 * Arguments
 *   q and out [total_draft + batch][q_heads][head_dim]; k and v
 *   data[page][position in page][head][head_dim] (batch_stride: elements between pages), all of
 *   shape->dtype, strides in elements, the last dimension contiguous.
 *   page_table int32 [batch][max_pages] with table_stride entries between rows, or NULL:
 *   sequence b's one page is page b (max_pages = 1, pages >= batch).  page_size is a
 *   multiple of 16 with a page_table, any number without.
 *   q and the caches lie on 16-byte places (pointers, and strides of a multiple of 8
 *   elements), out on 8-byte ones.  out_lse (nullable) float [total_draft +
 *   batch][q_heads].  scale > 0 and finite.
 *   dtype SV_DTYPE_BF16 or SV_DTYPE_F16; head_dim 64, 128 or 256.
 *   Sums, softmax statistics and scores are fp32; the softmax weights are
 *   rounded to dtype for the product with v.
 * The workspace depends on the shape's rows, not on the caches' size.  Values that
 * are not finite and bad cu_draft entries are met as in spec_prefix_attention.
 * Errors as for spec_verify_sample; SV_ERR_INVALID_ARGUMENT also for q_heads no
 * multiple of kv_heads and for rows of out that overlap; SV_ERR_UNSUPPORTED also
 * for fp32, another head_dim, a page_size with a page_table that is no multiple of 16, more than 2^30 positions of a
 * sequence, positions more than 32 MB apart, strides whose extents 64 bits do not
 * count, batch * kv_heads * positions / 64 of 2^31 or more, or more than 2^32
 * threads.  out may be q itself; it may not overlap the inputs otherwise.
 */
typedef struct {
    int32_t batch;             /* B >= 1                                      */
    int32_t max_draft;         /* K, or the largest K_b when cu_draft != NULL */
    int32_t total_draft;       /* sum_b K_b                                   */
    int32_t q_heads;
    int32_t kv_heads;
    int32_t head_dim;
    int32_t pages;             /* pages of k and v                            */
    int32_t page_size;         /* positions per page                          */
    int32_t max_pages;         /* entries of a sequence's table               */
    sv_dtype_t dtype;
    int64_t table_stride;      /* entries between the tables' rows            */
    int64_t q_row_stride, q_head_stride;
    int64_t out_row_stride, out_head_stride;
    const int32_t* cu_draft;   /* device [B+1], or NULL          */
    const int32_t* parents;    /* device [total_draft], or NULL  */
    const int32_t* lengths;    /* device [B], or NULL            */
    const int32_t* page_table; /* device [B][max_pages], or NULL */
} sv_tree_shape_t;

SV_API sv_status_t spec_tree_attention(const sv_tree_shape_t* shape,
                                 const void* q,
                                 const sv_cache_t* k,
                                 const sv_cache_t* v,
                                 float scale,
                                 void* out,
                                 float* out_lse,
                                 void* workspace,
                                 size_t* workspace_bytes,
                                 hipStream_t stream);

/*
 * Caches in pages.  A pool holds the states of many sequences in pages of
 * page_size positions,
 *     pool[slab][page][head][position in page][0 .. row_bytes)
 * with any strides whose places are distinct: [layers, pages, page_size, heads *
 * dim] has heads = 1 and one slab per layer (keys and values in one allocation:
 * two), [layers, pages, heads, page_size, dim] has its heads.  A sequence's page
 * table lists its pages: position p lies in page table[b][p / page_size].  A table
 * entry outside [0, pages) is no page (-1 where a table ends).
 */
typedef struct {
    int32_t slabs;           /* >= 1: layers, or layers * 2      */
    int32_t pages;           /* >= 1                             */
    int32_t page_size;       /* >= 1 positions per page          */
    int32_t heads;           /* >= 1                             */
    int64_t row_bytes;       /* >= 1, contiguous, per position (and head) */
    int64_t slab_stride;     /* bytes                            */
    int64_t page_stride;     /* bytes                            */
    int64_t head_stride;     /* bytes                            */
    int64_t position_stride; /* bytes                            */
} sv_pool_t;

/*
 * The step of a paged cache after a verify: the rows of the accepted guesses move
 * to the places that follow the context, in place, and the sequence's new length
 * is formed.  Sequence b's cache holds lengths[b] positions, the last K_b + 1 of
 * them its newest rows (row 0 the newest token accepted before, row j + 1 guess j,
 * as spec_tree_attention read them); with first = lengths[b] - 1 - K_b,
 *     position first + i takes the state of position first + path[i], i = 1 .. n,
 *     out_lengths[b] = first + 1 + n,
 * n = num_accepted[b], path = the sequence's rows of out_path (spec_verify_tree_*).
 * Other positions keep their states: those from the new length on hold what they
 * held, or a row that moved.
 *   A path rises strictly from path[0] = 0 to at most K_b; at an entry that does not,
 *   the moves end.  n outside [0, K_b], as a verify's -1, and cu_draft entries out
 *   of range move nothing and give out_lengths[b] = lengths[b].  A move from or to
 *   a position below 0, or one without a page, is left out.  Lengths below 0
 *   count as 0, above max_pages * page_size as that; NULL lengths are that.
 *   out_lengths is at least 0.
 * Arguments
 *   data: the pool, read and written.  page_table int32 [batch][max_pages] with
 *   table_stride entries between rows, or NULL: sequence b's one page is page b
 *   (max_pages = 1, a cache with one piece per sequence).  path int32
 *   [total_draft + batch]; num_accepted, out_lengths int32 [batch].  None of
 *   these lies among the pool's bytes; out_lengths overlaps no input.  The pages
 *   that hold newest rows belong to one sequence each.
 * Errors: SV_ERR_INVALID_ARGUMENT (null or misaligned pointer, a count < 1, a
 * stride < 0, places that overlap, an overlap as above), SV_ERR_UNSUPPORTED
 * (max_draft > SV_MAX_DRAFT, a position of all slabs and heads of more than 2^31 - 1
 * pieces, a piece being 16, 4, 2 or 1 bytes as the alignment of data, row_bytes and
 * the strides allows, more than 2^30 positions of a sequence, or more than 2^32 threads), SV_ERR_HIP.
 * Execution as for spec_verify_sample; no workspace.
 */
typedef struct {
    sv_pool_t pool;
    int32_t batch;             /* B >= 1                                      */
    int32_t max_draft;         /* K, or the largest K_b when cu_draft != NULL */
    int32_t total_draft;       /* sum_b K_b                                   */
    int32_t max_pages;         /* entries of a sequence's table               */
    int64_t table_stride;      /* entries between the tables' rows            */
    const int32_t* cu_draft;   /* device [B+1], or NULL                       */
    const int32_t* page_table; /* device [B][max_pages], or NULL              */
} sv_compact_shape_t;

SV_API sv_status_t spec_cache_compact(const sv_compact_shape_t* shape,
                                void* data,
                                const int32_t* lengths,
                                const int32_t* path,
                                const int32_t* num_accepted,
                                int32_t* out_lengths,
                                hipStream_t stream);

/*
 * The page tables of sequences that continue others: beams after a selection,
 * samples of one prompt, or the same sequences with more or fewer positions.  Place w
 * continues sequence s = parents[w] of the old tables: it takes over the
 * lengths[s] positions that s holds, and pages for max(lengths[s],
 * new_lengths[w]) positions (at most max_pages of them).
 *   Whole pages below the length are shared: the place's table lists the parent's.
 *   The page that the length ends in will be written by its place.  The lowest
 *   place that takes it keeps it, unless anyone else holds it (a table outside this
 *   call, or a place for which it is a whole page); every other one gets a free page
 *   and a copy of the used positions, in all slabs and heads.
 *   Pages behind the length are free ones.  Free pages are given in rising order to
 *   the places in rising order, each place's in the order of its table.
 *   refs[page] counts the holders of each page: every entry of an old table is one,
 *   besides holders outside this call.  out_refs has the old tables' taken away and the new ones'
 *   added; a page is free if it has none after the old tables' have gone and the
 *   shared and kept ones have been added.  Sequences that nobody continues are
 *   thereby freed.
 *   A parent outside the old tables (-1) gives an empty table.  With beams > 0,
 *   parents[w] counts within w's group of `beams` sequences, as
 *   spec_beam_select returns them.  NULL parents: place w continues sequence w.
 *   Entries behind a table's last page are -1.  out_free = free pages left; below
 *   0, so many were missing: the last entries that found none are -1, and a copy into
 *   them is left out.
 * Arguments
 *   data: the pool, read and written (fresh pages only).  page_table int32
 *   [old][max_pages], out_table int32 [batch][max_pages], strides in entries; lengths
 *   int32 [old] (below 0 counts as 0, above max_pages * page_size as that); parents
 *   and new_lengths (nullable) int32 [batch]; refs and out_refs int32 [pages], which
 *   may be one array; out_free int32 [1].  The other outputs overlap no input, and
 *   none of these lies among the pool's bytes.
 * Memory, execution, workspace and errors as for spec_verify_sample;
 * SV_ERR_INVALID_ARGUMENT also as for spec_cache_compact, and for beams > 0 with batch or
 * old no multiple of it; SV_ERR_UNSUPPORTED also for more than 2^31 - 1 table entries,
 * old or new, more than 2^30 positions of a sequence, a page of all slabs and heads
 * of more than 2^31 - 1 pieces, and more than 2^32 threads.
 */
typedef struct {
    sv_pool_t pool;
    int32_t old;              /* sequences of page_table, >= 1               */
    int32_t batch;            /* places of out_table, >= 1                   */
    int32_t beams;            /* 0: parents count over all old sequences     */
    int32_t max_pages;        /* entries of a sequence's table, old and new  */
    int64_t table_stride;     /* entries between rows of page_table          */
    int64_t out_table_stride; /* entries between rows of out_table           */
} sv_fork_shape_t;

SV_API sv_status_t spec_page_fork(const sv_fork_shape_t* shape,
                            void* data,
                            const int32_t* page_table,
                            const int32_t* lengths,
                            const int32_t* parents,
                            const int32_t* new_lengths,
                            const int32_t* refs,
                            int32_t* out_table,
                            int32_t* out_refs,
                            int32_t* out_free,
                            void* workspace,
                            size_t* workspace_bytes,
                            hipStream_t stream);

/* A static, human-readable name for a status code. */
SV_API const char* spec_verify_status_string(sv_status_t status);

#ifdef __cplusplus
}
#endif

#endif /* SPECVERIFY_H */
