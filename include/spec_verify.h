/*
 * spec_verify.h - C interface of a lossless speculative-sampling verifier for
 * AMD MI355X (gfx950).
 *
 * The operation is one verification round of speculative decoding for a batch
 * of B independent requests:
 *   - "Speculative Decoding - Turn guesses into parallel work", section "One
 *     round and shifted logits": the drafter proposes gamma tokens together with
 *     their proposal distributions q; one target pass yields gamma+1 target
 *     distributions p (row i judges proposal i, row gamma serves the bonus token).
 *   - same page, section "Exact sampling: account for every probability", and
 *     "Speculative Token Decoupling ..." Equation 3.1: proposal i is accepted with
 *     probability min(1, p_i(x_i) / q_i(x_i)); here: accept iff u_i * q_i(x_i) <=
 *     p_i(x_i) with u_i uniform on (0, 1].
 *   - "Drafters and Speculative Decoding: Useful Tokens, Correct State", section
 *     "Sampling needs a correction rule": at the first rejection the replacement
 *     is drawn from norm(max(0, p - q)); every later proposal is discarded.
 *   - "Speculative Decoding" (specdec fundamentals), section "The Loop": if all
 *     gamma proposals survive, one bonus token is drawn from p_gamma; every round
 *     emits between 1 and gamma+1 tokens.
 *   - "Speculative Decoding - Turn guesses into parallel work", section "Greedy,
 *     sampling and the real sampler": temperature, truncation and token bans are
 *     part of p and q, and the greedy variant accepts while the proposal equals
 *     the target argmax ("Drafters and Speculative Decoding", section "Greedy
 *     verification").
 *
 * Conventions shared by every entry point
 *   - Every pointer argument is caller-owned memory. Logits, tokens, outputs and
 *     workspace are DEVICE pointers on the current HIP device; sampler structs
 *     are passed by value. The library allocates no device memory, frees
 *     nothing, and keeps no pointer after returning.
 *   - Calls are asynchronous on `stream` (a hipStream_t; NULL = the null stream)
 *     and never synchronise. Outputs are valid once the stream has reached the
 *     call. Outputs must not alias inputs; concurrent calls need distinct
 *     outputs and workspaces.
 *   - Argument errors are detected on the host before anything is launched and
 *     return a negative SV_E* code; nothing is written in that case. Problems
 *     that can only be seen in the data are reported per request through the
 *     SV_FLAG_* bits of out_flags.
 *   - Logit rows are contiguous with row stride V elements. A logit of -inf
 *     marks a token as impossible. NaN and +inf are data errors (flag
 *     SV_FLAG_NONFINITE); the tokens of such a request are unspecified.
 */
#ifndef SPEC_VERIFY_H
#define SPEC_VERIFY_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { SV_F32 = 0, SV_BF16 = 1 } sv_dtype;

/* Sampler settings of one distribution (target or draft may differ).
 *   temperature: > 0 and finite; logits are divided by it.
 *   top_k:       0 = off; otherwise keep every token whose logit is >= the
 *                k-th largest admissible logit (ties kept, so more than k
 *                tokens may survive). k >= number of admissible tokens is off.
 *   top_p:       1.0 = off; otherwise in (0, 1): keep token x when the tempered
 *                probability mass of tokens with a strictly larger logit is
 *                < top_p (the crossing token and its exact ties are kept).
 * Order of transforms: bans, temperature, top-k, top-p, renormalise. */
typedef struct {
  float temperature;
  int32_t top_k;
  float top_p;
} sv_sampler;

/* Return codes. */
#define SV_OK 0
#define SV_EINVAL (-1)     /* null required pointer, bad size or sampler field */
#define SV_EDTYPE (-2)     /* dtype not SV_F32 / SV_BF16 */
#define SV_EWORKSPACE (-3) /* workspace NULL or smaller than spec_verify_workspace_bytes */
#define SV_ESIZE (-4)      /* sizes overflow the supported index ranges */
#define SV_EHIP (-5)       /* a HIP launch or runtime call failed */
#define SV_ESCRATCH (-6)   /* spec_verify_sample_noalloc: the sizes need more workspace
                              than SV_NOALLOC_SCRATCH_BYTES */

/* Per-request flag bits written to out_flags. */
#define SV_FLAG_TOKEN_RANGE 1u    /* some draft token lies outside [0, V) */
#define SV_FLAG_Q_ZERO 2u         /* the proposal that ended the walk has q(x) = 0 */
#define SV_FLAG_NONFINITE 4u      /* NaN or +inf in one of the request's rows */
#define SV_FLAG_EMPTY 8u          /* a row has no admissible token; see out_tokens */
#define SV_FLAG_RESIDUAL_ZERO 16u /* residual mass was 0 at a rejection; drawn from p */
#define SV_FLAG_BAD_PARAM 32u     /* a per-request setting of sv_requests is out of range */

/* Largest n_banned (and sv_requests.n_banned_draft) accepted. */
#define SV_MAX_BANNED 2048
/* Largest sv_requests.n_history accepted. A row penalizes at most
 * SV_MAX_HISTORY + 63 distinct ids (its history and the proposals before it);
 * the kernels keep them in an on-chip hash set of 4096 slots that this bound
 * keeps at most half full. */
#define SV_MAX_HISTORY 1984

/* Per-request settings of a mixed batch ("Speculative Decoding - Turn guesses
 * into parallel work", section "Implementation roadmap and tests": continuous
 * batching keeps per-request metadata on the GPU). Every array is DEVICE
 * memory of B entries (banned_draft: B rows of n_banned_draft); a NULL array
 * keeps the call-wide value. Passed to spec_verify_sample by host pointer.
 *   gamma         proposals of each request, 0 <= gamma[b] <= gamma: request b
 *                 uses target rows 0..gamma[b], draft rows and draft tokens
 *                 0..gamma[b]-1, acceptance uniforms (slots) 0..gamma[b]-1 and
 *                 the final-draw uniform of slot gamma; its out_tokens row has
 *                 at most gamma[b]+1 tokens.
 *   target        target sampler of each request. Temperature 0 makes the
 *                 request greedy: proposals are kept while they equal the
 *                 argmax of their target row (banned_ids applied, NaN excluded,
 *                 lowest id on ties), as in spec_verify_greedy; its draft rows
 *                 and uniforms are not read.
 *   draft         draft sampler of each request (ignored for greedy requests).
 *   banned_draft  [B][n_banned_draft] bans of the draft rows; banned_ids then
 *                 applies to the target rows only (same list rules).
 *   history       [B][n_history] tokens each request generated before this
 *                 round (-1 or ids outside [0, V) are padding), for the
 *                 repetition penalty; n_history <= SV_MAX_HISTORY.
 *   penalty       [B] repetition penalty theta >= 1 of the target rows (1:
 *                 off); penalty_draft [B] likewise for the draft rows. Row i
 *                 of a request penalizes its history and the proposals
 *                 x_0 .. x_{i-1} before position i (the tokens its sampler had
 *                 seen), each id once, banned ids excepted: a logit z becomes
 *                 z / theta if z > 0, else z * theta (Keskar et al. 2019,
 *                 "CTRL", section 4.1, sign-aware form), computed in float32
 *                 and rounded to bf16 for bf16 logits; the penalty comes after
 *                 the bans and before temperature and truncation.
 * A request whose gamma[b], sampler fields or penalties are out of range (the
 * ranges of sv_sampler; temperature 0 only as a target; a penalty below 1 or
 * not finite) is not verified: flag
 * SV_FLAG_BAD_PARAM, no accepted proposal, out_tokens row all -1. Rows a
 * request does not use report NaN in out_target_lse / out_draft_lse, and so
 * do the rows of greedy requests; out_overlap is NaN at positions a request
 * does not have and for greedy requests. */
typedef struct {
  const int32_t* gamma;
  const sv_sampler* target;
  const sv_sampler* draft;
  const int32_t* banned_draft;
  int32_t n_banned_draft;
  const int32_t* history;
  int32_t n_history;
  const float* penalty;
  const float* penalty_draft;
} sv_requests;

/* Workspace bytes needed by spec_verify_sample for these sizes (0 when B < 1,
 * gamma outside [1, 63], V < 1 or the sizes overflow the supported index
 * ranges). The workspace needs no initialisation and may be reused by later
 * calls on the same stream; calls that run concurrently need separate
 * workspaces. */
size_t spec_verify_workspace_bytes(int32_t B, int32_t gamma, int32_t V);

/* Speculative-sampling verification.
 *   target_logits  [B][gamma+1][V] of dtype; row i is the target distribution
 *                  after the prefix and proposals 0..i-1, row gamma the bonus row.
 *   draft_logits   [B][gamma][V] of dtype; row i is the distribution proposal i
 *                  was sampled from (it must be the distribution that actually
 *                  produced the token, after the drafter's own transforms).
 *   draft_tokens   [B][gamma] int32 proposals.
 *   banned_ids     [B][n_banned] int32 token ids removed from p AND q of every
 *                  row of the request; -1 or any id outside [0, V) is padding;
 *                  duplicates are allowed. NULL only when n_banned == 0.
 *   target, draft  sampler settings for p and q respectively.
 *   requests       per-request settings of a mixed batch (sv_requests above),
 *                  or NULL for a batch that shares gamma, samplers and bans.
 *   seed, offset   select the uniforms when `uniforms` is NULL: for request b
 *                  and slot j (j < gamma: acceptance of proposal j; j == gamma:
 *                  the single final draw) u = ((r >> 11) + 1) * 2^-53 with r the
 *                  first output word of Philox4x64-10 at counter (j, b, offset, 0)
 *                  and key (seed, 0) (Salmon et al., SC'11).
 *   uniforms       [B][gamma+1] double in (0, 1] used instead of Philox, or NULL.
 * Outputs:
 *   out_tokens       [B][gamma+1] int32: the n accepted proposals, then the
 *                    correction (n < gamma) or bonus (n == gamma) token, then -1
 *                    padding. The emitted token is -1 when the distribution it
 *                    must be drawn from is empty (SV_FLAG_EMPTY).
 *   out_num_accepted [B] int32 n in [0, gamma].
 *   out_flags        [B] uint32 SV_FLAG_* bits, or NULL.
 *   out_target_lse   [B][gamma+1] float log-normaliser of each tempered target
 *                    row over its kept set (-inf if empty), or NULL.
 *   out_draft_lse    [B][gamma] float, same for the draft rows, or NULL.
 *   out_overlap      [B][gamma] double, or NULL (then not computed): the overlap
 *                    sum_x min(p_i(x), q_i(x)) = 1 - TV(p_i, q_i) of target row
 *                    i and draft row i after every sampler transform; with x_i
 *                    drawn from q_i it is the probability that proposal i is
 *                    accepted once the walk reaches it ("Speculative
 *                    Decoding - Turn guesses into parallel work", sections
 *                    "Confidence and verification admission" and "Accepted
 *                    length is not speed"). 0 when either row is empty; unspecified for a
 *                    request flagged SV_FLAG_NONFINITE. Computing it reads the
 *                    rows 0..gamma-1 once more (only the kept groups of the
 *                    other row when one of the two is truncated).
 *   out_accept_hist  [gamma+1] uint32, or NULL: out_accept_hist[n] = number of
 *                    requests of this call with n accepted proposals (an
 *                    accepted-prefix histogram, same page, section "Read the
 *                    benchmark contract"). Overwritten by each call. Requests
 *                    that reached position i number sum_{n >= i} hist[n], and
 *                    sum_{n > i} hist[n] of them accepted it.
 *   workspace        device scratch of at least spec_verify_workspace_bytes(...)
 *                    bytes, 256-byte aligned.
 * Limits: 1 <= B, 1 <= gamma <= 63, 1 <= V < 2^31, B*(2*gamma+1) < 2^31,
 * n_banned <= SV_MAX_BANNED; logit pointers aligned to their element size. */
int spec_verify_sample(const void* target_logits, const void* draft_logits, sv_dtype dtype,
                       const int32_t* draft_tokens, const int32_t* banned_ids,
                       int32_t n_banned, int32_t B, int32_t gamma, int32_t V,
                       sv_sampler target, sv_sampler draft, const sv_requests* requests,
                       uint64_t seed, uint64_t offset,
                       const double* uniforms, int32_t* out_tokens, int32_t* out_num_accepted,
                       uint32_t* out_flags, float* out_target_lse, float* out_draft_lse,
                       double* out_overlap, uint32_t* out_accept_hist,
                       void* workspace, size_t workspace_bytes, void* stream);

/* spec_verify_sample without a workspace argument, for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc). Arguments, outputs and errors are those of
 * spec_verify_sample; the workspace is a static device array of
 * SV_NOALLOC_SCRATCH_BYTES bytes inside the library, one per GPU, held until
 * the process ends. The call allocates nothing. When
 * spec_verify_workspace_bytes exceeds SV_NOALLOC_SCRATCH_BYTES, the call runs
 * without the final draw's lists of kept tokens (the last part of that size:
 * 388 bytes per request and 2048-token sub-chunk), with the same outputs;
 * sizes whose remaining workspace still exceeds the array return SV_ESCRATCH
 * (c5-sized batches, B = 128, gamma = 8, V = 151936, need about 4.0 MB with
 * the lists and 0.3 MB without). The first call on a device resolves that
 * device's array address (SV_EHIP if it cannot). Every call on one GPU shares its array: calls that
 * may overlap on one GPU (different streams, or different host threads)
 * race and must be serialised by the caller; calls in order on one stream are
 * safe. Nothing needs clearing: every call initialises what it reads. */
#define SV_NOALLOC_SCRATCH_BYTES (8u << 20)
int spec_verify_sample_noalloc(const void* target_logits, const void* draft_logits,
                               sv_dtype dtype, const int32_t* draft_tokens,
                               const int32_t* banned_ids, int32_t n_banned, int32_t B,
                               int32_t gamma, int32_t V, sv_sampler target, sv_sampler draft,
                               const sv_requests* requests, uint64_t seed, uint64_t offset,
                               const double* uniforms, int32_t* out_tokens,
                               int32_t* out_num_accepted, uint32_t* out_flags,
                               float* out_target_lse, float* out_draft_lse, double* out_overlap,
                               uint32_t* out_accept_hist, void* stream);

/* Greedy verification ("Drafters and Speculative Decoding", section "Greedy
 * verification"): proposal i is kept while it equals the argmax of target row i
 * (largest logit, lowest token id on exact ties, -0 == +0); the first mismatch
 * emits that row's argmax, and if all gamma match the argmax of row gamma is
 * appended. Needs no workspace: out_tokens doubles as scratch.
 *   target_logits [B][gamma+1][V], draft_tokens [B][gamma];
 *   banned_ids [B][n_banned] ids that are never an argmax (the sampler's bans
 *   are part of greedy decoding too: "Speculative Decoding - Turn guesses into
 *   parallel work", section "Greedy, sampling and the real sampler"); same list
 *   rules as for spec_verify_sample; NULL only when n_banned == 0;
 *   out_tokens [B][gamma+1] (n matches, argmax, then -1), out_num_accepted [B],
 *   out_flags [B] or NULL (SV_FLAG_TOKEN_RANGE, SV_FLAG_NONFINITE, and
 *   SV_FLAG_EMPTY when the emitted token's row has no admissible id: that token
 *   is then -1),
 *   out_accept_hist [gamma+1] or NULL: accepted-prefix histogram of the call,
 *   as for spec_verify_sample.
 * NaN logits are not candidates and are flagged; a row whose admissible
 * logits are all -inf has the lowest such id as its argmax. */
int spec_verify_greedy(const void* target_logits, sv_dtype dtype, const int32_t* draft_tokens,
                       const int32_t* banned_ids, int32_t n_banned,
                       int32_t B, int32_t gamma, int32_t V, int32_t* out_tokens,
                       int32_t* out_num_accepted, uint32_t* out_flags,
                       uint32_t* out_accept_hist, void* stream);

/* Chain KV-commit metadata of one verification round ("Speculative Decoding -
 * Turn guesses into parallel work", section "Committed tokens versus cached
 * states"; "Drafters and Speculative Decoding: Useful Tokens, Correct State",
 * section "Committing state after rejection"), from the outputs of
 * spec_verify_sample or spec_verify_greedy, on the same stream.
 * gamma_b [B] (device) gives each request's number of proposals as in
 * sv_requests (NULL: all gamma); below, gamma stands for gamma_b[b].
 * Convention: before the round request b has kv_len[b] = K materialised target
 * KV rows, and its last committed token (the anchor) is pending: it has no row
 * yet. The verification pass ran the gamma+1 inputs (anchor, x_0, ...,
 * x_{gamma-1}) at positions K .. K+gamma and wrote their rows; slots[b][j] is
 * the physical KV slot of position K + j. After the round:
 *   new_kv_len[b] = K + 1 + n   the anchor's row and the n accepted rows are
 *                               committed history (logical length = new_kv_len + 1);
 *   anchor[b] = out_tokens[b][n]  the correction or bonus token, pending until
 *                               the next pass computes its row (-1 if the
 *                               verifier emitted none, see SV_FLAG_EMPTY);
 *   n_free[b] = gamma - n       rows of the rejected proposals x_n .. x_{gamma-1};
 *   free_slots[b][0 .. gamma-n-1] = slots[b][n+1 .. gamma], then -1.
 * Pointers: out_tokens [B][gamma+1], out_num_accepted [B], kv_len [B] (inputs,
 * device); new_kv_len [B], anchor [B] (required outputs); n_free [B] or NULL;
 * free_slots [B][gamma] or NULL, which needs slots [B][gamma+1]. A request
 * whose accepted count lies outside [0, gamma_b[b]], or whose gamma_b[b] lies
 * outside [0, gamma], is left unchanged (new_kv_len =
 * kv_len, anchor -1, nothing freed). The caller keeps kv_len + gamma + 1 within
 * int32. Returns SV_EINVAL for a missing required pointer, free_slots without
 * slots, B < 1 or gamma outside [1, 63]; SV_ESIZE if B*(gamma+1) overflows. */
int spec_verify_commit(const int32_t* out_tokens, const int32_t* out_num_accepted,
                       const int32_t* kv_len, const int32_t* slots, const int32_t* gamma_b,
                       int32_t B, int32_t gamma,
                       int32_t* new_kv_len, int32_t* anchor, int32_t* n_free,
                       int32_t* free_slots, void* stream);

/* ------------------------------------------------- training the drafter
 *
 * What a drafter is trained with, over the same vocabulary rows: the record of
 * a target row that a drafter learns from, the distillation loss against it,
 * and the cross entropy of a linear head whose logits are never stored.
 *
 * Conventions of these calls
 *   - Matrices are given by a pointer and a row stride in elements, at least the
 *     row's length; elements of a row are consecutive. Any stride and any
 *     alignment to the element size is accepted; rows that all start on 16
 *     bytes are fastest.
 *   - Sums, maxima and losses are float32 whatever the inputs' type; gradients
 *     are rounded once to the type of what they are gradients of.
 *   - No result depends on the order in which workgroups run: a call repeated on
 *     the same inputs gives the same bits.
 *   - Workspaces need no initialisation, are 256-byte aligned, hold nothing
 *     between calls, and may be reused by later calls on the same stream; calls
 *     (and captured graphs) that may run concurrently need separate ones.
 *     A workspace of 0 bytes may be NULL. */

/* Largest number of kept logits per row. */
#define SV_MAX_TOP 1024

/* The K largest logits of every row, in descending order, the lower id first
 * among equal values (-0 == +0), and the log-normaliser of the whole row.
 *   logits      [R][V] of dtype, row stride logits_stride >= V; the target
 *               logits of spec_verify_sample are R = B*(gamma+1) rows.
 *   temperature > 0, finite and not subnormal; only out_lse depends on it.
 *   out_ids     [R][K] int32 ids, out_values [R][K] float their logits (not
 *               tempered). -inf and NaN logits are not candidates: a row with
 *               fewer than K candidates is filled up with id -1, value -inf.
 *   out_lse     [R] float log sum_v exp(logit_v / temperature), or NULL; -inf
 *               for a row of -inf only, NaN for a row holding NaN or +inf.
 * Limits: 1 <= K <= SV_MAX_TOP, K <= V < 2^31, 1 <= R <= 2^22 (SV_ESIZE beyond). */
size_t spec_verify_top_logits_workspace_bytes(int32_t R, int32_t V, int32_t K, sv_dtype dtype);
int spec_verify_top_logits(const void* logits, int64_t logits_stride, sv_dtype dtype, int32_t R,
                           int32_t V, int32_t K, float temperature, int32_t* out_ids,
                           float* out_values, float* out_lse, void* workspace,
                           size_t workspace_bytes, void* stream);

/* Distillation from a teacher's kept logits. With T = temperature,
 *   p_k = exp(teacher_logits_k / T - L),
 *   L   = log sum_k exp(teacher_logits_k / T) over the row's slots, or
 *         teacher_lse[r] (then the kept slots keep their share of the whole row),
 *   q   = softmax(logits / T) over the vocabulary, P = sum_k p_k:
 *   loss = sum_k p_k (log p_k - log q_{id_k}),
 *   d loss / d logit_v = (P q_v - sum_{k: id_k = v} p_k) / T.
 *   logits         [R][V] of dtype: the drafter's (student's) rows.
 *   teacher_ids    [R][K] int32, teacher_logits [R][K] float, contiguous, in any
 *                  order, as spec_verify_top_logits writes them. A slot whose id
 *                  lies outside [0, V) or whose logit is -inf is empty;
 *                  an id may appear more than once: its masses add up.
 *   teacher_lse    [R] float (spec_verify_top_logits at the same temperature), or
 *                  NULL.
 *   row_weight     [R] float weights of out_grad (d total / d loss_r), or NULL (1).
 *   out_loss       [R] float, not weighted.
 *   out_stats      [R][2] float: the row's largest logit m, and
 *                  log sum_v exp((logit_v - m) / T).
 *   out_grad       [R][V] of dtype, row stride grad_stride >= V, or NULL (loss only).
 *                  It may be `logits` itself with the same stride (every value is
 *                  read before it is overwritten); any other overlap is an error
 *                  of the caller. Elements behind V are left as they are.
 * A row without a filled slot has loss 0 and gradient 0, whatever its logits. A row whose
 * logits are all -inf has gradient 0, and loss +inf against a filled slot, as
 * has a row that gives a kept token of positive mass -inf. NaN or +inf among a
 * row's logits, or NaN in its slots, make its loss and gradient NaN.
 * Limits: 1 <= K <= SV_MAX_TOP, 1 <= V < 2^31, 1 <= R <= 2^22 (SV_ESIZE beyond). */
size_t spec_verify_distill_workspace_bytes(int32_t R, int32_t V, sv_dtype dtype);
int spec_verify_distill(const void* logits, int64_t logits_stride, sv_dtype dtype, int32_t R,
                        int32_t V, const int32_t* teacher_ids, const float* teacher_logits,
                        const float* teacher_lse, int32_t K, float temperature,
                        const float* row_weight, float* out_loss, float* out_stats, void* out_grad,
                        int64_t grad_stride, void* workspace, size_t workspace_bytes, void* stream);

/* The gradient alone, from the statistics an earlier spec_verify_distill call
 * wrote for the same rows, teacher and temperature; grad_loss [R] float is the
 * gradient of each row's loss (NULL: 1). Needs no workspace. */
int spec_verify_distill_backward(const void* logits, int64_t logits_stride, sv_dtype dtype,
                                 int32_t R, int32_t V, const int32_t* teacher_ids,
                                 const float* teacher_logits, const float* teacher_lse, int32_t K,
                                 float temperature, const float* stats, const float* grad_loss,
                                 void* out_grad, int64_t grad_stride, void* stream);

/* Softmax cross entropy of a linear head over the vocabulary, without storing
 * the logits z = hidden weight^T:
 *   loss_n = log sum_v exp(z_nv) - z_{n, label_n}.
 *   hidden [N][D] and weight [V][D] of dtype (row strides >= D), labels [N] int32.
 *   A row whose label lies outside [0, V) (such as -100) is left out: loss 0, no
 *   gradient.
 *   out_loss  [N] float; out_stats [N][2] float: the row's largest logit m, and
 *             log sum_v exp(z_nv - m), also for the rows left out.
 * bfloat16 products are exact and summed in float32. float32 products are made by the
 * float32 matrix instructions for up to 384 states; for more, operands are taken as
 * three bfloat16 parts each, whose products down to 2^-24 of the largest are summed
 * in float32.
 * Inputs are finite; NaN or infinities make the rows (and with them the
 * gradients) they meet NaN.
 * Limits: 1 <= N <= 2^22, 1 <= D <= 2^22, 1 <= V < 2^31 - 1024, and 2^23 tiles of
 * 256 x 256 in N x V and N x D (64 x 32 up to 32 rows, 128 x 64 up to 128, 256 x 128 in
 * float32); SV_ESIZE beyond. Matrices whose rows start on 16 bytes and are whole groups of 16
 * bytes (D a multiple of 8 in bfloat16, of 4 in float32), at strides of at most 2^22, are read
 * in place, but for float32 of more than 384 states; others are copied into the workspace
 * first, the weight a piece at a time. The workspace holds whatever the strides need: for few
 * states about 128 MB, up to 1 GiB where D is not whole groups of 16 bytes. */
size_t spec_verify_linear_ce_workspace_bytes(int32_t N, int32_t D, int32_t V, sv_dtype dtype);
int spec_verify_linear_ce(const void* hidden, int64_t hidden_stride, const void* weight,
                          int64_t weight_stride, sv_dtype dtype, const int32_t* labels, int32_t N,
                          int32_t D, int32_t V, float* out_loss, float* out_stats, void* workspace,
                          size_t workspace_bytes, void* stream);

/* Its gradients, from the statistics an earlier spec_verify_linear_ce call wrote
 * for the same inputs. The logits are made again, a piece of the vocabulary at a
 * time: with dz_nv = grad_loss_n (softmax(z)_nv - [v = label_n]),
 *   out_grad_hidden [N][D] = dz weight,  out_grad_weight [V][D] = dz^T hidden,
 * both of dtype, with row strides >= D; either may be NULL (then not computed),
 * not both. grad_loss [N] float, or NULL (1).
 * For bfloat16, dz is taken as two bfloat16 parts, which hold it to 2^-16, and its
 * products are summed in float32. Outputs must not overlap inputs. Elements behind D are left as
 * they are. */
size_t spec_verify_linear_ce_backward_workspace_bytes(int32_t N, int32_t D, int32_t V,
                                                      sv_dtype dtype, int want_grad_hidden,
                                                      int want_grad_weight);
int spec_verify_linear_ce_backward(const void* hidden, int64_t hidden_stride, const void* weight,
                                   int64_t weight_stride, sv_dtype dtype, const int32_t* labels,
                                   const float* stats, const float* grad_loss, int32_t N, int32_t D,
                                   int32_t V, void* out_grad_hidden, int64_t grad_hidden_stride,
                                   void* out_grad_weight, int64_t grad_weight_stride,
                                   void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------- the verification pass's rows
 *
 * What a serving program does to the rows that a verification round reads, before
 * and after the target model's own layers: rotary positions of queries and keys,
 * a paged 8-bit cache of keys and values written and read back, attention of a
 * round's rows over it, and the adjustments of logits that are part of the
 * sampler and have to be made to the target's and the drafter's rows alike.
 *
 * Conventions of these calls
 *   - A batch has B requests of N rows (N = gamma + 1 in a verification round, 1 for
 *     plain decoding). Row j of request b stands at position kv_len[b] + j, kv_len as
 *     in spec_verify_commit. `rows` [B] (device) gives each request's number of
 *     rows, 0 <= rows[b] <= N (NULL: N). Outputs of rows beyond it are left as
 *     they were.
 *   - kv_len, rows and page tables live on the device, so what is wrong in them is only
 *     seen there. A request whose kv_len or rows is out of range has NaN in all its N rows
 *     of the outputs, and nothing of it is written to the cache.
 *   - Sums, softmax statistics and products are float32 or wider whatever the
 *     inputs' type; results are rounded once. (Attention's matrix products take the factors that do not
 *     fit bfloat16 as sums of bfloat16 numbers, see there.)
 *   - No result depends on the order in which workgroups run. (How attention shares out a
 *     request's tokens follows from the lengths of the whole batch: in another batch its sums may
 *     be in another order.)
 *   - Workspaces as in the training calls: no initialisation, 256-byte aligned,
 *     nothing kept between calls, separate ones for calls that may run concurrently. */

/* Element strides of a [B][N][heads][D] tensor whose D elements are consecutive. Inputs may
 * take any strides >= 0; rows and heads of outputs must not overlap, and
 * each is stepped over whole by the next wider stride (dimensions in any order). */
typedef struct {
  int64_t request, row, head;
} sv_strides;

/* Rotary positions. The first rotary_dim = R dimensions of every head are turned in pairs:
 * with a_i = position * freqs[i],
 *   (x, y) -> (scale (x cos a_i - y sin a_i), scale (y cos a_i + x sin a_i)),
 * pairs (i, i + R/2), or (2i, 2i + 1) when `interleaved` is not 0; the other
 * dimensions are copied. `inverse` (not 0) turns by -a_i: the gradient's way back.
 *   q, k       [B][N][q_heads][head_dim] and [B][N][k_heads][head_dim] of dtype at any
 *              strides (both may be views of one fused projection); k may be NULL
 *              with k_heads 0.
 *   freqs      [R/2] double on the device, radians a position: base^(-2i/R), scaled for long
 *              contexts as the caller's model does. Angles are made in float64.
 *   scale      finite; the factor on the rotated dimensions alone that some scalings
 *              for long contexts carry, else 1.
 *   kv_len     [B], or NULL (positions from 0); any int32 value is a position.
 *   out_q, out_k  like q and k at strides of their own; each may be its input
 *              at the input's strides. Any other overlap is an error of the caller.
 * Limits: head_dim >= 1, R even, 0 <= R <= head_dim <= 1024, q_heads >= 1; B*N < 2^31 and
 * q_heads + k_heads <= 2^15 (SV_ESIZE beyond). */
int spec_verify_rotate(const void* q, sv_strides q_strides, const void* k, sv_strides k_strides,
                       sv_dtype dtype, int32_t B, int32_t N, int32_t q_heads, int32_t k_heads,
                       int32_t head_dim, int32_t rotary_dim, int interleaved, int inverse,
                       const double* freqs, float scale, const int32_t* kv_len,
                       const int32_t* rows, void* out_q, sv_strides out_q_strides, void* out_k,
                       sv_strides out_k_strides, void* stream);

/* A paged cache of keys and values in 8 bits (e4m3: no infinities, largest value 448).
 * Position p of request b lies in page page_table[b][p / page_size], token p % page_size.
 * A block is 32 consecutive tokens of a page and one head, and has one scale for its keys and
 * one for its values: value = scale * code.
 *   k, v              [pages][heads][page_size / 32] blocks of 1024 * ceil(head_dim / 32)
 *                     bytes. A block is made of bricks of 32 dimensions; within a brick
 *                     the code of token s and dimension d (both 0..31) is
 *                       keys:   byte 256 (d / 8) + 16 (4 (s / 8) + s % 4) + 8 (s / 4 % 2) + d % 8
 *                       values: byte 256 (s / 8) + 16 (d % 16) + 8 (d / 16) + s % 8,
 *                     the order in which a wavefront takes an operand of its matrix
 *                     instruction, 16 consecutive bytes a lane.
 *   k_scale, v_scale  [pages][heads][page_size / 32] float, not negative.
 *   page_size         a power of two from 32 to 65536.
 * Fresh memory needs no initialisation: what no call has written is never used. */
typedef struct {
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  int32_t pages, heads, page_size, head_dim;
} sv_cache;

/* Bytes of k (and of v); 0 when a size is out of range. */
size_t spec_verify_cache_bytes(int32_t pages, int32_t heads, int32_t page_size, int32_t head_dim);

/* Writes the keys and values of a batch's rows, positions kv_len[b] .. kv_len[b] + rows[b] - 1.
 * The scale of a block is the smallest power of two 2^e, e >= -126, with max |x| <= 448 * 2^e
 * over what it holds up to its last new row (1 if that is all zero): the new rows, and the
 * rows before kv_len[b] in the same block, whose codes are taken over, at the new
 * scale, rounded to nearest even as the new ones. So the scale is a function of what the block
 * holds: a proposal that was rejected leaves no trace in the scale once its slot is
 * rewritten, and writing the same rows again changes nothing. Codes do not come back: rows that are 2^k times
 * the largest value L of the rows before them in the block round those below 2^(k - 13) L more coarsely (by at
 * most 2^(k - 17) L), and these stay so when the large rows are rejected. A call that begins at the block's
 * first position takes nothing over, so a program whose committed keys and values must not depend on rejected
 * proposals writes the last block's committed rows again, from its own copies, in front of the new ones. And all
 * rows of a call are rounded before any attends: an earlier row of a round sees the block at the scale
 * that later proposals of the round gave it. NaN and infinities are stored as
 * NaN and left out of the scale; numbers that would round to 2^128 (from 248 * 2^120 on), which
 * float32 does not hold, are stored as 240 * 2^120. Slots behind the last new row keep their bytes, whose values
 * follow the scale.
 *   k, v        [B][N][cache heads][head_dim] of dtype at any strides.
 *   page_table  [B][table_width] int32. A row whose page lies outside [0, pages) is not written.
 *               A block may be written at one position only: requests that share pages must own
 *               the block they write into, and a page stands in a table once.
 * A request is out of range (nothing written) when kv_len[b] < 0, rows[b] is not in 0..N, or
 * kv_len[b] + rows[b] > table_width * page_size.
 * Limits: 1 <= head_dim <= 256; table_width * page_size <= 2^30, N <= 2^30 and
 * B * heads * ceil((N + 31) / 32) < 2^22 (SV_ESIZE beyond). */
int spec_verify_cache_write(const sv_cache* cache, const int32_t* page_table, int32_t table_width,
                            const int32_t* kv_len, const int32_t* rows, const void* k,
                            sv_strides k_strides, const void* v, sv_strides v_strides,
                            sv_dtype dtype, int32_t B, int32_t N, void* stream);

/* Reads positions first[b] .. first[b] + rows[b] - 1 (first NULL: from 0) back: scale * code,
 * rounded once to dtype. out_k, out_v [B][N][heads][head_dim]; either may be NULL, not both.
 * Positions in a page outside [0, pages) read as NaN; a request is out of range, and sizes are
 * limited, as in spec_verify_cache_write. */
int spec_verify_cache_read(const sv_cache* cache, const int32_t* page_table, int32_t table_width,
                           const int32_t* first, const int32_t* rows, void* out_k,
                           sv_strides k_strides, void* out_v, sv_strides v_strides, sv_dtype dtype,
                           int32_t B, int32_t N, void* stream);

/* Attention of a round's rows over the cache, which already holds them (call
 * spec_verify_cache_write first). Query head h reads cache head h / (q_heads / heads). Row j
 * of request b, at p = kv_len[b] + j, sees positions max(0, p - window + 1) .. p (window 0: all
 * up to p):
 *   out = sum_t softmax_t(scale q . k_t) v_t,   out_lse = log sum_t exp(scale q . k_t).
 *   q        [B][N][q_heads][head_dim] of dtype at any strides; scale finite.
 *   out      like q, of dtype, at its strides, over no part of q; out_lse [B][N][q_heads] float, or
 *            NULL.
 * bfloat16: products of q and k are exact; a weight enters its product with v as the sum of two
 * bfloat16 numbers (off by 2^-17 of itself, however small it is), and blocks whose v_scale lies 2^-100 below
 * another's of the request lose precision. float32: q and the weights times v_scale as sums of three
 * (2^-25; less where such a product is below 2^-100). The sums are divided at the end: where a value times
 * 256 times the number of tokens passes 2^128, they may be infinite.
 * NaN in a position that a row does not see does not reach it. A row that sees a position in a
 * page outside [0, pages) is NaN; pages that no row of the request sees (all before its window)
 * are not read. Requests out of range as in spec_verify_cache_write.
 * Limits: 1 <= N <= 64, q_heads a multiple of the cache's heads (at most 4096 of them to one, SV_ESIZE
 * beyond), head_dim <= 256, window >= 0; B * N * q_heads < 2^31 (SV_ESIZE beyond) and, with the
 * N * q_heads / heads columns of a cache head counted in tiles of 16, a launch of B * heads * tiles: up
 * to 2^19 always, SV_ESIZE where they take more than 2^23 workgroups. The workspace holds the parts of requests that
 * several workgroups share; `tokens` is table_width * page_size, or window + N + 31 where that is less
 * (window not 0). Up to 1120 tokens the call is taken without a usable one too, and the function gives more than 0 only
 * where many rows or wide heads of few requests are faster with it. */
#define SV_MAX_ROWS 64
size_t spec_verify_attention_workspace_bytes(int32_t B, int32_t N, int32_t q_heads, int32_t heads,
                                             int32_t head_dim, int64_t tokens, sv_dtype dtype);
int spec_verify_attention(const void* q, sv_strides q_strides, sv_dtype dtype, int32_t B, int32_t N,
                          int32_t q_heads, const sv_cache* cache, const int32_t* page_table,
                          int32_t table_width, const int32_t* kv_len, const int32_t* rows,
                          float scale, int32_t window, void* out, sv_strides out_strides,
                          float* out_lse, void* workspace, size_t workspace_bytes, void* stream);

/* Adjusts the logits of a batch's rows before they are compared or drawn from. For row j of
 * request b let c_v be how often token v occurs in history[b] and in tokens[b][0 .. j-1]
 * (the proposals before row j), and seen_v whether c_v > 0 or v occurs in prompt[b]. In float32:
 *   z1 = seen_v ? (z > 0 ? z / repetition[b] : z * repetition[b]) : z
 *   z2 = c_v > 0 ? z1 - (frequency[b] * c_v + presence[b]) : z1
 *   z3 = z2 + bias_v                                 (tokens with a bias)
 *   out = bit v of allowed[b][j] is set ? z3 : -inf
 * rounded once to dtype; a logit that none of these touches keeps its bits.
 *   logits, out  [B][N][V] of dtype, rows of V at strides >= V elements (request and row; `head`
 *                is not used). out may be logits itself at the same strides; any other overlap is
 *                an error of the caller.
 *   tokens       [B][n_tokens] int32, n_tokens >= N - 1, or NULL with n_tokens 0 (no proposals).
 *   history, prompt  [B][n_history], [B][n_prompt] int32, or NULL with 0.
 *                Ids outside [0, V), such as -1, are padding in all lists.
 *   repetition, frequency, presence  [B] float, or NULL (1, 0, 0). They are taken as
 *                they are: a repetition of 0 divides by it.
 *   bias_ids, bias  [B][n_bias] int32 and float, or NULL with 0; the last entry of an id that
 *                occurs more than once counts.
 *   allowed      [B][N][ceil(V / 32)] words, token v at bit v % 32 of word v / 32, or NULL. A row
 *                without a set bit becomes all -inf (SV_FLAG_EMPTY in the verifier).
 * A request whose rows[b] is not in 0..N has NaN in all its rows.
 * Limits: V < 2^31 - 2^16, n_history, n_prompt and n_bias < 2^24, B * N * ceil(V / 4096) < 2^23
 * (SV_ESIZE beyond). */
int spec_verify_adjust_logits(const void* logits, sv_strides strides, sv_dtype dtype, int32_t B,
                              int32_t N, int32_t V, const int32_t* rows, const int32_t* tokens,
                              int32_t n_tokens, const int32_t* history, int32_t n_history,
                              const int32_t* prompt, int32_t n_prompt, const float* repetition,
                              const float* frequency, const float* presence,
                              const int32_t* bias_ids, const float* bias, int32_t n_bias,
                              const uint32_t* allowed, void* out, sv_strides out_strides,
                              void* stream);

/* Static description of a status code. */
const char* spec_verify_strerror(int status);


#ifdef __cplusplus
}
#endif

#endif /* SPEC_VERIFY_H */
