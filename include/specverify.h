/*
 * specverify.h -- C ABI of the batched speculative-decoding verification
 * library (libspecverify.so, CUDA kernels for sm_103a).
 *
 * The operation (one verification round per sequence) is the rule stated in
 *   - nextadmin.net lesson "Speculative Decoding (دیکودینگ گمانه‌زن)",
 *     § Core algorithm, steps 4-6, and § Step 1 (accept/reject), § Step 2
 *     (residual distribution), § Step 3 (one speculative step);
 *   - aiengineeringfromscratch.com Phase 10 lesson 25 "Speculative Decoding",
 *     § The exact rule and § Greedy case;
 *   - runelab.ai "Küçük bir model büyük olanı nasıl hızlandırır?", § the
 *     exact rule (points 1-3 and the bonus token);
 *   - for the shortlisted draft, the DynaSpec summary (lowest.today, "DynaSpec:
 *     Context-aware Dynamic Speculative Sampling for Large-Vocabulary Language
 *     Models"), § Abstract and § Method 3: the drafter works on a
 *     per-context shortlist, verification keeps the full vocabulary.
 * Notation: q = target distribution, p = draft distribution, d_i = drafted
 * tokens (i = 1..K), V = vocabulary size, T = temperature.
 *
 * For each sequence b, with q_i = softmax(target[b][i-1] / T) and
 * p_i = softmax(draft[b][i-1] / T) (or the given draft probabilities):
 *   for i = 1..K, left to right, accept d_i iff u_i < min(1, q_i(d_i)/p_i(d_i))
 *   (always when p_i(d_i) == 0); at the first rejection j emit a token drawn
 *   from (q_j - p_j)_+ / R_j (R_j its total; q_j itself when R_j == 0) and stop;
 *   if all K are accepted emit a bonus token drawn from q_{K+1}.
 *   T == 0 is greedy: accept d_i while d_i == argmax q_i (lowest index on
 *   ties), then emit argmax q_j at the first mismatch (argmax q_{K+1} if none).
 * Uniforms: Philox4x32-10 (Salmon et al., SC'11) with counter
 *   (position i-1, sequence b, 0, 0) and key (seed & 0xffffffff, seed >> 32);
 *   word 0 gives u_i, word 1 gives the sampling uniform v; a word w maps to
 *   ((w >> 8) + 0.5) * 2^-24.  Sampling is inverse-CDF in ascending token
 *   order: the smallest x with sum_{y<=x} r(y) > v * R.
 *
 * Conventions for every entry point:
 *   - All array pointers are DEVICE pointers owned by the caller; rows are
 *     contiguous and row-major.  Rows whose start is 16-byte aligned (row
 *     length times element size a multiple of 16 and a 16-byte aligned base)
 *     take the bulk-copy path; other shapes are correct but slower.
 *   - `workspace` is caller-owned device scratch of at least
 *     spec_workspace_bytes(B, K, V, S) bytes.  It must be zero-filled before
 *     its first use with given sizes (B, K, V, S); a call that returns SPEC_OK
 *     leaves it ready for the next call with the same sizes.  Before reusing it
 *     with other sizes, zero-fill it again: its control words sit at offsets
 *     that depend on the sizes.  One workspace per call in flight: two calls
 *     that overlap on the GPU must not share one.
 *   - Calls are asynchronous on `stream` (a cudaStream_t; NULL is the legacy
 *     default stream).  Argument errors are returned synchronously, before
 *     anything is launched.  Data errors are found on the device, in the rows
 *     the left-to-right rule examines: that sequence gets out_accept_len[b] =
 *     -code and out_tokens[b][*] = -1, and aux->device_status (if given)
 *     receives the code of one failing sequence after the kernel ends.  The
 *     device never traps.
 *   - out_tokens[b] holds the accepted draft tokens followed by one target
 *     token; out_accept_len[b] is the number of accepted draft tokens (0..K),
 *     so out_accept_len[b] + 1 tokens are emitted; unused slots are -1.
 */
#ifndef SPECVERIFY_H
#define SPECVERIFY_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    SPEC_OK = 0,
    SPEC_ERR_INVALID_ARG = 1,  /* bad size, pointer, dtype, temperature or workspace size */
    SPEC_ERR_NONFINITE = 2,    /* NaN / +inf logit, all -inf row, or bad draft probability */
    SPEC_ERR_TOKEN_RANGE = 3,  /* a drafted token outside [0, V) */
    SPEC_ERR_SHORTLIST = 4,    /* shortlist not ascending and unique inside [0, V) */
    SPEC_ERR_UNSUPPORTED = 5,  /* no usable sm_103a device, or a shape the entry point does not take */
    SPEC_ERR_CUDA = 6,         /* a CUDA runtime call or launch failed */
    SPEC_ERR_TIMEOUT = 7       /* a bounded on-device wait ran out (the kernel gave up) */
} spec_status_t;

typedef enum { SPEC_F32 = 0, SPEC_BF16 = 1 } spec_dtype_t;

/* Optional per-call outputs.  Any NULL member is not written.  Asking for
 * q_draft, p_draft or row_lse makes the call evaluate every position (it then
 * reads every row), not only the positions up to the first rejection.
 * All pointers are device pointers.                                          */
typedef struct {
    float *q_draft;          /* [B][K]     q_i(d_i); NaN where row or token is invalid   */
    float *p_draft;          /* [B][K]     p_i(d_i); NaN where row or token is invalid   */
    float *residual_mass;    /* [B]        total R of the distribution the last token was
                                           drawn from (residual, or q_{K+1} for a bonus) */
    float *row_lse;          /* [B][2K+1]  log sum exp(z / T): target rows 0..K, then draft
                                           rows 0..K-1 (NaN for draft probabilities)      */
    int32_t *device_status;  /* [1]        0, or the code of one failing sequence         */
} spec_aux_t;

/* Bytes of device workspace a call with these sizes needs (S = 0 without a
 * shortlist).  Returns 0 for sizes the library rejects.                      */
size_t spec_workspace_bytes(int B, int K, int V, int S);

/* Stochastic verification; T == 0 runs the greedy rule.
 *   target_logits  [B][K+1][V]  dtype `tdt`
 *   draft          [B][K][V]    logits of dtype `tdt`, or float32 probabilities
 *                               when draft_is_probs != 0 (ddt must then be SPEC_F32)
 *   draft_tokens   [B][K]       int32
 *   out_tokens     [B][K+1]     int32;  out_accept_len [B] int32
 * Limits: B >= 1, 1 <= K <= 31, V >= 1, T finite and >= 0.                     */
spec_status_t spec_verify(const void *target_logits, spec_dtype_t tdt,
                          const void *draft, spec_dtype_t ddt, int draft_is_probs,
                          const int32_t *draft_tokens,
                          int B, int K, int V, float T, uint64_t seed,
                          int32_t *out_tokens, int32_t *out_accept_len,
                          void *workspace, size_t workspace_bytes,
                          const spec_aux_t *aux, void *stream);

/* Greedy verification (aiengineeringfromscratch.com lesson 25, § Greedy case):
 * only the target logits are read. */
spec_status_t spec_verify_greedy(const void *target_logits, spec_dtype_t tdt,
                                 const int32_t *draft_tokens, int B, int K, int V,
                                 int32_t *out_tokens, int32_t *out_accept_len,
                                 void *workspace, size_t workspace_bytes,
                                 const spec_aux_t *aux, void *stream);

/* Verification with a draft defined on a per-sequence shortlist (DynaSpec):
 *   draft_sl       [B][K][S]  logits (dtype `tdt`) or float32 probabilities over
 *                             the shortlisted tokens; p is 0 off the shortlist
 *   shortlist_idx  [B][S]     int32, strictly ascending, each in [0, V)
 * The target distribution and the residual stay over the full vocabulary.
 * A drafted token outside its shortlist has p_i(d_i) = 0 and is accepted.    */
spec_status_t spec_verify_shortlist(const void *target_logits, spec_dtype_t tdt,
                                    const void *draft_sl, spec_dtype_t ddt, int draft_is_probs,
                                    const int32_t *shortlist_idx, int S,
                                    const int32_t *draft_tokens,
                                    int B, int K, int V, float T, uint64_t seed,
                                    int32_t *out_tokens, int32_t *out_accept_len,
                                    void *workspace, size_t workspace_bytes,
                                    const spec_aux_t *aux, void *stream);

/* Verification with a shortlisted draft whose list may depend on the position
 * (DynaSpec summary, § Method 3: the position-aware budget k_c(t) sets how
 * many clusters, hence tokens, the drafter uses at draft step t; a static
 * list shared by every sequence and position, as in FR-Spec, is the same
 * layout with both strides 0).
 *   draft_sl       [B][K][S]  draft logits of dtype `tdt` (ddt == tdt); row (b, i)
 *                             holds shortlist_len[i] logits, for the tokens of
 *                             list (b, i)
 *   shortlist_idx  list (b, i) starts at shortlist_idx + b * sl_seq_stride +
 *                  i * sl_pos_stride (entries): strictly ascending, each in [0, V)
 *                  (per position: strides K*S and S; per sequence: S and 0;
 *                  shared: 0 and 0)
 *   shortlist_len  HOST array of K entry counts, each in [1, S], or NULL (all S)
 * p_i is 0 off list (b, i); the target and the residual stay over the full
 * vocabulary; a drafted token off its list has p_i(d_i) = 0 and is accepted.
 * A list that is not strictly ascending inside [0, V) is an error
 * (SPEC_ERR_SHORTLIST) at the position that uses it, found only if the rule
 * reaches that position.  Draft probabilities are not accepted here.
 * The workspace is spec_workspace_bytes(B, K, V, S).  T == 0 runs the greedy
 * rule (the draft is not read).  Served by the row-parallel kernels.         */
spec_status_t spec_verify_shortlist_pos(const void *target_logits, spec_dtype_t tdt, const void *draft_sl,
                                        spec_dtype_t ddt, const int32_t *shortlist_idx, long long sl_seq_stride,
                                        long long sl_pos_stride, const int32_t *shortlist_len, int S,
                                        const int32_t *draft_tokens, int B, int K, int V, float T, uint64_t seed,
                                        int32_t *out_tokens, int32_t *out_accept_len, void *workspace,
                                        size_t workspace_bytes, const spec_aux_t *aux, void *stream);

/* Verification with no caller workspace (the pages have no counterpart: this
 * is an interface for callers that cannot allocate device memory, or cannot
 * hold a workspace per call, e.g. code with a fixed memory plan).  Arguments
 * and results are those of spec_verify (T == 0: greedy, draft_logits may be
 * NULL) with draft logits only.
 *   Scratch: a 256-byte device array inside the library holds the kernel's
 *   control words.  It is zero when the library loads, and every call that
 *   completes leaves it zero.  The call allocates nothing; it is served by
 *   the cluster kernel alone.
 *   Limits: rows 16-byte aligned (V * element size a multiple of 16, aligned
 *   bases), one CTA's slice of a position within that kernel's shared-memory
 *   budget (about V <= 289280 bfloat16 / 144640 float32 logits with draft
 *   rows, twice that for greedy), and no q_draft / p_draft / row_lse outputs.
 *   Any other call returns SPEC_ERR_UNSUPPORTED without launching;
 *   spec_verify serves it.
 *   Overlapping calls race: all calls on a device share the scratch, so they
 *   must be ordered on the GPU (one stream, or events between streams).
 *   Every call looks up the scratch's device address with a CUDA runtime
 *   call (a host-side lookup, not a stream operation), so the address stays
 *   right after a cudaDeviceReset.  The first call on a device also loads the
 *   library's kernels there; make that first call outside any stream capture. */
spec_status_t spec_verify_static(const void *target_logits, spec_dtype_t tdt, const void *draft_logits,
                                 const int32_t *draft_tokens, int B, int K, int V, float T, uint64_t seed,
                                 int32_t *out_tokens, int32_t *out_accept_len, const spec_aux_t *aux,
                                 void *stream);

/* Fused draft-token sampler: the drafting step that precedes verification
 * (nextadmin.net lesson "Speculative Decoding", § Core algorithm step 2 and
 * § Build it, spec_step: each drafted token is drawn from the draft
 * distribution and its probability p_dist[d] is kept for the acceptance test;
 * aiengineeringfromscratch.com lesson 25, § Build it: softmax of the logits
 * divided by the temperature).
 *   draft_logits  [B][K][V]  dtype `ddt`; row (b, i) is the drafter's output at
 *                            position i of sequence b (already conditioned on
 *                            the earlier drafts)
 *   out_tokens    [B][K]     int32: d_i = the smallest x whose running sum of
 *                            softmax(z / T) in ascending token order exceeds
 *                            v * R (R the total), v = word 0 of Philox4x32-10
 *                            with counter (i, b, 1, 0) and key (seed low, seed
 *                            high), mapped by ((w >> 8) + 0.5) * 2^-24
 *   out_prob      [B][K]     float: p_i(d_i) (may be NULL)
 *   device_status [1]        set to 0, or SPEC_ERR_NONFINITE when some row has a
 *                            NaN or +inf logit or is -inf everywhere (that row
 *                            gets token -1 and probability NaN); may be NULL
 * T == 0 drafts greedily: the first index of the largest logit, probability 1.
 * Limits: B, K, V >= 1, B * K <= 2^30, V <= 2093056, T finite and >= 0.
 * No workspace; the call is asynchronous on `stream`.                         */
spec_status_t spec_draft_sample(const void *draft_logits, spec_dtype_t ddt, int B, int K, int V, float T,
                                uint64_t seed, int32_t *out_tokens, float *out_prob, int32_t *device_status,
                                void *stream);

/* What requests ask for beside the temperature: device arrays of B entries, one
 * per sequence; NULL: off for all.  A row's tokens in descending order of the
 * logit z, the lowest index first among equals, have the weights
 * w = e^((z - max z) / T).  In turn:
 *   top_k  keeps the first k (k <= 0: all);
 *   top_p  keeps, of those, a token if the sum of the weights ahead of it is
 *          less than p times the sum of what top_k left (p >= 1: all);
 *   min_p  keeps w >= min_p (min_p <= 0: all).
 * The first token stays in any case; what is kept is normalised.  T == 0 is the
 * first token alone.  A temperature that is negative, infinite or NaN, a top_p of
 * NaN and a min_p above 1 or NaN are data errors (SPEC_ERR_INVALID_ARG) of the
 * sequence.  Temperatures below 2^-100 count as that, above 2^100 as that.
 * Weights are whole numbers of 2^-43 of the row's largest, right to half of one and
 * to 2^-31 of their own (those below 2^-43.75 of the largest are none), so sums of
 * them are exact.  The total that top-p takes its share of is right to 2^-29 of
 * itself.  Results do not depend on how the work is split, but for a top-p border
 * that lies nearer than that.                                                 */
typedef struct {
    const float *temperature;   /* NULL: 1 */
    const int32_t *top_k;
    const float *top_p;
    const float *min_p;
} spec_filters_t;

/* Tokens drawn from filtered rows of logits by given random numbers (the
 * drafting step of spec_draft_sample's sections, and plain decoding):
 *   logits        [B][K][V]  dtype `ldt`; row (b, i) under sequence b's filters
 *   uniforms      [B][K]     float32 in [0, 1)
 *   filters       NULL: none
 *   out_tokens    [B][K]     int32: the smallest x whose running sum of kept weights
 *                            in ascending token order exceeds uniform * their total
 *   out_prob      [B][K]     float: the token's probability among the kept (may be NULL)
 *   device_status [1]        set to 0, or the code of one failing row; may be NULL
 * A row with a NaN or +inf logit, or -inf everywhere (SPEC_ERR_NONFINITE), with
 * filters as above or a uniform outside [0, 1) (SPEC_ERR_INVALID_ARG) gets token -1
 * and probability NaN.  -inf logits are never drawn.
 * Limits: B, K, V >= 1, B * K <= 2^26, V <= 524288.  No workspace; one launch,
 * asynchronous on `stream`.                                                   */
spec_status_t spec_filter_sample(const void *logits, spec_dtype_t ldt, const float *uniforms, int B, int K, int V,
                                 const spec_filters_t *filters, int32_t *out_tokens, float *out_prob,
                                 int32_t *device_status, void *stream);

/* Verification between filtered distributions (the rule of the top of this
 * file, with q_i the target's row i under `filters` and p_i the draft's row i
 * under `draft_filters`): accept d_i iff u_i p_i(d_i) < q_i(d_i), so a token that
 * neither keeps is rejected; at the first rejection j a token from (q_j - p_j)+,
 * from q_j itself when that is nothing; after K accepted drafts one from q_{K+1}.
 *   target_logits  [B][K+1][V], draft_logits [B][K][V]  dtype `tdt`
 *   draft_tokens   [B][K]       int32, drawn from p_i (spec_filter_sample)
 *   uniforms       [B][K+1][2]  float32 in [0, 1): u_i, and the number that the
 *                               emitted token is drawn with when the round ends at i
 *   draft_filters  NULL: the same as `filters`
 *   out_tokens     [B][K+1], out_accept_len [B]  as spec_verify's, with its data errors:
 *                  those of the rows and uniforms that the left-to-right rule
 *                  reaches, and of filters (SPEC_ERR_INVALID_ARG, as uniforms)
 *   workspace      device scratch of spec_filter_workspace_bytes(B, K, V) bytes (no
 *                  zero-fill needed), 16-byte aligned; one per call in flight
 *   device_status  [1] set to 0, or the code of one failing sequence; may be NULL
 * Drawing is spec_filter_sample's.  Limits: B >= 1, 1 <= K <= 31, 1 <= V <= 524288,
 * B (2K + 1) <= 2^26.  Two launches, asynchronous on `stream`.                 */
size_t spec_filter_workspace_bytes(int B, int K, int V);
spec_status_t spec_verify_filtered(const void *target_logits, spec_dtype_t tdt, const void *draft_logits,
                                   const int32_t *draft_tokens, const float *uniforms, int B, int K, int V,
                                   const spec_filters_t *filters, const spec_filters_t *draft_filters,
                                   int32_t *out_tokens, int32_t *out_accept_len, void *workspace,
                                   size_t workspace_bytes, int32_t *device_status, void *stream);

/* KV-cache commit (and rollback) after verification (nextadmin.net lesson
 * "Speculative Decoding", § KV cache management: the verification pass
 * appends the K drafts' entries; when drafts are rejected the cache returns
 * to the accepted prefix, production systems staging the K entries and
 * committing the accepted ones; § Exercises item 4 fixes the outcome).
 *   cache       [NL][B][L][entry_bytes]  the KV cache: NL layers, capacity L
 *                                        entries per sequence, entry_bytes
 *                                        bytes per entry and layer (keys and
 *                                        values of all heads, any dtype)
 *   staged      [NL][B][K][entry_bytes]  the K new entries of the verification
 *                                        pass, or NULL when they were written in
 *                                        place at [seq_len[b], seq_len[b] + K)
 *   accept_len  [B]   spec_verify's out_accept_len (accepted drafts, or < 0
 *                     for a sequence in error)
 *   seq_len     [B]   in/out: cache lengths
 * For a = accept_len[b] >= 0: entries 0..a-1 of staged[l][b] are copied to
 * cache[l][b][seq_len[b]..] for every layer and seq_len[b] += a; the drafts'
 * other entries are dropped (rolled back).  a < 0 changes nothing.  a > K, or
 * seq_len[b] + a > L, changes nothing and sets *device_status to
 * SPEC_ERR_INVALID_ARG (device_status is set to 0 first; it may be NULL).
 * Device pointers; staged must not overlap cache.  16-byte aligned buffers
 * with entry_bytes a multiple of 16 take the vector path.  Asynchronous on
 * `stream`; two launches (one in place).  The token emitted at the rejection
 * (or the bonus token) has no entry yet: it is the next round's input.       */
spec_status_t spec_kv_commit(void *cache, const void *staged, int NL, int B, int K, int L, size_t entry_bytes,
                             const int32_t *accept_len, int32_t *seq_len, int32_t *device_status,
                             void *stream);

/* The KV cache in 8 bits.  An entry of a layer is [2][Hkv][D]: the keys, then
 * the values, of Hkv heads of D elements (D = 64 or 128).  Quantised, it is D
 * e4m3 codes per head (1 sign, 4 exponent, 3 mantissa bits, largest number
 * 448) and one scale byte per head in an array of its own, [2][Hkv] per entry:
 *   element = code * 2^(byte - 127); byte 255: every element of the head is NaN.
 * A head with the largest magnitude amax gets the least e >= -126 with
 * amax <= 448 * 2^e, byte e + 127 (127 when amax == 0), and the codes
 * e4m3(x * 2^-e), rounded to nearest even; a head with a NaN or an infinity
 * gets byte 255.  Read back, an element is exact in float32 up to that type's
 * largest number (bytes to 246, whatever the code), and in bfloat16 from byte 3 on
 * as well: bfloat16's smallest step is 2^-133, a code's at byte 0 2^-136.
 *
 * spec_kv_commit_quant commits the accepted entries of a verification pass as
 * spec_kv_commit does (the same sections), quantising them on the way:
 *   cache       [NL][B][L][2][Hkv][D]  e4m3 codes
 *   scale       [NL][B][L][2][Hkv]     scale bytes
 *   staged      [NL][B][K][2][Hkv][D]  the K new entries, dtype `sdt`
 *   nodes       [B][K]  staged entries after the lead, in the order of the
 *               commit (out_nodes of spec_verify_tree_greedy), or NULL (in order)
 *   accept_len  [B]     accepted drafts, or < 0 for a sequence in error
 *   seq_len     [B]     in/out: cache lengths
 *   lead        staged entries that are committed ahead of the accepted ones:
 *               0, or 1 when entry 0 is that of the last emitted token, the
 *               pass's first input (a tree's root)
 * For a = accept_len[b] >= 0, n = lead + a entries go to positions
 * seq_len[b].. of every layer and seq_len[b] += n: entry i < lead is staged
 * entry i, a later one is staged entry i, or nodes[b][i - lead].  a < 0 changes
 * nothing.  n > K, seq_len[b] outside [0, L - n] or a used node outside [0, K)
 * changes nothing and sets *device_status to SPEC_ERR_INVALID_ARG
 * (device_status is set to 0 first; it may be NULL).  16-byte aligned arrays
 * (scale: any); staged must not overlap cache.  Asynchronous on `stream`, two
 * launches.                                                                   */
spec_status_t spec_kv_commit_quant(void *cache, uint8_t *scale, const void *staged, spec_dtype_t sdt,
                                   const int32_t *nodes, int lead, int NL, int B, int K, int L, int Hkv, int D,
                                   const int32_t *accept_len, int32_t *seq_len, int32_t *device_status,
                                   void *stream);

/* Reads entries of an 8-bit cache back:
 *   out [NL][B][count][2][Hkv][D], dtype `odt`: entry i of sequence b is the
 *   cache's entry start[b] + i (start NULL: 0), zero at and past seq_len[b].
 * seq_len[b] outside [0, L] or start[b] < 0 gives zeros and sets *device_status
 * to SPEC_ERR_INVALID_ARG (set to 0 first; may be NULL).  Elements that
 * `odt` does not hold are rounded to it, past its largest number to infinity.  16-byte
 * aligned arrays (scale: any).  Asynchronous on `stream`, one launch.          */
spec_status_t spec_kv_read_quant(const void *cache, const uint8_t *scale, const int32_t *start,
                                 const int32_t *seq_len, int NL, int B, int L, int count, int Hkv, int D, void *out,
                                 spec_dtype_t odt, int32_t *device_status, void *stream);

/* Attention of the verification pass (nextadmin.net lesson "Speculative
 * Decoding", § KV cache management: one target forward pass over the drafts
 * extends the cache; aiengineeringfromscratch.com Phase 10 lesson 25, § Tree
 * attention verification: each node of a draft tree sees only its ancestors).
 * The T query tokens of sequence b (the last emitted token and K drafts, a
 * tree's N nodes, or the single token of plain decoding) attend to
 *   - a prefix of P entries that every sequence of the batch shares,
 *   - the sequence's own cache entries [0, seq_len[b]),
 *   - the T entries of this pass, not yet committed: entry j for token t where
 *     mask[b][t][j] != 0 (spec_tree_mask's layout), without a mask where j <= t.
 * For query head hq, which reads key/value head hq / (Hq / Hkv):
 *   out = sum_j w_j v_j / sum_j w_j,  w_j = exp(sm_scale q . k_j),
 *   lse = ln sum_j w_j, over the visible entries.
 * A row that sees nothing has out = 0 and lse = -inf.  Entries that a row does
 * not see are never part of its result, whatever they hold.
 *   q             [B][T][Hq][D]       bfloat16
 *   prefix        [P][2][Hkv][D]      bfloat16, or e4m3 codes when quant != 0; NULL when P == 0
 *   prefix_scale  [P][2][Hkv]         scale bytes (quant != 0), else NULL
 *   cache         [B][L][2][Hkv][D]   one layer of the cache, of the prefix's type; NULL when L == 0
 *   cache_scale   [B][L][2][Hkv]      scale bytes (quant != 0), else NULL
 *   seq_len       [B]                 int32
 *   staged        [B][T][2][Hkv][D]   bfloat16, or NULL: no entries of this pass (mask NULL too)
 *   mask          [B][T][T]           uint8, or NULL
 *   out           [B][T][Hq][D]       bfloat16
 *   lse           [B][T][Hq]          float32 (may be NULL)
 *   workspace     device scratch of spec_attention_workspace_bytes(...) bytes (no
 *                 zero-fill needed), 16-byte aligned; one per call in flight
 *   device_status [1] set to 0, or the code of one failing sequence; may be NULL
 * seq_len[b] outside [0, L] is an error (SPEC_ERR_INVALID_ARG): that
 * sequence's outputs are NaN.  So are the rows that a CTA leaves unfinished when a
 * bounded wait of its own runs out (SPEC_ERR_TIMEOUT).  Scores, softmax
 * statistics and sums are float32; a weight below 2^-117 of its row's largest may
 * count as 0.
 * What is rounded to fewer bits on the way: the weights where they meet prefix
 * and cache values, to bfloat16, by 2^-8 of a weight at most.  With 8-bit entries:
 *   - the weights to float16, by 2^-11 of a weight, or 2^-36 of the row's largest
 *     where that is more (a weight counts here times the largest value scale of
 *     its unit of 128 entries, heads of zeros left out);
 *   - values of heads whose scale is far below that of their unit, 2^s: from
 *     2^(s-23) on by 2^-40 of 448 * 2^s, and from 2^(s-32) on they are taken for
 *     0 (s < -100 counts as -100);
 *   - elements of q below 2^-10 of their row's largest, by 2^-18 of that.
 * Key scales above 2^103 may take a score out of float32's range.  An 8-bit
 * prefix under B T Hq / Hkv >= 1024 rows is read back to bfloat16 in the
 * workspace, as spec_kv_read_quant does, and then counts as bfloat16 here.
 * Limits: D = 64 or 128, Hq a multiple of Hkv, Hq / Hkv <= 128, sm_scale finite
 * and > 0, P, L >= 0, T <= 2048, B T Hq <= 2^30.  All arrays but the scales, mask and
 * lse 16-byte aligned.  One launch without prefix and cache, else two, four when
 * the prefix is read back (three without a cache).  Asynchronous on `stream`.  */
size_t spec_attention_workspace_bytes(int B, int T, int Hq, int Hkv, int D, int P, int L);
spec_status_t spec_verify_attention(const void *q, const void *prefix, const uint8_t *prefix_scale, const void *cache,
                                    const uint8_t *cache_scale, int quant, const int32_t *seq_len,
                                    const void *staged, const uint8_t *mask, int B, int T, int Hq, int Hkv, int D,
                                    int P, int L, float sm_scale, void *out, float *lse, void *workspace,
                                    size_t workspace_bytes, int32_t *device_status, void *stream);

/* The same for a layer whose tokens see a sliding window and a few first tokens
 * (sinks).  A token's entries, in order, are its sequence's cache entries
 * [0, seq_len[b]) and those of this pass that mask shows it (without a mask j <= t),
 * itself included; it sees the first `sinks` and the last `window` of them, and
 * nothing else is read into its result, whatever it holds.  There is no shared
 * prefix: the sinks lie in the sequence's own cache.  Of a long cache, only the
 * entries that some token sees are read, beside up to 127 behind each of the two
 * stretches.
 * Arguments, results, errors and roundings are spec_verify_attention's, with the
 * workspace of spec_attention_workspace_bytes(B, T, Hq, Hkv, D, 0, L); weights of
 * cache entries that not all of a sequence's tokens see are not rounded, nor those
 * of sinks ahead of entries that no or not every token sees, where sinks x
 * min(T x Hq / Hkv, 256) <= 640.  Limits: window >= 1, sinks >= 0.  Two launches, one
 * more with a mask (without a cache: one).  Asynchronous on `stream`.
 * Made for the passes of a verification, a chain or a tree.  A longer one, a part of
 * a prompt, is taken too, but slowly: what only some tokens' windows reach, and the
 * pass's own entries, are added row by row, T x min(T, window) of them to a head
 * (one sequence, 32/8 heads of 128, windows of 4096 over 8192 entries: 61 tokens 61
 * us, 128 113 us, 512 363 us, 2048 3.9 ms, under a mask 4.3 ms).              */
spec_status_t spec_verify_window_attention(const void *q, const void *cache, const uint8_t *cache_scale, int quant,
                                           const int32_t *seq_len, const void *staged, const uint8_t *mask, int window,
                                           int sinks, int B, int T, int Hq, int Hkv, int D, int L, float sm_scale,
                                           void *out, float *lse, void *workspace, size_t workspace_bytes,
                                           int32_t *device_status, void *stream);

/* Greedy tree verification (aiengineeringfromscratch.com Phase 10 lesson 25,
 * § Tree attention verification: one target pass over a draft tree under a
 * mask where each token sees only its ancestors; the output is the longest
 * accepted prefix along any path; § Greedy case: a draft is accepted when it
 * is the target's argmax).  The stochastic multi-branch rule is not on the
 * pages and is not offered.
 *   target_logits  [B][N][V]  dtype `tdt`; row n: the target's prediction after
 *                             node n's token
 *   tree_tokens    [B][N]     int32: node n's drafted token (node 0, the root,
 *                             is the last accepted token and is not read)
 *   parent         [B][N]     int32: parent[0] == -1, parent[n] in [0, n)
 *   out_tokens     [B][N]     int32: the accepted path's drafts, then the
 *                             argmax of its last node's row; -1 after
 *   out_nodes      [B][N]     int32: the path's node indices (root excluded); -1 after
 *   out_accept_len [B]        int32: accepted drafts (the path's depth), or
 *                             -code on a data error in an examined place:
 *                             1 malformed parent array, 2 NaN / +inf / all -inf
 *                             row of an accepted node, 3 token outside [0, V)
 *                             at a child of an accepted node
 * A child is accepted iff its parent is accepted and its token equals the
 * first index of the maximum of the parent's row.  The path ends at the
 * deepest accepted node, the lowest node index among equally deep ones.
 *   workspace      device scratch of spec_tree_workspace_bytes(B, N, V) bytes
 *                  (no zero-fill needed), 16-byte aligned
 *   device_status  [1] set to 0, or the code of one failing sequence; may be NULL
 * Limits: B, N, V >= 1, N <= 2048, B * N <= 2^30, V <= 2093056.  Two launches,
 * asynchronous on `stream`.                                                   */
size_t spec_tree_workspace_bytes(int B, int N, int V);
spec_status_t spec_verify_tree_greedy(const void *target_logits, spec_dtype_t tdt, const int32_t *tree_tokens,
                                      const int32_t *parent, int B, int N, int V, int32_t *out_tokens,
                                      int32_t *out_nodes, int32_t *out_accept_len, void *workspace,
                                      size_t workspace_bytes, int32_t *device_status, void *stream);

/* Tree attention mask (the same section): mask[b][i][j] = 1 iff node j is
 * node i or one of its ancestors, else 0; uint8 [B][N][N], device pointers.
 * A malformed parent array sets *device_status to 1 (it is set to 0 first;
 * may be NULL) and leaves that row's walk cut short.  One launch.            */
spec_status_t spec_tree_mask(const int32_t *parent, int B, int N, uint8_t *mask, int32_t *device_status,
                             void *stream);

/* Philox4x32-10 words as the verification kernels draw them, for checking:
 * out[(b * P + pos) * 4 + w] = word w of Philox(counter (pos, b, tag, 0),
 * key (seed low, seed high)) for b < B, pos < P.  `out` is a device pointer of
 * B * P * 4 uint32 entries.                                                   */
spec_status_t spec_philox_words(uint64_t seed, uint32_t tag, int B, int P, uint32_t *out,
                                void *stream);

/* Number of kernels this library has launched in this process, over every
 * entry point and device: a successful spec_verify* call launches one kernel,
 * or two to four when the row-parallel kernels serve it (large stochastic
 * batches: two from 1024 rows with aligned rows, where the residual pass runs
 * inside the statistics stream); spec_draft_sample and spec_philox_words
 * launch one each, spec_kv_commit two (one in place), spec_kv_commit_quant two,
 * spec_kv_read_quant one, spec_verify_attention one to four, spec_filter_sample
 * one, spec_verify_filtered two, spec_verify_window_attention one to three.  For
 * accounting;
 * thread-safe.                                                               */
uint64_t spec_launch_count(void);

/* A static description of a status code. */
const char *spec_status_string(spec_status_t status);

#ifdef __cplusplus
}
#endif
#endif /* SPECVERIFY_H */
