/*
 * pa_q8.h -- C ABI of a step with drafted tokens: new rows of q, K and V
 * normalised, rotated and appended to the paged cache, a paged cache held in 8
 * bits with the attention of one or several query tokens per sequence over it,
 * and the verification of drafted tokens.  Part of libpa_gb300.so; status
 * values, dtypes, device error bits and the rules on ownership, streams and
 * `device_error` are those of pa.h and pa_q4.h.
 *
 * ---- The 8-bit cache --------------------------------------------------------
 *   k_cache   e4m3 codes [num_pages, Hkv, 16, D]   (v_cache the same; pa_decode's
 *             layout with one byte an element)
 *   k_scales  fp32 [num_pages, Hkv]                (v_scales the same)
 * A code c of KV head h in page p stands for k_scales[p][h] * c.  e4m3 is the
 * 8-bit float with 4 exponent and 3 mantissa bits, largest value 448, NaN 0x7F and
 * 0xFF, no infinities (torch.float8_e4m3fn).  pa_q8_decode takes any
 * positive scales up to 2^126 with which V's values are finite in fp32; those that
 * pa_q8_append makes are powers of two, so that a scale costs no precision and raising it
 * later is a shift of the exponent.
 */
#ifndef PA_GB300_Q8_H
#define PA_GB300_Q8_H

#include "pa_q4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* One more bit of the device error word. */
#define PA_DEVERR_BAD_TOKEN 32u   /* a drafted token outside the vocabulary, a number of
                                     drafts out of bounds, or a row of probabilities
                                     without any weight (pa_verify_drafts) */

/*
 * New rows of q, K and V on their way into a step: heads of q and k normalised
 * and rotated in one pass, q written to q_out, k and v into the paged cache of
 * pa_decode by slot.  For a row x of a head (D elements):
 *     y = x * w / sqrt(mean(x^2) + eps)      with a norm weight w, else y = x
 *     dims i and i + R/2, i < R/2, R = rotary_dim, turned by
 *         positions[t] * theta^(-2 i / R)    (dims R .. D - 1 as they are)
 * v is copied.  All of it is fp32 (angles, from frequencies of 64 bits, with cosines and
 * sines within 2^-23.6), rounded once.
 *   q, k, v      T [num_tokens, Hq or Hkv, D], T = fp16, bf16 or fp32; consecutive
 *                tokens *_stride elements apart (columns of a fused projection's
 *                rows), 16-byte aligned, strides multiples of 16 bytes
 *   q_norm, k_norm  T [D], 16-byte aligned, or NULL: not normalised
 *   theta        > 0, or 0: not rotated (rotary_dim and positions are not used)
 *   positions    int32 [num_tokens], any value
 *   slots        int64 [num_tokens]: page * 16 + position in the page, -1 for a row
 *                of which only q is wanted.  A slot outside [-1, num_pages * 16) is
 *                left out too and reported as PA_DEVERR_BAD_SLOT.  Slots must be
 *                distinct: of two rows with one slot either may be kept, even in part
 *   q_out        T [num_tokens, Hq, D] with a stride of its own; may equal q with the
 *                same stride, must not overlap anything else
 *   k_cache, v_cache  T [num_pages, Hkv, 16, D], 16-byte aligned
 * num_q_heads may be 0 (then q, q_norm and q_out are not used), num_tokens too.
 * head_dim 64, 96, 128 or 256; rotary_dim a multiple of 16, at most head_dim.
 */
int pa_append(int num_tokens, int num_q_heads, int num_kv_heads, int head_dim, int rotary_dim,
              int page_size, int num_pages, int dtype, float theta, float eps, const void* q,
              long long q_stride, const void* k, long long k_stride, const void* v,
              long long v_stride, const void* q_norm, const void* k_norm,
              const int32_t* positions, const int64_t* slots, void* q_out,
              long long q_out_stride, void* k_cache, void* v_cache, uint32_t* device_error,
              void* stream);

/*
 * pa_append into an 8-bit cache.  With a the largest magnitude of the elements
 * of the page's rows so far (K and V apart, after norm and rotation, in fp32),
 * the scale of a (page, KV head) is
 *     the least 2^e, e >= -120, with a <= 448 * 2^e
 * and an element's code is e4m3(x / scale), to nearest even.  Infinities and NaN
 * get the code NaN and do not count for the scale.  Rows come in order: a call's
 * rows of one page are next to one another among its rows, at ascending positions
 * without gaps.  If the first of them is at position 0 the page begins anew;
 * otherwise the rows before it are kept, the scale is the larger of what was
 * there and what the new rows need, and if it rises the kept rows' codes are
 * rounded to it (exactly, but for values below 2^-6 of the new scale).  What lies
 * in the page behind the call's rows (drafts that were not accepted, say) is not
 * kept up when the scale rises.  Of two runs of rows in one page of one call
 * either may be kept, even in part.
 */
int pa_q8_append(int num_tokens, int num_q_heads, int num_kv_heads, int head_dim, int rotary_dim,
                 int page_size, int num_pages, int dtype, float theta, float eps, const void* q,
                 long long q_stride, const void* k, long long k_stride, const void* v,
                 long long v_stride, const void* q_norm, const void* k_norm,
                 const int32_t* positions, const int64_t* slots, void* q_out,
                 long long q_out_stride, void* k_cache, void* v_cache, float* k_scales,
                 float* v_scales, uint32_t* device_error, void* stream);

/*
 * Rows of K and V that an 8-bit cache stands for, by slot: scale * code in fp32,
 * rounded to T.  A row whose slot is -1 is filled with zeros, one with a bad slot
 * with NaN (PA_DEVERR_BAD_SLOT).  Slots may repeat.  k, v, strides as k and v of
 * pa_append; k and v must not overlap.
 */
int pa_q8_read(int num_tokens, int num_kv_heads, int head_dim, int page_size, int num_pages,
               int dtype, const void* k_cache, const void* v_cache, const float* k_scales,
               const float* v_scales, const int64_t* slots, void* k, long long k_stride, void* v,
               long long v_stride, uint32_t* device_error, void* stream);

typedef struct pa_q8_plan {
    int batch;              /* B, at most 4096 */
    int num_q_heads;        /* Hq */
    int num_kv_heads;       /* Hkv */
    int head_dim;           /* D */
    int page_size;          /* 16 */
    int num_pages;          /* pages in the cache */
    int max_pages_per_seq;  /* row length of block_tables */
    int max_context_len;    /* upper bound on every context_lens[b]; at most 2^31 - 16 */
    int window;             /* sliding window in tokens, 0 = whole context */
    int max_query_len;      /* query tokens of a sequence, at most (1 to 16) */
    int dtype;              /* PA_DTYPE_F16 or PA_DTYPE_BF16: q and out */
    int num_sms;            /* SM count the plan was made for */
    int heads_per_cta;      /* query heads one CTA serves: a divisor of Hq / Hkv */
    int ctas_per_group;     /* CTAs that share the batch's pages of one KV head and head
                               chunk; without clusters a caller may lower it (to 1 or
                               more) */
    int ctas;               /* CTAs in all */
    int ctrl_bytes;         /* leading workspace bytes that must be zero before the first
                               call (error word, counters); every call leaves the
                               counters zero */
    size_t workspace_bytes; /* device workspace of pa_q8_decode */
    int test_stall_bytes;   /* test hook, 0 in normal use (at most 4096): each warp's
                               first copy expects this many bytes more than it carries,
                               so the bounded wait on it runs out after 1 s
                               (PA_DEVERR_TIMEOUT, NaN rows) */
    int cluster;            /* 2 to 8: so many CTAs share each sequence as a thread-block
                               cluster and merge in it (ctas_per_group is batch times
                               that); 0: the batch's pages are cut into ranges of about
                               equal work.  A caller may set 0 */
} pa_q8_plan_t;

/*
 * Plan decode calls over an 8-bit cache (host only, no device access unless
 * num_sms == 0, which queries the current device).  The query heads of a KV head
 * go in the fewest equal chunks of G heads with G * max_query_len <= 32 (16 at
 * head_dim 256), each of which reads the cache once.
 */
int pa_q8_plan(int batch, int num_q_heads, int num_kv_heads, int head_dim, int page_size,
               int num_pages, int max_pages_per_seq, int max_context_len, int window,
               int max_query_len, int num_sms, int dtype, pa_q8_plan_t* plan);

/*
 * Attention of one or several query tokens per sequence over an 8-bit cache.
 * Sequence b's query tokens are rows starts[b] .. starts[b + 1] - 1 of q, its
 * last T_b tokens: with L = context_lens[b] (they are counted in it and lie in
 * the cache), query t attends to tokens 0 .. L - T_b + t, of these to the last
 * `window` where there is one.
 *   q, out       T [num_rows, Hq, D], lse fp32 [num_rows, Hq], T = fp16 or bf16,
 *                16-byte aligned (lse 4-byte)
 *   starts       int32 [B + 1], ascending, 0 <= T_b <= max_query_len (as
 *                pa_extend_tables makes them); NULL: one query token per sequence,
 *                row b (num_rows is at least B then)
 * Rows that no sequence has are left as they were.  A query that attends to
 * nothing (its sequence is shorter than its query tokens) gives out = 0, lse =
 * -inf.  Cells of tokens that a query does not attend to do not change its row,
 * whatever they hold.  A bad page id, length or start gives NaN rows and a bit of
 * the workspace's error word, as in pa_decode (PA_DEVERR_BAD_LENGTH for starts more
 * than max_query_len apart too, and for starts that do not ascend or lie outside
 * [0, num_rows], where it is not known which rows the sequence has: none is written).
 * Precision: the codes of K and V and q are exact in the products (bf16 rows of q are
 * scaled by a power of two; elements below 2^-28 of their row's largest are rounded, by at
 * most 2^-39 of it), scores, maxima and sums fp32.  Scores are these products times one
 * fp32 factor, the call's scale times log2(e), K's scale and q's power of two: a factor
 * that overflows makes its rows NaN, a score that does to -inf weighs nothing.  In the
 * product with V a weight, times its page's V scale relative to the greatest met, is two
 * fp16 numbers, a head and a rest (22 bits; what is below 2^-33 of the row's greatest
 * weight is nothing); products are summed in fp32 and normalised by the fp32 sum of the
 * weights, which lse has too.
 * workspace as for pa_q4_decode.
 */
int pa_q8_decode(const pa_q8_plan_t* plan, int num_rows, const void* q, const int32_t* starts,
                 const void* k_cache, const void* v_cache, const float* k_scales,
                 const float* v_scales, const int32_t* block_tables,
                 const int32_t* context_lens, float scale, int window, void* out, float* lse,
                 void* workspace, void* stream);

/*
 * Verification of drafted tokens.  Sequence b has n = num_drafts[b] drafts x_0 ..
 * x_(n-1); p_t and q_t are the target's and the draft's probabilities at draft t,
 * p_n the target's behind the last.  Drafts are accepted while
 *     accept_u[b][t] * q_t(x_t) < p_t(x_t)
 * up to the first that is not, j (n if all are); then one token is drawn from the
 * weights
 *     w(y) = max(p_j(y) - q_j(y), 0)  for j < n,   p_n(y)  for j = n
 * as the least y whose cumulated weight exceeds sample_u[b] times the total.  With
 * random numbers from [0, 1) tokens then have the target's distribution, whatever
 * the draft's is (and the number of drafts may be 0: a plain draw).
 *   target_probs  T [B, max_drafts + 1, V], draft_probs T [B, max_drafts, V], T =
 *                 fp16, bf16 or fp32, rows one after the other.  draft_probs NULL:
 *                 each draft was certain, q_t(x_t) = 1 and 0 for other tokens
 *   draft_tokens  int32 [B, max_drafts];  num_drafts int32 [B], NULL: max_drafts each
 *   accept_u      fp32 [B, max_drafts];   sample_u fp32 [B]
 *   accepted      int32 [B]: j
 *   tokens        int32 [B, max_drafts + 1]: the accepted drafts, the drawn token, -1
 * Exactly: probabilities are limited to [0, 1], NaN counts as 0; the test takes the
 * products in 64 bits; w is p - q in fp32, counted in whole units of 2^-44 (to
 * nearest), so that sums do not depend on their order; the drawn token is the least
 * y with sum_(i <= y) w_i > floor(sample_u * total), sample_u limited to [0, 1),
 * the product in 64-bit floating point.  If no weight is left at j < n, the draw is
 * from p_j; if there is none either, the token is -1 (PA_DEVERR_BAD_TOKEN).  A
 * draft outside [0, V) is not accepted (PA_DEVERR_BAD_TOKEN); a number of drafts is
 * limited to [0, max_drafts] (PA_DEVERR_BAD_TOKEN).
 * max_drafts 0 to 32, V 1 to 524288.
 * (A loop with pa_extend_tables: its next call counts pages by the tokens that are kept,
 * so the caller gives back those that only drafts that were not accepted had begun, entries
 * ceil(kept / 16) .. ceil(context_len / 16) - 1 of a sequence's row.)
 */
#define PA_VERIFY_MAX_DRAFTS 32
int pa_verify_drafts(int batch, int max_drafts, int vocab, int dtype, const void* target_probs,
                     const void* draft_probs, const int32_t* draft_tokens,
                     const int32_t* num_drafts, const float* accept_u, const float* sample_u,
                     int32_t* accepted, int32_t* tokens, uint32_t* device_error, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PA_GB300_Q8_H */
