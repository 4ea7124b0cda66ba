/*
 * pa_q4.h -- C ABI of the operators around a decode step: a paged KV cache
 * held in 4 bits with the attention that reads it, the block tables and slots
 * of a step, and rotary positions with several axes.  Part of
 * libpa_gb300.so; status values, dtypes, device error bits and the rules on
 * ownership and streams are those of pa.h: every pointer is caller-owned
 * device memory, no call allocates, calls are asynchronous on the given
 * stream, arguments are checked on the host before anything is launched, and
 * values found bad on the device are never read or written through.
 *
 * Where a call takes `device_error` it is the address of a 32-bit word (or
 * NULL) in which the kernel sets PA_DEVERR_* bits; the word accumulates and
 * can be read with pa_get_error / pa_get_error_ex, so the head of a workspace
 * serves.
 *
 * ---- The 4-bit cache --------------------------------------------------------
 * A token's K (or V) row of one KV head, D elements of type T (fp16 or bf16),
 * is held as D 4-bit codes and, for every group of 32 consecutive dims, a
 * scale s and an offset z of type T.  Code c in 0..15 of a group stands for
 *     RN_T(s * (16 + c) + z)            (one rounding to nearest even)
 * and a row is quantised, with exact arithmetic before each rounding, as
 *     mn, mx = least and greatest element of the group, limited to
 *              [-M, M] with M = 16384 (fp16) or 2^120 (bf16)
 *     s = RN_T((mx - mn) / 15)
 *     z = RN_T(mn - 16 s)
 *     c = min(15, max(0, rint((x - z) / s - 16))), ties to even; 0 if s = 0
 * so that an element within the limits comes back within about half a step s,
 * and the value itself is rounded.  Rounding z and s moves the grid's ends,
 * where the group straddles zero and s is a normal number of T, by at most
 *     fp16: s / 64 at the low end, s / 43 at the high end
 *     bf16: s / 8 at the low end, s / 5 at the high end
 * (u = 2^-11 or 2^-8 being half a step of rounding: z, at most 31 s (1 + u / 2),
 * is off by u of that, and at the high end come 15 times s's own u s).
 * Elements beyond the limits, infinities among them, come back as the grid's
 * ends; a group that holds a NaN comes back as NaN.  The 16 in 16 + c is the
 * leading bit of a 16-bit float whose mantissa holds c, so the kernels make
 * the value with one multiply-add.
 *
 * cache: uint8 [num_pages, Hkv, 20 D], 16-byte aligned, pages of 16 tokens.
 * The block of one (page, KV head) holds, for token r (0..15) and dim d:
 *   K codes    at 0:    4 bits; byte (d / W) 8 W + r W/2 + (d % W) / 2 with
 *                       W = min(D, 128), even d in the low half
 *   V codes    at 8 D:  32-bit words, each two bytes of token 2j (its low 16
 *                       bits) and two of token 2j + 1, four dims of each,
 *                       lowest dim in the lowest bits.  The words lie as lane
 *                       l = 4 (column) + j % 4 of a warp reads them:
 *                       byte (j / 4) 4 D + (w / V) 128 V + 4 V l + 4 (w % V)
 *                       V = 4 (D 128, 256), 2 (D 64), 1 (D 96) words a read;
 *                       column and word w of dim d: d / (D / 8) and
 *                       (d % (D / 8)) / 4, for D 96 (d % 32) / 4 and d / 32
 *   K scales   at 16 D: T (s, z) pairs; with N = W / 32, group n:
 *                       4 (((n / N) 16 + r) N + n % N)
 *   V scales   at 18 D: T [8 token pairs][D / 32][s of 2j, s of 2j + 1,
 *                       z of 2j, z of 2j + 1]
 * Every token of a page owns whole bytes, so rows of one page may be written
 * by one call in any order.  The element type is not recorded: a cache is
 * read with the type that it was written with.
 *
 * Supported: head_dim 64, 96, 128, 256; page_size 16; fp16 and bf16.
 */
#ifndef PA_GB300_Q4_H
#define PA_GB300_Q4_H

#include "pa.h"

#ifdef __cplusplus
extern "C" {
#endif

/* More bits of the device error word. */
#define PA_DEVERR_BAD_SLOT 8u    /* a slot outside [-1, num_pages * page_size) */
#define PA_DEVERR_NO_PAGES 16u   /* the free list ran out (pa_extend_tables) */

/* Bytes of one (page, KV head) block of a 4-bit cache, 20 * head_dim; 0 for a
 * head_dim that is not supported. */
int pa_q4_page_bytes(int head_dim);

/*
 * Quantise num_tokens rows of K and V into the cache.
 *   k, v        T [num_tokens, Hkv, D]; consecutive tokens k_stride (v_stride)
 *               elements apart (at least Hkv * D, a multiple of 8), so that
 *               they may be columns of a fused projection's rows; 16-byte
 *               aligned
 *   slots       int64 [num_tokens]: page * 16 + position in the page, -1 for
 *               a row that is to be left out (a padded batch).  A slot outside
 *               [-1, num_pages * 16) is left out too and reported as
 *               PA_DEVERR_BAD_SLOT.  The rows' slots must be distinct: of two
 *               rows with one slot either may be kept, even in part
 * Only the rows' own codes and scales are written.  num_tokens may be 0.
 */
int pa_q4_write(int num_tokens, int num_kv_heads, int head_dim, int page_size, int num_pages,
                int dtype, const void* k, long long k_stride, const void* v, long long v_stride,
                const int64_t* slots, void* cache, uint32_t* device_error, void* stream);

/*
 * The reverse: rows of K and V that the cache stands for, by slot.  A row
 * whose slot is -1 is filled with zeros, one with a bad slot with NaN
 * (PA_DEVERR_BAD_SLOT).  Slots may repeat.  k, v, strides as in pa_q4_write;
 * k and v must not overlap.
 */
int pa_q4_read(int num_tokens, int num_kv_heads, int head_dim, int page_size, int num_pages,
               int dtype, const void* cache, const int64_t* slots, void* k, long long k_stride,
               void* v, long long v_stride, uint32_t* device_error, void* stream);

typedef struct pa_q4_plan {
    int batch;              /* B, at most 4096 */
    int num_q_heads;        /* Hq */
    int num_kv_heads;       /* Hkv */
    int head_dim;           /* D */
    int page_size;          /* 16 */
    int num_pages;          /* pages in the cache */
    int max_pages_per_seq;  /* row length of block_tables */
    int max_context_len;    /* upper bound on every context_lens[b]; at most 2^31 - 16 */
    int window;             /* sliding window in tokens, 0 = whole context */
    int dtype;              /* PA_DTYPE_F16 or PA_DTYPE_BF16: q, out, the cache's values */
    int num_sms;            /* SM count the plan was made for */
    int heads_per_cta;      /* query heads one CTA serves (a divisor of Hq / Hkv, at most 8) */
    int ctas_per_group;     /* CTAs that share the batch's pages of one KV head and head
                               chunk; without clusters a caller may lower it (to 1 or
                               more) */
    int ctas;               /* CTAs in all */
    size_t workspace_bytes; /* device workspace of pa_q4_decode */
    int ctrl_bytes;         /* its leading bytes that must be zero before the first call
                               (error word, counters); every call leaves the counters
                               zero */
    int test_stall_bytes;   /* test hook, 0 in normal use (at most 4096): each warp's
                               first copy expects this many bytes more than it carries,
                               so the bounded wait on it runs out after 1 s
                               (PA_DEVERR_TIMEOUT, NaN rows) */
    int cluster;            /* 2 to 8: so many CTAs share each sequence as a thread-block
                               cluster and merge in it (ctas_per_group is batch times
                               that); 0: the batch's pages are cut into ranges of about
                               equal work.  A caller may set 0 */
} pa_q4_plan_t;

/*
 * Plan decode calls over a 4-bit cache (host only, no device access unless
 * num_sms == 0, which queries the current device).  The arguments mean what
 * they mean to pa_plan_ex.  More than 8 query heads per KV head go in the fewest
 * equal chunks of at most 8, each of which reads the cache once: 9 as 3 x 3, 15
 * as 3 x 5, 16 as 2 x 8; a prime above 8 is PA_ERR_UNSUPPORTED.
 */
int pa_q4_plan(int batch, int num_q_heads, int num_kv_heads, int head_dim, int page_size,
               int num_pages, int max_pages_per_seq, int max_context_len, int window,
               int num_sms, int dtype, pa_q4_plan_t* plan);

/*
 * pa_decode over a 4-bit cache: the same result as pa_decode on a cache of
 * type T that holds the values the 4-bit cache stands for, with the same
 * arguments, windows, empty sequences (out = 0, lse = -inf), error word and
 * NaN rows for a bad page id or length.  Cells of tokens outside a sequence's
 * attended range are not used, whatever they hold.
 * Precision, as pa_decode's: scores, maxima, sums and the lse are fp32.  In the
 * product with V the weights are rounded, to fp16 (11 bits) for fp16 caches and
 * to two bf16, a head and a rest (16 bits), for bf16 ones, and normalised by the
 * sum of the rounded weights; the sums are fp32 and rounded to T once.  (fp16 rows
 * of normal values measured 2.4e-4 to 2.9e-4 of their norm off, of which 2e-4
 * are their own rounding.)
 * The work of the whole batch is shared out over the CTAs on the device, from
 * the actual lengths (see ctas_per_group and cluster).
 * workspace: plan->workspace_bytes, 16-byte aligned, the first plan->ctrl_bytes
 * zero before the first call; concurrent calls must not share one, and one that
 * served another plan must have its ctrl_bytes zeroed first.
 */
int pa_q4_decode(const pa_q4_plan_t* plan, const void* q, const void* cache,
                 const int32_t* block_tables, const int32_t* context_lens, float scale,
                 int window, void* out, float* lse, void* workspace, void* stream);

/*
 * The block tables, lengths and slots of a step, from the requests' lengths.
 * Request b holds past_lens[b] tokens and gets new_lens[b] more (0 or more).
 * With have = ceil(past / 16) and need = ceil((past + new) / 16), pages
 * have .. need - 1 of its row of block_tables are taken from free_pages in
 * order: first the pages of request 0, then those of request 1, and so on.
 *   past_lens, new_lens  int32 [batch]
 *   free_pages           int32 [num_free]
 *   block_tables         int32 [batch, max_pages_per_seq], updated in place
 *                        (only the entries of new pages are written)
 *   context_lens         int32 [batch]      past + new (not past_lens itself)
 *   starts               int32 [batch + 1]  exclusive sums of new_lens: request
 *                        b's new tokens are rows starts[b] .. starts[b + 1] - 1
 *                        of the step's packed tokens
 *   slots                int64 [token_capacity]  page * 16 + position in the page of
 *                        every new token, -1 behind the last
 *   positions            int32 [token_capacity]  position in its request, 0 behind the last
 *   pages_taken          int32 [1]  free pages used
 * Refused on the device, with a bit of *device_error: a request with a
 * negative length, past + new beyond the row, or tokens beyond token_capacity
 * (PA_DEVERR_BAD_LENGTH), and one that the free list no longer serves
 * (PA_DEVERR_NO_PAGES; later requests are served if they need no page).  A
 * refused request keeps its length and row, takes no page, and its tokens get
 * slot -1 (they keep their rows in the packed order; a negative new length
 * has none).  A page id outside [0, num_pages) in free_pages or in the row is
 * reported (PA_DEVERR_BAD_PAGE) and gives slot -1; one taken from free_pages
 * is written to the row as -1.
 * batch at most 8192, and may be 0; the outputs must not overlap the inputs.
 */
int pa_extend_tables(int batch, int max_pages_per_seq, int page_size, int num_pages,
                     int num_free, int token_capacity, const int32_t* past_lens,
                     const int32_t* new_lens, const int32_t* free_pages, int32_t* block_tables,
                     int32_t* context_lens, int32_t* starts, int64_t* slots, int32_t* positions,
                     int32_t* pages_taken, uint32_t* device_error, void* stream);

/*
 * Rotary embedding of q and k whose pairs take their position from one of
 * several axes (time, height and width of an image's or video's tokens).
 * The rotate-half pairing of pa_plan_t.rope_theta: dims i and i + R/2 for
 * i < R/2, R = rotary_dim, are turned by positions[a][t] * theta^(-2 i / R)
 * where a is pair i's axis; dims R .. D - 1 are copied.
 *   sections     int [num_axes] (host memory), pairs per axis, their sum R/2.
 *     interleaved 0: the first sections[0] pairs go by axis 0, the next by axis 1, ...
 *     interleaved 1: pair i goes by axis i % num_axes while that axis has pairs left
 *                    (i < num_axes * sections[i % num_axes]), else by axis 0
 *   inverse      1: turn by the negative angle (the gradient of the rotation, or
 *                keys turned back)
 *   q, k         T [num_tokens, Hq or Hkv, D], T = fp16, bf16 or fp32;
 *                consecutive tokens q_stride (k_stride) elements apart; 16-byte
 *                aligned, strides multiples of 16 bytes
 *   q_out, k_out the same, with strides of their own; may equal q and k
 *                (in place) with the same strides, must not overlap them otherwise,
 *                nor each other
 *   positions    int32 [num_axes, num_tokens], any value
 * num_q_heads or num_kv_heads may be 0 (then q or k is not used).
 * rotary_dim: a multiple of 16, at most head_dim (at most 256, a multiple of
 * 16).  Angles are reduced modulo one turn in 64-bit integers and rounded to
 * fp32 once; the rotation is fp32, rounded once to T.
 */
#define PA_ROPE_MAX_AXES 4
int pa_rope_axes(int num_tokens, int num_q_heads, int num_kv_heads, int head_dim, int rotary_dim,
                 int num_axes, const int* sections, int interleaved, int inverse, float theta,
                 int dtype, const void* q, long long q_stride, const void* k, long long k_stride,
                 const int32_t* positions, void* q_out, long long q_out_stride, void* k_out,
                 long long k_out_stride, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PA_GB300_Q4_H */
