/*
 * dflash_paged.h -- C ABI of the paged-cache operators for one GB300 GPU (sm_103a).
 *
 * The draft's ring (dflash_ring.h) holds a fixed window.  The model that verifies the
 * drafted block keeps its whole context, in pages that a block table strings together; the
 * operators here serve that side: turn a projection's heads into cache rows
 * (paged_norm_rope, paged_append), read rows back (paged_gather), and let new tokens attend
 * to the pages (paged_attend): a single token, a verify block, a token tree, a chunk of a
 * prompt, or all of them in one ragged batch.
 *
 * Conventions (as in dflash_ring.h where not said otherwise)
 *   - Every function returns RING_OK or a negative RING_E* code and never aborts;
 *     paged_last_error() has the calling thread's last message.
 *   - Nothing is allocated and nothing is kept between calls: every buffer is the caller's,
 *     on the current device, and stays alive until the work queued on `stream` is done.
 *     Calls only enqueue work; they may be captured into a CUDA graph, whose replays read
 *     the then current contents of the device arrays.  Calls on different streams are
 *     independent of each other as long as they write different memory (the workspace of
 *     paged_attend included: one per call that may run at the same time).
 *   - Host checks see shapes, strides, alignment and pointers.  What the device arrays hold
 *     (lengths, page numbers) is checked by the kernels: nothing out of range is followed.
 *     Rows that such an entry names are not written, or read as zeros, and a bit is set in
 *     the device error word (paged_device_error).
 *   - An empty batch or tensor is nothing to do, its pointers are not looked at.
 *   - "Rows" tensors are [n_rows][heads][head_dim] with the innermost index contiguous and
 *     positive row and head strides (in elements) that keep every head 16-byte aligned, so that
 *     queries, keys and values may be slices of one projection's output.
 */
#ifndef DFLASH_PAGED_H
#define DFLASH_PAGED_H

#include "dflash_ring.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of rows and of pages. */
enum {
    PAGED_F16 = 0,
    PAGED_BF16 = 1,
    PAGED_F32 = 2,   /* rows of paged_norm_rope only */
    PAGED_INT8 = 3,  /* pages only: code * scale, one F32 scale per token and kv head */
    PAGED_E4M3 = 4   /* pages only: likewise with 8-bit floats (4 exponent, 3 mantissa bits) */
};

/* Which cached positions a new token sees (see paged_attend). */
enum { PAGED_CAUSAL = 0, PAGED_FULL = 1, PAGED_TREE = 2 };

/* Which elements of a head form a rotated pair. */
enum {
    PAGED_HALF = 0,        /* (i, i + rotary_dim / 2)  */
    PAGED_INTERLEAVED = 1  /* (2 i, 2 i + 1)           */
};

/* Bits of the device error word. */
enum {
    PAGED_ERR_WAIT = 1, /* a wait inside a kernel ran out (2 s); the call's output is not valid */
    PAGED_ERR_PAGE = 2  /* a page number outside the pool, a position outside the block table,
                           or lengths that contradict each other                               */
};

/*
 * One layer's K and V pages.  Pools are [n_pages][n_head_kv][page_size][head_dim] in any
 * order of strides with the innermost index contiguous (pages of [page_size][n_head_kv]
 * rows, or K and V pages side by side in one pool, are strides too).
 *   format      PAGED_F16, PAGED_BF16, PAGED_INT8 or PAGED_E4M3.
 *   head_dim    64 or 128.
 *   page_size   16, 32, 64, 128 or 256 tokens.
 *   *_stride    elements; the same for k and v; multiples of 16 bytes.
 *   k_scale, v_scale   PAGED_INT8 and PAGED_E4M3: device F32 [n_pages][n_head_kv][page_size]
 *                      with the given page and head strides (floats, multiples of 4), rows
 *                      of a page contiguous; else NULL.  All bases 16-byte aligned.
 */
typedef struct paged_cache {
    void *k, *v;
    float *k_scale, *v_scale;
    int64_t page_stride, head_stride, row_stride;
    int64_t scale_page_stride, scale_head_stride;
    int32_t n_pages, page_size, n_head_kv, head_dim, format, reserved;
} paged_cache;

/*
 * A ragged batch of new tokens: rows q_start[s] .. q_start[s+1]-1 of the rows tensors are
 * sequence s's newest tokens, at positions kv_len[s] - n .. kv_len[s] - 1 (n of them; kv_len
 * counts them).  Position p lives in row p % page_size of page pages[s][p / page_size].
 *   q_start  device int32 [n_seq + 1], not decreasing (paged_attend reports one that is,
 *            PAGED_ERR_PAGE; paged_append and paged_gather look rows up as if it were not, and so may
 *            serve a row at another place of the block table, or not at all).  Rows from q_start[n_seq] on (a padded
 *            batch) are not written, and what they hold changes nothing (their memory may be read).
 *   kv_len   device int32 [n_seq].
 *   pages    device int32 [n_seq][pages_stride]; entries of pages that a call has no need of
 *            (past the end, or in front of a window) are not looked at.
 *   max_q    upper bound of n over the sequences: paged_attend chooses its kernel by it (and a
 *            sequence of more new tokens is left alone there, PAGED_ERR_PAGE); the other calls
 *            do not look at it.
 *   max_kv   upper bound of kv_len, at most max_pages * page_size (0: that product): bounds
 *            paged_attend's grid and workspace.
 */
typedef struct paged_batch {
    const int32_t *q_start, *kv_len, *pages;
    int64_t pages_stride;
    int32_t n_seq, max_pages, max_q, max_kv;
} paged_batch;

/*
 * Position rotation: a pair (x1, x2) at position p turns to
 *   magnitude * (x1 cos a - x2 sin a, x1 sin a + x2 cos a),  a = p * inv_freq[i],
 * for the rotary_dim / 2 pairs of a head's first rotary_dim elements; the others stay.
 *
 * paged_rope_init -- fill *rope.  inv_freq: host double [rotary_dim / 2], 0 <= f < 1e6 (scaled
 * frequencies are the caller's); rotary_dim: a multiple of 16 up to 128 (and up to head_dim where
 * it is used).  The struct holds frequencies as turns per position in units of 2^-64: a product
 * with a position loses its whole turns in 64-bit integers, so far positions keep their angle to
 * float32 precision.  No CUDA call.  Errors: EINVAL.
 */
typedef struct paged_rope {
    uint64_t turns[64];
    float magnitude;
    int32_t rotary_dim, layout, reserved;
} paged_rope;
int paged_rope_init(paged_rope *rope, const double *inv_freq, double magnitude, int32_t rotary_dim, int32_t layout);

/*
 * paged_norm_rope -- per head: y = x / sqrt(mean(x^2) + eps) * w (w = q_norm / k_norm, F32
 * [head_dim]; NULL: no norm), then the rotation at positions[row] (rope NULL: none), in
 * float32, rounded once to the rows' type.
 *   q, q_out   rows [n_rows][n_head_q][head_dim] (n_head_q = 0: none); q_out may be q with
 *              the same strides, and may not overlap it otherwise.
 *   k, k_out   likewise with n_head_k heads.
 *   dtype      PAGED_F16, PAGED_BF16 or PAGED_F32, of all four.  head_dim 64 or 128.
 *   positions  device int32 [n_rows] (NULL only without a rope).
 * Errors: EINVAL, ECUDA.
 */
typedef struct paged_norm_rope_args {
    const void *q, *k;
    void *q_out, *k_out;
    int64_t q_row_stride, q_head_stride, k_row_stride, k_head_stride;
    int64_t qo_row_stride, qo_head_stride, ko_row_stride, ko_head_stride;
    const float *q_norm, *k_norm;
    const int32_t *positions;
    const paged_rope *rope;
    int64_t n_rows;
    float eps;
    int32_t n_head_q, n_head_k, head_dim, dtype;
} paged_norm_rope_args;
int paged_norm_rope(const paged_norm_rope_args *args, void *stream);

/*
 * paged_append -- write the batch's K and V rows to their pages.
 *   k, v       rows [n_rows][n_head_kv][head_dim], PAGED_F16 or PAGED_BF16.
 *   k_norm, rope   K is normed and turned first, as in paged_norm_rope, at its position in
 *              the sequence, or at positions[row] where given (a token tree's depths).
 *   q, q_out   optional (n_head_q > 0): queries normed (q_norm) and turned in the same pass;
 *              q_out may be q with the same strides.
 * Quantised pages: per row, A = max|x| in float32, scale = A / 127 (int8) or A / 448 (e4m3),
 * codes = x * (127 / A) or x * (448 / A) rounded to nearest even; a row with A < 1e-30 gets
 * scale 0 and codes 0, a row with an infinity or NaN gets scale NaN and codes 0 and reads
 * back as NaN.  K is quantised from its float32 rotated value.
 * A row whose page number is outside the pool, or whose position is outside the block table,
 * is not written (PAGED_ERR_PAGE).  Two rows for one place (one page named twice): either.
 * Errors: EINVAL, ECUDA.
 */
typedef struct paged_append_args {
    const paged_cache *cache;
    const paged_batch *batch;
    const void *k, *v, *q;
    void *q_out;
    int64_t k_row_stride, k_head_stride, v_row_stride, v_head_stride;
    int64_t q_row_stride, q_head_stride, qo_row_stride, qo_head_stride;
    const float *k_norm, *q_norm;
    const int32_t *positions;
    const paged_rope *rope;
    int64_t n_rows;
    float eps;
    int32_t n_head_q, dtype;
} paged_append_args;
int paged_append(const paged_append_args *args, void *stream);

/*
 * paged_gather -- read the batch's K and V rows back from their pages into rows tensors
 * [n_rows][n_head_kv][head_dim] of type PAGED_F16 or PAGED_BF16 (codes times scale in
 * float32, rounded once).  A whole sequence is read by a batch whose rows are all of its
 * positions.  Unmapped rows read as zeros (PAGED_ERR_PAGE).  Errors: EINVAL, ECUDA.
 */
typedef struct paged_gather_args {
    const paged_cache *cache;
    const paged_batch *batch;
    void *k, *v;
    int64_t k_row_stride, k_head_stride, v_row_stride, v_head_stride;
    int64_t n_rows;
    int32_t dtype, reserved;
} paged_gather_args;
int paged_gather(const paged_gather_args *args, void *stream);

/*
 * paged_attend -- attention of the batch's new tokens over their sequences' pages (the new
 * tokens' own K and V rows included: append first).  Token i of sequence s, with context
 * c = kv_len[s] - n, sees position p < kv_len[s] if
 *   PAGED_CAUSAL  p <= c + i, and, with window > 0, p > c + i - window;
 *   PAGED_FULL    always (the new tokens see each other both ways), with window > 0 only
 *                 p >= c - window;
 *   PAGED_TREE    p < c (with window > 0: and p >= c - window), or bit p - c of tree[row]
 *                 is set (n <= 64).
 * Per query head h (kv head h / (n_head / n_head_kv)):
 *   o = sum_p softmax_p(q . k_p * scale) v_p;  a token that sees nothing gets 0.
 * Products on the tensor cores with float32 accumulation, softmax in float32;
 * probabilities round to the operand type.  Quantised pages: codes are exact F16 operands and K's
 * scales multiply the scores in float32; a probability times its V scale rounds to F16, off by 2^-11 of
 * itself or by 2^-15 of the row's largest such product, whichever is more (scales that the row does not
 * see, or gives no weight, take nothing from it, up to 2^100 above the others).  Scores (q . k * scale)
 * above some 10^7 are beyond float32's steps, and the output may be NaN there.
 * A sequence whose lengths contradict each other (more new tokens than kv_len or than max_q, a
 * length beyond the block table) is left alone: its rows of o and lse stay as they were.
 *   q, o     rows [n_rows][n_head][head_dim], PAGED_F16 or PAGED_BF16; pages of a 16-bit
 *            format have the same type.  n_head a multiple of n_head_kv, up to 64 query
 *            heads per kv head.  o may not overlap q.
 *   scale    0: 1 / sqrt(head_dim); at most 2e38.
 *   window   0: none; one past every position is none too.
 *   tree     PAGED_TREE: device int64 [n_rows], else NULL.
 *   lse      NULL, or device F32 [n_rows][n_head]: ln of the softmax's denominator (of
 *            exp(score)), -inf for a token that sees nothing.
 *   workspace   device memory of paged_attend_workspace() bytes, 256-byte aligned; its
 *            contents before and after the call mean nothing.
 * Positions that no token of the batch sees may hold anything, infinities and NaN included.
 * A V row that some token of a sequence sees reaches every query row that shares its tile if
 * it holds an infinity or NaN (0 * inf), also rows that do not see it.
 * Errors: EINVAL, ECUDA.
 */
typedef struct paged_attend_args {
    const paged_cache *cache;
    const paged_batch *batch;
    const void *q;
    void *o;
    int64_t q_row_stride, q_head_stride, o_row_stride, o_head_stride;
    const int64_t *tree;
    float *lse;
    void *workspace;
    int64_t workspace_bytes, n_rows;
    float scale;
    int32_t n_head, dtype, mask, window, reserved;
} paged_attend_args;
int paged_attend(const paged_attend_args *args, void *stream);

/* Bytes of workspace that paged_attend needs for this cache, batch and number of query
 * heads, whatever its other arguments and the contents of the device arrays. */
int paged_attend_workspace(const paged_cache *cache, const paged_batch *batch, int32_t n_head,
                           int64_t *bytes);

/*
 * paged_attend_shared -- paged_attend for a batch whose sequences share beginnings (samples of one
 * prompt, questions about one document, requests behind one system prompt).  A prefix's K and V
 * are read once for all its rows: a first pass attends to the prefixes, a second one to
 * the sequences' own pages and joins the two softmaxes, exactly as over one context.
 *   args->batch   as in paged_attend, of each sequence's own part: kv_len counts the positions
 *            behind its prefix, the new tokens included, and pages holds them from the first on (a part of
 *            a page that the prefix fills does not go on here: the own part begins in a page of its
 *            own).  mask, tree and c refer to own positions; every token sees its whole prefix.
 *   prefix   rows q_start[i] .. q_start[i+1]-1 (n_seq prefixes; bounds of rows, over any number of
 *            sequences) begin with the kv_len[i] >= 0 positions of pages[i].  max_q: upper bound of one
 *            prefix's rows; max_kv of their lengths.  Rows that no prefix has stand for themselves.
 *   window   0 (EINVAL otherwise).
 *   lse      of both parts.
 *   workspace   paged_attend_shared_workspace() bytes.
 * A prefix whose bounds contradict each other (see paged_attend; its length may be below its number of rows)
 * is left out, PAGED_ERR_PAGE: its rows get their own part alone.
 * Beside bounds that decrease, sequences and prefixes whose own ones are right are served all the same; two of
 * them that have rows in common may end with anything.
 * With paged_append and paged_norm_rope, positions[] counts the prefix.  Errors: EINVAL, ECUDA.
 */
int paged_attend_shared(const paged_attend_args *args, const paged_batch *prefix, void *stream);
int paged_attend_shared_workspace(const paged_cache *cache, const paged_batch *batch, const paged_batch *prefix,
                                  int64_t n_rows, int32_t n_head, int64_t *bytes);

/* paged_device_error -- synchronise, read and clear the current device's error word of these
 * operators.  RING_OK, or RING_EDEVICE with the bits in *bits (may be NULL). */
int paged_device_error(uint32_t *bits);

/* Message of the calling thread's last failing call.  Never NULL. */
const char *paged_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* DFLASH_PAGED_H */
