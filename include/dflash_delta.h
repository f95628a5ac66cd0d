/*
 * dflash_delta.h -- C ABI of the gated delta rule for one GB300 GPU (sm_103a).
 *
 * Models that verify drafted blocks mix attention over a paged cache (dflash_paged.h) with
 * recurrent layers, whose context is one matrix per head instead of rows per token.  The
 * operator here runs such a layer's recurrence for a ragged batch: a token each, drafted blocks
 * whose state can be taken back, whole prompts.
 *
 * Conventions (as in dflash_paged.h where not said otherwise)
 *   - Every function returns RING_OK or a negative RING_E* code and never aborts;
 *     delta_last_error() has the calling thread's last message.
 *   - Nothing is allocated and nothing is kept between calls: every buffer is the caller's, on
 *     the current device, and stays alive until the work queued on `stream` is done.  Calls
 *     only enqueue work; they may be captured into a CUDA graph, whose replays read the then
 *     current contents of the device arrays.  Calls on different streams are independent of each
 *     other as long as they write different memory (the workspace included: one per call that
 *     may run at the same time).
 *   - Host checks see shapes, strides, alignment and pointers.  What the device arrays hold
 *     (row bounds, slot numbers) is checked by the kernels: nothing out of range is followed, and
 *     a bit is set in the device error word (delta_device_error).
 *   - An empty batch is nothing to do, its pointers are not looked at.
 */
#ifndef DFLASH_DELTA_H
#define DFLASH_DELTA_H

#include "dflash_paged.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bits of the device error word. */
enum {
    DELTA_ERR_BATCH = 1, /* row bounds that decrease, pass the rows, or hold more than max_q */
    DELTA_ERR_SLOT = 2,  /* a slot number past the pool                                       */
    DELTA_ERR_WAIT = 4   /* a wait inside a kernel ran out (2 s); the call's output is not valid */
};

/*
 * A pool of states: slot i, head h is float32 [dim_v][dim_k] at
 * data + i * slot_stride + h * head_stride (in floats, positive multiples of 4; data 16-byte
 * aligned), its rows contiguous.  Row j holds the state's weights of value element j over the
 * key's elements.
 *   dim_k, dim_v   64 or 128 each.
 */
typedef struct delta_state {
    float *data;
    int64_t slot_stride, head_stride;
    int32_t n_slots, n_head, dim_k, dim_v;
} delta_state;

/*
 * A ragged batch: rows q_start[s] .. q_start[s+1]-1 of the rows tensors are sequence s's new
 * tokens, in order.
 *   q_start   device int32 [n_seq + 1], not decreasing.  Rows from q_start[n_seq] on (a padded
 *             batch) are not written, and what they hold changes nothing.
 *   slot_in   device int32 [n_seq]: the slot that holds the state in front of the first token;
 *             negative: zeros.  Sequences may read one slot (branches of one prompt).
 *   slot_out  device int32 [n_seq]: the slot that gets the state behind the last token;
 *             negative: it is not kept.  It may be slot_in[s].  A sequence without new tokens
 *             has its state copied.
 *   save      NULL, or device int32 [n_rows]: the slot that gets the state behind that row's
 *             token, negative: none.  (A drafted block whose tail is rejected goes on from the
 *             state behind its last accepted token.)  A call with it goes token by token, whatever the lengths and even
 *             where no state is kept (32 heads of 128 x 128, 16,381 tokens: 12.5 ms, 0.76 without): prompts
 *             want a call of their own.
 *   max_q     upper bound of the sequences' new tokens, now and at every replay of a captured
 *             call.  How the work is shared out goes by it: far above the lengths it costs speed.
 * Sequences that have rows in common (bounds that decrease between them, which is reported) may end
 * with anything.
 * A slot that one sequence writes may be read by that sequence, as its slot_in, and by no
 * other of the call; a slot that is written twice holds either state, or rows of both.
 */
typedef struct delta_batch {
    const int32_t *q_start, *slot_in, *slot_out, *save;
    int32_t n_seq, max_q;
} delta_batch;

/*
 * delta_rule -- for each sequence and head h (key head h / (n_head / n_head_k)), token by token:
 *     S <- exp(g) S
 *     u  = beta (v - S k)
 *     S <- S + u k^T
 *     o  = scale S q
 *   q, k     rows [n_rows][n_head_k][dim_k], PAGED_F16 or PAGED_BF16; with `normalise` both
 *            are divided by sqrt(sum of squares + eps) first.
 *   v, o     rows [n_rows][n_head][dim_v] of the same type.  o may not overlap the inputs.
 *   g, beta  device float32 [n_rows][n_head] with row strides in floats (heads contiguous).  g
 *            is a log decay, up to 0 in use; below -1e4 it counts as -1e4 (the state is gone
 *            either way).
 *   scale    0: 1 / sqrt(dim_k).
 *   n_head   of the state pool; a multiple of n_head_k.
 *   workspace   device memory of delta_rule_workspace() bytes, 256-byte aligned (NULL where
 *               that is 0); its contents before and after the call mean nothing.
 * States, sums and norms are float32.  A batch with max_q up to 12, or with `save`, goes token by token in float32.  In others
 * sequences of more than 8 tokens go 32 tokens at a time through the tensor cores, whose operands are F16:
 *   - keys and queries one each, after a power of two by their norm: exact but for elements below 2^-14 of it, off by up to 2^-25;
 *     one whose square sum is 0 in float32 counts as zero;
 *   - states, updates u and what weighs tokens against one another two each, 22 bits together, in units that go by the value
 *     element, whatever its neighbours hold.  One unit serves its 32 updates beta (v - S k): those 2^10 and more below the largest
 *     lose bits, which end at 2^-30 of that;
 *   - for BF16 outputs the state's first part alone in S q, 11 bits: beside its own rounding an output is off by up to
 *     2^-11 exp(G) |S| |q| then, S the value element's weights in front of the 32 tokens, G the log decays since.
 * Keys that are not normalised want beta |k|^2 of at most 2, as the recurrence itself does: beyond, it grows with every token.
 * An infinity or NaN in a token's rows reaches the token's value elements (in v) or all of its head (in the
 * others) from there on, and in a batch with max_q above 12 the same elements of up to 31 in front of it, as
 * NaN: what is a number there is right.
 * A sequence whose row bounds contradict each other (DELTA_ERR_BATCH), or whose slot_in is past the pool
 * (DELTA_ERR_SLOT), is left alone: its rows of o and its slots stay as they were.  A slot past
 * the pool in slot_out or save is not written (DELTA_ERR_SLOT).
 * Errors: EINVAL, ECUDA.
 */
typedef struct delta_rule_args {
    const delta_state *state;
    const delta_batch *batch;
    const void *q, *k, *v;
    void *o;
    int64_t q_row_stride, q_head_stride, k_row_stride, k_head_stride;
    int64_t v_row_stride, v_head_stride, o_row_stride, o_head_stride;
    const float *g, *beta;
    int64_t g_row_stride, beta_row_stride;
    void *workspace;
    int64_t workspace_bytes, n_rows;
    float scale, eps;
    int32_t n_head_k, dtype, normalise, reserved;
} delta_rule_args;
int delta_rule(const delta_rule_args *args, void *stream);

/* Bytes of workspace that delta_rule needs for this pool, batch and number of rows and key
 * heads, whatever its other arguments and the contents of the device arrays (0: none). */
int delta_rule_workspace(const delta_state *state, const delta_batch *batch, int64_t n_rows, int32_t n_head_k,
                         int64_t *bytes);

/* delta_device_error -- synchronise, read and clear the current device's error word of this
 * operator.  RING_OK, or RING_EDEVICE with the bits in *bits (may be NULL). */
int delta_device_error(uint32_t *bits);

/* Message of the calling thread's last failing call.  Never NULL. */
const char *delta_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* DFLASH_DELTA_H */
