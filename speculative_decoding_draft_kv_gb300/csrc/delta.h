// Internal declarations shared by the gated delta rule's CUDA translation units.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "dflash_delta.h"

namespace dflash {

struct DeltaArgs {
    const uint16_t *q, *k, *v;
    uint16_t *o;
    int64_t q_rs, q_hs, k_rs, k_hs, v_rs, v_hs, o_rs, o_hs;
    const float *g, *beta;
    int64_t g_rs, beta_rs;
    float *state;
    int64_t slot_stride, head_stride;
    const int *q_start, *slot_in, *slot_out, *save;
    uint32_t *err;
    int64_t n_rows;
    float scale, eps;
    int n_seq, max_q, n_slots, n_head, n_head_k, group;   // group: heads of a key head
    int normalise;
    int split;                           // sequences of up to kDeltaFew tokens (and unprepared ones) are one kernel's, longer ones the other's
    // chunks of many tokens: what k_delta_prep leaves for k_delta_scan
    uint8_t *tiles;                      // [chunks][n_head_k][K, Q] F16 tiles of 32 rows
    uint8_t *heads;                      // [chunks][n_head] blocks of kDeltaHeadBytes
};

constexpr int kDeltaChunk = 32;          // tokens
constexpr int kDeltaHeadBytes = 2 * 6 * 32 * 16 + 2 * 16 * 16 + 32 * 4 + 16;
// Chunks, with room for each sequence's ragged last one: sequence s has those from q_start[s] / 32 + s on.
inline int64_t delta_chunks(int64_t n_rows, int n_seq) { return n_rows / kDeltaChunk + n_seq; }

// A batch of up to kDeltaTokens tokens a sequence goes token by token: above it chunks are faster (32 sequences of 32
// heads of 128 x 128, us: 9 tokens each 57 by tokens and 68 by chunks, 12 tokens 68 and 66, 16 tokens 85 and 67; heads
// of 64 x 64: 21 and 29, 23 and 29, 29 and 29).  In a batch with longer ones, whose chunks are to be prepared and
// walked anyway, only up to kDeltaFew do (32 sequences of 1 to 16 tokens, us: 58 with 8, 60 with 10 and with 12).
constexpr int kDeltaTokens = 12;
constexpr int kDeltaFew = 8;
constexpr float kDeltaLeast = -1e4f;     // log decays below it count as it: exp() of both is 0

// A sequence's rows and the slot that it begins from, as far as the arrays can be believed.
struct DeltaSeq {
    int row0, n, slot;                   // slot negative: zeros
    bool ok;
};
__device__ __forceinline__ DeltaSeq delta_seq(const DeltaArgs &a, int s, uint32_t &bits) {
    DeltaSeq q;
    const int64_t r0 = a.q_start[s], r1 = a.q_start[s + 1];
    q.slot = a.slot_in[s];
    const bool rows = r0 >= 0 && r0 <= r1 && r1 <= a.n_rows && r1 - r0 <= a.max_q, slot = q.slot < a.n_slots;
    bits = (rows ? 0u : (uint32_t)DELTA_ERR_BATCH) | (slot ? 0u : (uint32_t)DELTA_ERR_SLOT);
    q.ok = rows && slot;
    q.row0 = rows ? (int)r0 : 0;
    q.n = rows ? (int)(r1 - r0) : 0;
    return q;
}

// Where a sequence's chunks begin among all (see delta_chunks).
__device__ __forceinline__ int delta_base(int row0, int s) { return row0 / kDeltaChunk + s; }

// The sequence that chunks at .. to are prepared for: the last one whose chunks begin at them or in front of them, as long as bounds
// do not decrease; -1 where at and to find different ones.  Whole warps, a lane looking at every 32nd part of what is left.
__device__ __forceinline__ int delta_owner(const DeltaArgs &a, int at, int to) {
    const int lane = threadIdx.x & 31;
    int seq = 0;
    for (int left = a.n_seq; left > 1;) {
        const int part = (left + 31) >> 5, from = lane * part;
        const int begin = lane == 0 ? INT32_MIN : from < left ? delta_base(a.q_start[seq + from], seq + from) : INT32_MAX;
        const int last = 31 - __clz((int)__ballot_sync(0xffffffffu, begin <= at));
        if (to != at && __any_sync(0xffffffffu, lane > last && begin <= to)) return -1;
        seq += last * part;
        left = min(part, left - last * part);
    }
    return seq;
}

// Whether sequence s, in order and of some tokens, has its chunks prepared.  Where bounds decrease (which is reported), the search may
// find another sequence in its place for some of them: then it goes token by token.  (Found for its first chunk and for its
// last one, it is found for all between: a lane's answer only ever turns to yes as `at` grows.)
__device__ __forceinline__ bool delta_prepared(const DeltaArgs &a, int s, const DeltaSeq &q) {
    const int base = delta_base(q.row0, s);
    return delta_owner(a, base, base + (q.n - 1) / kDeltaChunk) == s;
}

cudaError_t delta_chunk_setup();
// The kernels of a long batch, each beside the end of the one in front: prep, k_delta_step (split), scan.
cudaError_t launch_delta_prep(const DeltaArgs &a, int dtype, int dim_k, cudaStream_t st);
cudaError_t launch_delta_scan(const DeltaArgs &a, int dtype, int dim_k, int dim_v, int sms, cudaStream_t st);
cudaError_t launch_delta_step(const DeltaArgs &a, int dtype, int dim_k, int dim_v, cudaStream_t st);

}  // namespace dflash
