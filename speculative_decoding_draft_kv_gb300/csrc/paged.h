// Internal declarations shared by the paged-cache operators' CUDA translation units.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "dflash_paged.h"

namespace dflash {

constexpr int kPagedMaxDim = 128;
constexpr int kPagedMaxGroup = 64;     // query heads per kv head

// One layer's pools; strides of codes and 16-bit values in elements, of scales in floats.
struct PagedPool {
    uint8_t *k, *v;
    float *ks, *vs;
    int64_t page_stride, head_stride, row_stride, s_page_stride, s_head_stride;
    int n_pages, page_shift, n_head_kv, format;
};

struct PagedBatchDev {
    const int *q_start, *kv_len, *pages;
    int64_t pages_stride, n_rows;
    int n_seq, max_pages;
};

// A sequence's new rows and lengths, as far as the arrays can be believed: rows within
// [0, n_rows), a length within the block table.  ok is false where they were not.  prefix: the length does
// not count the rows, which all come behind it.
struct PagedSeq {
    int row0, n, kv;
    bool ok;
};

__device__ __forceinline__ PagedSeq paged_seq(const PagedBatchDev &b, int page_shift, int s, bool prefix = false) {
    PagedSeq q;
    const int64_t r0 = b.q_start[s], r1 = b.q_start[s + 1];
    const int64_t kv = b.kv_len[s], cap = (int64_t)b.max_pages << page_shift;
    const int64_t lo = r0 < 0 ? 0 : (r0 > b.n_rows ? b.n_rows : r0);
    const int64_t hi = r1 < lo ? lo : (r1 > b.n_rows ? b.n_rows : r1);
    q.row0 = (int)lo;
    q.n = (int)(hi - lo);
    q.kv = (int)(kv < 0 ? 0 : (kv > cap ? cap : kv));
    q.ok = lo == r0 && hi == r1 && q.kv == kv && (prefix || q.n == 0 || kv >= q.n);
    return q;
}

// ---- launchers ----
struct PagedRowsArgs {
    const void *q, *k, *v;            // inputs (NULL: none of that kind)
    void *qo, *ko, *vo;               // rows outputs; ko, vo NULL: into the pages
    int64_t q_rs, q_hs, k_rs, k_hs, v_rs, v_hs, qo_rs, qo_hs, ko_rs, ko_hs;
    const float *q_norm, *k_norm;
    const int *positions;
    PagedPool pool;
    PagedBatchDev batch;
    uint32_t *err;
    int64_t n_rows;
    float eps, magnitude;
    int nq, nk, nv;                   // heads of each kind
    int rot, layout;                  // rot 0: no rotation
    int steps_q, steps_k, steps_v;    // warp steps of a token's queries, keys, values (set at launch)
    int iters, tasks;                 // warp steps per task, tasks per token
    uint64_t turn[kPagedMaxDim / 2];  // turns per position, in 2^-64
};
cudaError_t launch_paged_rows(const PagedRowsArgs &a, int dtype, int head_dim, bool paged, cudaStream_t st);

struct PagedGatherArgs {
    void *k, *v;
    int64_t k_rs, k_hs, v_rs, v_hs;
    PagedPool pool;
    PagedBatchDev batch;
    uint32_t *err;
    int steps, iters, chunks;         // warp steps of a token's K (or V), steps per task, tasks per token
};
cudaError_t launch_paged_gather(const PagedGatherArgs &a, int dtype, int head_dim, cudaStream_t st);

// Attention: what every CTA needs to find its share of the work.
struct PagedAttendArgs {
    const uint16_t *q;
    uint16_t *o;
    float *lse;
    const int64_t *tree;
    int64_t q_rs, q_hs, o_rs, o_hs;
    PagedPool pool;
    PagedBatchDev batch;
    uint32_t *err;
    float *part_acc;                  // [ctas][2][rows][head_dim] numerators
    float2 *part_ml;                  // [ctas][2][rows] (max in log2 units, sum)
    int4 *desc;                       // [ctas] the item whose first part is the CTA's last one
    int n_head, group, mask, window, max_q;
    int ctas, min_tiles, item_cost;   // fewest units of a share; units of an item beyond its tiles
    int tile_tokens, tile_rows;       // tokens and rows (tokens times group, at most) of an item
    float scale_log2;
    // A batch whose sequences share beginnings is attended to in two passes, all rows of a prefix over its
    // positions (kPrefix, the mask a full one) and each sequence over its own (kOwn), which k_paged_levels joins.
    // A pass writes down where an item's states are, and those of items that are not cut beside the cut ones'.
    int level;
    float *level_acc;                 // [n_rows][n_head][head_dim] numerators
    float2 *level_ml;                 // [n_rows][n_head] (max in log2 units, sum)
    int2 *level_items;                // [n_rows][kv heads] of an item's first row: the CTAs with its first and last
                                      // tile; .y negative: not cut, its states are in the arrays above
    int *level_broken;                // 1 where some sequence (or prefix) contradicts itself, else 0
    const PagedAttendArgs *first;     // kOwn, on the host: the first pass's, whose join goes behind this one
    int sms;
};
enum { kOnly = 0, kPrefix = 1, kOwn = 2 };

template <int T> cudaError_t paged_attend_setup_t();
template <int T>
cudaError_t launch_paged_attend_t(const PagedAttendArgs &a, const CUtensorMap &tm_k, const CUtensorMap &tm_v,
                                  int head_dim, cudaStream_t st);

template <int T> cudaError_t paged_prefill_setup_t();
template <int T>
cudaError_t launch_paged_prefill_t(const PagedAttendArgs &a, const CUtensorMap &tm_k, const CUtensorMap &tm_v,
                                   const CUtensorMap &tm_q, int head_dim, cudaStream_t st);

}  // namespace dflash
