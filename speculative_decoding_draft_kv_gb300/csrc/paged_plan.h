// How the attention kernels of a paged cache share out their work, and how a CTA finds its
// share.
//
// An item is (sequence, row tile, kv head): a run of query rows -- the tokens of the sequence
// times the query heads of one kv head, token by token -- and the key tiles that some row of
// it sees.  All key tiles of all items, laid end to end (sequence, head, row tile, key tile),
// are cut into equal shares, one per CTA.  So ragged lengths, a few long sequences among many
// short ones, and causal row tiles of uneven length all load the CTAs alike, with a grid that
// depends on nothing but bounds known to the host.  An item inside one share is finished by
// its CTA; an item cut by a share's border leaves one partial softmax state in each CTA that
// has a piece of it, and the combine kernel joins them.
//
// A share is one run of tiles, so a CTA holds at most two such pieces: the end (or middle) of
// an item begun earlier, slot 0, and the beginning of one that goes on, slot 1.
#pragma once

#include "paged.h"
#include "paged_ptx.h"

namespace dflash {

// Row tiles and key ranges of one sequence; TR query rows a row tile, KT keys a key tile.
template <int KT>
struct PagedShape {
    PagedSeq q;
    int group, tile_rows, mask, window, ctx, heads;

    __device__ __forceinline__ void load(const PagedAttendArgs &a, int s, int rows_per_tile) {
        q = paged_seq(a.batch, a.pool.page_shift, s);
        group = a.group;
        tile_rows = rows_per_tile;
        mask = a.mask;
        window = a.window;
        ctx = q.kv - q.n;
        heads = a.pool.n_head_kv;
    }
    __device__ __forceinline__ int row_tiles() const { return (q.n * group + tile_rows - 1) / tile_rows; }
    __device__ __forceinline__ int first_token(int rt) const { return rt * tile_rows / group; }
    __device__ __forceinline__ int last_token(int rt) const {
        return min(q.n - 1, (rt * tile_rows + tile_rows - 1) / group);
    }
    // positions that some row of the tile sees lie in [lo, hi)
    __device__ __forceinline__ int lo(int rt) const {
        if (window == 0) return 0;
        return max(0, mask == PAGED_CAUSAL ? ctx + first_token(rt) - window + 1 : ctx - window);
    }
    __device__ __forceinline__ int hi(int rt) const {
        return mask == PAGED_CAUSAL ? max(0, min(q.kv, ctx + last_token(rt) + 1)) : q.kv;
    }
    // every row tile has a key tile at least, so that rows seeing nothing get their zeros
    __device__ __forceinline__ int tile0(int rt) const { return lo(rt) / KT; }
    __device__ __forceinline__ int tiles(int rt) const {
        const int t0 = tile0(rt), t1 = (hi(rt) + KT - 1) / KT;
        return max(1, t1 - t0);
    }
    __device__ __forceinline__ int64_t head_tiles() const {
        int64_t w = 0;
        const int n = row_tiles();
        for (int rt = 0; rt < n; ++rt) w += tiles(rt);
        return w;
    }
};

struct PagedShare {
    int64_t begin, end, seq_begin;   // this CTA's tiles, and the first tile of sequence seq
    int64_t per;                     // tiles per CTA
    int seq;
};

// Block-wide: every thread calls it, every thread gets the CTA's share.  scratch: shared
// memory of 40 int64.
template <int KT, int THREADS>
__device__ __forceinline__ PagedShare paged_share(const PagedAttendArgs &a, int tile_rows, int64_t *scratch) {
    constexpr int WARPS = THREADS / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per_thread = (a.batch.n_seq + THREADS - 1) / THREADS;
    const int s0 = min(a.batch.n_seq, tid * per_thread), s1 = min(a.batch.n_seq, s0 + per_thread);
    PagedShape<KT> sh;
    int64_t sum = 0;
    bool ok = true;
    for (int s = s0; s < s1; ++s) {
        sh.load(a, s, tile_rows);
        ok = ok && sh.q.ok;
        sum += sh.head_tiles() * sh.heads;
    }
    if (!ok && blockIdx.x == 0) atomicOr(a.err, (uint32_t)PAGED_ERR_PAGE);
    int64_t incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += v;
    }
    if (lane == 31) scratch[warp] = incl;
    if (tid == 0) scratch[WARPS + 1] = -1;
    __syncthreads();
    int64_t base = 0, total = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        if (w == warp) base = total;
        total += scratch[w];
    }
    const int64_t mine = base + incl - sum;       // tiles in front of this thread's sequences
    PagedShare r;
    r.per = max((int64_t)a.min_tiles, (total + a.ctas - 1) / a.ctas);
    r.begin = min(total, (int64_t)blockIdx.x * r.per);
    r.end = min(total, r.begin + r.per);
    if (r.begin < r.end && mine <= r.begin && r.begin < mine + sum) {
        int64_t at = mine;
        for (int s = s0; s < s1; ++s) {
            sh.load(a, s, tile_rows);
            const int64_t w = sh.head_tiles() * sh.heads;
            if (r.begin < at + w) {
                scratch[WARPS] = at;
                scratch[WARPS + 1] = s;
                break;
            }
            at += w;
        }
    }
    __syncthreads();
    r.seq_begin = scratch[WARPS];
    r.seq = (int)scratch[WARPS + 1];
    if (r.seq < 0) r.end = r.begin;
    return r;
}

// Walks a share item by item.  Every warp role runs its own copy over the same share.
template <int KT>
struct PagedWalk {
    PagedShape<KT> sh;
    int64_t cur, end, per;
    int seq, head, rt, off;          // the item, and the tile of it that comes next
    // the piece at hand
    int t0, nt, item_tiles;          // first key tile (absolute), their number; the item's
    bool first, last;                // the piece has the item's first / last tile

    __device__ __forceinline__ void init(const PagedAttendArgs &a, const PagedShare &r, int tile_rows) {
        cur = r.begin;
        end = r.end;
        per = r.per;
        seq = r.seq;
        head = rt = off = 0;
        if (cur >= end) return;
        sh.load(a, seq, tile_rows);
        const int64_t per_head = sh.head_tiles();
        int64_t rem = cur - r.seq_begin;
        head = (int)(rem / per_head);
        rem -= head * per_head;
        while (rem >= sh.tiles(rt)) {
            rem -= sh.tiles(rt);
            ++rt;
        }
        off = (int)rem;
    }
    __device__ __forceinline__ bool next(const PagedAttendArgs &a, int tile_rows) {
        if (cur >= end) return false;
        if (off < 0) {                               // the item before this one is done
            off = 0;
            if (++rt >= sh.row_tiles()) {
                rt = 0;
                if (++head >= sh.heads) {
                    head = 0;
                    do {
                        if (++seq >= a.batch.n_seq) return false;
                        sh.load(a, seq, tile_rows);
                    } while (sh.q.n == 0);
                }
            }
        }
        item_tiles = sh.tiles(rt);
        t0 = sh.tile0(rt) + off;
        nt = (int)min((int64_t)(item_tiles - off), end - cur);
        first = off == 0;
        last = off + nt == item_tiles;
        cur += nt;
        off = last ? -1 : off + nt;
        return true;
    }
    // the CTA that has the item's last tile, for the piece at hand (off already advanced)
    __device__ __forceinline__ int last_cta() const {
        return last ? (int)blockIdx.x : (int)((cur + (item_tiles - off) - 1) / per);
    }
};

}  // namespace dflash
