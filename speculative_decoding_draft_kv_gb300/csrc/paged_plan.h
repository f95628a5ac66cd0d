// How the attention kernels of a paged cache share out their work, and how a CTA finds its
// share.
//
// An item is (sequence, row tile, kv head): a run of query rows -- the tokens of the sequence
// times the query heads of one kv head, token by token -- and the key tiles that some row of
// it sees.  All key tiles of all items, laid end to end (sequence, head, row tile, key tile), are
// cut into equal shares, one per CTA; an item counts for item_cost tiles more than it has, which is
// what its beginning and end were measured to take.  So ragged lengths, a few long sequences among many
// short ones, and causal row tiles of uneven length all load the CTAs alike, with a grid that
// depends on nothing but bounds known to the host.  An item inside one share is finished by
// its CTA; an item cut by a share's border leaves one partial softmax state in each CTA that
// has a piece of it, and the combine kernel joins them.
//
// (What it is worth in either kernel: see plan_of.)
//
// A share is one run of tiles, so a CTA holds at most two such pieces: the end (or middle) of
// an item begun earlier, slot 0, and the beginning of one that goes on, slot 1.
#pragma once

#include "paged.h"
#include "paged_ptx.h"

namespace dflash {

// 64-bit numbers here are nearly always small ones, and a 64-bit division is a long way
__device__ __forceinline__ int64_t small_div(int64_t a, int64_t b) {
    return (a | b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// sum over i < n of floor((a i + b) / m), 0 <= a, b < 2^31, 0 < m, n a' < 2^32 for a' = a mod m (n is a
// number of row tiles, m of keys in a tile): whole parts of a / m and b / m first, then the lattice
// points under the line counted along the other axis
__device__ __forceinline__ int64_t floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b) {
    int64_t sum = 0;
    while (true) {
        if (a >= m) {
            sum += (int64_t)n * (n - 1) / 2 * (a / m);
            a %= m;
        }
        if (b >= m) {
            sum += (int64_t)n * (b / m);
            b %= m;
        }
        const uint64_t y = (uint64_t)a * n + b;
        if (y < m) return sum;
        n = (uint32_t)small_div((int64_t)y, m);
        b = (uint32_t)(y - (uint64_t)n * m);
        const uint32_t t = m;
        m = a;
        a = t;
    }
}

// Row tiles and key ranges of one sequence: a.tile_tokens tokens a row tile, KT keys a key tile.
template <int KT>
struct PagedShape {
    PagedSeq q;
    int ctx;

    // a sequence whose lengths contradict each other has no tiles: its rows stay as they are
    __device__ __forceinline__ void load(const PagedAttendArgs &a, int s) {
        q = paged_seq(a.batch, a.pool.page_shift, s, a.level == kPrefix);
        q.ok = q.ok && q.n <= a.max_q;
        if (!q.ok) q.n = 0;
        ctx = q.kv - q.n;
    }
    __device__ __forceinline__ int row_tiles(const PagedAttendArgs &a) const {
        return (q.n + a.tile_tokens - 1) / a.tile_tokens;
    }
    // positions that some row of the tile sees lie in [lo, hi); 0 <= lo < hi (a prefix may be empty)
    __device__ __forceinline__ int lo(const PagedAttendArgs &a, int rt) const {
        if (a.window == 0) return 0;
        return max(0, a.mask == PAGED_CAUSAL ? ctx + rt * a.tile_tokens - a.window + 1 : ctx - a.window);
    }
    __device__ __forceinline__ int hi(const PagedAttendArgs &a, int rt) const {
        return a.mask == PAGED_CAUSAL ? min(q.kv, ctx + (rt + 1) * a.tile_tokens) : q.kv;
    }
    __device__ __forceinline__ int tile0(const PagedAttendArgs &a, int rt) const { return lo(a, rt) / KT; }
    __device__ __forceinline__ int tiles(const PagedAttendArgs &a, int rt) const {
        return (hi(a, rt) + KT - 1) / KT - lo(a, rt) / KT;
    }
    // units of work: an item's key tiles and what starting and ending it costs, in tiles
    __device__ __forceinline__ int units(const PagedAttendArgs &a, int rt) const { return tiles(a, rt) + a.item_cost; }
    __device__ __forceinline__ int64_t head_units(const PagedAttendArgs &a) const {
        const int n = row_tiles(a);
        if (n == 0) return 0;
        if (n == 1 || a.mask != PAGED_CAUSAL) return (int64_t)n * units(a, 0);
        return head_tiles(a, n) + (int64_t)n * a.item_cost;
    }
    __device__ __forceinline__ int64_t head_tiles(const PagedAttendArgs &a, int n) const {
        // ceil(hi / KT) of all row tiles but the last, whose hi is kv ...
        int64_t w = floor_sum(n - 1, KT, a.tile_tokens, ctx + a.tile_tokens + KT - 1) + (q.kv + KT - 1) / KT;
        // ... less floor(lo / KT) of those whose lo is above 0
        if (a.window) {
            const int first = ctx - a.window + 1;
            const int i0 = first >= 0 ? 0 : (-first + a.tile_tokens - 1) / a.tile_tokens;
            if (i0 < n) w -= floor_sum(n - i0, KT, a.tile_tokens, first + i0 * a.tile_tokens);
        }
        return w;
    }
};

struct PagedShare {
    int64_t rem;                     // the CTA's first unit, counted from sequence seq's first
    int units, per;                  // this CTA's units, and those of a full share
    int seq;
    PagedSeq q;                      // of sequence seq
};

// Block-wide: every thread calls it, every thread gets the CTA's share.  scratch: shared
// memory of THREADS / 32 + 4 int64.
template <int KT, int THREADS>
__device__ __forceinline__ PagedShare paged_share(const PagedAttendArgs &a, int64_t *scratch) {
    constexpr int WARPS = THREADS / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (a.batch.n_seq <= 32) {
        // every warp for itself, a sequence to a lane; the barrier is for the caller's sake
        PagedShape<KT> sh;
        sh.q = PagedSeq{0, 0, 0, true};
        int64_t mine = 0;
        if (lane < a.batch.n_seq) {
            sh.load(a, lane);
            mine = sh.head_units(a) * a.pool.n_head_kv;
            if (!sh.q.ok && blockIdx.x == 0 && warp == 0) atomicOr(a.err, (uint32_t)PAGED_ERR_PAGE);
        }
        if (a.level != kOnly && blockIdx.x == 0 && warp == 0) {
            const bool broken = __any_sync(0xffffffffu, !sh.q.ok);
            if (lane == 0) *a.level_broken = broken;
        }
        int64_t incl = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += v;
        }
        const int64_t total = __shfl_sync(0xffffffffu, incl, 31);
        const int64_t per = max((int64_t)a.min_tiles, small_div(total + a.ctas - 1, a.ctas));
        const int64_t begin = min(total, (int64_t)blockIdx.x * per), end = min(total, begin + per);
        const uint32_t beyond = __ballot_sync(0xffffffffu, begin < incl);
        PagedShare r;
        r.seq = beyond ? __ffs(beyond) - 1 : 0;
        r.rem = begin - __shfl_sync(0xffffffffu, incl - mine, r.seq);
        r.units = beyond ? (int)(end - begin) : 0;
        r.per = (int)per;
        r.q.row0 = __shfl_sync(0xffffffffu, sh.q.row0, r.seq);
        r.q.n = __shfl_sync(0xffffffffu, sh.q.n, r.seq);
        r.q.kv = __shfl_sync(0xffffffffu, sh.q.kv, r.seq);
        r.q.ok = true;
        __syncthreads();
        return r;
    }
    const int per_thread = (a.batch.n_seq + THREADS - 1) / THREADS;
    const int s0 = min(a.batch.n_seq, tid * per_thread), s1 = min(a.batch.n_seq, s0 + per_thread);
    PagedShape<KT> sh;
    int64_t sum = 0;
    bool ok = true;
    for (int s = s0; s < s1; ++s) {
        sh.load(a, s);
        ok = ok && sh.q.ok;
        sum += sh.head_units(a) * a.pool.n_head_kv;
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
    if (a.level != kOnly) {
        const int broken = __syncthreads_or(!ok);
        if (blockIdx.x == 0 && tid == 0) *a.level_broken = broken;
    } else {
        __syncthreads();
    }
    int64_t base = 0, total = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        if (w == warp) base = total;
        total += scratch[w];
    }
    const int64_t mine = base + incl - sum;       // units in front of this thread's sequences
    // a share of 2^31 tiles would take hours: 32 bits are enough for one
    const int64_t per = max((int64_t)a.min_tiles, small_div(total + a.ctas - 1, a.ctas));
    const int64_t begin = min(total, (int64_t)blockIdx.x * per), end = min(total, begin + per);
    if (begin < end && mine <= begin && begin < mine + sum) {
        int64_t at = mine;
        for (int s = s0; s < s1; ++s) {
            sh.load(a, s);
            const int64_t w = sh.head_units(a) * a.pool.n_head_kv;
            if (begin < at + w) {
                scratch[WARPS] = begin - at;
                scratch[WARPS + 1] = s;
                scratch[WARPS + 2] = (int64_t)sh.q.n << 32 | (uint32_t)sh.q.row0;
                scratch[WARPS + 3] = sh.q.kv;
                break;
            }
            at += w;
        }
    }
    __syncthreads();
    PagedShare r;
    r.rem = scratch[WARPS];
    r.seq = (int)scratch[WARPS + 1];
    r.units = r.seq < 0 ? 0 : (int)(end - begin);
    r.per = (int)per;
    r.q.row0 = (int)scratch[WARPS + 2];
    r.q.n = (int)(scratch[WARPS + 2] >> 32);
    r.q.kv = (int)scratch[WARPS + 3];
    r.q.ok = true;
    return r;
}

// Walks a share item by item.  Every warp role runs its own copy over the same share; init takes
// whole warps.
template <int KT>
struct PagedWalk {
    PagedShape<KT> sh;
    int left, per;                   // units to come, units of a full share
    int seq, head, rt, off;          // the item, and the unit of it that comes next
    // the piece at hand
    int t0, nt, rest;                // first key tile (absolute), their number; units beyond them
    bool first, last;                // the piece has the item's first / last tile

    __device__ __forceinline__ void init(const PagedAttendArgs &a, const PagedShare &r) {
        left = r.units;
        per = r.per;
        seq = r.seq;
        head = rt = off = 0;
        if (left == 0) return;
        sh.q = r.q;
        sh.ctx = r.q.kv - r.q.n;
        const int64_t per_head = sh.head_units(a);
        int64_t rem = r.rem;
        head = (int)small_div(rem, per_head);
        rem -= head * per_head;
        if (per_head == sh.units(a, 0)) {            // one row tile
            off = (int)rem;
            return;
        }
        // the row tile that holds unit rem of the head, 32 row tiles at a time
        const int lane = threadIdx.x & 31, n = sh.row_tiles(a);
        while (true) {
            const int mine = rt + lane < n ? sh.units(a, rt + lane) : 0;
            int64_t incl = mine;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int64_t v = __shfl_up_sync(0xffffffffu, incl, d);
                if (lane >= d) incl += v;
            }
            const uint32_t beyond = __ballot_sync(0xffffffffu, rem < incl);
            if (beyond) {
                const int at = __ffs(beyond) - 1;
                off = (int)(rem - __shfl_sync(0xffffffffu, incl - mine, at));
                rt += at;
                return;
            }
            rem -= __shfl_sync(0xffffffffu, incl, 31);
            rt += 32;
            if (rt >= n) {                           // not reached: rem < per_head
                left = 0;
                return;
            }
        }
    }
    __device__ __forceinline__ bool next(const PagedAttendArgs &a) {
        while (left > 0) {
            if (off < 0) {                           // the item before this one is done
                off = 0;
                if (++rt >= sh.row_tiles(a)) {
                    rt = 0;
                    if (++head >= a.pool.n_head_kv) {
                        head = 0;
                        do {
                            if (++seq >= a.batch.n_seq) return false;
                            sh.load(a, seq);
                        } while (sh.q.n == 0);
                    }
                }
            }
            // the item's first item_cost units stand for no tile
            const int units = sh.units(a, rt), n = min(units - off, left);
            const int from = max(0, off - a.item_cost), to = max(0, off + n - a.item_cost);
            t0 = sh.tile0(a, rt) + from;
            nt = to - from;
            first = from == 0;
            rest = units - off - n;
            last = rest == 0;
            left -= n;
            off = last ? -1 : off + n;
            if (nt > 0) return true;
        }
        return false;
    }
    // an item's first piece of one of two passes: where the join finds its states
    __device__ __forceinline__ void note(const PagedAttendArgs &a) const {
        a.level_items[(int64_t)(sh.q.row0 + rt * a.tile_tokens) * a.pool.n_head_kv + head] =
            make_int2((int)blockIdx.x, last ? -1 : last_cta());
    }
    // the CTA that has the item's last tile (a piece that leaves some ends its CTA's share)
    __device__ __forceinline__ int last_cta() const { return (int)blockIdx.x + (rest + per - 1) / per; }
};

}  // namespace dflash
