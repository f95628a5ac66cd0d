// Attention of new tokens over a paged cache: the kernel for many query rows per kv head (prompt
// chunks, large trees, mixed batches), on the 5th-generation tensor cores.
//
// With 128 query rows and more a cached byte takes part in 128 flops and up, and the pass is
// bound by the tensor cores, then by the exponentials beside them.  An item is up to 256 query
// rows -- two blocks of 128 TMEM lanes, a row being a (token, query head) of one kv head -- and
// its key tiles of 128.  Per tile and block, with all accumulators in tensor memory:
//   S = Q K^T   128 x 128 in TMEM, A and B from shared memory;
//   P = 2^(S scale - m) by the block's four softmax warps, a thread per row, written back over S
//               as 16-bit values;
//   O += P V    A = P from TMEM, B = V from shared memory as it lies (rows along the keys).
// The two blocks take turns: while the tensor cores work for one, the softmax warps of the other
// have the exponentials.  One thread issues, per tile, O0 += P0 V, S0 = Q0 K', O1 += P1 V,
// S1 = Q1 K': the tensor pipe runs them in that order, so S may overwrite the P that the product
// in front of it reads, and a block's S being there means its O is up to date.
//
// The softmax reference moves only when a row outgrows it by 2^8 (see paged_attend.cuh), so O is
// read back and rescaled in few tiles.
//
// An item of at most 128 rows (a verify block, a tree, a single token in a mixed batch) fills one
// block only: then both blocks take the same queries, block 0 the even key tiles and block 1 the
// odd ones, so that products and exponentials still take turns, and block 0 joins the two states at
// the end.  A batch with no larger item runs the variant with memory for one block of queries.
//
// Quantised pages: four more warps turn codes into F16 tiles in shared memory, exactly, a thread per key; K's
// scales are multiplied on the scores and V's on the probabilities, in float32, as the streaming kernel does,
// with units that the F16 products are in: common ones, then the rows' own (apart_tile).  Rows of code
// times scale rounded to F16 would spare the rows' threads three products a score (mixed batch below 202 us),
// but a row whose scale is 2^-14 of its tile's largest would lose bits, and with F16 outputs they doubled
// the error.  bf16 queries are turned to F16 in shared memory, a power of two per row taken out, by the
// threads that own the rows.
//
// Measured, 32 query and 8 kv heads: a chunk of 2,048 tokens at the end of 32,768, heads of 128, bf16:
// 792 us, 1.35 PFLOP/s, the tensor pipe active 62 % of the time (a block's chain S -> softmax -> P -> O
// is longer than the other block's products); 64 verify blocks of up to 9 tokens (36 rows, dealt) over
// 2.2 GB: 355 us, 6.2 TB/s, bound by memory; two prompts of 4,097 tokens, heads of 64: 214 us, bound by the
// same chain (P lies over S, so the next S waits for O += P V; the exponentials alone would be 55 us, the
// tensor pipe is active 31 % of the time); 16 trees of up to 31 nodes over int8: 123 us, and chunks of 1,024
// among single tokens, e4m3, window 2,048: 238 us, both chains of copy, conversion, S, softmax, P and O,
// where neither memory nor the tensor cores nor the issue slots are full.
// What the kernel's parts run at the same time has to fit the instruction cache: over quantised pages and one
// block the rows' loops are unrolled twice, not eight times (trees 162 -> 130 us), over 16-bit pages whole (two
// prompts: 214 us, 229 unrolled twice).  Two blocks over quantised pages lie between: F16 queries whole (a
// chunk of 619 tokens at 23,810 281 us, the second loop unrolled twice 297; the mixed batch 243 and 232), bf16
// ones with the second loop unrolled twice (mixed batch 237 us, whole 256; chunk 296 and 285).
// Tried and not faster: eight converting warps (640 threads), waits that sleep or poll otherwise; one pass
// over S with the reference moved where needed was slower (914 us for the chunk, where two passes took
// 793).
//
// Roles: warps 0-3 and 4-7 the blocks' rows, warps 8 and 10 copies (queries by one box of heads x
// tokens, K and V a box per page), warp 9 issues products, warps 12-15 convert codes.
#pragma once

#include "paged_attend.cuh"

namespace dflash {

constexpr int kPreTile = 128;
constexpr int kScaleRing = 8;            // key tiles whose scales or units are kept (see below)

template <int D, int FMT, int T, bool ONE>
struct PreCfg {
    static constexpr bool kCodes = FMT != kFmt16;
    static constexpr int kThreads = kCodes ? 512 : 352;
    // With scales on the scores and two blocks of rows, those are what holds the kernel: their 256 threads
    // take 168 registers, the others 88 (together the 65,536 of the launch, 512 times 128), and pieces of
    // 32 scores (a chunk of 619 tokens at 23,810, heads of 64, int8: 314 -> 257 us).  One block: no gain
    // (trees 130 -> 137 us).
    static constexpr bool kMore = kCodes && !ONE;
    static constexpr int kManyRegs = 168, kFewRegs = 88;
    static constexpr int kHalves = D / 64;                       // 128-byte columns of a 16-bit row
    static constexpr int kHalfBytes = kPreTile * 128;
    static constexpr int kSlotBytes = kHalves * kHalfBytes;      // 128 rows of D 16-bit values
    static constexpr int kBlocks = ONE ? 1 : 2;                  // of queries
    // K and V tiles in turn: what fits
    static constexpr int kSlots = kCodes ? (D == 128 && !ONE ? 3 : 4) : (D == 128 ? (ONE ? 6 : 5) : 10);
    static constexpr int kCodeBytes = kPreTile * D;
    static constexpr int kCodeSlots = kCodes ? 3 : 0;
    static constexpr int kOffQ = kSlots * kSlotBytes;
    static constexpr int kOffCodes = kOffQ + kBlocks * kSlotBytes;
    static constexpr int kOffCodeScale = kOffCodes + kCodeSlots * kCodeBytes;   // as loaded, per code slot
    static constexpr int kOffScale = kOffCodeScale + kCodeSlots * kPreTile * 4;  // [ring][K, V][128]
    static constexpr int kOffUnit = kOffScale + (kCodes ? kScaleRing * 2 * kPreTile * 4 : 0);   // [ring]
    // a dealt item's odd tiles: maxima and sums; its queries' powers of two (in a place of their own: block 0
    // writes those of the next item while its slower warps may still read the sums of this one)
    static constexpr int kOffOdd = kOffUnit + (kCodes ? kScaleRing * 4 : 0);
    static constexpr int kOffExp = kOffOdd + 128 * 8;
    static constexpr int kOffBars = kOffExp + (kCodes && T == PAGED_BF16 ? 128 : 0);
    static constexpr int kOffPlan = kOffBars + 304;                // what else is shared: the plan, then words
    static constexpr int kSmem = kOffPlan + 24 * 8 + 16;
    static_assert(kSmem <= 227 * 1024, "one CTA per SM");
};

// two float32 at a time
__device__ __forceinline__ uint64_t pk2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void upk2(uint64_t x, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// What a row sees: positions [lo, hi) and, for a tree, bits of its word from ctx on, below kv.
struct RowSight {
    int lo, hi, ctx, kv;
    bool tree;
    uint64_t word;

    // bit e: position p + e
    __device__ __forceinline__ uint32_t bits(int p) const {
        // positions below x of the 32 from p on
        auto below = [&](int x) { return x - p >= 32 ? ~0u : (x <= p ? 0u : (1u << (x - p)) - 1u); };
        uint32_t b = below(hi) & ~below(lo);
        if (tree) {
            const int at = p - ctx;                        // the word's bit that p is
            const uint32_t nodes = at >= 64 ? 0u : (at >= 0 ? (uint32_t)(word >> at) : (at > -32 ? (uint32_t)word << -at : 0u));
            b |= nodes & below(kv);
        }
        return b;
    }
};

// A row's numerators (dim columns from `to` on) times a factor.
__device__ __forceinline__ void scale_numerators(uint32_t to, int dim, float by) {
#pragma unroll 1
    for (int c = 0; c < dim; c += 16) {
        uint32_t u[16];
        tmem_ld16(to + c, u);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(__uint_as_float(u[e]) * by);
        tmem_st16(to + c, u);
    }
}

// A row's tile over quantised pages where the item's V scales are far apart: its scores (ts) to probabilities
// times V scales, as F16 values in a unit of the row's own.  The unit is at most the row's largest such
// product, and not below 2^-10 of that: what is lost below F16's smallest step is small beside what counts
// most, whatever scales the row does not see or gives no weight.  When the reference m moves the unit moves
// with it and O stays.  (m, l, vref) before and after; vref: the unit, with a minus sign.  Rare, and in a loop of
// its own, so that it takes no room between the loops that are not (there it cost two blocks 5 to 20 %).  Blocks
// of up to 9 tokens over int8, one V row in 5,000 of zeros: 793 us, 414 without; chunks 2.1 times as long.
__device__ __forceinline__ float3 apart_tile(uint32_t ts, uint32_t to, int dim, bool more, RowSight sight, int base, const float4 *ks4,
                                          float tscale, bool valid, float m, float l, float vref) {
    const float4 *vs4 = ks4 + kPreTile / 4;
    // fn(piece of 16, scores, masked by -inf, V scales)
    auto pieces = [&](auto &&fn) {
#pragma unroll 1
        for (int c = 0; c < kPreTile / 16; ++c) {
            uint32_t u[16];
            tmem_ld16(ts + 16 * c, u);
            tmem_ld_wait();
            const uint32_t bits = sight.bits(base + 16 * c);
            float x[16], v[16];
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
                const float4 k = ks4[4 * c + e / 4], w = vs4[4 * c + e / 4];
                x[e] = __uint_as_float(u[e]) * k.x;
                x[e + 1] = __uint_as_float(u[e + 1]) * k.y;
                x[e + 2] = __uint_as_float(u[e + 2]) * k.z;
                x[e + 3] = __uint_as_float(u[e + 3]) * k.w;
                v[e] = w.x; v[e + 1] = w.y; v[e + 2] = w.z; v[e + 3] = w.w;
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = bits & (1u << e) ? x[e] : -INFINITY;
            fn(c, x, v);
        }
    };
    float mx = -INFINITY;
    pieces([&](int, const float (&x)[16], const float (&)[16]) {
#pragma unroll
        for (int e = 0; e < 16; ++e) mx = fmaxf(mx, x[e]);
    });
    mx *= tscale;
    float unit = fabsf(vref);
    if (valid && mx > m + kLazyMove) {
        const float alpha = exp2f(m - mx);
        m = mx;
        l *= alpha;
        unit *= alpha;                                     // in place of O
    }
    const float mu = m == -INFINITY ? 0.f : m;
    float wt = 0.f;                                        // the tile's largest product (NaN is passed over)
    pieces([&](int, const float (&x)[16], const float (&v)[16]) {
#pragma unroll
        for (int e = 0; e < 16; ++e) wt = fmaxf(wt, fabsf(ex2_approx(fmaf(x[e], tscale, -mu)) * v[e]));
    });
    wt = fminf(wt, 0x1p126f);
    // A unit from before, common to the item's rows: no scale was below 2^-10 of it then, so the row's largest
    // product was not either, if it has seen any.
    const bool first = !signbit(vref);
    const float least = !first ? unit : (l > 0.f ? unit * 0x1p-10f : 0.f);
    float now = least;
    if (wt > 0.f && (first || wt > 1024.f * least || least < 0x1p-126f)) now = fmaxf(fmaxf(wt, least), 0x1p-126f);
    const float by = now > 0.f ? (first && !(l > 0.f) ? 0.f : unit / now) : 1.f;
    if (more && __any_sync(0xffffffffu, by != 1.f)) scale_numerators(to, dim, by);
    const float inv = now >= 0x1p-126f ? 1.f / now : 0.f;
    float sum = 0.f;
    pieces([&](int c, const float (&x)[16], const float (&v)[16]) {
        uint32_t u[8];
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
            const float p0 = ex2_approx(fmaf(x[e], tscale, -mu)), p1 = ex2_approx(fmaf(x[e + 1], tscale, -mu));
            sum += p0 + p1;
            u[e / 2] = pack_half2(p0 * v[e] * inv, p1 * v[e + 1] * inv);
        }
        tmem_st(ts + 8 * c, u);                            // over scores that have been read
    });
    return make_float3(m, l + sum, -now);
}

template <int D, int FMT, int T, bool ONE>
__global__ void __launch_bounds__(PreCfg<D, FMT, T, ONE>::kThreads, 1)
k_paged_prefill(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ PagedAttendArgs a) {
    using C = PreCfg<D, FMT, T, ONE>;
    constexpr int NS = C::kSlots;
    constexpr bool kCodes = C::kCodes;
    constexpr int OT = kCodes ? PAGED_F16 : T;                       // operand type
    constexpr bool kQTurned = kCodes && T == PAGED_BF16;
    constexpr uint32_t kIdescQK = tc_idesc(128, kPreTile, OT == PAGED_BF16, false);
    constexpr uint32_t kIdescPV = tc_idesc(128, D, OT == PAGED_BF16, true);
    constexpr int CODE_ROW = D < 128 ? D : 128;                      // bytes of a row of codes
    // no static shared memory beside this, so its start is the CTA's, aligned for any swizzle
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t bars = smem_u32(smem + C::kOffBars);
    const uint32_t full = bars, empty = bars + 8 * NS;               // [NS] each
    const uint32_t q_full = bars + 16 * NS, q_empty = q_full + 8, q_ready = q_full + 16;
    const uint32_t s_full = q_full + 24, p_full = s_full + 16, o_full = p_full + 16;   // [2] each
    const uint32_t landed = o_full + 16, drain = landed + 8, odd_done = landed + 16, odd_free = landed + 24;
    const uint32_t c_full = landed + 32, c_empty = c_full + 8 * C::kCodeSlots;
    int64_t *s_plan = reinterpret_cast<int64_t *>(smem + C::kOffPlan);
    uint32_t &s_tmem = *reinterpret_cast<uint32_t *>(smem + C::kOffPlan + 24 * 8);
    volatile int &s_abort = *reinterpret_cast<volatile int *>(smem + C::kOffPlan + 24 * 8 + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (smem_u32(smem) & 1023u) {                          // never: tiles would be read in another order
        if (threadIdx.x == 0) {
            atomicOr(a.err, (uint32_t)PAGED_ERR_WAIT);
            a.desc[blockIdx.x] = make_int4(-1, 0, 0, 0);
        }
        return;
    }

    if (threadIdx.x == 0) {
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
        prefetch_tensormap(&tm_q);
        for (int k = 0; k < NS; ++k) {
            mbar_init(full + 8 * k, kCodes ? 4 : 1);     // the converting warps, or the copy
            mbar_init(empty + 8 * k, 1);
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, 9);                           // the products, and the rows' eight warps
        mbar_init(q_ready, 8);                           // the rows' warps (a dealt item: block 0's, twice)
        for (int b = 0; b < 2; ++b) {
            mbar_init(s_full + 8 * b, 1);
            mbar_init(p_full + 8 * b, 4);
            mbar_init(o_full + 8 * b, 1);
        }
        mbar_init(landed, 1);
        mbar_init(drain, 1);
        mbar_init(odd_done, 4);
        mbar_init(odd_free, 4);
        for (int k = 0; k < C::kCodeSlots; ++k) {
            mbar_init(c_full + 8 * k, 33);
            mbar_init(c_empty + 8 * k, 4);
        }
        s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 9) {
        tmem_alloc(smem_u32(&s_tmem), 512);
        tmem_relinquish();
    }
    pdl_trigger();                       // the join may settle; it waits for this grid's end
    tc_fence_before();
    const PagedShare share = paged_share<kPreTile, C::kThreads>(a, s_plan);   // synchronises
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    const int block_tokens = a.tile_tokens / C::kBlocks, block_rows = block_tokens * a.group;
    auto timed_out = [&]() {
        atomicOr(a.err, (uint32_t)PAGED_ERR_WAIT);
        s_abort = 1;
    };

    PagedWalk<kPreTile> w;
    w.init(a, share);
    // the item has rows for one block only: its key tiles are dealt to both
    auto dealt = [&]() { return ONE || w.sh.q.n - w.rt * a.tile_tokens <= block_tokens; };
    // some position of key tile t that no token of the sequence sees (its V row is cleared)
    auto ragged = [&](int t) {
        const int base = t * kPreTile;
        return base < w.sh.lo(a, 0) || base + kPreTile > w.sh.q.kv || (a.mask == PAGED_TREE && base + kPreTile > w.sh.ctx);
    };
    // tree positions that some token of the sequence sees (whole warp)
    auto tree_union = [&]() {
        if (a.mask != PAGED_TREE) return ~0ull;
        uint32_t lo32 = 0, hi32 = 0;
        for (int i = lane; i < w.sh.q.n; i += 32) {
            const uint64_t x = (uint64_t)a.tree[w.sh.q.row0 + i];
            lo32 |= (uint32_t)x;
            hi32 |= (uint32_t)(x >> 32);
        }
        lo32 = __reduce_or_sync(0xffffffffu, lo32);
        hi32 = __reduce_or_sync(0xffffffffu, hi32);
        return (unsigned long long)((uint64_t)hi32 << 32 | lo32);
    };
    auto seen = [&](int p, uint64_t any_word) {
        if (p < w.sh.lo(a, 0) || p >= w.sh.q.kv) return false;
        const int t = p - w.sh.ctx;
        return a.mask != PAGED_TREE || t < 0 || (t < 64 && ((any_word >> t) & 1ull));
    };

    auto fewer = [&]() {
        if constexpr (C::kMore) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kFewRegs));
    };
    if (warp == 8 || warp == 10) {
        fewer();
        // ---------------- copies: warp 8 queries and K, warp 10 V ----------------
        // (two, since boxes leave a warp one lane after the other: 16 of them, of pages of 16, took
        // one warp longer than memory takes for their bytes)
        constexpr int N = kCodes ? C::kCodeSlots : NS;           // stages of this ring
        constexpr int BYTES = kCodes ? C::kCodeBytes : C::kSlotBytes;
        constexpr int HALVES = kCodes ? 1 : C::kHalves;
        const uint32_t ring_full = kCodes ? c_full : full, ring_empty = kCodes ? c_empty : empty;
        const int kv = warp == 10;
        const CUtensorMap *tm = kv ? &tm_v : &tm_k;
        const int ps = a.pool.page_shift;
        const int br = min(1 << ps, kPreTile), nb = kPreTile / br, boxes = nb * HALVES;
        int turn = kv, items = 0;        // place in the order K0 V0 K1 V1 ...
        uint32_t lph = 0;                // parity of the cleared tiles
        bool alive = true;
        while (alive && w.next(a)) {
            const PagedSeq &q = w.sh.q;
            const int hi = w.sh.hi(a, w.rt), lo = w.sh.lo(a, w.rt), nblk = dealt() ? 1 : 2;
            const int64_t row = (int64_t)w.seq * a.batch.pages_stride;
            if (!kv && lane == 0) {
                if (!mbar_wait(q_empty, ((uint32_t)items & 1u) ^ 1u)) timed_out();
                if (!s_abort) {
                    mbar_expect_tx(q_full, (uint32_t)(nblk * C::kHalves * block_rows * 128));
                    for (int b = 0; b < nblk; ++b)
                        for (int h = 0; h < C::kHalves; ++h)
                            tma_load_3d(smem_u32(smem + C::kOffQ) + b * C::kSlotBytes + h * C::kHalfBytes, &tm_q, h * 64,
                                        w.head * a.group, q.row0 + w.rt * a.tile_tokens + b * block_tokens, q_full);
                }
            }
            ++items;
            auto lookup = [&](int t) {
                const int p = t * kPreTile + lane * br;
                if (lane >= nb || p >= hi || p + br <= lo) return -1;
                const int id = a.batch.pages[row + (p >> ps)];
                if (id < 0 || id >= a.pool.n_pages) {
                    atomicOr(a.err, (uint32_t)PAGED_ERR_PAGE);
                    return -1;
                }
                return id;
            };
            const uint64_t any_word = !kCodes && kv ? tree_union() : 0ull;
            int id = lookup(w.t0);
            for (int j = 0; j < w.nt; ++j) {
                const int t = w.t0 + j;
                const int id_now = id;
                id = j + 1 < w.nt ? lookup(t + 1) : -1;
                const int u = lane % boxes, b = u % nb, h = u / nb;
                const int page = __shfl_sync(0xffffffffu, id_now, b);
                const int slot = turn % N;
                const uint32_t par = (uint32_t)(turn / N) & 1u;
                turn += 2;
                // a V tile with rows to clear lands on a barrier of this warp's own first (codes are
                // cleared where they are converted)
                const bool clear = !kCodes && kv && ragged(t);
                const uint32_t bar = clear ? landed : ring_full + 8 * slot;
                int ok = 1;
                if (lane == 0) {
                    if (!mbar_wait(ring_empty + 8 * slot, par ^ 1u)) timed_out();
                    ok = !s_abort;
                    if (ok) mbar_expect_tx(bar, BYTES);
                }
                if (!__shfl_sync(0xffffffffu, ok, 0)) {
                    alive = false;
                    turn -= 2;                             // not issued
                    break;
                }
                uint8_t *dst = smem + (kCodes ? C::kOffCodes : 0) + slot * BYTES;
                if (lane < boxes)
                    tma_load_4d(smem_u32(dst) + h * C::kHalfBytes + b * br * (kCodes ? CODE_ROW : 128), tm, h * 64,
                                (t * kPreTile) & ((1 << ps) - 1), w.head, page < 0 ? a.pool.n_pages : page, bar);
                if constexpr (kCodes) {
                    const int key = lane * 4;
                    const int kp = __shfl_sync(0xffffffffu, id_now, key / br);
                    const float *src = (kv ? a.pool.vs : a.pool.ks) + (int64_t)max(kp, 0) * a.pool.s_page_stride +
                                       (int64_t)w.head * a.pool.s_head_stride + ((t * kPreTile + key) & ((1 << ps) - 1));
                    cp_async16(smem_u32(smem + C::kOffCodeScale + slot * kPreTile * 4) + key * 4, src, kp < 0 ? 0 : 16);
                    cp_async_arrive(bar);
                }
                if (clear) {
                    // what nobody sees must not reach the product: 0 * NaN
                    if (!__all_sync(0xffffffffu, mbar_wait(landed, lph))) {
                        if (lane == 0) timed_out();
                        alive = false;
                        break;
                    }
                    lph ^= 1u;
                    for (int r = lane; r < kPreTile; r += 32)
                        if (!seen(t * kPreTile + r, any_word))
                            for (int c = 0; c < C::kHalves * 8; ++c)
                                *reinterpret_cast<uint4 *>(dst + (c >> 3) * C::kHalfBytes + r * 128 + (c & 7) * 16) =
                                    make_uint4(0, 0, 0, 0);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) mbar_arrive(full + 8 * slot);
                }
            }
        }
        // no copy may land after the CTA is gone: every one that was issued has been waited for by
        // its reader, but on the way out of a failure.  (A tile for clearing lands elsewhere: there
        // the wait for its slot just runs its 50 ms.)
        if (lane == 0 && s_abort) {
            for (int k = 1; k <= N; ++k) {                 // this warp's last turns
                const int n = turn - 2 * k;
                if (n >= 0) mbar_wait(ring_full + 8 * (n % N), (uint32_t)(n / N) & 1u, 50000000ull);
            }
            if (!kv && items > 0) mbar_wait(q_full, (uint32_t)(items - 1) & 1u, 50000000ull);
        }
        __syncwarp();
    } else if (warp == 9) {
        fewer();
        // ---------------- products ----------------
        // The whole warp keeps the order and waits; one lane issues.  Descriptors differ by constants
        // from one base per operand: an address step adds its sixteenth to the low word (computed
        // anew for each product they took longer than the products).
        int slot = 0, items = 0;
        uint32_t wrap = 0, pph[2] = {0, 0};      // parity of the slots' use, and of the blocks' P
        bool alive = true;
        auto wait = [&](uint32_t bar, uint32_t parity) {
            if (!alive) return;
            if (!__all_sync(0xffffffffu, mbar_wait(bar, parity))) {
                if (lane == 0) timed_out();
                alive = false;
            }
            if (__any_sync(0xffffffffu, s_abort)) alive = false;
            tc_fence_after();
        };
        auto step = [&]() {
            if (++slot == NS) {
                slot = 0;
                wrap ^= 1u;
            }
        };
        auto commit = [&](uint32_t bar) {
            if (elect_one()) tc_commit(bar);
        };
        const uint64_t q_desc = tc_desc_sw128(smem_u32(smem + C::kOffQ));
        const uint64_t k_desc = tc_desc_sw128(smem_u32(smem));
        const uint64_t v_desc = tc_desc_mn_sw128(smem_u32(smem), C::kHalfBytes);
        // block b's S from queries qb and slot s
        auto qk = [&](int b, int qb, int s) {
            const uint64_t qd = q_desc + (uint32_t)(qb * (C::kSlotBytes >> 4));
            const uint64_t kd = k_desc + (uint32_t)(s * (C::kSlotBytes >> 4));
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = ((kk >> 2) * C::kHalfBytes + (kk & 3) * 32) >> 4;
                    tc_mma_f16(tmem + b * 128, qd + off, kd + off, kIdescQK, kk != 0);
                }
                tc_commit(s_full + 8 * b);
            }
            __syncwarp();
        };
        auto pv = [&](int b, int s, bool acc) {
            wait(p_full + 8 * b, pph[b]);
            pph[b] ^= 1u;
            if (!alive) return;
            const uint64_t vd = v_desc + (uint32_t)(s * (C::kSlotBytes >> 4));
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < kPreTile / 16; ++kk)
                    tc_mma_ts(tmem + 256 + b * 128, tmem + b * 128 + kk * 8, vd + (uint32_t)(kk * (2048 >> 4)), kIdescPV,
                              kk != 0 || acc);
            }
            __syncwarp();
        };
        while (alive && w.next(a)) {
            wait(kQTurned ? q_ready : q_full, (uint32_t)items & 1u);
            ++items;
            if (!dealt()) {
                wait(full + 8 * slot, wrap);
                if (!alive) break;
                qk(0, 0, slot);
                qk(1, 1, slot);
                commit(empty + 8 * slot);
                step();
                if (w.nt == 1) commit(q_empty);
                for (int j = 0; j < w.nt && alive; ++j) {
                    const int vs = slot;
                    const uint32_t vw = wrap;
                    step();
                    const bool more = j + 1 < w.nt;
                    wait(full + 8 * vs, vw);
                    pv(0, vs, j > 0);
                    if (more) wait(full + 8 * slot, wrap);
                    if (!alive) break;
                    if (more) qk(0, 0, slot);
                    else commit(o_full);
                    pv(1, vs, j > 0);
                    if (!alive) break;
                    commit(empty + 8 * vs);
                    if (more) {
                        qk(1, 1, slot);
                        commit(empty + 8 * slot);
                        step();
                        if (j + 2 == w.nt) commit(q_empty);
                    } else {
                        commit(o_full + 8);
                    }
                }
            } else {
                // slots in the order K0 V0 K1 V1 ...; products in the order QK0 QK1 PV0 QK2 PV1 QK3 ...
                const int s0 = slot;
                const uint32_t w0 = wrap;
                auto at = [&](int n, uint32_t &par) {          // slot and parity of the item's n-th tile
                    const int x = s0 + n;
                    par = w0 ^ ((uint32_t)(x / NS) & 1u);
                    return x % NS;
                };
                auto qk_of = [&](int j) {
                    uint32_t par;
                    const int s = at(2 * j, par);
                    wait(full + 8 * s, par);
                    if (!alive) return;
                    qk(j & 1, 0, s);
                    commit(empty + 8 * s);
                    if (j == w.nt - 1) commit(q_empty);
                };
                qk_of(0);
                if (w.nt > 1) qk_of(1);
                for (int j = 0; j < w.nt && alive; ++j) {
                    uint32_t par;
                    const int s = at(2 * j + 1, par);
                    wait(full + 8 * s, par);
                    pv(j & 1, s, j > 1);
                    if (!alive) break;
                    commit(empty + 8 * s);
                    if (j + 2 < w.nt) qk_of(j + 2);
                    else commit(o_full + 8 * (j & 1));
                }
                uint32_t par;
                slot = at(2 * w.nt, par);
                wrap = par;
            }
        }
        commit(drain);
        if (!mbar_wait(drain, 0) && lane == 0) timed_out();
        __syncwarp();
    } else if (kCodes && warp >= 12) {
        fewer();
        // ---------------- codes to F16 ----------------
        // A row's codes become F16 exactly.  Its scale goes to the rows' threads, K's as it is, V's in units of a
        // power of two, the largest so far of the item, which O is kept in.  Once the item has a V scale below
        // 2^-10 of that (a row of zeros too), V's go as they are, and the unit as -1: see apart_tile.
        // The ring of units needs no barrier of its own: the V slot of the tile that the slower
        // block's rows are at is taken, and with it every later one, so with 4 slots the tile at hand
        // here is at most 2 ahead of that one.
        const int r = (int)threadIdx.x - 384;              // the thread's key
        // 16-byte pieces of a row at a time: all of them (trees 130 us, 135 two at a time)
        constexpr int kChunks = D / 16;
        int slot = 0, cs = 0;
        uint32_t wrap = 0, cwrap = 0;
        int tile = 0;                                      // tiles so far: its place in the ring
        bool alive = true;
        while (alive && w.next(a)) {
            const uint64_t any_word = tree_union();
            uint32_t v_unit = 0;
            float v_low = INFINITY;                        // the smallest of the V scales that this lane has met
            bool far = false;
            for (int j = 0; j < w.nt && alive; ++j, ++tile) {
                const int t = w.t0 + j;
                // positions that no row of the item sees (some lie in pages that were not fetched for it) count
                // for nothing
                const int lo = w.sh.lo(a, w.rt), hi = w.sh.hi(a, w.rt);
                const bool edge = t * kPreTile < lo || (t + 1) * kPreTile > hi || ragged(t);
                auto counts = [&](int p) { return p >= lo && p < hi && seen(p, any_word); };
                for (int kv = 0; kv < 2; ++kv) {
                    const bool ok = mbar_wait(c_full + 8 * cs, cwrap) && mbar_wait(empty + 8 * slot, wrap ^ 1u);
                    if (!__all_sync(0xffffffffu, ok && !s_abort)) {
                        if (lane == 0) timed_out();
                        alive = false;
                        break;
                    }
                    const uint8_t *src = smem + C::kOffCodes + cs * C::kCodeBytes;
                    uint8_t *dst = smem + slot * C::kSlotBytes;
                    const float *scales = reinterpret_cast<const float *>(smem + C::kOffCodeScale) + cs * kPreTile;
                    const bool live = !edge || counts(t * kPreTile + r);
                    const float own = scales[r];
                    float inv = 1.f;
                    if (kv) {
                        // the tile's largest and smallest scale among the rows that count (four to a lane)
                        const float4 four = reinterpret_cast<const float4 *>(scales)[lane];
                        const float f[4] = {fabsf(four.x), fabsf(four.y), fabsf(four.z), fabsf(four.w)};
                        float most = fmaxf(fmaxf(f[0], f[1]), fmaxf(f[2], f[3]));           // NaN is passed over
                        if (!edge) {
                            v_low = fminf(v_low, fminf(fminf(f[0], f[1]), fminf(f[2], f[3])));
                        } else {
                            most = 0.f;
#pragma unroll 1
                            for (int i = 0; i < 4; ++i)
                                if (counts(t * kPreTile + 4 * lane + i)) {
                                    const float x = fabsf(scales[4 * lane + i]);
                                    most = fmaxf(most, x);
                                    v_low = fminf(v_low, x);
                                }
                        }
                        const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(most));
                        // the power of two above it, at most 2^127, and its inverse; 0 stays
                        v_unit = max(v_unit, top ? min((top & 0x7f800000u) + 0x00800000u, 0x7f000000u) : 0u);
                        far = __any_sync(0xffffffffu, far || v_low < __uint_as_float(v_unit) * 0x1p-10f);
                        if (!far) inv = v_unit == 0 ? 0.f : (v_unit == 0x7f000000u ? 0x1p-127f : __uint_as_float(0x7f000000u - v_unit));
                        if (warp == 12 && lane == 0)
                            reinterpret_cast<float *>(smem + C::kOffUnit)[tile % kScaleRing] = far ? -1.f : __uint_as_float(v_unit);
                    }
                    const float sc = live ? own * inv : 0.f;
                    reinterpret_cast<float *>(smem + C::kOffScale)[((tile % kScaleRing) * 2 + kv) * kPreTile + r] = sc;
#pragma unroll 1
                    for (int c0 = 0; c0 < D / 16; c0 += kChunks) {
                        uint4 row[kChunks];                // loads first: stores might be to the same place
#pragma unroll
                        for (int i = 0; i < kChunks; ++i)
                            row[i] = *reinterpret_cast<const uint4 *>(src + swz_row<CODE_ROW>(r, c0 + i));
#pragma unroll
                        for (int i = 0; i < kChunks; ++i) {
                            const int ch = c0 + i;
                            if (!live) row[i] = make_uint4(0, 0, 0, 0);        // (an e4m3 NaN times 0)
                            const uint32_t xs[4] = {row[i].x, row[i].y, row[i].z, row[i].w};
                            uint32_t y[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                if constexpr (FMT == kFmtInt8) y[k] = int8_pair(xs[k >> 1] ^ 0x80808080u, k & 1 ? 0x7362u : 0x5140u);
                                else y[k] = e4m3_pair_f16(xs[k >> 1] >> (16 * (k & 1)));
                            }
                            uint8_t *at = dst + (ch >> 2) * C::kHalfBytes;
                            *reinterpret_cast<uint4 *>(at + swz_row<128>(r, (2 * ch) & 7)) = make_uint4(y[0], y[1], y[2], y[3]);
                            *reinterpret_cast<uint4 *>(at + swz_row<128>(r, (2 * ch + 1) & 7)) = make_uint4(y[4], y[5], y[6], y[7]);
                        }
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(full + 8 * slot);
                        mbar_arrive(c_empty + 8 * cs);
                    }
                    if (++slot == NS) {
                        slot = 0;
                        wrap ^= 1u;
                    }
                    if (++cs == C::kCodeSlots) {
                        cs = 0;
                        cwrap ^= 1u;
                    }
                }
            }
        }
    } else if (warp < 8) {
        if constexpr (C::kMore) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kManyRegs));
        // ---------------- softmax rows ----------------
        constexpr int CH = kCodes && !C::kMore ? 16 : 32;               // scores of a row at a time: more would spill
        const int blk = warp >> 2, r = (warp & 3) * 32 + lane;
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lane_base + blk * 128, to = tmem + lane_base + 256 + blk * 128;
        uint8_t *row_exp = smem + C::kOffExp;                                         // [128] biased exponents
        float2 *odd_ml = reinterpret_cast<float2 *>(smem + C::kOffOdd);               // [128]
        float *odd_ref = reinterpret_cast<float *>(smem + C::kOffPlan + 24 * 8 + 8);
        uint32_t sph = 0, oph = 0, dph = 0;
        bool began = false;                                 // this CTA starts an item that another finishes
        bool owed = false;                                 // block 0 has yet to read this block's state
        int items = 0, tile0 = 0;                          // pieces and tiles so far
        int vslot = 1;                                     // running number of tile tile0's V in the slots
        while (w.next(a)) {
            const bool deal = dealt();
            if (owed) {
                if (!__all_sync(0xffffffffu, mbar_wait(odd_free, dph))) {
                    if (lane == 0) timed_out();
                    break;
                }
                dph ^= 1u;
                owed = false;
            }
            const PagedSeq &q = w.sh.q;
            const int my_blk = deal ? 0 : blk;             // whose rows these are
            const int local = my_blk * block_rows + r, f = w.rt * a.tile_tokens * a.group + local;
            const int tok = f / a.group;
            const bool valid = r < block_rows && f < q.n * a.group;
            const bool busy = __any_sync(0xffffffffu, valid);
            float qscale = a.scale_log2;
            // Every warp waits for every item's queries, whether it reads them or not, before it says
            // that they may go: else a block without a tile (block 1 of a dealt item of one) would
            // run on and speak twice for one item.
            if (!__all_sync(0xffffffffu, mbar_wait(q_full, (uint32_t)items & 1u))) {
                if (lane == 0) timed_out();
                break;
            }
            if constexpr (kQTurned) {
                // This block's queries to F16, unless the other block does it, which then leaves the rows'
                // powers of two here.  (They stand until every warp has said that this item's queries may
                // go: the next ones are not looked at before.  Loops not unrolled, for the instruction cache's sake:
                // two prompts of 4,097 tokens 421 us, 466 whole.)
                int e = 127;
                if (my_blk == blk) {
                    uint8_t *qr = smem + C::kOffQ + blk * C::kSlotBytes;
                    uint32_t top = 0;
#pragma unroll 1
                    for (int ch = 0; ch < D / 8; ++ch) {
                        const uint4 x = *reinterpret_cast<const uint4 *>(qr + (ch >> 3) * C::kHalfBytes + swz_row<128>(r, ch & 7));
                        const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) top = max(top, max(xs[i] & 0x7fffu, (xs[i] >> 16) & 0x7fffu));
                    }
                    if (top) e = min(254, max(1, (int)(top >> 7)));
                    const float down = e == 254 ? 0x1p-127f : __uint_as_float((uint32_t)(254 - e) << 23);
#pragma unroll 1
                    for (int ch = 0; ch < D / 8; ++ch) {
                        uint4 *at = reinterpret_cast<uint4 *>(qr + (ch >> 3) * C::kHalfBytes + swz_row<128>(r, ch & 7));
                        const uint4 x = *at;
                        uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            xs[i] = pack_half2(__uint_as_float(xs[i] << 16) * down, __uint_as_float(xs[i] & 0xffff0000u) * down);
                        *at = make_uint4(xs[0], xs[1], xs[2], xs[3]);
                    }
                    if (deal) row_exp[r] = (uint8_t)e;
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(q_ready);
                        if (deal) mbar_arrive(q_ready);
                    }
                }
                if (!__all_sync(0xffffffffu, mbar_wait(q_ready, (uint32_t)items & 1u))) {
                    if (lane == 0) timed_out();
                    break;
                }
                if (my_blk != blk) e = row_exp[r];
                qscale *= __uint_as_float((uint32_t)e << 23);
                __syncwarp();                              // read by every lane before lane 0 says so
            }
            ++items;
            // the queries may go with the last product
            if (lane == 0) mbar_arrive(q_empty);
            // what the row sees: [rlo, rhi) and, for a tree, bits from ctx on
            const int ctx = w.sh.ctx;
            int rlo = 0, rhi = 0;
            uint64_t word = 0;
            if (valid) {
                if (a.mask == PAGED_CAUSAL) {
                    rlo = a.window ? max(0, ctx + tok - a.window + 1) : 0;
                    rhi = min(q.kv, ctx + tok + 1);
                } else {
                    rlo = a.window ? max(0, ctx - a.window) : 0;
                    rhi = a.mask == PAGED_FULL ? q.kv : min(ctx, q.kv);
                    if (a.mask == PAGED_TREE) word = (uint64_t)a.tree[q.row0 + tok];
                }
            }
            const int all_lo = __reduce_max_sync(0xffffffffu, valid ? rlo : 0);
            const int all_hi = __reduce_min_sync(0xffffffffu, valid ? rhi : 0x7fffffff);
            float m = -INFINITY, l = 0.f, vref = 0.f;      // vref: the unit that O is in
            bool alive = true;
            const int j0 = deal ? blk : 0, dj = deal ? 2 : 1;
            auto wait_scores = [&](int j) {
                bool ok = mbar_wait(s_full + 8 * blk, sph);
                if constexpr (kCodes) {
                    // the tile's V scales (K's came with S)
                    const int vn = vslot + 2 * j;
                    ok = ok && mbar_wait(full + 8 * (vn % NS), (uint32_t)(vn / NS) & 1u);
                }
                if (!__all_sync(0xffffffffu, ok)) {
                    if (lane == 0) timed_out();
                    alive = false;
                    return;
                }
                sph ^= 1u;
                tc_fence_after();
            };
            auto hand_over = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + 8 * blk);
            };
            const RowSight sight{rlo, rhi, w.sh.ctx, q.kv, a.mask == PAGED_TREE, word};
            // (never 0, which would make NaN of what the mask leaves out; scores that small are 0)
            const float tscale = kCodes ? fmaxf(qscale, 0x1p-120f) : qscale;
            int j = j0;
            for (; j < w.nt; j += dj) {
                const int base = (w.t0 + j) * kPreTile;
                wait_scores(j);
                if (!alive) break;
                if (busy) {
                    // quantised: the tile's scales, and the unit of V's
                    const int ring = (tile0 + j) % kScaleRing;
                    float unit = 0.f;
                    if constexpr (kCodes) {
                        unit = reinterpret_cast<const float *>(smem + C::kOffUnit)[ring];
                        if (unit < 0.f) break;             // from here on V scales are far apart: below
                    }
                    const float4 *ks4 = reinterpret_cast<const float4 *>(smem + C::kOffScale) + ring * (kPreTile / 2);
                    const float4 *vs4 = ks4 + kPreTile / 4;
                    const bool partly = base < all_lo || base + kPreTile > all_hi;
                    // O times a factor per row
                    auto rescale = [&](float by) {
#pragma unroll 1
                        for (int c = 0; c < D / 16; ++c) {     // rare: small pieces spare registers
                            uint32_t u[16];
                            tmem_ld16(to + 16 * c, u);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(__uint_as_float(u[e]) * by);
                            tmem_st16(to + 16 * c, u);
                        }
                    };
                    // The row twice, CH scores at a time: its maximum, then, against a reference that
                    // is settled, its probabilities, without a branch to hold up the exponentials.
                    // bit e: the row sees position p + e
                    uint32_t raw[2][CH];                   // the piece at hand and, with registers to spare, the next
                    auto begin = [&]() {
                        tmem_ld(ts, raw[0]);
                    };
                    auto scores = [&](int c, const bool masked, uint64_t (&s)[CH / 2]) {
                        const bool ahead = !masked;
                        const int at = ahead ? c & 1 : 0;
                        if (!ahead) tmem_ld(ts + CH * c, raw[0]);
                        tmem_ld_wait();
                        if (ahead && c + 1 < 128 / CH) tmem_ld(ts + CH * (c + 1), raw[at ^ 1]);
#pragma unroll
                        for (int e = 0; e < CH / 2; ++e)
                            s[e] = pk2(__uint_as_float(raw[at][2 * e]), __uint_as_float(raw[at][2 * e + 1]));
                        if constexpr (kCodes) {
#pragma unroll
                            for (int e = 0; e < CH / 4; ++e) {
                                const float4 k = ks4[c * (CH / 4) + e];
                                s[2 * e] = mul2(s[2 * e], pk2(k.x, k.y));
                                s[2 * e + 1] = mul2(s[2 * e + 1], pk2(k.z, k.w));
                            }
                        }
                        if (masked) {
                            const uint32_t bits = sight.bits(base + CH * c);
#pragma unroll
                            for (int e = 0; e < CH / 2; ++e) {
                                float x, y;
                                upk2(s[e], x, y);
                                s[e] = pk2(bits & (1u << (2 * e)) ? x : -INFINITY, bits & (2u << (2 * e)) ? y : -INFINITY);
                            }
                        }
                    };
                    float factor = 1.f;                    // what O needs for this tile's reference
                    if (kCodes && unit != vref) {
                        factor = vref / unit;
                        vref = unit;
                    }
                    const uint64_t scale2 = pk2(tscale, tscale);
                    auto tile = [&](auto kind) {
                        constexpr bool masked = kind.value;
                        constexpr int kUnroll = masked ? 1 : (kCodes && !C::kMore ? 2 : 128 / CH);   // (see above; the masked one is rare)
                        constexpr int kProducts = masked ? 1 : (kCodes && (!C::kMore || kQTurned) ? 2 : 128 / CH);
                        float x0 = -INFINITY, x1 = x0;
                        if (!masked) begin();
#pragma unroll kUnroll
                        for (int c = 0; c < 128 / CH; ++c) {
                            uint64_t s[CH / 2];
                            scores(c, masked, s);
#pragma unroll
                            for (int e = 0; e < CH / 2; e += 2) {
                                float y0, y1, y2, y3;
                                upk2(s[e], y0, y1);
                                upk2(s[e + 1], y2, y3);
                                x0 = max3(x0, y0, y1);
                                x1 = max3(x1, y2, y3);
                            }
                        }
                        const float mx = fmaxf(x0, x1) * tscale;
                        if (!masked) begin();
                        const bool move = valid && mx > m + kLazyMove;
                        if (__any_sync(0xffffffffu, move || factor != 1.f)) {
                            const float mnew = move ? mx : m;
                            const float alpha = move ? exp2f(m - mnew) : 1.f;
                            m = mnew;
                            l *= alpha;
                            if (j > j0) rescale(alpha * factor);
                        }
                        const float mu = m == -INFINITY ? 0.f : m;
                        const uint64_t minus2 = pk2(-mu, -mu);
                        uint64_t sa = pk2(0.f, 0.f), sb = sa;
#pragma unroll kProducts
                        for (int c = 0; c < 128 / CH; ++c) {
                            uint64_t s[CH / 2];
                            scores(c, masked, s);
                            uint32_t u[CH / 2];
#pragma unroll
                            for (int e = 0; e < CH / 2; ++e) {
                                float x, y;
                                upk2(fma2(s[e], scale2, minus2), x, y);
                                uint64_t p2 = pk2(ex2_approx(x), ex2_approx(y));
                                if (e & 1) sb = add2(sb, p2);
                                else sa = add2(sa, p2);
                                if constexpr (kCodes) {
                                    const float4 v = vs4[c * (CH / 4) + e / 2];
                                    p2 = mul2(p2, e & 1 ? pk2(v.z, v.w) : pk2(v.x, v.y));
                                }
                                upk2(p2, x, y);
                                u[e] = pack16<OT>(x, y);
                            }
                            tmem_st(ts + c * (CH / 2), u);     // over scores that have been read
                        }
                        float s0, s1;
                        upk2(add2(sa, sb), s0, s1);
                        l += s0 + s1;
                    };
                    if (partly) tile(std::true_type{});
                    else tile(std::false_type{});
                    tmem_st_wait();
                }
                hand_over();
            }
            if constexpr (kCodes) {
                // the item's other tiles, the first of them waited for
                for (bool here = true; alive && j < w.nt; j += dj, here = false) {
                    if (!here) wait_scores(j);
                    if (!alive) break;
                    const float4 *ks4 = reinterpret_cast<const float4 *>(smem + C::kOffScale) + (tile0 + j) % kScaleRing * (kPreTile / 2);
                    const float3 x = apart_tile(ts, to, D, j > j0, sight, (w.t0 + j) * kPreTile, ks4, tscale, valid, m, l, vref);
                    m = x.x;
                    l = x.y;
                    vref = x.z;
                    tmem_st_wait();
                    hand_over();
                }
            }
            tile0 += w.nt;
            vslot += 2 * w.nt;
            if (__any_sync(0xffffffffu, !alive || s_abort)) break;     // one answer for the warp
            const bool mine = j0 < w.nt;                   // this block had a tile
            if (mine) {
                if (!__all_sync(0xffffffffu, mbar_wait(o_full + 8 * blk, oph))) {
                    if (lane == 0) timed_out();
                    break;
                }
                oph ^= 1u;
                tc_fence_after();
            }
            // dealt items: block 0 joins the two states; both blocks' lanes are the same, so it reads
            // the odd tiles' numerators where they are
            if (deal && blk == 1) {
                if (w.nt > 1) {
                    if (kCodes && busy && signbit(vref)) { // units of the rows' own are taken out: there is room for one
                        scale_numerators(to, D, fabsf(vref));
                        tmem_st_wait();
                        vref = 1.f;
                    }
                    odd_ml[r] = make_float2(m, l);
                    if (kCodes && threadIdx.x == 128) *odd_ref = vref;
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(odd_done);
                    owed = true;
                }
                continue;
            }
            const bool joins = deal && w.nt > 1;
            if (joins) {
                if (!__all_sync(0xffffffffu, mbar_wait(odd_done, dph))) {
                    if (lane == 0) timed_out();
                    break;
                }
                dph ^= 1u;
                tc_fence_after();
            }
            if (busy) {
                float keep = 1.f, add = 0.f;               // weights of this block's numerators and the odd ones
                if (kCodes) keep = fabsf(vref);
                if (joins) {
                    const float2 x = odd_ml[r];
                    const float mm = fmaxf(m, x.x), mu = mm == -INFINITY ? 0.f : mm;
                    const float e0 = m == -INFINITY ? (l != l ? l : 0.f) : exp2f(m - mu);
                    add = x.x == -INFINITY ? (x.y != x.y ? x.y : 0.f) : exp2f(x.x - mu);
                    l = l * e0 + x.y * add;
                    keep *= e0;
                    m = mm;
                    if (kCodes) add *= *odd_ref;
                }
                const bool whole = w.first && w.last;
                const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
                const int head = w.head * a.group + f - tok * a.group;
                const int64_t part = ((int64_t)blockIdx.x * 2 + (w.first ? 1 : 0)) * a.tile_rows + local;
                uint16_t *o = a.o + (int64_t)(q.row0 + tok) * a.o_rs + (int64_t)head * a.o_hs;
                float *acc = a.part_acc + part * D;
                if (whole) {
                    keep *= inv;
                    add *= inv;
                }
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t u[32], v[32];
                    __syncwarp();
                    tmem_ld32(to + 32 * c, u);
                    if (joins) tmem_ld32(to + 128 + 32 * c, v);
                    tmem_ld_wait();
                    if (!valid) continue;
                    float x[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] = __uint_as_float(u[e]) * keep;
                    if (joins) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) x[e] = fmaf(__uint_as_float(v[e]), add, x[e]);
                    }
                    if (whole) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
                            *reinterpret_cast<uint4 *>(o + 32 * c + e) =
                                make_uint4(pack16<T>(x[e], x[e + 1]), pack16<T>(x[e + 2], x[e + 3]),
                                           pack16<T>(x[e + 4], x[e + 5]), pack16<T>(x[e + 6], x[e + 7]));
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<float4 *>(acc + 32 * c + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
                    }
                }
                if (valid) {
                    if (whole) {
                        if (a.lse)
                            a.lse[(int64_t)(q.row0 + tok) * a.n_head + head] =
                                l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
                    } else {
                        a.part_ml[part] = make_float2(m, l);
                    }
                }
                tc_fence_before();
            }
            if (joins) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(odd_free);
            }
            if (threadIdx.x == 0 && w.first && !w.last) {
                began = true;
                a.desc[blockIdx.x] = make_int4(w.seq, w.head, w.rt, w.last_cta());
            }
        }
        if (threadIdx.x == 0 && !began) a.desc[blockIdx.x] = make_int4(-1, 0, 0, 0);
    } else {
        fewer();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace dflash
