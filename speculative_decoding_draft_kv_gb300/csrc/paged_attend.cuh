// Attention of new tokens over a paged cache: the kernel for few query rows per kv head
// (single tokens, verify blocks, token trees), and the join of partial results.
//
// o = sum_p softmax_p(q . k_p * scale) v_p over the pages of a sequence.  With R query rows
// per kv head a 16-bit K or V byte takes part in R flops, so up to R = 32 the pass is bound by
// the bytes of the cache, each of which is fetched once: the query heads of a kv head ride
// together, one pass over the keys with a running maximum and sum.  Tensor work goes to
// mma.sync (m16n8k16): at R = 16 it needs a fifth of that unit's rate.
//
// Shape: 4 consumer warps and one copy warp, two CTAs per SM, key tiles of 64.  The copy warp
// looks the tile's pages up and fetches K and V by TMA, a box per page (or part of one),
// 128-byte swizzle, into a ring of stages of about 96 KiB; rows past a page's last live
// position are fetched with their page and masked, V rows nobody sees are cleared in shared
// memory before the product (0 * NaN).  Consumer warp w owns row block w % MT and key slice
// w / MT of every tile; the slices' softmax states meet in shared memory when an item is done.
//
// The softmax keeps a reference maximum per row that moves only when a row outgrows it by
// 2^8 (probabilities up to 256 are as exact in F16 as those up to 1, and the quotient does not
// depend on the reference), so most tiles rescale nothing.
//
// Quantised pages: codes become F16 operands exactly (int8: byte permutes and a subtraction;
// e4m3: one conversion), whatever the queries' type; K's scale multiplies the score, V's the
// probability.  The product of those two becomes an F16 operand in a unit that keeps it in range: the power
// of two above the largest V scale so far, while none of the item's is below 2^-10 of that, which
// every row's largest product is then not far below either.  Once one is (a row of zeros too), each row has
// a unit of its own, which follows the row's largest product: what is lost below F16's smallest step is
// small beside what counts most, whatever scales the row does not see or gives no weight.  (Units by the
// row from the start: 4 tokens over int8 338 us instead of 291; one unit for all always: 284.)  bf16
// queries enter as F16 after a power of two per row brings the row's largest value to [1, 2): exact but
// for values 2^-17 below it, which are off by 2^-25 of it at most.
//
// Measured, bf16, 32 query and 8 kv heads of 128, pages of 16, 64 sequences of 9 to 16,384 tokens
// (2.2 GB): one token each 353 us, 6.3 TB/s (93 % of the copy rate); 4 tokens (16 rows) 367 us.  With
// 32 rows it took 382 us, where the products' instructions show, against the tensor-core kernel's 371:
// 16-bit pages come here with up to 16 rows, quantised ones with up to 32 (4 tokens over int8 291 us, 3.9
// TB/s; 8 tokens 455 us: turning codes into operands is what counts).  One token over 4,096: 12 us with the
// join, of which bytes are 2.5: the rest is a chain of lookups (plan, page numbers), one round of
// copies, the slices' merge and the join.
#pragma once

#include "paged_plan.h"

namespace dflash {

constexpr int kDecTile = 64;
constexpr float kLazyMove = 8.f;

enum { kFmt16 = 0, kFmtInt8 = 1, kFmtE4m3 = 2 };

template <int D, int MT, int FMT>
struct DecCfg {
    static constexpr int kThreads = 160;
    static constexpr int ES = FMT == kFmt16 ? 2 : 1;
    static constexpr int kTileBytes = kDecTile * D * ES;
    static constexpr int kStageBytes = 2 * kTileBytes;
    static constexpr int kStages = FMT == kFmt16 ? 96 * 1024 / kStageBytes : (D == 128 ? 6 : 11);
    static constexpr int kRowBytes = D * ES < 128 ? D * ES : 128;      // one TMA box row
    static constexpr int kHalves = D * ES / kRowBytes;                 // boxes side by side
    static constexpr int kRows = 16 * MT;
    static constexpr int kSlices = 4 / MT;
    static constexpr int kKeys = kDecTile / kSlices;                   // per warp and tile
    static constexpr int kNT = kKeys / 8;
    static constexpr int kScaleBytes = FMT == kFmt16 ? 0 : 2 * kDecTile * 4;   // K, then V
    static constexpr int kOffScale = kStages * kStageBytes;
    // the queries (until their fragments are in registers), then the slices' numerators
    static constexpr int kXBytes = (kSlices - 1) * MT * 32 * 32 * 4;
    static constexpr int kQBytes = kRows * D * 2;
    static constexpr int kOffX = kOffScale + kStages * kScaleBytes;
    static constexpr int kOffMl = kOffX + (kXBytes > kQBytes ? kXBytes : kQBytes);
    static constexpr int kOffBars = kOffMl + 4 * 16 * 8;
    static constexpr int kSmem = 1024 + kOffBars + 2 * kStages * 8;
    static_assert(kSmem <= 113 * 1024, "two CTAs per SM");
};

// byte offset of 16-byte chunk ch of row r in a tile of rows of RB bytes as TMA's swizzle
// of that width leaves it
template <int RB>
__device__ __forceinline__ uint32_t swz_row(int r, int ch) {
    const int x = RB == 128 ? (r & 7) : ((r >> 1) & 3);
    return (uint32_t)(r * RB + ((ch ^ x) << 4));
}

// the largest of a row's four lanes
__device__ __forceinline__ float quad_max(float x) {
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}

template <int T>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    if constexpr (T == PAGED_F16) return pack_half2(lo, hi);
    else return pack_bf162(lo, hi);
}

template <int D, int MT, int FMT, int T>
__global__ void __launch_bounds__(160, 2)
k_paged_attend(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
               const __grid_constant__ PagedAttendArgs a) {
    using C = DecCfg<D, MT, FMT>;
    constexpr int S = C::kStages;
    // operands are F16 for quantised pages, else of the queries' type
    constexpr int OT = FMT == kFmt16 ? T : PAGED_F16;
    constexpr bool kQScaled = FMT != kFmt16 && T == PAGED_BF16;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t bar0 = smem_u32(smem + C::kOffBars);       // full[S], empty[S]
    __shared__ int64_t s_plan[9];
    __shared__ volatile int s_abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
        for (int k = 0; k < S; ++k) {
            mbar_init(bar0 + 8 * k, FMT == kFmt16 ? 1 : 33);
            mbar_init(bar0 + 8 * (S + k), 4);
        }
        s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    pdl_trigger();                       // the join may settle; it waits for this grid's end
    const PagedShare share = paged_share<kDecTile, C::kThreads>(a, s_plan);
    if (threadIdx.x == 0 && share.units == 0) a.desc[blockIdx.x] = make_int4(-1, 0, 0, 0);
    if (share.units == 0) {
        if (a.level == kOwn) pdl_wait();
        return;
    }

    PagedWalk<kDecTile> w;
    w.init(a, share);
    int it = 0;                          // tiles so far: stage it % S, use it / S

    if (warp == 4) {
        // ---------------- copies ----------------
        const int ps = a.pool.page_shift;
        const int br = min(1 << ps, kDecTile);                 // rows per box
        const int nb = kDecTile / br;                          // boxes along a tile
        const int boxes = nb * C::kHalves;                     // per tensor
        bool alive = true;
        while (alive && w.next(a)) {
            const int hi = w.sh.hi(a, w.rt), lo = w.sh.lo(a, w.rt);
            const int64_t row = (int64_t)w.seq * a.batch.pages_stride;
            // lane b: the page of box b of tile t (-1: not needed, or not to be had)
            auto lookup = [&](int t) {
                const int p = t * kDecTile + lane * br;
                if (lane >= nb || p >= hi || p + br <= lo) return -1;
                const int id = a.batch.pages[row + (p >> ps)];
                if (id < 0 || id >= a.pool.n_pages) {
                    atomicOr(a.err, (uint32_t)PAGED_ERR_PAGE);
                    return -1;
                }
                return id;
            };
            int id = lookup(w.t0);
            for (int j = 0; j < w.nt; ++j, ++it) {
                const int t = w.t0 + j, stg = it % S;
                const int id_next = j + 1 < w.nt ? lookup(t + 1) : -1;
                int ok = 1;
                if (lane == 0) {
                    if (!mbar_wait(bar0 + 8 * (S + stg), ((uint32_t)(it / S) & 1u) ^ 1u)) {
                        atomicOr(a.err, (uint32_t)PAGED_ERR_WAIT);
                        s_abort = 1;
                    }
                    ok = !s_abort;
                    if (ok) mbar_expect_tx(bar0 + 8 * stg, C::kStageBytes);
                }
                if (!__shfl_sync(0xffffffffu, ok, 0)) {
                    alive = false;
                    break;
                }
                const uint32_t full = bar0 + 8 * stg;
                const uint32_t dst = smem_u32(smem + stg * C::kStageBytes);
                const int u = lane % boxes, b = u % nb, h = u / nb;
                const int page = __shfl_sync(0xffffffffu, id, b);
                if (lane < 2 * boxes) {
                    const bool is_v = lane >= boxes;
                    // a page that is not to be had reads as zeros: past the pool's end
                    tma_load_4d(dst + (is_v ? C::kTileBytes : 0) + (h * kDecTile + b * br) * C::kRowBytes,
                                is_v ? &tm_v : &tm_k, h * (C::kRowBytes / C::ES),
                                (t * kDecTile) & ((1 << ps) - 1), w.head, page < 0 ? a.pool.n_pages : page, full);
                }
                if constexpr (FMT != kFmt16) {
                    // lanes 0-15: K scales of four keys each, lanes 16-31: V scales
                    const int key = (lane & 15) * 4;
                    const int kp = __shfl_sync(0xffffffffu, id, key / br);
                    const int slot = (t * kDecTile + key) & ((1 << ps) - 1);
                    const float *base = lane < 16 ? a.pool.ks : a.pool.vs;
                    const float *src = base + (int64_t)max(kp, 0) * a.pool.s_page_stride +
                                       (int64_t)w.head * a.pool.s_head_stride + slot;
                    cp_async16(smem_u32(smem + C::kOffScale + stg * C::kScaleBytes) + (lane >> 4) * kDecTile * 4 + key * 4,
                               src, kp < 0 ? 0 : 16);
                    cp_async_arrive(full);
                }
                id = id_next;
            }
        }
        // no copy may land after the CTA is gone
        if (lane == 0)
            for (int k = max(0, it - S); k < it; ++k)
                if (!mbar_wait(bar0 + 8 * (k % S), (uint32_t)(k / S) & 1u)) {
                    atomicOr(a.err, (uint32_t)PAGED_ERR_WAIT);
                    break;
                }
        __syncwarp();
        return;
    }

    // ---------------- consumers ----------------
    const int mb = warp % MT, ksl = warp / MT;
    const int g = lane >> 2, c = lane & 3;
    const int key0 = ksl * C::kKeys;
    uint8_t *sq = smem + C::kOffX;
    float *sx = reinterpret_cast<float *>(smem + C::kOffX);
    float2 *sml = reinterpret_cast<float2 *>(smem + C::kOffMl);
    bool began = false;                  // this CTA starts an item that another one finishes
    while (w.next(a)) {
        const PagedSeq &q = w.sh.q;
        const int flat_n = q.n * a.group;            // a row is (token, query head), token by token
        float qscale[2] = {a.scale_log2, a.scale_log2};
        // queries of this kv head into shared memory; rows that are not there are zeros
        for (int u = threadIdx.x; u < C::kRows * (D / 8); u += 128) {
            const int r = u / (D / 8), ch = u % (D / 8), f = r;
            uint4 x = make_uint4(0, 0, 0, 0);
            if (f < flat_n) {
                const int tok = f / a.group, hh = f - tok * a.group;
                x = *reinterpret_cast<const uint4 *>(a.q + (int64_t)(q.row0 + tok) * a.q_rs +
                                                     (int64_t)(w.head * a.group + hh) * a.q_hs + ch * 8);
            }
            *reinterpret_cast<uint4 *>(sq + swz(r, ch * 8, C::kRows)) = x;
        }
        bar_sync(1, 128);
        uint32_t qf[D / 16][4];
        const int r0 = mb * 16 + g, r1 = r0 + 8;
        if constexpr (FMT == kFmt16) {
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
                ldsm_x4(smem_u32(sq) + swz(mb * 16 + (lane & 15), ks * 16 + ((lane >> 4) << 3), C::kRows), qf[ks][0],
                        qf[ks][1], qf[ks][2], qf[ks][3]);
        } else {
            // codes come four consecutive dimensions to a thread, which fill the product's k
            // slots 2c, 2c+1, 2c+8, 2c+9; the queries take the same order
            uint32_t top[2] = {0u, 0u};
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                const int col = ks * 16 + 4 * c;
                const uint2 x = *reinterpret_cast<const uint2 *>(sq + swz(r0, col & ~7, C::kRows) + (col & 7) * 2);
                const uint2 y = *reinterpret_cast<const uint2 *>(sq + swz(r1, col & ~7, C::kRows) + (col & 7) * 2);
                qf[ks][0] = x.x;
                qf[ks][1] = y.x;
                qf[ks][2] = x.y;
                qf[ks][3] = y.y;
                if constexpr (kQScaled) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        top[e & 1] = max(top[e & 1], max(qf[ks][e] & 0x7fffu, (qf[ks][e] >> 16) & 0x7fffu));
                }
            }
            if constexpr (kQScaled) {
                // bf16 -> F16: the row's largest value brought to [1, 2) by a power of two
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    top[j] = max(top[j], __shfl_xor_sync(0xffffffffu, top[j], 1));
                    top[j] = max(top[j], __shfl_xor_sync(0xffffffffu, top[j], 2));
                    const int e = top[j] ? min(254, max(1, (int)(top[j] >> 7))) : 127;   // biased exponent
                    const float down = e == 254 ? 0x1p-127f : __uint_as_float((uint32_t)(254 - e) << 23);
                    const float up = __uint_as_float((uint32_t)e << 23);
                    // (never 0, which would make NaN of what the mask leaves out; scores that small are 0)
                    qscale[j] = fmaxf(a.scale_log2 * up, 0x1p-120f);
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                        for (int i = j; i < 4; i += 2) {
                            const uint32_t v = qf[ks][i];
                            qf[ks][i] = pack_half2(__uint_as_float(v << 16) * down, __uint_as_float(v & 0xffff0000u) * down);
                        }
                }
            }
        }

        // what this thread's two rows see: [rlo, rhi) and, for a tree, bits from ctx on
        int rlo[2], rhi[2];
        uint64_t word[2] = {0ull, 0ull};
        int all_lo = 0, all_hi = 0x7fffffff;
        const int ctx = w.sh.ctx, item_lo = w.sh.lo(a, w.rt), item_hi = w.sh.hi(a, w.rt);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int f = j ? r1 : r0, tok = f / a.group;
            rlo[j] = rhi[j] = 0;
            if (f < flat_n) {
                if (a.mask == PAGED_CAUSAL) {
                    rlo[j] = a.window ? max(0, ctx + tok - a.window + 1) : 0;
                    rhi[j] = min(q.kv, ctx + tok + 1);
                } else {
                    rlo[j] = a.window ? max(0, ctx - a.window) : 0;
                    rhi[j] = a.mask == PAGED_FULL ? q.kv : min(ctx, q.kv);
                    if (a.mask == PAGED_TREE) word[j] = (uint64_t)a.tree[q.row0 + tok];
                }
                all_lo = max(all_lo, rlo[j]);
                all_hi = min(all_hi, rhi[j]);
            }
        }
        all_lo = __reduce_max_sync(0xffffffffu, all_lo);
        all_hi = __reduce_min_sync(0xffffffffu, all_hi);
        // tree positions that some row of the item sees
        uint64_t any_word = ~0ull;
        if (a.mask == PAGED_TREE) {
            uint32_t lo32 = 0, hi32 = 0;
            const int f = lane;
            if (lane < C::kRows && f < flat_n) {
                const uint64_t x = (uint64_t)a.tree[q.row0 + f / a.group];
                lo32 = (uint32_t)x;
                hi32 = (uint32_t)(x >> 32);
            }
            lo32 = __reduce_or_sync(0xffffffffu, lo32);
            hi32 = __reduce_or_sync(0xffffffffu, hi32);
            any_word = (uint64_t)hi32 << 32 | lo32;
        }
        auto seen_by_any = [&](int p) {
            if (p < item_lo || p >= item_hi) return false;
            return a.mask != PAGED_TREE || p < ctx || (p - ctx < 64 && ((any_word >> (p - ctx)) & 1ull));
        };

        float oacc[D / 8][4];
#pragma unroll
        for (int n = 0; n < D / 8; ++n) oacc[n][0] = oacc[n][1] = oacc[n][2] = oacc[n][3] = 0.f;
        float mrow[2] = {-INFINITY, -INFINITY}, lrow[2] = {0.f, 0.f};
        // quantised: the unit that the numerators are in; far: each row has its own, at most its largest
        // probability times V scale so far (negative: one from before, which may be above that)
        float vref[2] = {0.f, 0.f};
        float low = INFINITY;            // the smallest of the V scales that this lane has met
        bool far = false;
        for (int j = 0; j < w.nt; ++j, ++it) {
            const int stg = it % S, base = (w.t0 + j) * kDecTile;
            if (!__all_sync(0xffffffffu, mbar_wait(bar0 + 8 * stg, (uint32_t)(it / S) & 1u))) {
                if (lane == 0) atomicOr(a.err, (uint32_t)PAGED_ERR_WAIT);
                s_abort = 1;
                break;
            }
            uint8_t *tk = smem + stg * C::kStageBytes, *tv = tk + C::kTileBytes;
            const uint32_t sk = smem_u32(tk), sv = smem_u32(tv);
            // some position of the tile that no row sees: clear its V row
            const bool ragged = base < item_lo || base + kDecTile > item_hi || (a.mask == PAGED_TREE && base + kDecTile > ctx);
            if (ragged) {
                for (int u = lane; u < C::kKeys * (C::kRowBytes / 16) * C::kHalves; u += 32) {
                    const int r = key0 + u / ((C::kRowBytes / 16) * C::kHalves);
                    const int ch = u % ((C::kRowBytes / 16) * C::kHalves);
                    if (!seen_by_any(base + r))
                        *reinterpret_cast<uint4 *>(tv + (ch / (C::kRowBytes / 16)) * kDecTile * C::kRowBytes +
                                                   r * C::kRowBytes + (ch % (C::kRowBytes / 16)) * 16) =
                            make_uint4(0, 0, 0, 0);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
            }

            // S = Q K^T
            float sc[C::kNT][4];
#pragma unroll
            for (int n = 0; n < C::kNT; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.f;
            if constexpr (FMT == kFmt16) {
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                    for (int np = 0; np < C::kNT / 2; ++np) {
                        const int key = key0 + np * 16 + (lane & 7) + ((lane >> 4) << 3);
                        uint32_t b0, b1, b2, b3;
                        ldsm_x4(sk + swz(key, ks * 16 + (((lane >> 3) & 1) << 3), kDecTile), b0, b1, b2, b3);
                        if constexpr (OT == PAGED_F16) {
                            mma16816(sc[np * 2], qf[ks], b0, b1);
                            mma16816(sc[np * 2 + 1], qf[ks], b2, b3);
                        } else {
                            mma16816_bf16(sc[np * 2], qf[ks], b0, b1);
                            mma16816_bf16(sc[np * 2 + 1], qf[ks], b2, b3);
                        }
                    }
            } else {
                const float *kscale = reinterpret_cast<const float *>(smem + C::kOffScale + stg * C::kScaleBytes);
#pragma unroll
                for (int np = 0; np < C::kNT / 2; ++np) {
                    const int lkey = key0 + np * 16 + 8 * ((lane >> 3) & 1) + (lane & 7);
#pragma unroll
                    for (int kp = 0; kp < D / 32; ++kp) {
                        uint32_t x[4];
                        ldsm_x4(sk + swz_row<C::kRowBytes>(lkey, 2 * kp + (lane >> 4)), x[0], x[1], x[2], x[3]);
#pragma unroll
                        for (int m = 0; m < 2; ++m)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                uint32_t b0, b1;
                                if constexpr (FMT == kFmtInt8) {
                                    const uint32_t xf = x[2 * h + m] ^ 0x80808080u;
                                    b0 = int8_pair(xf, 0x5140u);
                                    b1 = int8_pair(xf, 0x7362u);
                                } else {
                                    b0 = e4m3_pair_f16(x[2 * h + m]);
                                    b1 = e4m3_pair_f16(x[2 * h + m] >> 16);
                                }
                                mma16816(sc[2 * np + m], qf[2 * kp + h], b0, b1);
                            }
                    }
                }
#pragma unroll
                for (int n = 0; n < C::kNT; ++n) {
                    const float2 f = *reinterpret_cast<const float2 *>(kscale + key0 + n * 8 + 2 * c);
                    sc[n][0] *= f.x;
                    sc[n][1] *= f.y;
                    sc[n][2] *= f.x;
                    sc[n][3] *= f.y;
                }
            }
            if (base < all_lo || base + kDecTile > all_hi) {
#pragma unroll
                for (int n = 0; n < C::kNT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int p = base + key0 + n * 8 + 2 * c + (e & 1), jj = e >> 1;
                        bool vis = p >= rlo[jj] && p < rhi[jj];
                        if (a.mask == PAGED_TREE && p >= ctx && p < q.kv && p - ctx < 64)
                            vis = (word[jj] >> (p - ctx)) & 1ull;
                        if (!vis) sc[n][e] = -INFINITY;
                    }
            }

            // softmax in log2 units against a lazily moved reference
            float mx[2];
            bool move = false;
#pragma unroll
            for (int jj = 0; jj < 2; ++jj) {
                float x = -INFINITY;
#pragma unroll
                for (int n = 0; n < C::kNT; ++n) x = fmaxf(x, fmaxf(sc[n][2 * jj], sc[n][2 * jj + 1]));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                mx[jj] = x * qscale[jj];
                move |= mx[jj] > mrow[jj] + kLazyMove;
            }
            if (__any_sync(0xffffffffu, move)) {
                float alpha[2];
#pragma unroll
                for (int jj = 0; jj < 2; ++jj) {
                    const float mnew = fmaxf(mrow[jj], mx[jj]);
                    alpha[jj] = mnew == -INFINITY ? 1.f : exp2f(mrow[jj] - mnew);
                    mrow[jj] = mnew;
                    lrow[jj] *= alpha[jj];
                    if (FMT != kFmt16 && far) {          // the unit moves in the numerators' place
                        vref[jj] *= alpha[jj];
                        alpha[jj] = 1.f;
                    }
                }
#pragma unroll
                for (int n = 0; n < D / 8; ++n) {
                    oacc[n][0] *= alpha[0];
                    oacc[n][1] *= alpha[0];
                    oacc[n][2] *= alpha[1];
                    oacc[n][3] *= alpha[1];
                }
            }
#pragma unroll
            for (int jj = 0; jj < 2; ++jj) {
                const float muse = mrow[jj] == -INFINITY ? 0.f : mrow[jj];
                float rs = 0.f;
#pragma unroll
                for (int n = 0; n < C::kNT; ++n) {
                    const float p0 = ex2_approx(fmaf(sc[n][2 * jj], qscale[jj], -muse));
                    const float p1 = ex2_approx(fmaf(sc[n][2 * jj + 1], qscale[jj], -muse));
                    sc[n][2 * jj] = p0;
                    sc[n][2 * jj + 1] = p1;
                    rs += p0 + p1;
                }
                lrow[jj] += rs;
            }

            // O += P V
            if constexpr (FMT != kFmt16) {
                const float *vscale = reinterpret_cast<const float *>(smem + C::kOffScale + stg * C::kScaleBytes) + kDecTile;
                float2 f[C::kNT];
                float top = 0.f;                         // the tile's largest (NaN is passed over)
#pragma unroll
                for (int n = 0; n < C::kNT; ++n) f[n] = *reinterpret_cast<const float2 *>(vscale + key0 + n * 8 + 2 * c);
                if (ragged) {
#pragma unroll
                    for (int n = 0; n < C::kNT; ++n) {
                        const int p = base + key0 + n * 8 + 2 * c;
                        if (seen_by_any(p)) low = fminf(low, fabsf(f[n].x));
                        else f[n].x = 0.f;
                        if (seen_by_any(p + 1)) low = fminf(low, fabsf(f[n].y));
                        else f[n].y = 0.f;
                    }
                } else {
#pragma unroll
                    for (int n = 0; n < C::kNT; ++n) low = fminf(low, fminf(fabsf(f[n].x), fabsf(f[n].y)));
                }
                float inv[2];
                if (!far) {
#pragma unroll
                    for (int n = 0; n < C::kNT; ++n) top = fmaxf(top, fmaxf(fabsf(f[n].x), fabsf(f[n].y)));
                    top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
                    const bool apart = low < fmaxf(top, vref[0]) * 0x1p-10f;         // (also with an infinity among them)
                    if (__any_sync(0xffffffffu, apart || top > vref[0])) {
                        far = __any_sync(0xffffffffu, apart);
                        // the next power of two (the exponent field plus one, at most 2^127)
                        const float vnew = fmaxf(vref[0], __uint_as_float(min((__float_as_uint(top) & 0x7f800000u) + 0x00800000u, 0x7f000000u)));
                        const float r = far ? 1.f : vref[0] / vnew;
                        vref[0] = vref[1] = far ? -vref[0] : vnew;
#pragma unroll
                        for (int n = 0; n < D / 8; ++n)
#pragma unroll
                            for (int e = 0; e < 4; ++e) oacc[n][e] *= r;
                    }
                }
                if (far) {
#pragma unroll
                    for (int jj = 0; jj < 2; ++jj) {
                        float wt = 0.f, omax = 0.f;
#pragma unroll
                        for (int n = 0; n < C::kNT; ++n) {
                            sc[n][2 * jj] *= f[n].x;
                            sc[n][2 * jj + 1] *= f[n].y;
                            wt = fmaxf(wt, fmaxf(fabsf(sc[n][2 * jj]), fabsf(sc[n][2 * jj + 1])));
                        }
                        wt = fminf(quad_max(wt), 0x1p126f);
                        // (a unit that followed the reference's moves below F32's smallest is set anew too)
                        const bool move = wt > 0.f && (wt > 1024.f * vref[jj] || vref[jj] < 0x1p-126f);
                        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
                            for (int n = 0; n < D / 8; ++n) omax = fmaxf(omax, fmaxf(fabsf(oacc[n][2 * jj]), fabsf(oacc[n][2 * jj + 1])));
                            omax = quad_max(omax);
                            // 2^-60 of the numerators is less than any product in them, and keeps them in range
                            const float vold = fabsf(vref[jj]);
                            const float vnew = move ? fmaxf(fmaxf(wt, 0x1p-126f), fminf(omax * vold, 0x1p126f) * 0x1p-60f) : vref[jj];
                            if (move) {
                                vref[jj] = vnew;
#pragma unroll
                                for (int n = 0; n < D / 8; ++n) {
                                    oacc[n][2 * jj] = oacc[n][2 * jj] * vold * (1.f / vnew);
                                    oacc[n][2 * jj + 1] = oacc[n][2 * jj + 1] * vold * (1.f / vnew);
                                }
                            }
                        }
                        inv[jj] = vref[jj] >= 0x1p-126f ? 1.f / vref[jj] : 0.f;
                    }
#pragma unroll
                    for (int n = 0; n < C::kNT; ++n) f[n] = make_float2(1.f, 1.f);
                } else {
                    inv[0] = inv[1] = vref[0] > 0.f ? 1.f / vref[0] : 0.f;
                }
#pragma unroll
                for (int n = 0; n < C::kNT; ++n) {
                    sc[n][0] *= f[n].x * inv[0];
                    sc[n][1] *= f[n].y * inv[0];
                    sc[n][2] *= f[n].x * inv[1];
                    sc[n][3] *= f[n].y * inv[1];
                }
            }
#pragma unroll
            for (int kk = 0; kk < C::kKeys / 16; ++kk) {
                uint32_t pa[4];
                pa[0] = pack16<OT>(sc[2 * kk][0], sc[2 * kk][1]);
                pa[1] = pack16<OT>(sc[2 * kk][2], sc[2 * kk][3]);
                pa[2] = pack16<OT>(sc[2 * kk + 1][0], sc[2 * kk + 1][1]);
                pa[3] = pack16<OT>(sc[2 * kk + 1][2], sc[2 * kk + 1][3]);
                const int key = key0 + kk * 16 + (lane & 7) + (((lane >> 3) & 1) << 3);
                if constexpr (FMT == kFmt16) {
#pragma unroll
                    for (int dp = 0; dp < D / 16; ++dp) {
                        uint32_t b0, b1, b2, b3;
                        ldsm_x4_t(sv + swz(key, dp * 16 + ((lane >> 4) << 3), kDecTile), b0, b1, b2, b3);
                        if constexpr (OT == PAGED_F16) {
                            mma16816(oacc[dp * 2], pa, b0, b1);
                            mma16816(oacc[dp * 2 + 1], pa, b2, b3);
                        } else {
                            mma16816_bf16(oacc[dp * 2], pa, b0, b1);
                            mma16816_bf16(oacc[dp * 2 + 1], pa, b2, b3);
                        }
                    }
                } else {
                    // 16 codes of a key transposed as pairs: a thread holds keys (2c, 2c+1) at
                    // dimensions (2g, 2g+1) of a chunk; even dimensions make one column block,
                    // odd ones the next (undone where O is written)
#pragma unroll
                    for (int qp = 0; qp < D / 32; ++qp) {
                        uint32_t x[4];
                        ldsm_x4_t(sv + swz_row<C::kRowBytes>(key, 2 * qp + (lane >> 4)), x[0], x[1], x[2], x[3]);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t e0, e1, d0, d1;
                            if constexpr (FMT == kFmtInt8) {
                                const uint32_t xa = x[2 * h] ^ 0x80808080u, xb = x[2 * h + 1] ^ 0x80808080u;
                                e0 = int8_pair(xa, 0x6240u);
                                e1 = int8_pair(xb, 0x6240u);
                                d0 = int8_pair(xa, 0x7351u);
                                d1 = int8_pair(xb, 0x7351u);
                            } else {
                                const uint32_t xa = prmt(x[2 * h], 0u, 0x3120u), xb = prmt(x[2 * h + 1], 0u, 0x3120u);
                                e0 = e4m3_pair_f16(xa);
                                e1 = e4m3_pair_f16(xb);
                                d0 = e4m3_pair_f16(xa >> 16);
                                d1 = e4m3_pair_f16(xb >> 16);
                            }
                            const int ch = 2 * qp + h;
                            mma16816(oacc[2 * ch], pa, e0, e1);
                            mma16816(oacc[2 * ch + 1], pa, d0, d1);
                        }
                    }
                }
            }
            // (the next copy into the stage writes through another proxy: behind the reads still on their way; no cost measured)
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(bar0 + 8 * (S + stg));
        }

        // ---- the slices' states meet ----
#pragma unroll
        for (int jj = 0; jj < 2; ++jj) {
            lrow[jj] += __shfl_xor_sync(0xffffffffu, lrow[jj], 1);
            lrow[jj] += __shfl_xor_sync(0xffffffffu, lrow[jj], 2);
        }
        if (c == 0) {
            sml[warp * 16 + g] = make_float2(mrow[0], lrow[0]);
            sml[warp * 16 + g + 8] = make_float2(mrow[1], lrow[1]);
        }
        // a wait that ran out, here or in the copy warp (which may say so at any time): all four warps leave
        if (bar_any(1, 128, s_abort != 0)) break;
        float M[2], L[2];
#pragma unroll
        for (int jj = 0; jj < 2; ++jj) {
            M[jj] = -INFINITY;
            L[jj] = 0.f;
#pragma unroll
            for (int s = 0; s < C::kSlices; ++s) M[jj] = fmaxf(M[jj], sml[(s * MT + mb) * 16 + g + 8 * jj].x);
#pragma unroll
            for (int s = 0; s < C::kSlices; ++s) {
                const float2 x = sml[(s * MT + mb) * 16 + g + 8 * jj];
                L[jj] += x.x == -INFINITY ? x.y : x.y * exp2f(x.x - M[jj]);   // x.y: 0, or NaN
            }
            // (one factor after the other: a small unit goes with large numerators)
            const float f = mrow[jj] == -INFINITY ? 0.f : exp2f(mrow[jj] - M[jj]), unit = FMT != kFmt16 ? fabsf(vref[jj]) : 1.f;
#pragma unroll
            for (int n = 0; n < D / 8; ++n) {
                oacc[n][2 * jj] = oacc[n][2 * jj] * unit * f;
                oacc[n][2 * jj + 1] = oacc[n][2 * jj + 1] * unit * f;
            }
        }
        // 64 columns at a time through shared memory, conflict-free
#pragma unroll
        for (int hf = 0; hf < D / 64; ++hf) {
            if (ksl > 0) {
                float *dst = sx + ((ksl - 1) * MT + mb) * 1024 + lane;
#pragma unroll
                for (int n = 0; n < 8; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) dst[(n * 4 + e) * 32] = oacc[hf * 8 + n][e];
            }
            bar_sync(1, 128);
            if (ksl == 0) {
#pragma unroll
                for (int s = 0; s < C::kSlices - 1; ++s) {
                    const float *src = sx + (s * MT + mb) * 1024 + lane;
#pragma unroll
                    for (int n = 0; n < 8; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) oacc[hf * 8 + n][e] += src[(n * 4 + e) * 32];
                }
            }
            bar_sync(1, 128);
        }
        if (ksl == 0) {
            // column of accumulator (n, e): 16-bit pages n * 8 + 2c + e; codes in the even / odd
            // order, 16 (n / 2) + 4c + 2e + (n & 1)
            const bool uncut = w.first && w.last, whole = uncut && a.level == kOnly;
            const int64_t part = ((int64_t)blockIdx.x * 2 + (w.first ? 1 : 0)) * C::kRows;
#pragma unroll
            for (int jj = 0; jj < 2; ++jj) {
                const int r = jj ? r1 : r0, f = r;
                if (f >= flat_n) continue;
                if (whole) {
                    const float inv = L[jj] > 0.f || L[jj] != L[jj] ? 1.f / L[jj] : 0.f;
                    const int tok = f / a.group, head = w.head * a.group + f - tok * a.group;
                    uint16_t *o = a.o + (int64_t)(q.row0 + tok) * a.o_rs + (int64_t)head * a.o_hs;
#pragma unroll
                    for (int n = 0; n < D / 8; n += 2) {
                        const float x0 = oacc[n][2 * jj] * inv, x1 = oacc[n][2 * jj + 1] * inv;
                        const float y0 = oacc[n + 1][2 * jj] * inv, y1 = oacc[n + 1][2 * jj + 1] * inv;
                        if constexpr (FMT == kFmt16) {
                            *reinterpret_cast<uint32_t *>(o + n * 8 + 2 * c) = pack16<T>(x0, x1);
                            *reinterpret_cast<uint32_t *>(o + n * 8 + 8 + 2 * c) = pack16<T>(y0, y1);
                        } else {
                            *reinterpret_cast<uint2 *>(o + n * 8 + 4 * c) = make_uint2(pack16<T>(x0, y0), pack16<T>(x1, y1));
                        }
                    }
                    if (a.lse && c == 0)
                        a.lse[(int64_t)(q.row0 + tok) * a.n_head + head] =
                            L[jj] == 0.f ? -INFINITY : (M[jj] + log2f(L[jj])) * 0.6931471805599453f;
                } else {
                    float *acc = a.part_acc + (part + r) * D;
                    float2 *ml = a.part_ml + part + r;
                    if (uncut) {
                        const int64_t at = (int64_t)(q.row0 + f / a.group) * a.n_head + w.head * a.group + f % a.group;
                        acc = a.level_acc + at * D;
                        ml = a.level_ml + at;
                    }
#pragma unroll
                    for (int n = 0; n < D / 8; n += 2) {
                        if constexpr (FMT == kFmt16) {
                            *reinterpret_cast<float2 *>(acc + n * 8 + 2 * c) = make_float2(oacc[n][2 * jj], oacc[n][2 * jj + 1]);
                            *reinterpret_cast<float2 *>(acc + n * 8 + 8 + 2 * c) =
                                make_float2(oacc[n + 1][2 * jj], oacc[n + 1][2 * jj + 1]);
                        } else {
                            *reinterpret_cast<float4 *>(acc + n * 8 + 4 * c) =
                                make_float4(oacc[n][2 * jj], oacc[n + 1][2 * jj], oacc[n][2 * jj + 1], oacc[n + 1][2 * jj + 1]);
                        }
                    }
                    if (c == 0) *ml = make_float2(M[jj], L[jj]);
                }
            }
            if (a.level != kOnly && w.first && threadIdx.x == 0) w.note(a);
            if (w.first && !w.last) {
                began = true;
                if (threadIdx.x == 0) a.desc[blockIdx.x] = make_int4(w.seq, w.head, w.rt, w.last_cta());
            }
        }
    }
    if (threadIdx.x == 0 && !began) a.desc[blockIdx.x] = make_int4(-1, 0, 0, 0);
    // (the second of two passes begins beside the first: what waits for it waits for both)
    if (a.level == kOwn) pdl_wait();
}

// Join of the items that a share's border cut: block (c, y) takes rows of the item that CTA c began
// and did not finish; the pieces lie in CTAs c (slot 1), c + 1, ... (slot 0).  W warps share a row's
// pieces: all eight after the streaming kernel, whose few rows are cut into many pieces (one token over
// 4,096 positions, 16 pieces and more a row: 12.6 us with the kernel before it, 16.4 with a warp a row),
// one after the tensor-core kernel, where it is the other way round.  Bound by latency: its bytes come
// out of L2, where the attention just left them.
template <int D, int T, int W>
__global__ void __launch_bounds__(256)
k_paged_join(const __grid_constant__ PagedAttendArgs a) {
    constexpr int N = D / 32;
    __shared__ float s_acc[W > 1 ? W : 1][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    const int4 d = a.desc[blockIdx.x];
    if (d.x < 0) return;
    const int r = blockIdx.y * (8 / W) + warp / W, part = warp % W;
    const PagedSeq q = paged_seq(a.batch, a.pool.page_shift, d.x);
    const int f = d.z * a.tile_rows + r;
    if (r >= a.tile_rows || f >= q.n * a.group) return;    // whole blocks with W = 8
    const int tok = f / a.group, head = d.y * a.group + f - tok * a.group;
    const int c0 = blockIdx.x, c1 = min(d.w, a.ctas - 1);
    auto slot = [&](int cc) { return ((int64_t)cc * 2 + (cc == c0 ? 1 : 0)) * a.tile_rows + r; };
    // 32 pieces' maxima and sums at a time, one to a lane
    float m = -INFINITY, l = 0.f, acc[N];
#pragma unroll
    for (int e = 0; e < N; ++e) acc[e] = 0.f;
    for (int cb = c0; cb <= c1; cb += 32) {
        const int n = min(32, c1 - cb + 1);
        const float2 ml = lane < n ? a.part_ml[slot(cb + lane)] : make_float2(-INFINITY, 0.f);
        // this warp's numerators of the 32, four at a time, on their way before the weights are known
        constexpr int PER = 32 / W, U = PER < 4 ? PER : 4;
        float x[U][N];
        auto fetch = [&](int i) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int p = part + (i + u) * W;
                if (p >= n) continue;
                const float *src = a.part_acc + slot(cb + p) * D + lane * N;
                if constexpr (N == 4) {
                    const float4 v = *reinterpret_cast<const float4 *>(src);
                    x[u][0] = v.x; x[u][1] = v.y; x[u][2] = v.z; x[u][3] = v.w;
                } else {
                    const float2 v = *reinterpret_cast<const float2 *>(src);
                    x[u][0] = v.x; x[u][1] = v.y;
                }
            }
        };
        fetch(0);
        float top = ml.x;
#pragma unroll
        for (int s = 16; s; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
        const float mnew = fmaxf(m, top);
        const float mu = mnew == -INFINITY ? 0.f : mnew;
        const float wgt = ml.x == -INFINITY ? (ml.y != ml.y ? ml.y : 0.f) : exp2f(ml.x - mu);
        float sum = ml.y * wgt;
#pragma unroll
        for (int s = 16; s; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
        const float keep = m == -INFINITY ? 0.f : exp2f(m - mu);
        l = l * keep + sum;
#pragma unroll
        for (int e = 0; e < N; ++e) acc[e] *= keep;
        m = mnew;
        for (int i = 0; part + i * W < n; i += U) {
            if (i) fetch(i);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int p = part + (i + u) * W;
                const float f4 = __shfl_sync(0xffffffffu, wgt, p & 31);
                if (p >= n) continue;
#pragma unroll
                for (int e = 0; e < N; ++e) acc[e] = fmaf(x[u][e], f4, acc[e]);
            }
        }
    }
    if constexpr (W > 1) {
#pragma unroll
        for (int e = 0; e < N; ++e) s_acc[warp][lane * N + e] = acc[e];
        __syncthreads();
        if (warp) return;
#pragma unroll
        for (int e = 0; e < N; ++e) {
            acc[e] = 0.f;
#pragma unroll
            for (int i = 0; i < W; ++i) acc[e] += s_acc[i][lane * N + e];
        }
    }
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
    uint16_t *o = a.o + (int64_t)(q.row0 + tok) * a.o_rs + (int64_t)head * a.o_hs + lane * N;
    if constexpr (N == 4)
        *reinterpret_cast<uint2 *>(o) = make_uint2(pack16<T>(acc[0] * inv, acc[1] * inv), pack16<T>(acc[2] * inv, acc[3] * inv));
    else
        *reinterpret_cast<uint32_t *>(o) = pack16<T>(acc[0] * inv, acc[1] * inv);
    if (a.lse && lane == 0)
        a.lse[(int64_t)(q.row0 + tok) * a.n_head + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// Join of two passes over a batch whose sequences share beginnings: a block takes `rows` rows of one kv head, looks
// up once per row the items that hold its states over its prefix and over its own positions, and joins all
// their pieces as k_paged_join does, `wide` warps to a (row, query head).  Bound by latency with few rows (row bounds,
// items, maxima, numerators: loads one behind another), by L2 with many; a look-up per warp and query head took
// 16 us for 64 rows of 32 heads behind 16,384 positions and 54 us for 2,048 rows, this takes 10 and 43.
template <int D, int T>
__global__ void __launch_bounds__(256)
k_paged_levels(const __grid_constant__ PagedAttendArgs prefix, const __grid_constant__ PagedAttendArgs own, int rows, int wide) {
    constexpr int N = D / 32, U = 4;
    __shared__ float s_acc[8][D];
    // a pass's pieces of a row: .y of them, the first in CTA .x; .y = 0: none, .x negative: in the level's arrays;
    // .z: the row in its item
    __shared__ int3 s_piece[2][16];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = warp % wide;
    const int kvh = own.pool.n_head_kv, hk = blockIdx.x % kvh, first = blockIdx.x / kvh * rows;
    // (what the passes do not write is looked up beside them: 1.5 of 80 us for 64 rows)
    const int level = threadIdx.x / rows, mine = threadIdx.x % rows;
    const PagedAttendArgs &a = level ? own : prefix;
    int64_t item = -1;
    int3 piece = make_int3(0, 0, 0);
    const int row = first + mine;
    // whether the row is one of sequence s
    auto is_of = [&](int s) {
        const PagedSeq q = paged_seq(a.batch, a.pool.page_shift, s, level == 0);
        if (!q.ok || q.n > a.max_q || row < q.row0 || row >= q.row0 + q.n) return false;
        const int tok = row - q.row0, rt = tok / a.tile_tokens;
        if (q.kv > 0) item = (int64_t)(q.row0 + rt * a.tile_tokens) * kvh + hk;
        piece.z = (tok - rt * a.tile_tokens) * a.group;
        return true;
    };
    bool found = level >= 2;
    if (level < 2) {
        // the last sequence that begins at the row or in front of it
        int s = 0, end = a.batch.n_seq;
        while (end - s > 1) {
            const int mid = (s + end) >> 1;
            if (a.batch.q_start[mid] <= row) s = mid;
            else end = mid;
        }
        found = is_of(s);
    }
    pdl_wait();
    // (where bounds decrease the search may miss the row's sequence: one after the other then)
    if (!found && *a.level_broken)
        for (int s = 0; s < a.batch.n_seq && !is_of(s); ++s) {
        }
    if (level < 2) {
        if (item >= 0) {
            const int2 c = a.level_items[item];
            // (in range, should the pass have given up)
            piece.x = c.y < 0 ? -1 : min(max(c.x, 0), a.ctas - 1);
            piece.y = c.y < 0 ? 1 : max(1, min(c.y, a.ctas - 1) - piece.x + 1);
        }
        s_piece[level][mine] = piece;
    }
    __syncthreads();
    for (int u0 = 0; u0 < rows * own.group; u0 += 8 / wide) {
        const int u = u0 + warp / wide, i = min(u / own.group, rows - 1), hh = u % own.group, row = first + i;
        const int3 pp = s_piece[0][i], po = s_piece[1][i];
        // (po.y = 0: not in the batch, or left alone)
        const int total = u < rows * own.group && po.y ? pp.y + po.y : 0;
        const int64_t at = (int64_t)row * own.n_head + hk * own.group + hh;
        // where piece k is: numerators (of a lane) or maximum and sum
        auto slot = [&](int k, bool &cut, bool &mine) {
            mine = k >= pp.y;
            const int3 p = mine ? po : pp;
            if (mine) k -= pp.y;
            cut = p.x >= 0;
            return cut ? ((int64_t)(p.x + k) * 2 + (k == 0 ? 1 : 0)) * (mine ? own.tile_rows : prefix.tile_rows) + p.z + hh : at;
        };
        float m = -INFINITY, l = 0.f, acc[N];
#pragma unroll
        for (int e = 0; e < N; ++e) acc[e] = 0.f;
        for (int base = 0; base < total; base += 32) {
            const int n = min(32, total - base);
            float2 ml = make_float2(-INFINITY, 0.f);
            if (lane < n) {
                bool cut, mine;
                const int64_t to = slot(base + lane, cut, mine);
                ml = (mine ? (cut ? own.part_ml : own.level_ml) : (cut ? prefix.part_ml : prefix.level_ml))[to];
            }
            float x[U][N];
            auto fetch = [&](int k) {
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    const int p = part + (k + j) * wide;
                    if (p >= n) continue;
                    bool cut, mine;
                    const int64_t to = slot(base + p, cut, mine);
                    const float *src = (mine ? (cut ? own.part_acc : own.level_acc) : (cut ? prefix.part_acc : prefix.level_acc)) + to * D + lane * N;
                    if constexpr (N == 4) {
                        const float4 v = *reinterpret_cast<const float4 *>(src);
                        x[j][0] = v.x; x[j][1] = v.y; x[j][2] = v.z; x[j][3] = v.w;
                    } else {
                        const float2 v = *reinterpret_cast<const float2 *>(src);
                        x[j][0] = v.x; x[j][1] = v.y;
                    }
                }
            };
            fetch(0);
            float top = ml.x;
#pragma unroll
            for (int s = 16; s; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
            const float mnew = fmaxf(m, top);
            const float mu = mnew == -INFINITY ? 0.f : mnew;
            const float wgt = ml.x == -INFINITY ? (ml.y != ml.y ? ml.y : 0.f) : exp2f(ml.x - mu);
            float sum = ml.y * wgt;
#pragma unroll
            for (int s = 16; s; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
            const float keep = m == -INFINITY ? 0.f : exp2f(m - mu);
            l = l * keep + sum;
#pragma unroll
            for (int e = 0; e < N; ++e) acc[e] *= keep;
            m = mnew;
            for (int k = 0; part + k * wide < n; k += U) {
                if (k) fetch(k);
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    const int p = part + (k + j) * wide;
                    const float f4 = __shfl_sync(0xffffffffu, wgt, p & 31);
                    if (p >= n) continue;
#pragma unroll
                    for (int e = 0; e < N; ++e) acc[e] = fmaf(x[j][e], f4, acc[e]);
                }
            }
        }
        if (wide > 1) {
            if (u0) __syncthreads();
#pragma unroll
            for (int e = 0; e < N; ++e) s_acc[warp][lane * N + e] = acc[e];
            __syncthreads();
            if (part) continue;
            for (int w = 1; w < wide; ++w)
#pragma unroll
                for (int e = 0; e < N; ++e) acc[e] += s_acc[warp + w][lane * N + e];
        }
        if (total == 0) continue;
        const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
        uint16_t *o = own.o + (int64_t)row * own.o_rs + (int64_t)(hk * own.group + hh) * own.o_hs + lane * N;
        if constexpr (N == 4)
            *reinterpret_cast<uint2 *>(o) = make_uint2(pack16<T>(acc[0] * inv, acc[1] * inv), pack16<T>(acc[2] * inv, acc[3] * inv));
        else
            *reinterpret_cast<uint32_t *>(o) = pack16<T>(acc[0] * inv, acc[1] * inv);
        if (own.lse && lane == 0) own.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
    }
}

}  // namespace dflash
