// Head rows on their way into and out of a paged cache: RMS norm and position rotation
// (paged_norm_rope), the same with quantisation and the scatter into pages (paged_append),
// and the way back (paged_gather).
//
// A row is one head of one token: head_dim values, eight to a lane (16 bytes of a 16-bit
// type), so 16 lanes hold a row of 128 and a warp two of them.  A warp's task is one token
// and a run of its query, key or value heads; everything that belongs to the token (its
// sequence, position, page, and the cosines and sines of its angles) is worked out once per
// task and serves all the heads of it.
//
// Angles: position times frequency, less whole turns.  A frequency is held as turns per
// position in units of 2^-64, so the product's whole turns fall off the top of a 64-bit
// integer multiplication, exactly, and float32 sees only the rest (at most half a turn, in two parts):
// no float64 and no large arguments, for any position.
//
// Bytes are all that these operators cannot do without, each read and written once.  Measured, 32 query
// and 8 kv heads of 128: norm and rotation of 16,384 bf16 tokens 67 us (5.0 TB/s, 74 % of the copy
// rate); 22,600 F16 tokens to int8 and back 69 us (4.0 TB/s); 270,000 tokens back from e4m3 286 us (5.9
// TB/s, 88 %).  What holds them is instructions and their latency together: 0.64 to 0.74 a clock and scheduler
// with 33 to 45 % of the warps, and nothing of a warp's next steps in flight while it works on these; when
// quantising, two divisions a row on every lane of it besides.  Small calls (a verify block, 64 of them) are bound by the host's call, 7 to 9 us.
#include "paged.h"
#include "paged_ptx.h"

#include <algorithm>
#include <type_traits>

namespace dflash {
namespace {

constexpr int kRowThreads = 128, kRowBlocks = 6, kGatherBlocks = 8;

template <int T> struct RowType;
template <> struct RowType<PAGED_F16> { using type = __half; };
template <> struct RowType<PAGED_BF16> { using type = __nv_bfloat16; };
template <> struct RowType<PAGED_F32> { using type = float; };

// Eight consecutive values as loaded (one or two 16-byte words).
template <int T> struct Raw8 { uint4 w[T == PAGED_F32 ? 2 : 1]; };

template <int T>
__device__ __forceinline__ Raw8<T> load8(const void *base, int64_t elem) {
    Raw8<T> r;
    const uint4 *p = reinterpret_cast<const uint4 *>(reinterpret_cast<const typename RowType<T>::type *>(base) + elem);
    r.w[0] = __ldcs(p);
    if constexpr (T == PAGED_F32) r.w[1] = __ldcs(p + 1);
    return r;
}

__device__ __forceinline__ float2 unpack2(uint32_t w, std::integral_constant<int, PAGED_F16>) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
__device__ __forceinline__ float2 unpack2(uint32_t w, std::integral_constant<int, PAGED_BF16>) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack2(float a, float b, std::integral_constant<int, PAGED_F16>) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, std::integral_constant<int, PAGED_BF16>) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

template <int T>
__device__ __forceinline__ void widen(const Raw8<T> &r, float (&x)[8]) {
    if constexpr (T == PAGED_F32) {
        const float *f = reinterpret_cast<const float *>(&r);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = f[e];
    } else {
        const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 f = unpack2(w[e], std::integral_constant<int, T>{});
            x[2 * e] = f.x;
            x[2 * e + 1] = f.y;
        }
    }
}

template <int T>
__device__ __forceinline__ void store8(void *base, int64_t elem, const float (&x)[8]) {
    uint4 *p = reinterpret_cast<uint4 *>(reinterpret_cast<typename RowType<T>::type *>(base) + elem);
    if constexpr (T == PAGED_F32) {
        p[0] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
        p[1] = make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7]));
    } else {
        const std::integral_constant<int, T> t{};
        *p = make_uint4(pack2(x[0], x[1], t), pack2(x[2], x[3], t), pack2(x[4], x[5], t), pack2(x[6], x[7], t));
    }
}

__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// Where row t lives: its sequence (the last s with q_start[s] <= t) and position, and the page and
// row in it; found false for a row in front of the first or behind the last sequence, mapped false
// where the arrays name no place for it.  A lane loads all that belongs to a sequence, 32 sequences
// at a time, so that only the page number has to wait for another load.
struct Place {
    bool found, mapped;
    int pos, page, slot;
};
__device__ __forceinline__ Place place_of(const PagedBatchDev &b, const PagedPool &pool, int t, int lane) {
    int count = 0, r0 = 0, r1 = 0, kv = 0;
    for (int i = 0; i < b.n_seq; i += 32) {
        const bool in = i + lane < b.n_seq;
        const int x0 = in ? b.q_start[i + lane] : 0x7fffffff, x1 = in ? b.q_start[i + lane + 1] : 0, x2 = in ? b.kv_len[i + lane] : 0;
        const int n = __popc(__ballot_sync(0xffffffffu, x0 <= t));
        if (n) {
            r0 = x0;
            r1 = x1;
            kv = x2;
        }
        count += n;
    }
    Place p{};
    if (count == 0) return p;
    const int s = count - 1;
    r0 = __shfl_sync(0xffffffffu, r0, s & 31);
    r1 = __shfl_sync(0xffffffffu, r1, s & 31);
    kv = __shfl_sync(0xffffffffu, kv, s & 31);
    if (r0 > t || t >= r1) return p;
    p.found = true;
    const int64_t cap = (int64_t)b.max_pages << pool.page_shift, n = (int64_t)r1 - r0;
    p.pos = (int)(kv - n + (t - r0));
    p.mapped = r0 >= 0 && r1 <= b.n_rows && kv >= n && kv <= cap;
    if (p.mapped) {
        p.page = b.pages[(int64_t)s * b.pages_stride + (p.pos >> pool.page_shift)];
        p.slot = p.pos & ((1 << pool.page_shift) - 1);
        p.mapped = p.page >= 0 && p.page < pool.n_pages;
    }
    return p;
}

// cos and sin (times the magnitude) of p * turn, turn in 2^-64 turns.  The angle's top 20 bits are exact
// in float32; the other 12, at most 6e-6, follow by the derivative (a float32 angle would be off by up to
// 1e-7: of 226 million e4m3 codes 13 fell on the other side of a rounding border that way, 8 this way).
__device__ __forceinline__ float2 turn_cs(int p, uint64_t turn, float magnitude) {
    const int32_t frac = (int32_t)((uint64_t)(int64_t)p * turn >> 32);   // whole turns gone
    const float low = (float)(frac & 0xfff) * 1.4629180792671596e-9f;    // pi 2^-31
    float sn, cs;
    sincospif((float)(frac & ~0xfff) * 0x1p-31f, &sn, &cs);
    return make_float2(fmaf(-sn, low, cs) * magnitude, fmaf(cs, low, sn) * magnitude);
}

// Norm and rotation of one row spread over LPR lanes (lane c: values 8c .. 8c+7).  With inv =
// 1 / sqrt(mean(x^2) + eps) and x' an element's partner in its pair, both steps together are
//   y = inv (x A + x' B),   A = w cos,  B = -+ w' sin  (A = w, B = 0 where nothing turns),
// whose A and B belong to the token and the kind of head, not to the head.
template <int T, int D>
struct Turner {
    static constexpr int LPR = D / 8;
    float A[8], B[8];
    int c, shift;            // shift: lanes to the partner's (half layout; 0: in this lane, or none)
    bool norm, turns;        // turns: this lane's elements do

    // A and B at position p under weights wt (worked out anew for queries and keys: the cosines kept
    // between the two would spill)
    __device__ __forceinline__ void prepare(const PagedRowsArgs &a, const float *wt, int p, int lane) {
        norm = wt != nullptr;
        float w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = 1.f;
        if (norm) {
            const float4 x = reinterpret_cast<const float4 *>(wt)[2 * c], y = reinterpret_cast<const float4 *>(wt)[2 * c + 1];
            w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
            w[4] = y.x; w[5] = y.y; w[6] = y.z; w[7] = y.w;
        }
        const int e0 = 8 * c, half = a.rot / 2;
        const bool halves = a.layout == PAGED_HALF, first = e0 < half;
        turns = e0 < a.rot;
        shift = !turns || !halves ? 0 : (first ? half / 8 : -(half / 8));
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float far = __shfl_sync(0xffffffffu, w[e], lane + shift);
            B[e] = halves ? far : w[e ^ 1];
        }
        if (!turns) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                A[e] = w[e];
                B[e] = 0.f;
            }
        } else if (halves) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float2 r = turn_cs(p, a.turn[(first ? e0 : e0 - half) + e], a.magnitude);
                A[e] = w[e] * r.x;
                B[e] *= first ? -r.y : r.y;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 r = turn_cs(p, a.turn[e0 / 2 + e], a.magnitude);
                A[2 * e] = w[2 * e] * r.x;
                A[2 * e + 1] = w[2 * e + 1] * r.x;
                B[2 * e] *= -r.y;
                B[2 * e + 1] *= r.y;
            }
        }
    }
    __device__ __forceinline__ void apply(const PagedRowsArgs &a, const Raw8<T> &raw, float (&y)[8], int lane) const {
        float x[8];
        widen(raw, x);
        float inv = 1.f;
        if (norm) {
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
            for (int d = LPR / 2; d; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
            inv = rsqrtf(ss * (1.f / D) + a.eps);
        }
        if (a.rot == 0) {
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = x[e] * A[e] * inv;
        } else if (a.layout == PAGED_HALF) {
            Raw8<T> far = raw;
            uint32_t *f = reinterpret_cast<uint32_t *>(&far);
#pragma unroll
            for (int e = 0; e < (T == PAGED_F32 ? 8 : 4); ++e) f[e] = __shfl_sync(0xffffffffu, f[e], lane + shift);
            if (!turns) far = Raw8<T>{};                   // (an infinity times 0)
            float z[8];
            widen(far, z);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = fmaf(z[e], B[e], x[e] * A[e]) * inv;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = fmaf(turns ? x[e ^ 1] : 0.f, B[e], x[e] * A[e]) * inv;
        }
    }
};

// Eight values per lane of a row that is LPR lanes, quantised: codes and the row's scale.
// top: the largest magnitude's bits among this lane's values (as integers, magnitudes order as the
// floats do, and infinities and NaN are above all).
template <int LPR>
__device__ __forceinline__ uint2 quantise(const float (&x)[8], uint32_t top, bool int8, float *scale) {
#pragma unroll
    for (int d = LPR / 2; d; d >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
    const float full = int8 ? 127.f : 448.f;
    const float amax = __uint_as_float(top);
    const bool finite = top < 0x7f800000u, any = amax >= 1e-30f;
    const float inv = any && finite ? full / amax : 0.f;
    *scale = !finite ? __int_as_float(0x7fc00000) : (any ? amax / full : 0.f);
    uint2 w = make_uint2(0u, 0u);
    if (int8) {
        // |x inv| <= 127 + 2^-16: adding 1.5 2^23 leaves the code, rounded to even, in the low byte
        uint32_t b[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) b[e] = __float_as_uint(__fadd_rn(__fmul_rn(x[e], inv), 12582912.f));
        w.x = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
        w.y = __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
    } else {
        w.x = e4m3_pair(x[0] * inv, x[1] * inv) | e4m3_pair(x[2] * inv, x[3] * inv) << 16;
        w.y = e4m3_pair(x[4] * inv, x[5] * inv) | e4m3_pair(x[6] * inv, x[7] * inv) << 16;
    }
    if (!finite) w = make_uint2(0u, 0u);
    return w;
}

template <int T>
__device__ __forceinline__ uint32_t largest(const Raw8<T> &raw, const float (&x)[8], bool same) {
    uint32_t top = 0;
    if (T != PAGED_F32 && same) {
        // the values are the raw ones: two 16-bit magnitudes at a time
        const uint32_t m = 0x7fff7fffu;
        const uint32_t a = __vimax3_u16x2(raw.w[0].x & m, raw.w[0].y & m, raw.w[0].z & m);
        const uint32_t b = __vimax3_u16x2(a, raw.w[0].w & m, 0u);
        const uint32_t h = max(b & 0xffffu, b >> 16);
        if constexpr (T == PAGED_BF16) return h << 16;
        return __float_as_uint(__half2float(__ushort_as_half((unsigned short)h)));
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[e]) & 0x7fffffffu);
    return top;
}

// A warp step is RPW rows of one kind (queries, keys, values) of one token; a token's steps are laid
// end to end and a task is `iters` of them, all of them where there are tokens enough.  With plenty of
// tokens what a warp issues counts (about 0.7 instructions a clock and scheduler), so a
// step's addresses are two additions, and each kind has a loop of its own.
template <int T, int D, bool PAGED>
__global__ void __launch_bounds__(kRowThreads, kRowBlocks)
k_paged_rows(const __grid_constant__ PagedRowsArgs a) {
    using E = typename RowType<T>::type;
    constexpr int LPR = D / 8, RPW = 32 / LPR, U = 4;      // rows a warp step, steps in flight
    const int lane = threadIdx.x & 31;
    // (tokens times tasks stay below 2^31: several tasks a token only while they fit a wave)
    const uint32_t gw = blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
    const int t = (int)(gw / (uint32_t)a.tasks);
    if (t >= a.n_rows) return;
    const int s0 = (int)(gw - (uint32_t)t * a.tasks) * a.iters, s1 = min(a.steps_q + a.steps_k + a.steps_v, s0 + a.iters);
    const int sub = lane / LPR, c = lane % LPR;

    // one kind's steps of this task: [from, to) of the kind's own
    struct Run {
        const E *src;
        int64_t stride;      // per step
        int from, to, heads;
    };
    auto run_of = [&](const void *base, int64_t rs, int64_t hs, int before, int steps, int heads) {
        Run r;
        r.from = max(0, s0 - before);
        r.to = min(steps, s1 - before);
        r.heads = heads;
        r.stride = (int64_t)RPW * hs;
        r.src = reinterpret_cast<const E *>(base) + (int64_t)t * rs + (int64_t)(r.from * RPW + sub) * hs + 8 * c;
        return r;
    };
    Raw8<T> raw[U];
    auto load = [&](const Run &r, int st) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            raw[u] = Raw8<T>{};
            if (st + u < r.to && (st + u) * RPW + sub < r.heads) raw[u] = load8<T>(r.src, (int64_t)(st + u - r.from) * r.stride);
        }
    };
    const Run rq = run_of(a.q, a.q_rs, a.q_hs, 0, a.steps_q, a.nq);
    const Run rk = run_of(a.k, a.k_rs, a.k_hs, a.steps_q, a.steps_k, a.nk);
    const Run rv = run_of(a.v, a.v_rs, a.v_hs, a.steps_q + a.steps_k, a.steps_v, a.nv);

    // the first rows are on their way while the token's place is looked up
    if (rq.from < rq.to) load(rq, rq.from);
    else if (rk.from < rk.to) load(rk, rk.from);
    else load(rv, rv.from);
    bool loaded = true;

    int pos = 0;
    bool mapped = true;
    int64_t off = 0, soff = 0;
    if constexpr (PAGED) {
        const Place at = place_of(a.batch, a.pool, t, lane);
        if (!at.found) return;
        pos = at.pos;
        mapped = at.mapped;
        off = (int64_t)at.page * a.pool.page_stride + at.slot * a.pool.row_stride;
        soff = (int64_t)at.page * a.pool.s_page_stride + at.slot;
        if (!mapped && lane == 0) atomicOr(a.err, (uint32_t)PAGED_ERR_PAGE);
    }
    const int at = a.rot && a.positions ? a.positions[t] : pos;
    Turner<T, D> tr;
    tr.c = c;

    // steps of one kind, fn(row's head, raw, values, turned)
    auto walk = [&](const Run &r, bool turned, const float *wt, auto &&fn) {
        if (r.from >= r.to) return;
        if (turned) tr.prepare(a, wt, at, lane);
        for (int st = r.from; st < r.to; st += U) {
            if (!loaded) load(r, st);
            loaded = false;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (st + u >= r.to) break;                 // uniform over the warp
                float y[8];
                if (turned) tr.apply(a, raw[u], y, lane);
                else widen(raw[u], y);
                fn((st + u) * RPW + sub, raw[u], y);
            }
        }
    };
    const bool q_turns = a.rot || a.q_norm, k_turns = a.rot || a.k_norm;
    {
        E *dst = reinterpret_cast<E *>(a.qo) + (int64_t)t * a.qo_rs + 8 * c;
        walk(rq, q_turns, a.q_norm, [&](int h, const Raw8<T> &, const float (&y)[8]) {
            if (h < a.nq) store8<T>(dst, (int64_t)h * a.qo_hs, y);
        });
    }
    if constexpr (!PAGED) {
        E *dst = reinterpret_cast<E *>(a.ko) + (int64_t)t * a.ko_rs + 8 * c;
        walk(rk, k_turns, a.k_norm, [&](int h, const Raw8<T> &, const float (&y)[8]) {
            if (h < a.nk) store8<T>(dst, (int64_t)h * a.ko_hs, y);
        });
    } else {
        const bool wide = a.pool.format == PAGED_F16 || a.pool.format == PAGED_BF16, int8 = a.pool.format == PAGED_INT8;
        auto put = [&](uint8_t *pool, float *scales, bool turned) {
            return [=, &a](int h, const Raw8<T> &raw, const float (&y)[8]) {
                const bool live = h < a.nk && mapped;
                const int64_t e = off + (int64_t)h * a.pool.head_stride + 8 * c;
                if (wide) {
                    if (live) store8<T>(pool, e, y);
                    return;
                }
                float scale;
                const uint2 w = quantise<LPR>(y, largest<T>(raw, y, !turned), int8, &scale);
                if (live) {
                    *reinterpret_cast<uint2 *>(pool + e) = w;
                    if (c == 0) scales[soff + (int64_t)h * a.pool.s_head_stride] = scale;
                }
            };
        };
        walk(rk, k_turns, a.k_norm, put(a.pool.k, a.pool.ks, k_turns));
        walk(rv, false, nullptr, put(a.pool.v, a.pool.vs, false));
    }
}

// Rows of K and V read back: the same split of lanes and tasks over a token's K steps, then V steps.
template <int T, int D>
__global__ void __launch_bounds__(kRowThreads, kGatherBlocks)
k_paged_gather(const __grid_constant__ PagedGatherArgs a) {
    using E = typename RowType<T>::type;
    constexpr int LPR = D / 8, RPW = 32 / LPR, U = 4;
    const int lane = threadIdx.x & 31;
    const uint32_t gw = blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
    const int t = (int)(gw / (uint32_t)a.chunks);
    if (t >= a.batch.n_rows) return;
    const Place at = place_of(a.batch, a.pool, t, lane);
    if (!at.found) return;
    if (!at.mapped && lane == 0) atomicOr(a.err, (uint32_t)PAGED_ERR_PAGE);
    const int sub = lane / LPR, c = lane % LPR;
    const int s0 = (int)(gw - (uint32_t)t * a.chunks) * a.iters, s1 = min(2 * a.steps, s0 + a.iters);
    const int64_t off = (int64_t)at.page * a.pool.page_stride + at.slot * a.pool.row_stride + 8 * c;
    const int64_t soff = (int64_t)at.page * a.pool.s_page_stride + at.slot;
    const bool wide = a.pool.format == PAGED_F16 || a.pool.format == PAGED_BF16, int8 = a.pool.format == PAGED_INT8;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        const int from = max(0, s0 - kv * a.steps), to = min(a.steps, s1 - kv * a.steps), h0 = from * RPW + sub;
        const int64_t in_stride = (int64_t)RPW * a.pool.head_stride, sc_stride = (int64_t)RPW * a.pool.s_head_stride;
        const int64_t out_hs = kv ? a.v_hs : a.k_hs;
        const int64_t in0 = off + (int64_t)h0 * a.pool.head_stride;
        const uint8_t *src = (kv ? a.pool.v : a.pool.k) + (wide ? 2 * in0 : in0);
        const float *scales = (kv ? a.pool.vs : a.pool.ks) + soff + (int64_t)h0 * a.pool.s_head_stride;
        E *dst = reinterpret_cast<E *>(kv ? a.v : a.k) + (int64_t)t * (kv ? a.v_rs : a.k_rs) + (int64_t)h0 * out_hs + 8 * c;
        for (int st = from; st < to; st += U) {
            uint4 w[U];
            float sc[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int n = st + u - from;
                w[u] = make_uint4(0, 0, 0, 0);
                sc[u] = 0.f;
                if (st + u < to && h0 + n * RPW < a.pool.n_head_kv && at.mapped) {
                    if (wide) {
                        w[u] = __ldcs(reinterpret_cast<const uint4 *>(src + 2 * n * in_stride));
                    } else {
                        const uint2 x = __ldcs(reinterpret_cast<const uint2 *>(src + n * in_stride));
                        w[u].x = x.x;
                        w[u].y = x.y;
                        sc[u] = __ldg(scales + n * sc_stride);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int n = st + u - from;
                if (st + u >= to || h0 + n * RPW >= a.pool.n_head_kv) continue;
                if (wide) {
                    *reinterpret_cast<uint4 *>(dst + (int64_t)n * RPW * out_hs) = w[u];
                    continue;
                }
                float x[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t v = i < 2 ? w[u].x : w[u].y;
                    const uint32_t h = int8 ? int8_pair(v ^ 0x80808080u, i & 1 ? 0x7362u : 0x5140u) : e4m3_pair_f16(v >> (16 * (i & 1)));
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
                    x[2 * i] = f.x * sc[u];
                    x[2 * i + 1] = f.y * sc[u];
                }
                store8<T>(dst, (int64_t)n * RPW * out_hs, x);
            }
        }
    }
}

// Tasks per token: as many as fill one wave of `warps`, at most one per warp step, each of as near
// the same number of steps as can be.  Few tokens: single steps, or the few that keep the grid within
// the wave, since latency counts; many: whole tokens, whose angles are then worked out once.
int tasks_per_token(int64_t tokens, int steps, int warps) {
    return (int)std::max<int64_t>(1, std::min<int64_t>(steps, warps / std::max<int64_t>(tokens, 1)));
}

int sm_count() {
    int dev = 0, sms = 1;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms;
}

template <int T, int D>
cudaError_t rows_t(PagedRowsArgs a, bool paged, cudaStream_t st) {
    constexpr int rpw = 32 / (D / 8);
    a.steps_q = (a.nq + rpw - 1) / rpw;
    a.steps_k = (a.nk + rpw - 1) / rpw;
    a.steps_v = (a.nv + rpw - 1) / rpw;
    const int steps = a.steps_q + a.steps_k + a.steps_v;
    a.tasks = tasks_per_token(a.n_rows, steps, sm_count() * kRowBlocks * (kRowThreads / 32));
    a.iters = (steps + a.tasks - 1) / a.tasks;
    a.tasks = (steps + a.iters - 1) / a.iters;
    const int64_t warps = a.n_rows * a.tasks;
    const int64_t blocks = (warps + kRowThreads / 32 - 1) / (kRowThreads / 32);
    if (blocks <= 0) return cudaSuccess;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    if (paged) {
        if constexpr (T != PAGED_F32) k_paged_rows<T, D, true><<<(unsigned)blocks, kRowThreads, 0, st>>>(a);
    } else {
        k_paged_rows<T, D, false><<<(unsigned)blocks, kRowThreads, 0, st>>>(a);
    }
    return cudaGetLastError();
}

template <int T, int D>
cudaError_t gather_t(PagedGatherArgs a, cudaStream_t st) {
    constexpr int rpw = 32 / (D / 8);
    a.steps = (a.pool.n_head_kv + rpw - 1) / rpw;
    const int steps = 2 * a.steps;
    a.chunks = tasks_per_token(a.batch.n_rows, steps, sm_count() * kGatherBlocks * (kRowThreads / 32));
    a.iters = (steps + a.chunks - 1) / a.chunks;
    a.chunks = (steps + a.iters - 1) / a.iters;
    const int64_t warps = a.batch.n_rows * a.chunks;
    const int64_t blocks = (warps + kRowThreads / 32 - 1) / (kRowThreads / 32);
    if (blocks <= 0) return cudaSuccess;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    k_paged_gather<T, D><<<(unsigned)blocks, kRowThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_rows(const PagedRowsArgs &a, int dtype, int head_dim, bool paged, cudaStream_t st) {
    switch (dtype * 1000 + head_dim) {
    case PAGED_F16 * 1000 + 64: return rows_t<PAGED_F16, 64>(a, paged, st);
    case PAGED_F16 * 1000 + 128: return rows_t<PAGED_F16, 128>(a, paged, st);
    case PAGED_BF16 * 1000 + 64: return rows_t<PAGED_BF16, 64>(a, paged, st);
    case PAGED_BF16 * 1000 + 128: return rows_t<PAGED_BF16, 128>(a, paged, st);
    case PAGED_F32 * 1000 + 64: return rows_t<PAGED_F32, 64>(a, paged, st);
    case PAGED_F32 * 1000 + 128: return rows_t<PAGED_F32, 128>(a, paged, st);
    }
    return cudaErrorInvalidValue;
}

cudaError_t launch_paged_gather(const PagedGatherArgs &a, int dtype, int head_dim, cudaStream_t st) {
    switch (dtype * 1000 + head_dim) {
    case PAGED_F16 * 1000 + 64: return gather_t<PAGED_F16, 64>(a, st);
    case PAGED_F16 * 1000 + 128: return gather_t<PAGED_F16, 128>(a, st);
    case PAGED_BF16 * 1000 + 64: return gather_t<PAGED_BF16, 64>(a, st);
    case PAGED_BF16 * 1000 + 128: return gather_t<PAGED_BF16, 128>(a, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace dflash
