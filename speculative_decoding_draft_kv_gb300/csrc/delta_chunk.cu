// The gated delta rule over many tokens: 32 at a time, as matrix products.
//
// With G_i the sum of a chunk's log decays up to token i, S the state in front of the chunk, and every
// sum over tokens of the chunk, the recurrence's updates are the solution of a triangular system,
//   u_i = beta_i (v_i - exp(G_i) S k_i) - sum_{j<i} beta_i exp(G_i - G_j) (k_i . k_j) u_j,
// so U = T R with R = beta (V - exp(G) K S^T) and T the inverse of a unit lower triangular 32 x 32 matrix
// that does not depend on S.  Then
//   o_i = exp(G_i) S q_i + sum_{j<=i} exp(G_i - G_j) (q_i . k_j) u_j,
//   S  <- exp(G_last) S + sum_j u_j (exp(G_last - G_j) k_j)^T.
//
// k_delta_prep does what the state is not needed for, all chunks at once: norms, keys and queries as F16
// tiles, k . k and q . k, decays, T.  k_delta_scan walks a sequence's chunks with the state in registers.
// A warp has 16 value elements (rows of S) and shares nothing with the others: S as the A operand of
// S [K Q]^T, U of U T^T, U A^T and U K, are accumulators of the product before, in the same layout
// (mma.sync m16n8k16: its accumulators feed the next product without leaving the thread).  A form on tcgen05.mma, with
// 128 value elements as rows and the left operands in tensor memory, was built too: there a product of 16 steps along K
// takes some 98 cycles whatever its columns, 32 or 64, and a chunk has 40 of them and three hand-overs to the threads
// and back, 4,900 cycles for a head's chunk and SM.  It took 552 us for eight prompts and 1,136 for 48 heads of
// 14,142 tokens, which took 533 and 972 here then (546 and 950 now).  Chunks of more tokens, which would spread a product's
// time over more columns, were not tried.
//
// Bound by the walk's chain: a chunk of a head of 128 x 128 takes two warps to a group 1.3 us when they have the SM to
// themselves, two CTAs with a warp to a group 3.3 us for both, of which the tensor pipe is busy about half.
//
// Precision.  The state, its update and all sums are float32.  Operands are F16 pairs hi + lo, 22 bits together,
// after powers of two that bring them below 2^15.  Rows of S never meet, so each has units of its own, whatever its neighbours
// hold (a unit for a warp's 16 rows cost a row 2^-16 of its neighbour all but ten bits; eight prompts 530 us so, 544 now, one
// prompt 728 and 762): the state is kept times its unit, by a bound that each chunk's sum of exp(G_last - G) |u| moves and that is
// set right every eighth chunk; R's is by the row's largest of the chunk, and where a token's is 2^10 or more below that it loses
// bits, ending at 2^-30 of the largest; U's by R's and T's largest row sum.  Keys and queries
// are one F16 each, after a power of two by the row's norm: exact but for elements below 2^-14 of the norm, which
// are off by 2^-25 of it at most.  What a product adds up starts at zero and joins the state by one fused
// multiply-add: tensor-core sums are cut off, not rounded, and hundreds of chunks would add that up.  Decays are
// exponentials of sums over just the tokens between, so neither a long sequence nor a state that was dropped in front of
// their chunk costs later tokens their precision.
#include "delta.h"

#include "ring_internal.h"
#include "ptx.h"
#include "paged_ptx.h"

#include <algorithm>
#include <type_traits>

namespace dflash {
namespace {

constexpr int C = kDeltaChunk;                         // tokens of a chunk
static_assert(C == 32, "a lane per token");

template <int T> __device__ __forceinline__ float from16(uint32_t x) {
    if constexpr (T == PAGED_F16) return __half2float(__ushort_as_half((unsigned short)x));
    else return __uint_as_float(x << 16);
}
__device__ __forceinline__ float2 half2_floats(uint32_t x) { return __half22float2(*reinterpret_cast<const __half2 *>(&x)); }

// Byte offset of 16-byte chunk ch of row r in a tile of 32 rows of F16: runs of 64 columns one behind another, with the
// 128-byte swizzle, conflict-free for ldmatrix along rows as along columns.
__device__ __forceinline__ uint32_t tile_at(int r, int ch) { return (uint32_t)((ch >> 3) * C * 128 + r * 128 + (((ch & 7) ^ (r & 7)) << 4)); }

// Of T or A, the (token tile, key step) blocks with something in them, in the order of use.
constexpr int kBlocks = 6;
__host__ __device__ constexpr int block_n(int b) { return b < 4 ? b : b - 2; }     // 0 1 2 3 2 3
__host__ __device__ constexpr int block_k(int b) { return b < 4 ? 0 : 1; }

// What a head's chunk needs beside T and A.
struct HeadScalars {
    float4 r[C / 2];                                   // of tokens 2i, 2i+1: beta twice, -beta exp(G) |k| twice
    float4 o[C / 2];                                   // |q| twice, |q| exp(G) twice
    float w[C];                                        // exp(G_last - G) |k|
    float last, t_unit, a_unit, unused;                // exp(G_last); what T and A are to be multiplied by
};
// A head's part of a chunk in the workspace, for mma.sync: B operands of T and of A (exp(G_i - G_j) q_i . k_j), a lane's
// words beside one another (hi, hi, lo, lo).
struct HeadBlock {
    uint4 t[kBlocks][32], a[kBlocks][32];
    HeadScalars s;
};
static_assert(sizeof(HeadBlock) == kDeltaHeadBytes, "as the workspace is laid out");

// the power of two that brings m > 0 (as bits) to [2^12, 2^13), if that is 2^-115 to 2^115
__device__ __forceinline__ float unit_of(uint32_t bits) {
    const int e = (int)(bits >> 23);                   // biased
    return bits == 0u || e == 255 ? 1.f : __uint_as_float((uint32_t)min(242, max(12, 254 + 12 - e)) << 23);
}
// the same for m of kLeast to infinity
constexpr float kLeast = 0x1p-103f;
__device__ __forceinline__ float unit_above(float m) { return __uint_as_float((266u << 23) - (__float_as_uint(m) & 0x7f800000u)); }
__device__ __forceinline__ float inverse_unit(float u) { return __uint_as_float((254u << 23) - __float_as_uint(u)); }

// x0, x1 as two F16 pairs
__device__ __forceinline__ void split(float x0, float x1, uint32_t &hi, uint32_t &lo) {
    hi = pack_half2(x0, x1);
    const float2 h = half2_floats(hi);
    float l0, l1;
    upk2(fma2(pk2(h.x, h.y), pk2(-1.f, -1.f), pk2(x0, x1)), l0, l1);
    lo = pack_half2(l0, l1);
}
__device__ __forceinline__ void scale2(float &x0, float &x1, float f0, float f1) { upk2(mul2(pk2(x0, x1), pk2(f0, f1)), x0, x1); }

// ---------------------------------------------------------------- what the state is not needed for

// A CTA of two warps takes a chunk of a key head: both make the tiles and the products, then a warp has a head, a
// lane a token.  Decays between tokens, exp(G_i - G_j), are products of two factors with a border between
// the tokens: at the highest bit in which i and j differ, the sum up to i from the border on and that from j on up to
// it, both of at most 16 log decays and never a difference of long sums.  So a lane takes seven exponentials, not 32.
template <int T, int DK>
__global__ void __launch_bounds__(64, 8)
k_delta_prep(const __grid_constant__ DeltaArgs a) {
    constexpr int LP = 68;                                         // of two rows of the system, side by side
    // K and Q, then each warp's system (and T) and A
    __shared__ __align__(128) union {
        uint8_t tile[2][C * DK * 2];
        float la[2][2][C * 36];
    } s;
    __shared__ float s_kk[C * 33], s_qk[C * 33];
    __shared__ float s_kn[C], s_qn[C];                             // what the F16 rows are to be multiplied by
    __shared__ float s_b[2][5][C];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int hk = blockIdx.x % a.n_head_k, at = blockIdx.x / a.n_head_k;
    pdl_trigger();
    const int seq = delta_owner(a, at, at);
    uint32_t bits;
    const DeltaSeq q = delta_seq(a, seq, bits);
    const int t0 = (at - delta_base(q.row0, seq)) * C;
    if (!q.ok || q.n <= kDeltaFew || t0 < 0 || t0 >= q.n) return;
    const int nv = min(C, q.n - t0);

    // rows: four lanes to one, eight rows to a warp
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
        const int r = pass * 16 + warp * 8 + (lane >> 2), p = lane & 3;
        constexpr int N = DK / 32;                                 // 16-byte pieces of a lane
        uint4 x[2][N];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
#pragma unroll
            for (int j = 0; j < N; ++j) x[w][j] = make_uint4(0, 0, 0, 0);
            if (r < nv) {
                const int64_t row = q.row0 + t0 + r;
                const uint16_t *src = w ? a.q + row * a.q_rs + (int64_t)hk * a.q_hs : a.k + row * a.k_rs + (int64_t)hk * a.k_hs;
#pragma unroll
                for (int j = 0; j < N; ++j) x[w][j] = *reinterpret_cast<const uint4 *>(src + (p + 4 * j) * 8);
            }
        }
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            uint64_t ss2 = 0ull;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const uint32_t v[4] = {x[w][j].x, x[w][j].y, x[w][j].z, x[w][j].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint64_t f = pk2(from16<T>(v[e] & 0xffffu), from16<T>(v[e] >> 16));
                    ss2 = fma2(f, f, ss2);
                }
            }
            float ss, s1;
            upk2(ss2, ss, s1);
            ss += s1;
            ss += __shfl_xor_sync(0xffffffffu, ss, 1);
            ss += __shfl_xor_sync(0xffffffffu, ss, 2);
            float norm = a.normalise ? 1.f / sqrtf(ss + a.eps) : 1.f;
            // to a norm in [1, 2) by a power of two; a square sum past float32 makes the row 0, as its norm does
            const uint32_t e = __float_as_uint(sqrtf(ss)) >> 23;
            float down = e == 0u ? 1.f : (e == 255u ? 0x1p-126f : __uint_as_float((254u - min(e, 253u)) << 23));
            if (e == 255u && a.normalise) down = 0.f;
            norm = down == 0.f ? 1.f : norm * __uint_as_float((254u << 23) - __float_as_uint(down));
            // no length at all: its factor is of no row (1 / sqrt(eps) would count in the bounds of what the row adds), but for 0 / 0
            if (e == 0u) norm = norm < INFINITY ? 0.f : norm;
            uint8_t *tile = a.tiles + (((int64_t)at * a.n_head_k + hk) * 2 + w) * (C * DK * 2);
            const uint64_t down2 = pk2(down, down);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                uint32_t v[4] = {x[w][j].x, x[w][j].y, x[w][j].z, x[w][j].w};
#pragma unroll
                for (int e2 = 0; e2 < 4; ++e2) {
                    float f0, f1;
                    upk2(mul2(pk2(from16<T>(v[e2] & 0xffffu), from16<T>(v[e2] >> 16)), down2), f0, f1);
                    v[e2] = pack_half2(f0, f1);
                }
                const uint32_t off = tile_at(r, p + 4 * j);
                const uint4 y = make_uint4(v[0], v[1], v[2], v[3]);
                *reinterpret_cast<uint4 *>(s.tile[w] + off) = y;
                *reinterpret_cast<uint4 *>(tile + off) = y;
            }
            if (p == 0) (w ? s_qn : s_kn)[r] = r < nv ? (w ? norm * a.scale : norm) : 0.f;
        }
    }
    __syncthreads();
    {   // k . k and q . k: a warp has 16 columns, without what is above the diagonal; two sums, each cut off half as often
        float acc[2][2][2][2][4] = {};                             // K, Q; rows 0-15, 16-31; columns; even and odd steps
        const uint32_t k0 = smem_u32(s.tile[0]), q0 = smem_u32(s.tile[1]);
#pragma unroll
        for (int ks = 0; ks < DK / 16; ++ks) {
            uint32_t b[4], f[4];
            ldsm_x4(k0 + tile_at(warp * 16 + (lane & 7) + ((lane >> 4) << 3), ks * 2 + ((lane >> 3) & 1)), b[0], b[1], b[2], b[3]);
#pragma unroll
            for (int w = 0; w < 2; ++w)
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    if (m == 0 && warp) continue;
                    ldsm_x4((w ? q0 : k0) + tile_at(m * 16 + (lane & 15), ks * 2 + (lane >> 4)), f[0], f[1], f[2], f[3]);
                    mma16816(acc[w][m][0][ks & 1], f, b[0], b[1]);
                    mma16816(acc[w][m][1][ks & 1], f, b[2], b[3]);
                }
        }
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (m || !warp)
                            (w ? s_qk : s_kk)[(m * 16 + g + 8 * (e >> 1)) * 33 + warp * 16 + n * 8 + 2 * t + (e & 1)] =
                                acc[w][m][n][0][e] + acc[w][m][n][1][e];
    }
    __syncthreads();
    const int i = lane;
    float *l = s.la[warp][0], *am = s.la[warp][1];
    const float kn = s_kn[i], qn = s_qn[i];
    for (int hh = warp; hh < a.group; hh += 2) {
        const int h = hk * a.group + hh;
        float g = 0.f, beta = 0.f;
        if (i < nv) {
            const int64_t row = q.row0 + t0 + i;
            g = a.g[row * a.g_rs + h];
            if (g < kDeltaLeast) g = kDeltaLeast;
            beta = a.beta[row * a.beta_rs + h];
        }
        __syncwarp();                                              // the head before this one is written
        // of the aligned runs of 1, 2, 4, ... tokens: sums up to this token, from behind it on, and of all
        float upto = g, behind = 0.f, all = g, part[5];
#pragma unroll
        for (int v = 0; v < 5; ++v) {
            part[v] = expf(i >> v & 1 ? upto : behind);
            s_b[warp][v][i] = part[v] * kn;
            const float other = __shfl_xor_sync(0xffffffffu, all, 1 << v);
            if (i >> v & 1) upto += other;
            else behind += other;
            all += other;
        }
        const float gone = expf(upto), w = expf(behind) * kn, last = expf(all), bk = beta * kn;
        __syncwarp();
        float amax = fabsf(kn * s_qk[i * 33 + i]);
        am[i * 36 + i] = kn * s_qk[i * 33 + i];
#pragma unroll
        for (int v = 4; v >= 0; --v)
            if (i >> v & 1) {
                const int j0 = i >> (v + 1) << (v + 1);
#pragma unroll
                for (int d = 0; d < 1 << v; ++d) {
                    const int j = j0 + d;
                    const float x = part[v] * s_b[warp][v][j], y = x * s_qk[i * 33 + j];
                    l[(i >> 1) * LP + j * 2 + (i & 1)] = bk * x * s_kk[i * 33 + j];
                    am[i * 36 + j] = y;
                    amax = fmaxf(amax, fabsf(y));
                }
            }
        const float au = unit_of(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
        __syncwarp();
        // T by columns, a lane has one, and two rows at a time
        uint64_t nx[C];                                            // -x twice
        float x[C];
#pragma unroll
        for (int r = 0; r < C; r += 2) {
            uint64_t y0 = pk2(r == i ? 1.f : 0.f, r + 1 == i ? 1.f : 0.f), y1 = 0ull;
#pragma unroll
            for (int m = 0; m < r; m += 2) {
                const ulonglong2 f = *reinterpret_cast<const ulonglong2 *>(l + (r >> 1) * LP + m * 2);
                y0 = fma2(f.x, nx[m], y0);
                y1 = fma2(f.y, nx[m + 1], y1);
            }
            upk2(add2(y0, y1), x[r], x[r + 1]);
            x[r + 1] = fmaf(-l[(r >> 1) * LP + r * 2 + 1], x[r], x[r + 1]);
            nx[r] = pk2(-x[r], -x[r]);
            nx[r + 1] = pk2(-x[r + 1], -x[r + 1]);
        }
        __syncwarp();
#pragma unroll
        for (int r = 0; r < C; ++r) l[r * 36 + i] = x[r];
        __syncwarp();
        // the largest row sum of magnitudes, 1 at least, to [2^8, 2^9): with R below 2^6 U stays below 2^15, and neither
        // operand's low part falls below F16's smallest numbers before it is 2^-33 of the largest values
        float row = 0.f;
#pragma unroll
        for (int m = 0; m < C; m += 4) {
            const float4 f = *reinterpret_cast<const float4 *>(l + i * 36 + m);
            row += fabsf(f.x) + fabsf(f.y) + fabsf(f.z) + fabsf(f.w);
        }
        const float tu = unit_of(__reduce_max_sync(0xffffffffu, __float_as_uint(row))) * 0x1p-4f;
        HeadBlock *block = reinterpret_cast<HeadBlock *>(a.heads + ((int64_t)at * a.n_head + h) * kDeltaHeadBytes);
        HeadScalars *out = &block->s;
        const int gq = lane >> 2, tq = lane & 3;
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
            const int ri = block_n(b) * 8 + gq, ci = block_k(b) * 16 + 2 * tq, from = ri * 36 + ci;
            uint4 v;
            float2 lo = *reinterpret_cast<const float2 *>(l + from), hi = *reinterpret_cast<const float2 *>(l + from + 8);
            split(lo.x * tu, lo.y * tu, v.x, v.z);
            split(hi.x * tu, hi.y * tu, v.y, v.w);
            block->t[b][lane] = v;
            lo = *reinterpret_cast<const float2 *>(am + from);
            hi = *reinterpret_cast<const float2 *>(am + from + 8);
            if (block_n(b) < 2 || block_k(b)) {                // nothing above the diagonal has been written
                lo.x = ci <= ri ? lo.x : 0.f;
                lo.y = ci + 1 <= ri ? lo.y : 0.f;
                hi.x = ci + 8 <= ri ? hi.x : 0.f;
                hi.y = ci + 9 <= ri ? hi.y : 0.f;
            }
            split(lo.x * au, lo.y * au, v.x, v.z);
            split(hi.x * au, hi.y * au, v.y, v.w);
            block->a[b][lane] = v;
        }
        const int to = (i >> 1) * 4 + (i & 1);
        reinterpret_cast<float *>(out->r)[to] = beta;
        reinterpret_cast<float *>(out->r)[to + 2] = -(bk * gone);
        reinterpret_cast<float *>(out->o)[to] = qn;
        reinterpret_cast<float *>(out->o)[to + 2] = qn * gone;
        out->w[i] = w;
        if (i == 0) *reinterpret_cast<float4 *>(&out->last) = make_float4(last, inverse_unit(tu), inverse_unit(au), 0.f);
    }
}

// ---------------------------------------------------------------- the state's walk

// W groups of 16 value elements to a CTA, KS warps to a group: each has DK / KS of the key elements of the
// state, and makes the outputs of 32 / KS of a chunk's tokens.
template <int DK, int W, int KS>
struct ScanCfg {
    static constexpr int kWarps = W * KS;
    static constexpr int kThreads = (kWarps + 1) * 32;
    static constexpr int kTileBytes = 2 * C * DK * 2;
    static constexpr int kStageBytes = kTileBytes + (int)sizeof(HeadBlock);
    static constexpr int kVBytes = C * 32;                         // [C tokens][16 values], two to a group
    static constexpr int kOBytes = C / KS * 32;                    // a warp's outputs on their way
    static constexpr int kXWords = KS == 2 ? 6 * 4 * 32 : 0;       // what a warp hands its partner, two chunks' worth
    static constexpr int kStages = DK == 128 ? 3 : 4;
    static constexpr int kOffV = kStages * kStageBytes;
    static constexpr int kOffO = kOffV + W * 2 * kVBytes;
    static constexpr int kOffX = kOffO + kWarps * kOBytes;
    static constexpr int kOffBars = kOffX + kWarps * 2 * kXWords * 4;
    static constexpr int kSmem = kOffBars + 2 * kStages * 8;
    static_assert(kSmem <= 113 * 1024, "two CTAs per SM");
};

__device__ __forceinline__ uint32_t v_at(int r, int half) { return (uint32_t)(r * 32 + ((half ^ ((r >> 2) & 1)) << 4)); }

__device__ __forceinline__ void stsm_x2_t(uint32_t addr, uint32_t r0, uint32_t r1) {
    asm volatile("stmatrix.sync.aligned.m8n8.x2.trans.shared.b16 [%0], {%1, %2};" ::"r"(addr), "r"(r0), "r"(r1) : "memory");
}

// whether the phase is over, without waiting at all
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}

// mbar_wait of the copy warp, which has two chunks' time and leaves the issue slots to the warps beside it (eight prompts
// 567 us without a pause, 554 with 100 ns, 546 with 400)
__device__ __forceinline__ bool mbar_wait_idle(uint32_t bar, uint32_t parity) {
    const uint64_t t0 = global_ns();
    for (uint32_t it = 1; it < (1u << 30); ++it) {
        if (mbar_test(bar, parity)) return true;
        __nanosleep(400);
        if ((it & 255u) == 0 && global_ns() - t0 > kWaitNs) return false;
    }
    return false;
}

// A thread has parts of two rows, g and g + 8, the four threads of a quad the whole ones: their largest magnitudes, kLeast
// at least (NaN is passed over).
template <int N> __device__ __forceinline__ void row_tops(const float (&x)[N][4], float (&m)[2]) {
    m[0] = m[1] = kLeast;
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) m[i] = max3(m[i], fabsf(x[n][2 * i]), fabsf(x[n][2 * i + 1]));
#pragma unroll
    for (int d = 1; d < 4; d <<= 1)
#pragma unroll
        for (int i = 0; i < 2; ++i) m[i] = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], d));
}

// Accumulators of 32 columns as an A operand of two steps, in two parts.
__device__ __forceinline__ void operand(const float (&x)[4][4], uint32_t (&hi)[2][4], uint32_t (&lo)[2][4]) {
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) split(x[n][2 * e], x[n][2 * e + 1], hi[n >> 1][(n & 1) * 2 + e], lo[n >> 1][(n & 1) * 2 + e]);
}

constexpr int kSorted = 128;             // sequences

template <int T, int DK, int W, int KS>
__global__ void __launch_bounds__((W * KS + 1) * 32, KS == 1 ? 2 : 1)
k_delta_scan(const __grid_constant__ DeltaArgs a, int parts) {
    using F = ScanCfg<DK, W, KS>;
    static_assert(F::kThreads >= kSorted);
    constexpr int S = F::kStages, NT = DK / 8 / KS, STEPS = DK / 16 / KS;
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t full = smem_u32(smem + F::kOffBars), empty = full + 8 * S;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = blockIdx.x % parts, sh = blockIdx.x / parts, h = sh % a.n_head;
    int s = sh / a.n_head;
    // The longest sequences first, so that none begins when the others end (eight prompts of 239 to 4,096 tokens by rising
    // length, us: 645 as they come, 543 so; falling 541 and 544).  Each CTA counts the longer ones, as many
    // sequences as it has threads for; with more of them the last ones weigh less.
    if (a.n_seq > 1 && a.n_seq <= kSorted) {
        __shared__ int s_len[kSorted], s_seq;
        const int me = threadIdx.x;
        if (me < a.n_seq) s_len[me] = (int)((uint32_t)a.q_start[me + 1] - (uint32_t)a.q_start[me]);
        __syncthreads();
        if (me < a.n_seq) {
            int before = 0;
            for (int j = 0; j < a.n_seq; ++j) before += s_len[j] > s_len[me] || (s_len[j] == s_len[me] && j < me);
            if (before == s) s_seq = me;
        }
        __syncthreads();
        s = s_seq;
    }
    if (threadIdx.x == 0) {
        for (int k = 0; k < S; ++k) {
            mbar_init(full + 8 * k, 1);
            mbar_init(empty + 8 * k, F::kWarps);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    uint32_t bits;
    DeltaSeq q = delta_seq(a, s, bits);
    if (bits && threadIdx.x == 0 && h == 0 && part == 0) atomicOr(a.err, bits);
    q.ok = q.ok && q.n > kDeltaFew;                                // the others are k_delta_step's
    pdl_trigger();
    if (!q.ok && blockIdx.x) return;                               // (one waits for the kernel in front, as the one behind counts on)
    __shared__ bool s_prepared;
    if (warp == F::kWarps && q.ok) {
        const bool prepared = delta_prepared(a, s, q);
        if (lane == 0) s_prepared = prepared;
    }
    __syncthreads();
    q.ok = q.ok && s_prepared;                                     // unprepared ones too
    const int chunks = q.ok ? (q.n + C - 1) / C : 0;
    const int64_t base = delta_base(q.row0, s);
    auto timed_out = [&]() { atomicOr(a.err, (uint32_t)DELTA_ERR_WAIT); };

    if (warp == F::kWarps) {
        // ---------------- copies ----------------
        pdl_wait();                                                // the chunks are prepared
        if (lane == 0) {
            const int hk = h / a.group;
            int c = 0;
            for (; c < chunks; ++c) {
                const int k = c % S;
                if (!mbar_wait_idle(empty + 8 * k, ((uint32_t)(c / S) & 1u) ^ 1u)) {
                    timed_out();
                    break;
                }
                const uint32_t dst = smem_u32(smem + k * F::kStageBytes);
                mbar_expect_tx(full + 8 * k, F::kStageBytes);
                bulk_g2s(dst, a.tiles + ((base + c) * a.n_head_k + hk) * F::kTileBytes, F::kTileBytes, full + 8 * k);
                bulk_g2s(dst + F::kTileBytes, a.heads + ((base + c) * a.n_head + h) * kDeltaHeadBytes, (uint32_t)sizeof(HeadBlock), full + 8 * k);
            }
            // no copy may land after the CTA is gone
            for (int k = max(0, c - S); k < c; ++k)
                if (!mbar_wait(full + 8 * (k % S), (uint32_t)(k / S) & 1u)) {
                    timed_out();
                    break;
                }
        }
        __syncwarp();
        return;
    }
    if (!q.ok) return;

    // ---------------- the state ----------------
    const int g = lane >> 2, t = lane & 3, kp = warp % KS;
    const int row0 = (part * W + warp / KS) * 16;                  // the group's value elements: rows g and g + 8 of it
    auto place = [&](int slot) {
        return a.state + (int64_t)slot * a.slot_stride + (int64_t)h * a.head_stride + (int64_t)(row0 + g) * DK + kp * (DK / KS) + 2 * t;
    };
    float st[NT][4];
    {
        const float *src = q.slot < 0 ? nullptr : place(q.slot);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float2 x = make_float2(0.f, 0.f), y = x;
            if (src) {
                x = *reinterpret_cast<const float2 *>(src + n * 8);
                y = *reinterpret_cast<const float2 *>(src + 8 * DK + n * 8);
            }
            st[n][0] = x.x; st[n][1] = x.y; st[n][2] = y.x; st[n][3] = y.y;
        }
    }
    const uint32_t v0 = smem_u32(smem + F::kOffV + warp / KS * 2 * F::kVBytes), o0 = smem_u32(smem + F::kOffO + warp * F::kOBytes);
    float4 *xs = reinterpret_cast<float4 *>(smem + F::kOffX) + lane;
    // values of chunk c: two 16-byte pieces a token, zeros behind the last one
    auto fetch_v = [&](int c) {
        if (c < chunks) {
            const int nv = min(C, q.n - c * C);
#pragma unroll
            for (int e = kp; e < 2; e += KS) {
                const int r = (lane >> 1) + 16 * e, half = lane & 1;
                const uint16_t *src = a.v + (int64_t)(q.row0 + c * C + min(r, nv - 1)) * a.v_rs + (int64_t)h * a.v_hs + row0 + half * 8;
                cp_async16(v0 + (c & 1) * F::kVBytes + v_at(r, half), src, r < nv ? 16 : 0);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    fetch_v(0);
    bool alive = true;
    // each row times a power of two; what takes that back, and a bound of its magnitudes without it
    float si[2], sb[2];
    row_tops<NT>(st, sb);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float su = unit_above(sb[i]);
        si[i] = inverse_unit(su);
#pragma unroll
        for (int n = 0; n < NT; ++n) scale2(st[n][2 * i], st[n][2 * i + 1], su, su);
    }
    bool ready = false;                                            // the chunk was seen to be there while the one before it was worked on
    for (int c = 0; c < chunks; ++c) {
        const int k = c % S, nv = min(C, q.n - c * C);
        const bool here = __all_sync(0xffffffffu, ready) || __all_sync(0xffffffffu, mbar_wait(full + 8 * k, (uint32_t)(c / S) & 1u));
        if (!here && lane == 0) timed_out();
        if (KS == 1 && !here) {
            alive = false;
            break;
        }
        const uint32_t kt = smem_u32(smem + k * F::kStageBytes), qt = kt + C * DK * 2;
        const HeadBlock *hb = reinterpret_cast<const HeadBlock *>(smem + k * F::kStageBytes + F::kTileBytes);
        // S K^T and S Q^T: 16 value elements by 32 tokens each.  (lo's sum apart: it is small, and hi's is cut off half
        // as often.)  bf16 outputs take S's hi alone for S Q^T: off by 2^-11 of the products, an eighth of their
        // own rounding, for a seventh of a chunk's products.
        float pk[4][4] = {}, pl[4][4] = {}, pq[4][4] = {};
        uint32_t fk[2][2][4], fq[2][2][4];
        auto fetch = [&](int ks) {
#pragma unroll
            for (int np = 0; np < 2; ++np) {
                const uint32_t off = tile_at(np * 16 + (lane & 7) + ((lane >> 4) << 3), (kp * STEPS + ks) * 2 + ((lane >> 3) & 1));
                uint32_t (&x)[4] = fk[ks & 1][np], (&y)[4] = fq[ks & 1][np];
                ldsm_x4(kt + off, x[0], x[1], x[2], x[3]);
                ldsm_x4(qt + off, y[0], y[1], y[2], y[3]);
            }
        };
        fetch(0);
#pragma unroll
        for (int ks = 0; ks < STEPS; ++ks) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) split(st[2 * ks + (e >> 1)][2 * (e & 1)], st[2 * ks + (e >> 1)][2 * (e & 1) + 1], hi[e], lo[e]);
            if (ks + 1 < STEPS) fetch(ks + 1);
#pragma unroll
            for (int n = 0; n < 4; ++n) mma16816(pk[n], hi, fk[ks & 1][n >> 1][2 * (n & 1)], fk[ks & 1][n >> 1][2 * (n & 1) + 1]);
#pragma unroll
            for (int n = 0; n < 4; ++n) mma16816(pl[n], lo, fk[ks & 1][n >> 1][2 * (n & 1)], fk[ks & 1][n >> 1][2 * (n & 1) + 1]);
#pragma unroll
            for (int n = 0; n < 4; ++n) mma16816(pq[n], hi, fq[ks & 1][n >> 1][2 * (n & 1)], fq[ks & 1][n >> 1][2 * (n & 1) + 1]);
            if (T == PAGED_F16) {
#pragma unroll
                for (int n = 0; n < 4; ++n) mma16816(pq[n], lo, fq[ks & 1][n >> 1][2 * (n & 1)], fq[ks & 1][n >> 1][2 * (n & 1) + 1]);
            }
        }
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int e = 0; e < 4; e += 2) upk2(add2(pk2(pk[n][e], pk[n][e + 1]), pk2(pl[n][e], pl[n][e + 1])), pk[n][e], pk[n][e + 1]);
        asm volatile("cp.async.wait_all;" ::: "memory");           // this chunk's values
        constexpr int OT = 4 / KS;                                 // token tiles whose outputs are this warp's
        float ks1[2] = {si[0], si[1]};                             // what the sums are to be multiplied by
        if constexpr (KS == 2) {
            // the partner's half of the sums: of S K^T all, of S Q^T those of the 16 tokens whose outputs are this warp's
            ks1[0] = ks1[1] = 1.f;
            float4 *mine = xs + (warp * 2 + (c & 1)) * (F::kXWords / 4);
            const float4 *other = xs + ((warp ^ 1) * 2 + (c & 1)) * (F::kXWords / 4);
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                scale2(pk[n][0], pk[n][1], si[0], si[0]);
                scale2(pk[n][2], pk[n][3], si[1], si[1]);
                mine[n * 32] = make_float4(pk[n][0], pk[n][1], pk[n][2], pk[n][3]);
            }
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    scale2(pq[m][e], pq[m][e + 1], si[e / 2], si[e / 2]);
                    scale2(pq[2 + m][e], pq[2 + m][e + 1], si[e / 2], si[e / 2]);
                }
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                mine[(4 + m) * 32] = kp ? make_float4(pq[m][0], pq[m][1], pq[m][2], pq[m][3])
                                        : make_float4(pq[2 + m][0], pq[2 + m][1], pq[2 + m][2], pq[2 + m][3]);
                // (what stays, to the front)
#pragma unroll
                for (int e = 0; e < 4; ++e) pq[m][e] = kp ? pq[2 + m][e] : pq[m][e];
            }
            // (a wait that ran out in either: both leave)
            if (bar_any(1 + warp / 2, 64, !here)) {
                alive = false;
                break;
            }
            // (the same sums in both warps: addition does not mind the order of two)
            auto join = [](float (&x)[4], const float4 &y) {
                upk2(add2(pk2(x[0], x[1]), pk2(y.x, y.y)), x[0], x[1]);
                upk2(add2(pk2(x[2], x[3]), pk2(y.z, y.w)), x[2], x[3]);
            };
#pragma unroll
            for (int n = 0; n < 4; ++n) join(pk[n], other[n * 32]);
#pragma unroll
            for (int m = 0; m < OT; ++m) join(pq[m], other[(4 + m) * 32]);
        } else {
            __syncwarp();
        }
        fetch_v(c + 1);                                            // (the group is through with the chunk before)
        // R = beta V - beta exp(G) |k| (S K^T)
        const uint32_t vt = v0 + (c & 1) * F::kVBytes;
        float r[4][4];
#pragma unroll
        for (int np = 0; np < 2; ++np) {
            uint32_t v[4];
            ldsm_x4_t(vt + v_at(np * 16 + (lane & 7) + ((lane >> 4) << 3), (lane >> 3) & 1), v[0], v[1], v[2], v[3]);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const int n = 2 * np + m;
                const float4 f = hb->s.r[n * 4 + t];                 // beta, then -beta exp(G) |k| of tokens 8n + 2t, + 1
                const uint64_t b2 = pk2(f.x, f.y);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint64_t c2 = mul2(pk2(f.z, f.w), pk2(ks1[e], ks1[e]));
                    const uint64_t x = pk2(from16<T>(v[2 * m + e] & 0xffffu), from16<T>(v[2 * m + e] >> 16));
                    upk2(fma2(b2, x, mul2(c2, pk2(pk[n][2 * e], pk[n][2 * e + 1]))), r[n][2 * e], r[n][2 * e + 1]);
                }
            }
        }
        // U = R T^T, times the row's unit of R and T's, by which it is below 2^15
        float u[4][4] = {};
        uint32_t hi[2][4], lo[2][4];
        float ui[2];
        {
            float top[2];
            row_tops<4>(r, top);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float unit = unit_above(top[i]) * 0x1p-7f;
                ui[i] = inverse_unit(unit) * hb->s.t_unit;
                const float ru = fmaf(top[i], 0.f, unit);          // an infinity has no unit: NaN for all its row's tokens
#pragma unroll
                for (int n = 0; n < 4; ++n) scale2(r[n][2 * i], r[n][2 * i + 1], ru, ru);
            }
            uint4 f[kBlocks];
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) f[b] = hb->t[b][lane];
            operand(r, hi, lo);
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) mma16816(u[block_n(b)], hi[block_k(b)], f[b].x, f[b].y);
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) mma16816(u[block_n(b)], lo[block_k(b)], f[b].x, f[b].y);
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) mma16816(u[block_n(b)], hi[block_k(b)], f[b].z, f[b].w);
        }
        // The rows' next units: a row's bound is the old one's decayed and, with |k| below 2 a token, 2 sum(w |u|).  (It
        // may pass float32 where the state does not.)
        const float last = hb->s.last;
        float nu[2] = {};
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const float2 f = *reinterpret_cast<const float2 *>(&hb->s.w[n * 8 + 2 * t]);
#pragma unroll
            for (int i = 0; i < 2; ++i) nu[i] = fmaf(f.x, fabsf(u[n][2 * i]), fmaf(f.y, fabsf(u[n][2 * i + 1]), nu[i]));
        }
        float more[2];
        auto round = [&](int d) {
#pragma unroll
            for (int i = 0; i < 2; ++i) more[i] = __shfl_xor_sync(0xffffffffu, nu[i], d);
        };
        round(1);
        // o = |q| (exp(G) S q + A u)
        {
            operand(u, hi, lo);
            float x[OT][4] = {};
            uint4 f[OT][2];
#pragma unroll
            for (int m = 0; m < OT; ++m) {
                const int n = kp * OT + m;                         // blocks n and, from token 16 on, n + 2
                f[m][0] = hb->a[n][lane];
                if (n >= 2) f[m][1] = hb->a[n + 2][lane];
            }
            auto product = [&](int ks, const uint32_t (&op)[2][4], bool low) {
#pragma unroll
                for (int m = 0; m < OT; ++m)
                    if (ks == 0 || kp * OT + m >= 2) mma16816(x[m], op[ks], low ? f[m][ks].z : f[m][ks].x, low ? f[m][ks].w : f[m][ks].y);
            };
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                product(ks, hi, false);
                product(ks, lo, false);
                product(ks, hi, true);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) nu[i] += more[i];
            round(2);
            const float back[2] = {ui[0] * hb->s.a_unit, ui[1] * hb->s.a_unit};
            // through shared memory into rows
            uint32_t o16[OT][2];
#pragma unroll
            for (int m = 0; m < OT; ++m) {
                const float4 w = hb->s.o[(kp * OT + m) * 4 + t];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint64_t fa = mul2(pk2(w.x, w.y), pk2(back[e], back[e])), fs = mul2(pk2(w.z, w.w), pk2(ks1[e], ks1[e]));
                    float y0, y1;
                    upk2(fma2(fa, pk2(x[m][2 * e], x[m][2 * e + 1]), mul2(fs, pk2(pq[m][2 * e], pq[m][2 * e + 1]))), y0, y1);
                    o16[m][e] = T == PAGED_F16 ? pack_half2(y0, y1) : pack_bf162(y0, y1);
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                nu[i] += more[i];
                sb[i] = fminf(fmaf(last, sb[i], 2.f * (ui[i] * nu[i])), 3.4e38f);
                // (and not so small that what U is multiplied by would pass float32, should all that U adds vanish by decays)
                sb[i] = max3(sb[i], 0x1p-114f * ui[i], kLeast);
                nu[i] = unit_above(sb[i]);
            }
#pragma unroll
            for (int m = 0; m < OT; ++m) stsm_x2_t(o0 + v_at(m * 8 + (lane & 7), (lane >> 3) & 1), o16[m][0], o16[m][1]);
            __syncwarp();
#pragma unroll
            for (int e = 0; e < OT / 2; ++e) {
                const int row = (lane >> 1) + 16 * e, piece = lane & 1, token = kp * OT * 8 + row;
                uint4 y;
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(y.x), "=r"(y.y), "=r"(y.z), "=r"(y.w) : "r"(o0 + v_at(row, piece)) : "memory");
                if (token < nv)
                    *reinterpret_cast<uint4 *>(a.o + (int64_t)(q.row0 + c * C + token) * a.o_rs + (int64_t)h * a.o_hs + row0 + piece * 8) = y;
            }
        }
        // (the next chunk: the answer is there by the time it is asked for)
        ready = c + 1 < chunks && mbar_test(full + 8 * ((c + 1) % S), (uint32_t)((c + 1) / S) & 1u);
        // S <- exp(G_last) S + U (exp(G_last - G) |k| K), all times the new unit
        {
            float wf[2], keep[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                // (units far apart: the row has vanished, and their product alone may pass float32)
                const float step = si[i] * nu[i];
                keep[i] = step < INFINITY ? last * step : last * si[i] * nu[i];
                wf[i] = ui[i] * nu[i];
                si[i] = inverse_unit(nu[i]);
            }
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const float2 f = *reinterpret_cast<const float2 *>(&hb->s.w[n * 8 + 2 * t]);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float f0, f1;
                    upk2(mul2(pk2(f.x, f.y), pk2(wf[i], wf[i])), f0, f1);
                    scale2(u[n][2 * i], u[n][2 * i + 1], f0, f1);
                }
            }
            operand(u, hi, lo);
            // four key tiles at a time, their operands fetched ahead
            uint32_t f[2][2][2][4];                                // [buffer][step][pair of tiles]
            auto fetch_k = [&](int n4) {
#pragma unroll
                for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        uint32_t (&x)[4] = f[n4 & 1][ks][p];
                        ldsm_x4_t(kt + tile_at(ks * 16 + (lane & 15), kp * NT + n4 * 4 + p * 2 + (lane >> 4)), x[0], x[1], x[2], x[3]);
                    }
            };
            fetch_k(0);
            const uint64_t keep2[2] = {pk2(keep[0], keep[0]), pk2(keep[1], keep[1])};
#pragma unroll
            for (int n4 = 0; n4 < NT / 4; ++n4) {
                if (n4 + 1 < NT / 4) fetch_k(n4 + 1);
                float x[4][4] = {};
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
                    for (int m = 0; m < 4; ++m) mma16816(x[m], hi[ks], f[n4 & 1][ks][m >> 1][2 * (m & 1)], f[n4 & 1][ks][m >> 1][2 * (m & 1) + 1]);
#pragma unroll
                    for (int m = 0; m < 4; ++m) mma16816(x[m], lo[ks], f[n4 & 1][ks][m >> 1][2 * (m & 1)], f[n4 & 1][ks][m >> 1][2 * (m & 1) + 1]);
                }
#pragma unroll
                for (int m = 0; m < 4; ++m)
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {
                        float (&y)[4] = st[4 * n4 + m];
                        upk2(fma2(keep2[e / 2], pk2(y[e], y[e + 1]), pk2(x[m][e], x[m][e + 1])), y[e], y[e + 1]);
                    }
            }
        }
        // (the stage's next copy writes through another proxy: an arrival alone does not hold it back behind reads still
        // on their way, and a warp's last ones were overwritten when a new CTA's first loads delayed them; 8 of 728 us)
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(empty + 8 * k);
        if ((c & 7) == 7) {
            row_tops<NT>(st, sb);
            sb[0] *= si[0];
            sb[1] *= si[1];
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    const int out = a.slot_out[s];
    if (!alive || out < 0) return;
    if (out >= a.n_slots) {
        if (threadIdx.x == 0 && h == 0 && part == 0) atomicOr(a.err, (uint32_t)DELTA_ERR_SLOT);
        return;
    }
    float *dst = place(out);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        *reinterpret_cast<float2 *>(dst + n * 8) = make_float2(st[n][0] * si[0], st[n][1] * si[0]);
        *reinterpret_cast<float2 *>(dst + 8 * DK + n * 8) = make_float2(st[n][2] * si[1], st[n][3] * si[1]);
    }
}

constexpr int kAlone = 120 * 1024;       // more than half of an SM's shared memory

template <int T, int DK>
cudaError_t prep(const DeltaArgs &a, cudaStream_t st) {
    const int64_t chunks = delta_chunks(a.n_rows, a.n_seq);
    k_delta_prep<T, DK><<<(unsigned)(chunks * a.n_head_k), 64, 0, st>>>(a);
    return cudaGetLastError();
}

template <int T, int DK, int W, int KS>
cudaError_t scan(const DeltaArgs &a, int dv, bool alone, cudaStream_t st) {
    using F = ScanCfg<DK, W, KS>;
    const int parts = dv / (16 * W);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((int64_t)a.n_seq * a.n_head * parts), 1, 1);
    cfg.blockDim = dim3(F::kThreads);
    cfg.dynamicSmemBytes = alone ? kAlone : F::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_delta_scan<T, DK, W, KS>, a, parts);
}

// By the CTAs of four groups that all rows make when each takes as long as the longest sequence's: up to half the SMs'
// number, two warps to a group and half the groups to a CTA; up to little more than the SMs', each CTA has an SM to
// itself (beginning beside the kernel in front, two long ones would find room on one while others have none); then
// two to an SM.  32 heads of 128, us, in these three forms: one sequence of 2,000 tokens 101, 138, 199, with seven of
// 200 172, 152, 214, two 199, 155, 216, four of 2,000 to 500 231, 194, 223, three 295, 286, 228; of 64: two 97,
// 105, 120, three 176, 115, 155, six 275, 222, 186.
template <int T, int DK>
cudaError_t walk(const DeltaArgs &a, int dv, int sms, cudaStream_t st) {
    const int64_t rows = std::min(a.n_rows, (int64_t)a.n_seq * a.max_q), work = rows * a.n_head * dv / 64, one = (int64_t)a.max_q * sms;
    if (2 * work <= one) return scan<T, DK, 2, 2>(a, dv, true, st);
    return scan<T, DK, 4, 1>(a, dv, 10 * work <= 11 * one, st);
}

template <int T, int DK, int W, int KS> cudaError_t allow() {
    return cudaFuncSetAttribute(k_delta_scan<T, DK, W, KS>, cudaFuncAttributeMaxDynamicSharedMemorySize, kAlone);
}
template <int T> cudaError_t allow_all() {
    cudaError_t e = allow<T, 64, 2, 2>();
    if (e == cudaSuccess) e = allow<T, 64, 4, 1>();
    if (e == cudaSuccess) e = allow<T, 128, 2, 2>();
    if (e == cudaSuccess) e = allow<T, 128, 4, 1>();
    return e;
}

}  // namespace

cudaError_t delta_chunk_setup() {
    const cudaError_t e = allow_all<PAGED_F16>();
    return e == cudaSuccess ? allow_all<PAGED_BF16>() : e;
}

cudaError_t launch_delta_prep(const DeltaArgs &a, int dtype, int dim_k, cudaStream_t st) {
    if (dtype == PAGED_F16) return dim_k == 64 ? prep<PAGED_F16, 64>(a, st) : prep<PAGED_F16, 128>(a, st);
    return dim_k == 64 ? prep<PAGED_BF16, 64>(a, st) : prep<PAGED_BF16, 128>(a, st);
}
cudaError_t launch_delta_scan(const DeltaArgs &a, int dtype, int dim_k, int dim_v, int sms, cudaStream_t st) {
    if (dtype == PAGED_F16) return dim_k == 64 ? walk<PAGED_F16, 64>(a, dim_v, sms, st) : walk<PAGED_F16, 128>(a, dim_v, sms, st);
    return dim_k == 64 ? walk<PAGED_BF16, 64>(a, dim_v, sms, st) : walk<PAGED_BF16, 128>(a, dim_v, sms, st);
}

}  // namespace dflash
