// The gated delta rule token by token, the state in registers: the kernel for few new tokens per
// sequence, and for states that are kept behind single tokens.
//
//   S <- a S,  u = beta (v - S k),  S <- S + u k^T,  o = scale S q;   a = exp(g)
//
// Rows of S (one per value element) never meet, so a head's state is shared out by rows: a warp
// has four rows beside one another, eight lanes to a row, each lane a run of four key elements in
// every 32, so that a row is read and written in whole 128-byte lines.  S k and S q come out of one pass
// over the old state, o = a (S q) + (q . k) u, whose two sums over the eight lanes are the only words
// that lanes exchange.  Keys and queries are normed once per CTA, eight tokens at a time, in shared memory.
//
// Bound by the state's bytes, 64 KB read and written per head of 128 x 128, as long as a sequence has
// few tokens: a token takes 3 flops per state element beside 8 bytes of it.  What counts is bytes under way: eight
// CTAs to an SM (64 sequences of 32 heads, a token each: 62 us with five, 51 with eight; ten spill, 59), and states that
// pass through L2 as what is not read again (46 us; 5.8 TB/s, 87 % of the copy rate).  With states kept behind every
// token (64 branches of up to 9 tokens) the one that all read stays there: 103 us, 6.6 TB/s, and 108 otherwise.
#include "delta.h"

#include "ring_internal.h"
#include "ptx.h"
#include "paged_ptx.h"

namespace dflash {
namespace {

constexpr int kStepThreads = 128, kStepTokens = 8;

__device__ __forceinline__ float2 unpack2(uint64_t x) {
    float2 r;
    upk2(x, r.x, r.y);
    return r;
}

template <int T> __device__ __forceinline__ float from16(uint32_t x) {
    if constexpr (T == PAGED_F16) return __half2float(__ushort_as_half((unsigned short)x));
    else return __uint_as_float(x << 16);
}
template <int T> __device__ __forceinline__ uint16_t to16(float x) {
    if constexpr (T == PAGED_F16) return __half_as_ushort(__float2half_rn(x));
    else return __bfloat16_as_ushort(__float2bfloat16_rn(x));
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

// DK key elements, DV value elements
template <int T, int DK, int DV>
__global__ void __launch_bounds__(kStepThreads, DK == 64 ? 6 : 8)
k_delta_step(const __grid_constant__ DeltaArgs a) {
    constexpr int E = DK / 8;                          // of a lane's part of a row
    constexpr int J = 32 / E;                          // rows of a lane: 2 or 4
    constexpr int WHICH = J == 4 ? 1 : 2;              // of a lane's number among eight: whether it ends with a k . S or a q . S
    constexpr int kRows = 4 * 4 * J;                   // of a CTA
    constexpr int kParts = DV / kRows;
    constexpr int TB = kStepTokens;
    __shared__ float s_k[TB][DK], s_q[TB][DK], s_v[TB][kRows];
    __shared__ float s_decay[TB], s_beta[TB], s_qk[TB];
    __shared__ int s_save[TB];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = blockIdx.x % kParts, sh = blockIdx.x / kParts, h = sh % a.n_head, s = sh / a.n_head;
    uint32_t bits;
    const DeltaSeq q = delta_seq(a, s, bits);
    if (bits && threadIdx.x == 0 && h == 0 && part == 0) atomicOr(a.err, bits);
    // (between the kernels of longer sequences: what waits for this one waits for the one in front too)
    if (a.split) {
        pdl_trigger();
        if (threadIdx.x == 0 && blockIdx.x == 0) pdl_wait();
    }
    if (!q.ok || (a.split && q.n > kDeltaFew && delta_prepared(a, s, q))) return;
    const int sub = lane & 7, rg = lane >> 3;          // the lane's part of a row, its row of four
    const int row0 = part * kRows + warp * 4 * J;      // the warp's rows: row0 + 4 j + rg
    auto place = [&](int slot) {
        return a.state + (int64_t)slot * a.slot_stride + (int64_t)h * a.head_stride + (int64_t)(row0 + rg) * DK + sub * 4;
    };
    uint64_t st[J][E / 2];
    if (q.slot >= 0) {
        const float *src = place(q.slot);
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int e = 0; e < E / 4; ++e) {
                const float4 *from = reinterpret_cast<const float4 *>(src + j * 4 * DK + e * 32);
                const float4 x = a.save ? *from : __ldcs(from);
                st[j][2 * e] = pk2(x.x, x.y);
                st[j][2 * e + 1] = pk2(x.z, x.w);
            }
    } else {
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int e = 0; e < E / 2; ++e) st[j][e] = 0ull;
    }
    auto store = [&](int slot) {
        if (slot < 0) return;
        if (slot >= a.n_slots) {
            if (threadIdx.x == 0 && h == 0 && part == 0) atomicOr(a.err, (uint32_t)DELTA_ERR_SLOT);
            return;
        }
        float *dst = place(slot);
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int e = 0; e < E / 4; ++e) {
                const float2 x = unpack2(st[j][2 * e]), y = unpack2(st[j][2 * e + 1]);
                __stcs(reinterpret_cast<float4 *>(dst + j * 4 * DK + e * 32), make_float4(x.x, x.y, y.x, y.y));
            }
    };

    const int hk = h / a.group;
    for (int t0 = 0; t0 < q.n; t0 += TB) {
        const int nt = min(TB, q.n - t0);
        if (t0) __syncthreads();                       // the tokens before these have been read
        for (int i = warp; i < nt; i += 4) {
            const int64_t row = q.row0 + t0 + i;
            const uint16_t *kp = a.k + row * a.k_rs + (int64_t)hk * a.k_hs;
            const uint16_t *qp = a.q + row * a.q_rs + (int64_t)hk * a.q_hs;
            constexpr int N = DK / 32;                 // of a lane
            float kx[N], qx[N], kk = 0.f, qq = 0.f, qk = 0.f;
            uint32_t kw[N / 2], qw[N / 2];
            if constexpr (N == 4) {
                const uint2 x = *reinterpret_cast<const uint2 *>(kp + lane * 4), y = *reinterpret_cast<const uint2 *>(qp + lane * 4);
                kw[0] = x.x; kw[1] = x.y; qw[0] = y.x; qw[1] = y.y;
            } else {
                kw[0] = *reinterpret_cast<const uint32_t *>(kp + lane * 2);
                qw[0] = *reinterpret_cast<const uint32_t *>(qp + lane * 2);
            }
#pragma unroll
            for (int e = 0; e < N; ++e) {
                kx[e] = from16<T>(e & 1 ? kw[e / 2] >> 16 : kw[e / 2] & 0xffffu);
                qx[e] = from16<T>(e & 1 ? qw[e / 2] >> 16 : qw[e / 2] & 0xffffu);
                kk = fmaf(kx[e], kx[e], kk);
                qq = fmaf(qx[e], qx[e], qq);
            }
            float kr = 1.f, qr = a.scale;
            if (a.normalise) {
                kr = 1.f / sqrtf(warp_sum(kk) + a.eps);
                qr = a.scale / sqrtf(warp_sum(qq) + a.eps);
            }
#pragma unroll
            for (int e = 0; e < N; ++e) {
                kx[e] *= kr;
                qx[e] *= qr;
                qk = fmaf(kx[e], qx[e], qk);
                s_k[i][lane * N + e] = kx[e];
                s_q[i][lane * N + e] = qx[e];
            }
            qk = warp_sum(qk);
            if (lane == 0) {
                const float g = a.g[row * a.g_rs + h];
                s_decay[i] = expf(g < kDeltaLeast ? kDeltaLeast : g);
                s_beta[i] = a.beta[row * a.beta_rs + h];
                s_qk[i] = qk;
                s_save[i] = a.save ? a.save[row] : -1;
            }
        }
        for (int i = threadIdx.x; i < nt * kRows; i += kStepThreads) {
            const int t = i / kRows, r = i % kRows;
            s_v[t][r] = from16<T>(a.v[(int64_t)(q.row0 + t0 + t) * a.v_rs + (int64_t)h * a.v_hs + part * kRows + r]);
        }
        __syncthreads();
        for (int t = 0; t < nt; ++t) {
            uint64_t kd[E / 2], ks[J], qs[J];
#pragma unroll
            for (int j = 0; j < J; ++j) ks[j] = qs[j] = 0ull;
#pragma unroll
            for (int e = 0; e < E / 4; ++e) {
                const ulonglong2 kx = *reinterpret_cast<const ulonglong2 *>(&s_k[t][sub * 4 + e * 32]);
                const ulonglong2 qx = *reinterpret_cast<const ulonglong2 *>(&s_q[t][sub * 4 + e * 32]);
                kd[2 * e] = kx.x;
                kd[2 * e + 1] = kx.y;
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    ks[j] = fma2(kx.x, st[j][2 * e], ks[j]);
                    ks[j] = fma2(kx.y, st[j][2 * e + 1], ks[j]);
                    qs[j] = fma2(qx.x, st[j][2 * e], qs[j]);
                    qs[j] = fma2(qx.y, st[j][2 * e + 1], qs[j]);
                }
            }
            // 2 J sums over eight lanes: a round hands half of them over and keeps the other half, so that lane 2j WHICH (+ WHICH)
            // of the eight ends with row j's k . S (q . S): four or seven shuffles, where one sum after the other takes
            // three each.
            float x[2 * J];
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const float2 a0 = unpack2(ks[j]), a1 = unpack2(qs[j]);
                x[2 * j] = a0.x + a0.y;
                x[2 * j + 1] = a1.x + a1.y;
            }
#pragma unroll
            for (int d = 4, n = J; d; d >>= 1, n >>= 1) {
                if (n == 0) {
                    x[0] += __shfl_xor_sync(0xffffffffu, x[0], d);
                    continue;
                }
                const bool up = sub & d;
#pragma unroll
                for (int i = 0; i < n; ++i) {
                    const float give = up ? x[i] : x[i + n], keep = up ? x[i + n] : x[i];
                    x[i] = keep + __shfl_xor_sync(0xffffffffu, give, d);
                }
            }
            const float decay = s_decay[t], other = __shfl_xor_sync(0xffffffffu, x[0], WHICH);
            const float kS = sub & WHICH ? other : x[0], qS = sub & WHICH ? x[0] : other;
            const int r = warp * 4 * J + 4 * (sub / (2 * WHICH)) + rg;
            const float mine = s_beta[t] * (s_v[t][r] - decay * kS);
            if (sub % (2 * WHICH) == 0)
                a.o[(int64_t)(q.row0 + t0 + t) * a.o_rs + (int64_t)h * a.o_hs + part * kRows + r] = to16<T>(fmaf(s_qk[t], mine, decay * qS));
            const uint64_t decay2 = pk2(decay, decay);
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const float u = __shfl_sync(0xffffffffu, mine, (lane & 24) + 2 * WHICH * j);
                const uint64_t u2 = pk2(u, u);
#pragma unroll
                for (int e = 0; e < E / 2; ++e) st[j][e] = fma2(kd[e], u2, mul2(decay2, st[j][e]));
            }
            store(s_save[t]);
        }
    }
    store(a.slot_out[s]);
}

template <int T, int DK, int DV>
cudaError_t go(const DeltaArgs &a, cudaStream_t st) {
    constexpr int parts = DV / (4 * 4 * (32 / (DK / 8)));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((int64_t)a.n_seq * a.n_head * parts), 1, 1);
    cfg.blockDim = dim3(kStepThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.split ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, k_delta_step<T, DK, DV>, a);
}
template <int T>
cudaError_t pick(const DeltaArgs &a, int dk, int dv, cudaStream_t st) {
    if (dk == 64) return dv == 64 ? go<T, 64, 64>(a, st) : go<T, 64, 128>(a, st);
    return dv == 64 ? go<T, 128, 64>(a, st) : go<T, 128, 128>(a, st);
}

}  // namespace

cudaError_t launch_delta_step(const DeltaArgs &a, int dtype, int dim_k, int dim_v, cudaStream_t st) {
    return dtype == PAGED_F16 ? pick<PAGED_F16>(a, dim_k, dim_v, st) : pick<PAGED_BF16>(a, dim_k, dim_v, st);
}

}  // namespace dflash
