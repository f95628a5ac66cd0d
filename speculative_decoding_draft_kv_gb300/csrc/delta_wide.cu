// The gated delta rule over many tokens (formulas: delta_chunk.cu): a sequence's chunks walked on the 5th-generation
// tensor cores, for batches with a CTA for about every SM.
//
// A CTA has a head's whole state, 128 value elements by DK key elements.  All products have the value elements as
// rows, one to a TMEM lane:
//   S [K Q]^T, then U = R T^T, then S += U K and O += U A^T,
// with the left operand -- state, right-hand sides, updates, as F16 pairs hi + lo -- in tensor memory, where the
// threads that own the rows put it, and the right one in shared memory: K and Q as tiles of 32 tokens by 64 columns,
// read along their rows by the first product and along their columns by the state's update, T and A with hi beside lo.
// The state itself stays in registers, float32, two threads to a row: an accumulator in tensor memory would be cut off
// at every addition.  Rows share nothing, so each has a unit (power of two) of its own.
//
// Per chunk the threads and the tensor cores hand over three times (S -> R -> U -> S), which is the chain that bounds it;
// what the outputs need runs beside the next chunk's first product.
//
// Roles: warps 0-7 rows (warp w: lanes 32 (w % 4) on, key elements and tokens by halves w / 4), warp 8 issues products,
// warp 9 copies.
#include "delta_chunk.cuh"

namespace dflash {
namespace {

constexpr int kDV = 128;
template <int DK>
struct WideCfg {
    static constexpr int kThreads = 320;
    static constexpr int kStages = 4;
    static constexpr int kTileBytes = 2 * C * DK * 2;
    static constexpr int kOffT = kTileBytes, kOffA = kOffT + C * 128, kOffScalars = kOffA + C * 128;
    static constexpr int kBlockBytes = 2 * C * 128 + (int)sizeof(HeadScalars);
    static constexpr int kOffV = kOffScalars + 1024;               // [C tokens][kDV] 16-bit values
    static constexpr int kStageBytes = kOffV + C * kDV * 2;
    static constexpr int kOffX = kStages * kStageBytes;            // [2][2][8 warps][32]: what halves of a row tell each other
    static constexpr int kOffBars = kOffX + 2 * 2 * 8 * 32 * 4;
    static constexpr int kSmem = kOffBars + 256;
    static_assert(kStageBytes % 1024 == 0 && sizeof(HeadScalars) <= 1024 && kSmem <= 227 * 1024, "");
};
// columns of tensor memory
enum { kColHi = 0, kColLo = 64, kColDS = 128, kColPK = 256, kColPQ = 288, kColR = 352, kColU = 384, kColUOp = 416, kColWOp = 448,
       kColO = 480 };

template <int T, int DK>
__global__ void __launch_bounds__(320, 1)
k_delta_wide(const __grid_constant__ DeltaArgs a) {
    using F = WideCfg<DK>;
    constexpr int S = F::kStages, H = DK / 2;                      // key elements of a thread
    constexpr uint32_t kIdescTok = tc_idesc(128, C, false, false), kIdescKey = tc_idesc(128, DK, false, true);
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ uint32_t s_tmem;
    const uint32_t full = smem_u32(smem + F::kOffBars), empty = full + 8 * S;
    const uint32_t s_ready = empty + 8 * S, p_full = s_ready + 8, r_ready = s_ready + 16, u_full = s_ready + 24, w_ready = s_ready + 32;
    const uint32_t d_full = s_ready + 40, o_ready = s_ready + 48, o_full = s_ready + 56, drain = s_ready + 64;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.x % a.n_head, s = blockIdx.x / a.n_head;
    auto timed_out = [&]() { atomicOr(a.err, (uint32_t)DELTA_ERR_WAIT); };
    if (smem_u32(smem) & 1023u) {                                  // never: tiles would be read in another order
        if (threadIdx.x == 0) timed_out();
        if (threadIdx.x == 0) pdl_wait();
        return;
    }
    if (threadIdx.x == 0) {
        for (int k = 0; k < S; ++k) {
            mbar_init(full + 8 * k, 33);                           // the bulk copies, and the values' 32 lanes
            mbar_init(empty + 8 * k, 9);                           // the products, and the rows' eight warps
        }
        for (uint32_t b : {s_ready, r_ready, w_ready, o_ready}) mbar_init(b, 8);
        for (uint32_t b : {p_full, u_full, d_full, o_full, drain}) mbar_init(b, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 8) {
        tmem_alloc(smem_u32(&s_tmem), 512);
        tmem_relinquish();
    }
    uint32_t bits;
    DeltaSeq q = delta_seq(a, s, bits);
    if (bits && threadIdx.x == 0 && h == 0) atomicOr(a.err, bits);
    q.ok = q.ok && q.n > kDeltaFew;                                // the others are k_delta_step's
    pdl_trigger();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    const int chunks = q.ok ? (q.n + C - 1) / C : 0;

    if (warp == 9) {
        // ---------------- copies ----------------
        pdl_wait();                                                // the chunks are prepared
        const int64_t base = chunk_base(q.row0, s);
        const int hk = h / a.group;
        int c = 0;
        for (; c < chunks; ++c) {
            const int k = c % S, nv = min(C, q.n - c * C);
            if (!__all_sync(0xffffffffu, mbar_wait(empty + 8 * k, ((uint32_t)(c / S) & 1u) ^ 1u))) {
                if (lane == 0) timed_out();
                break;
            }
            const uint32_t dst = smem_u32(smem + k * F::kStageBytes);
            // values, zeros behind the last token: 16 pieces of 16 bytes a token
#pragma unroll 4
            for (int u = lane; u < C * 16; u += 32) {
                const int r = u >> 4, ch = u & 15;
                cp_async16(dst + F::kOffV + r * kDV * 2 + ch * 16,
                           a.v + (int64_t)(q.row0 + c * C + min(r, nv - 1)) * a.v_rs + (int64_t)h * a.v_hs + ch * 8, r < nv ? 16 : 0);
            }
            cp_async_arrive(full + 8 * k);
            if (lane == 0) {
                mbar_expect_tx(full + 8 * k, F::kTileBytes + F::kBlockBytes);
                bulk_g2s(dst, a.tiles + ((base + c) * a.n_head_k + hk) * F::kTileBytes, F::kTileBytes, full + 8 * k);
                bulk_g2s(dst + F::kOffT, a.heads + ((base + c) * a.n_head + h) * kDeltaHeadBytes, F::kBlockBytes, full + 8 * k);
            }
            __syncwarp();
        }
        // no copy may land after the CTA is gone
        for (int k = max(0, c - S); k < c; ++k)
            if (!__all_sync(0xffffffffu, mbar_wait(full + 8 * (k % S), (uint32_t)(k / S) & 1u))) {
                if (lane == 0) timed_out();
                break;
            }
    } else if (warp == 8) {
        // ---------------- products ----------------
        bool alive = true;
        auto wait = [&](uint32_t bar, uint32_t parity) {
            if (alive && !__all_sync(0xffffffffu, mbar_wait(bar, parity))) {
                if (lane == 0) timed_out();
                alive = false;
            }
            tc_fence_after();
            return alive;
        };
        int c = 0;
        for (; c < chunks; ++c) {
            const int k = c % S;
            const uint32_t ph = (uint32_t)c & 1u, at = smem_u32(smem + k * F::kStageBytes);
            const uint64_t kd = tc_desc_sw128(at), qd = tc_desc_sw128(at + C * DK * 2), td = tc_desc_sw128(at + F::kOffT);
            const uint64_t ad = tc_desc_sw128(at + F::kOffA), kn = tc_desc_mn_sw128(at, C * 128);
            auto step = [](int ks) { return (uint64_t)(uint32_t)(((ks >> 2) * C * 128 + (ks & 3) * 32) >> 4); };
            if (!wait(full + 8 * k, (uint32_t)(c / S) & 1u) || !wait(s_ready, ph)) break;
            if (elect_one()) {
                // lo first: what it adds up is small, and hi's sum is cut off no more often than it has steps
#pragma unroll
                for (int ks = 0; ks < DK / 16; ++ks) tc_mma_ts(tmem + kColPK, tmem + kColLo + ks * 8, kd + step(ks), kIdescTok, ks != 0);
#pragma unroll
                for (int ks = 0; ks < DK / 16; ++ks) tc_mma_ts(tmem + kColPK, tmem + kColHi + ks * 8, kd + step(ks), kIdescTok, 1);
                tc_commit(p_full);
                const uint32_t pq = tmem + kColPQ + ph * 32;
                if (T == PAGED_F16) {
#pragma unroll
                    for (int ks = 0; ks < DK / 16; ++ks) tc_mma_ts(pq, tmem + kColLo + ks * 8, qd + step(ks), kIdescTok, ks != 0);
                }
#pragma unroll
                for (int ks = 0; ks < DK / 16; ++ks) tc_mma_ts(pq, tmem + kColHi + ks * 8, qd + step(ks), kIdescTok, T == PAGED_F16 || ks != 0);
            }
            __syncwarp();
            // a 32-token operand (hi at op, lo 16 columns on) times hi and lo of T or A
            auto small = [&](uint32_t to, uint32_t op, uint64_t d) {
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) tc_mma_ts(to, op + ks * 8, d + (uint64_t)(uint32_t)((64 + ks * 32) >> 4), kIdescTok, ks != 0);
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) tc_mma_ts(to, op + 16 + ks * 8, d + (uint64_t)(uint32_t)((ks * 32) >> 4), kIdescTok, 1);
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) tc_mma_ts(to, op + ks * 8, d + (uint64_t)(uint32_t)((ks * 32) >> 4), kIdescTok, 1);
            };
            if (!wait(r_ready, ph)) break;
            if (elect_one()) {
                small(tmem + kColU, tmem + kColR, td);
                tc_commit(u_full);
            }
            __syncwarp();
            if (!wait(w_ready, ph)) break;
            if (elect_one()) {
#pragma unroll
                for (int ks = 0; ks < 2; ++ks)
                    tc_mma_ts(tmem + kColDS, tmem + kColWOp + 16 + ks * 8, kn + (uint64_t)(uint32_t)((ks * 16 * 128) >> 4), kIdescKey, ks != 0);
#pragma unroll
                for (int ks = 0; ks < 2; ++ks)
                    tc_mma_ts(tmem + kColDS, tmem + kColWOp + ks * 8, kn + (uint64_t)(uint32_t)((ks * 16 * 128) >> 4), kIdescKey, 1);
                tc_commit(d_full);
            }
            __syncwarp();
            if (!wait(o_ready, ph)) break;
            if (elect_one()) {
                small(tmem + kColO, tmem + kColUOp, ad);
                tc_commit(o_full);
                tc_commit(empty + 8 * k);
            }
            __syncwarp();
        }
        if (!alive) {                                              // products in flight end before their memory is given back
            if (elect_one()) tc_commit(drain);
            __syncwarp();
            mbar_wait(drain, 0);
        }
    } else {
        // ---------------- rows ----------------
        const int wq = warp & 3, hh = warp >> 2, row = wq * 32 + lane;
        const uint32_t tl = tmem + ((uint32_t)(wq * 32) << 16);
        float *xs = reinterpret_cast<float *>(smem + F::kOffX);
        bool alive = q.ok;
        auto wait = [&](uint32_t bar, uint32_t parity) {
            if (!__all_sync(0xffffffffu, mbar_wait(bar, parity))) {
                if (lane == 0) timed_out();
                alive = false;
            }
            tc_fence_after();
            return alive;
        };
        auto arrive = [&](uint32_t bar) {
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        auto place = [&](int slot) {
            return a.state + (int64_t)slot * a.slot_stride + (int64_t)h * a.head_stride + (int64_t)row * DK + hh * H;
        };
        float st[H];
        float smax = 0.f, su = 1.f, si = 1.f, sb = 0.f;
        if (alive) {
#pragma unroll
            for (int e = 0; e < H; ++e) st[e] = 0.f;
            if (q.slot >= 0) {
                const float *src = place(q.slot);
#pragma unroll
                for (int e = 0; e < H; e += 4) {
                    const float4 x = *reinterpret_cast<const float4 *>(src + e);
                    st[e] = x.x; st[e + 1] = x.y; st[e + 2] = x.z; st[e + 3] = x.w;
                }
            }
#pragma unroll
            for (int e = 0; e < H; ++e) smax = fmaxf(smax, fabsf(st[e]));
            // (the halves' buffers: maxima of R, then of S)
            xs[(1 * 2 + 1) * 256 + warp * 32 + lane] = smax;
            bar_sync(1 + wq, 64);
            sb = fmaxf(smax, xs[(1 * 2 + 1) * 256 + (warp ^ 4) * 32 + lane]);
            su = unit_of(__float_as_uint(sb));
            si = inverse_unit(su);
#pragma unroll
            for (int e = 0; e < H; e += 2) scale2(st[e], st[e + 1], su, su);
        }
        auto put_state = [&]() {
#pragma unroll
            for (int e = 0; e < H; e += 32) {
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int p = 0; p < 16; ++p) split(st[e + 2 * p], st[e + 2 * p + 1], hi[p], lo[p]);
                tmem_st(tl + kColHi + hh * (H / 2) + e / 2, hi);
                tmem_st(tl + kColLo + hh * (H / 2) + e / 2, lo);
            }
            arrive(s_ready);
        };
        // 16 values to the operand at col (hi, 16 columns on lo), this half's eight words of each
        auto put = [&](uint32_t col, const float (&x)[16]) {
            uint32_t hi[8], lo[8];
#pragma unroll
            for (int p = 0; p < 8; ++p) split(x[2 * p], x[2 * p + 1], hi[p], lo[p]);
            tmem_st(tl + col + hh * 8, hi);
            tmem_st(tl + col + 16 + hh * 8, lo);
        };
        if (alive) put_state();
        // (a wait that ran out in one half of the rows: both leave at their next meeting, which neither may miss)
        for (int c = 0; c < chunks; ++c) {
            const int k = c % S, nv = min(C, q.n - c * C);
            const uint32_t ph = (uint32_t)c & 1u;
            const uint8_t *stage = smem + k * F::kStageBytes;
            const HeadScalars *hb = reinterpret_cast<const HeadScalars *>(stage + F::kOffScalars);
            const uint16_t *vt = reinterpret_cast<const uint16_t *>(stage + F::kOffV) + row;
            float *xr = xs + ph * 256 + lane, *xm = xs + (2 + ph) * 256 + lane;
            const bool here = alive && wait(full + 8 * k, (uint32_t)(c / S) & 1u) && wait(p_full, ph);
            // R = beta V - beta exp(G) |k| (S K^T), of 16 tokens
            float r[16];
            float top = 0.f;
            {
                uint32_t x[16];
                tmem_ld(tl + kColPK + hh * 16, x);
                uint32_t v[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] = vt[(hh * 16 + j) * kDV];
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float4 f = hb->r[hh * 8 + j];
                    const uint64_t c2 = mul2(pk2(f.z, f.w), pk2(si, si));
                    upk2(fma2(pk2(f.x, f.y), pk2(from16<T>(v[2 * j]), from16<T>(v[2 * j + 1])),
                              mul2(c2, pk2(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1])))),
                         r[2 * j], r[2 * j + 1]);
                    top = fmaxf(top, fmaxf(fabsf(r[2 * j]), fabsf(r[2 * j + 1])));
                }
            }
            xr[warp * 32] = top;
            if ((c & 3) == 0) xm[warp * 32] = smax;
            if (bar_any(1 + wq, 64, !here)) {
                alive = false;
                break;
            }
            top = fmaxf(top, xr[(warp ^ 4) * 32]);
            if ((c & 3) == 0 && c) sb = fmaxf(smax, xm[(warp ^ 4) * 32]) * si;
            const float ru = unit_of(__float_as_uint(top)) * 0x1p-7f, ui = inverse_unit(ru) * hb->t_unit;
#pragma unroll
            for (int j = 0; j < 16; j += 2) scale2(r[j], r[j + 1], ru, ru);
            put(kColR, r);
            arrive(r_ready);
            // the state's next unit, by a bound (see delta_chunk.cu)
            const float last = hb->last;
            sb = fmaf(last, sb, 1024.f * hb->w_sum * (top * hb->t_unit));
            const float nu = unit_of(__float_as_uint(sb)), wf = ui * nu, keep = last * (si * nu);
            if (!wait(u_full, ph)) continue;
            {
                uint32_t x[16];
                tmem_ld(tl + kColU + hh * 16, x);
                tmem_ld_wait();
                float u[16], w[16];
#pragma unroll
                for (int j = 0; j < 16; j += 2) {
                    u[j] = __uint_as_float(x[j]);
                    u[j + 1] = __uint_as_float(x[j + 1]);
                    const float2 f = *reinterpret_cast<const float2 *>(&hb->w[hh * 16 + j]);
                    upk2(mul2(mul2(pk2(f.x, f.y), pk2(wf, wf)), pk2(u[j], u[j + 1])), w[j], w[j + 1]);
                }
                put(kColWOp, w);
                arrive(w_ready);
                put(kColUOp, u);
                arrive(o_ready);
            }
            if (!wait(d_full, ph)) continue;
            {
                const uint64_t keep2 = pk2(keep, keep);
                smax = 0.f;
#pragma unroll
                for (int e = 0; e < H; e += 32) {
                    uint32_t x[32];
                    tmem_ld32(tl + kColDS + hh * H + e, x);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; j += 2)
                        upk2(fma2(keep2, pk2(st[e + j], st[e + j + 1]), pk2(__uint_as_float(x[j]), __uint_as_float(x[j + 1]))), st[e + j], st[e + j + 1]);
                }
            }
            const float back = ui * hb->a_unit, so = si;
            si = inverse_unit(nu);
            if (c + 1 < chunks) put_state();
            if ((c & 3) == 3) {
#pragma unroll
                for (int e = 0; e < H; ++e) smax = fmaxf(smax, fabsf(st[e]));
            }
            // o = |q| (exp(G) S q + A u), of 16 tokens
            // (S Q^T has been there since d_full, which stands for all products in front of it.  Each of these barriers is
            // waited for before this warp gives what its next phase but one needs: none is overtaken.)
            if (!wait(o_full, ph)) continue;
            {
                uint32_t x[16], y[16];
                tmem_ld(tl + kColPQ + ph * 32 + hh * 16, x);
                tmem_ld(tl + kColO + hh * 16, y);
                tmem_ld_wait();
                uint16_t *to = a.o + (int64_t)(q.row0 + c * C + hh * 16) * a.o_rs + (int64_t)h * a.o_hs + row;
#pragma unroll
                for (int j = 0; j < 16; j += 2) {
                    const float4 f = hb->o[hh * 8 + j / 2];
                    float y0, y1;
                    upk2(fma2(mul2(pk2(f.x, f.y), pk2(back, back)), pk2(__uint_as_float(y[j]), __uint_as_float(y[j + 1])),
                              mul2(mul2(pk2(f.z, f.w), pk2(so, so)), pk2(__uint_as_float(x[j]), __uint_as_float(x[j + 1])))),
                         y0, y1);
                    const uint32_t o2 = T == PAGED_F16 ? pack_half2(y0, y1) : pack_bf162(y0, y1);
                    if (hh * 16 + j < nv) to[(int64_t)j * a.o_rs] = (uint16_t)o2;
                    if (hh * 16 + j + 1 < nv) to[(int64_t)(j + 1) * a.o_rs] = (uint16_t)(o2 >> 16);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(empty + 8 * k);
        }
        if (alive) {
            const int out = a.slot_out[s];
            if (out >= a.n_slots) {
                if (threadIdx.x == 0 && h == 0) atomicOr(a.err, (uint32_t)DELTA_ERR_SLOT);
            } else if (out >= 0) {
                float *dst = place(out);
#pragma unroll
                for (int e = 0; e < H; e += 4)
                    *reinterpret_cast<float4 *>(dst + e) = make_float4(st[e] * si, st[e + 1] * si, st[e + 2] * si, st[e + 3] * si);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int T, int DK> cudaError_t allow() {
    return cudaFuncSetAttribute(k_delta_wide<T, DK>, cudaFuncAttributeMaxDynamicSharedMemorySize, WideCfg<DK>::kSmem);
}

template <int T, int DK>
cudaError_t go(const DeltaArgs &a, cudaStream_t st) {
    using F = WideCfg<DK>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((int64_t)a.n_seq * a.n_head), 1, 1);
    cfg.blockDim = dim3(F::kThreads);
    cfg.dynamicSmemBytes = F::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_delta_wide<T, DK>, a);
}

}  // namespace

cudaError_t delta_wide_setup() {
    cudaError_t e = allow<PAGED_F16, 64>();
    if (e == cudaSuccess) e = allow<PAGED_F16, 128>();
    if (e == cudaSuccess) e = allow<PAGED_BF16, 64>();
    if (e == cudaSuccess) e = allow<PAGED_BF16, 128>();
    return e;
}

cudaError_t launch_delta_wide(const DeltaArgs &a, int dtype, int dim_k, cudaStream_t st) {
    if (dtype == PAGED_F16) return dim_k == 64 ? go<PAGED_F16, 64>(a, st) : go<PAGED_F16, 128>(a, st);
    return dim_k == 64 ? go<PAGED_BF16, 64>(a, st) : go<PAGED_BF16, 128>(a, st);
}

}  // namespace dflash
