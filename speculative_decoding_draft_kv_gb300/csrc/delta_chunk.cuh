// What the kernels of the gated delta rule over many tokens share.
#pragma once

#include "delta.h"

#include "ring_internal.h"
#include "ptx.h"
#include "paged_ptx.h"

namespace dflash {
namespace {

constexpr int C = kDeltaChunk;                         // tokens of a chunk
static_assert(C == 32, "a lane per token");

template <int T> __device__ __forceinline__ float from16(uint32_t x) {
    if constexpr (T == PAGED_F16) return __half2float(__ushort_as_half((unsigned short)x));
    else return __uint_as_float(x << 16);
}
__device__ __forceinline__ float2 half2_floats(uint32_t x) { return __half22float2(*reinterpret_cast<const __half2 *>(&x)); }

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

// Byte offset of 16-byte chunk ch of row r in a tile of 32 rows of F16: runs of 64 columns one behind another, with the
// 128-byte swizzle -- conflict-free for ldmatrix, and what tcgen05.mma reads along rows as along columns.
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
    float last, t_unit, a_unit, w_sum;                 // exp(G_last); what T and A are to be multiplied by; sum of w
};
// A head's part of a chunk in the workspace, for mma.sync: B operands of T and of A (exp(G_i - G_j) q_i . k_j), a lane's
// words beside one another (hi, hi, lo, lo).
struct HeadBlock {
    uint4 t[kBlocks][32], a[kBlocks][32];
    HeadScalars s;
};
// The same for tcgen05.mma: 32 rows of 64 columns, hi beside lo, with the 128-byte swizzle.
struct WideBlock {
    uint4 t[C][8], a[C][8];
    HeadScalars s;
};
static_assert(sizeof(HeadBlock) <= kDeltaHeadBytes && sizeof(WideBlock) <= kDeltaHeadBytes && kDeltaHeadBytes % 128 == 0, "as the workspace is laid out");

__device__ __forceinline__ int chunk_base(int row0, int s) { return row0 / C + s; }

// the power of two that brings m > 0 (as bits) to [2^12, 2^13), as far as float32 has it and its inverse
__device__ __forceinline__ float unit_of(uint32_t bits) {
    const int e = (int)(bits >> 23);                   // biased
    return bits == 0u || e == 255 ? 1.f : __uint_as_float((uint32_t)min(241, max(13, 254 + 12 - e)) << 23);
}
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

}  // namespace
}  // namespace dflash
