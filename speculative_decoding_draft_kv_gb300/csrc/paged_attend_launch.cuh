// Choice and launch of the attention kernels of one query type.
#pragma once

#include "paged_attend.cuh"

#include <algorithm>

namespace dflash {

// The join settles while the attention runs, and waits for its end.
template <int T, int W>
cudaError_t launch_join(const PagedAttendArgs &a, int head_dim, cudaStream_t st) {
    const int rows = std::min<int64_t>(a.tile_rows, (int64_t)a.max_q * a.group);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.ctas, (unsigned)((rows * W + 7) / 8), 1);
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return head_dim == 64 ? cudaLaunchKernelEx(&cfg, k_paged_join<64, T, W>, a)
                          : cudaLaunchKernelEx(&cfg, k_paged_join<128, T, W>, a);
}

// Two passes' join, which settles as the other one does.  Rows to a block: as few as leave one wave of blocks, five to
// an SM; warps to a (row, query head): what a block has left.
template <int T>
cudaError_t launch_levels(const PagedAttendArgs &prefix, const PagedAttendArgs &own, int head_dim, cudaStream_t st) {
    const int64_t n = own.batch.n_rows;
    int rows = 1, wide = 8;
    while (rows < 16 && (n + rows - 1) / rows * own.pool.n_head_kv > 5 * own.sms) rows *= 2;
    while (wide > 1 && rows * own.group * wide > 8) wide /= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((n + rows - 1) / rows * own.pool.n_head_kv), 1, 1);
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return head_dim == 64 ? cudaLaunchKernelEx(&cfg, k_paged_levels<64, T>, prefix, own, rows, wide)
                          : cudaLaunchKernelEx(&cfg, k_paged_levels<128, T>, prefix, own, rows, wide);
}

// What joins a pass's states: of the only one those of cut items, behind the second of two both passes'.
template <int T, int W>
cudaError_t launch_behind(const PagedAttendArgs &a, int head_dim, cudaStream_t st) {
    if (a.level == kOnly) return launch_join<T, W>(a, head_dim, st);
    return a.level == kOwn ? launch_levels<T>(*a.first, a, head_dim, st) : cudaSuccess;
}

// A pass of the attention.  The second of two may begin while the first one runs: it reads nothing of that.
template <class K, class... Args>
cudaError_t launch_pass(K kernel, const PagedAttendArgs &a, int threads, int smem, cudaStream_t st, const Args &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.ctas, 1, 1);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.level == kOwn ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// fn(kernel, its shared memory, threads, rows) for one of the instances
template <int T, int D, int MT, int FMT, class F>
cudaError_t with_attend(F &&fn) {
    using C = DecCfg<D, MT, FMT>;
    return fn(k_paged_attend<D, MT, FMT, T>, C::kSmem, C::kThreads, C::kRows);
}

template <int T, int D, class F>
cudaError_t pick_attend(int format, int mt, F &&fn) {
    // (16-bit pages come here with up to 16 rows only)
    if (format == PAGED_INT8) return mt == 1 ? with_attend<T, D, 1, kFmtInt8>(fn) : with_attend<T, D, 2, kFmtInt8>(fn);
    if (format == PAGED_E4M3) return mt == 1 ? with_attend<T, D, 1, kFmtE4m3>(fn) : with_attend<T, D, 2, kFmtE4m3>(fn);
    return with_attend<T, D, 1, kFmt16>(fn);
}

template <int T>
cudaError_t paged_attend_setup_t() {
    auto allow = [](auto kernel, int smem, int, int) {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    };
    const int formats[3] = {T, PAGED_INT8, PAGED_E4M3};
    for (int f : formats)
        for (int mt = 1; mt <= 2; ++mt) {
            cudaError_t e = pick_attend<T, 64>(f, mt, allow);
            if (e == cudaSuccess) e = pick_attend<T, 128>(f, mt, allow);
            if (e != cudaSuccess) return e;
        }
    return cudaSuccess;
}

template <int T>
cudaError_t launch_paged_attend_t(const PagedAttendArgs &a, const CUtensorMap &tm_k, const CUtensorMap &tm_v,
                                  int head_dim, cudaStream_t st) {
    auto go = [&](auto kernel, int smem, int threads, int) {
        const cudaError_t e = launch_pass(kernel, a, threads, smem, st, tm_k, tm_v, a);
        return e == cudaSuccess ? launch_behind<T, 8>(a, head_dim, st) : e;
    };
    const int mt = a.tile_rows <= 16 ? 1 : 2;
    return head_dim == 64 ? pick_attend<T, 64>(a.pool.format, mt, go) : pick_attend<T, 128>(a.pool.format, mt, go);
}

}  // namespace dflash
