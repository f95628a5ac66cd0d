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
        kernel<<<a.ctas, threads, smem, st>>>(tm_k, tm_v, a);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        return launch_join<T, 8>(a, head_dim, st);
    };
    const int mt = a.tile_rows <= 16 ? 1 : 2;
    return head_dim == 64 ? pick_attend<T, 64>(a.pool.format, mt, go) : pick_attend<T, 128>(a.pool.format, mt, go);
}

}  // namespace dflash
