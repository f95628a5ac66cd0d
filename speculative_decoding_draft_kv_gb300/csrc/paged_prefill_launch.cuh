// Choice and launch of the tensor-core attention kernels of one query type.
#pragma once

#include "paged_attend_launch.cuh"
#include "paged_prefill.cuh"

namespace dflash {

// one: every item fits a block
template <int T, class F>
cudaError_t pick_prefill(int head_dim, int format, bool one, F &&fn) {
    auto with = [&](auto d, auto fmt, auto single) {
        using C = PreCfg<d.value, fmt.value, T, single.value>;
        // registers a thread that the launch has to bring for the shares that its warps ask for
        constexpr int regs = C::kMore ? (256 * C::kManyRegs + (C::kThreads - 256) * C::kFewRegs) / C::kThreads : 0;
        return fn(k_paged_prefill<d.value, fmt.value, T, single.value>, C::kSmem, C::kThreads, regs);
    };
    auto blocks = [&](auto d, auto fmt) { return one ? with(d, fmt, std::true_type{}) : with(d, fmt, std::false_type{}); };
    auto dim = [&](auto fmt) {
        return head_dim == 64 ? blocks(std::integral_constant<int, 64>{}, fmt) : blocks(std::integral_constant<int, 128>{}, fmt);
    };
    if (format == PAGED_INT8) return dim(std::integral_constant<int, kFmtInt8>{});
    if (format == PAGED_E4M3) return dim(std::integral_constant<int, kFmtE4m3>{});
    return dim(std::integral_constant<int, kFmt16>{});
}

template <int T>
cudaError_t paged_prefill_setup_t() {
    auto allow = [](auto kernel, int smem, int, int regs) {
        cudaFuncAttributes at;
        const cudaError_t e = cudaFuncGetAttributes(&at, kernel);
        if (e != cudaSuccess) return e;
        if (at.numRegs < regs) return cudaErrorLaunchOutOfResources;   // its warps would wait for registers for ever
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    };
    const int formats[3] = {T, PAGED_INT8, PAGED_E4M3};
    for (int f : formats)
        for (int d = 64; d <= 128; d += 64)
            for (int one = 0; one < 2; ++one) {
                const cudaError_t e = pick_prefill<T>(d, f, one != 0, allow);
                if (e != cudaSuccess) return e;
            }
    return cudaSuccess;
}

template <int T>
cudaError_t launch_paged_prefill_t(const PagedAttendArgs &a, const CUtensorMap &tm_k, const CUtensorMap &tm_v,
                                   const CUtensorMap &tm_q, int head_dim, cudaStream_t st) {
    return pick_prefill<T>(head_dim, a.pool.format, a.tile_rows <= 128, [&](auto kernel, int smem, int threads, int) {
        kernel<<<a.ctas, threads, smem, st>>>(tm_k, tm_v, tm_q, a);
        const cudaError_t e = cudaGetLastError();
        return e == cudaSuccess ? launch_join<T, 1>(a, head_dim, st) : e;
    });
}

}  // namespace dflash
