// The tensor-core attention kernels for bf16 queries.
#include "paged_prefill_launch.cuh"

namespace dflash {
template cudaError_t paged_prefill_setup_t<PAGED_BF16>();
template cudaError_t launch_paged_prefill_t<PAGED_BF16>(const PagedAttendArgs &, const CUtensorMap &, const CUtensorMap &,
                                                 const CUtensorMap &, int, cudaStream_t);
}  // namespace dflash
