// The attention and join kernels for bf16 queries.
#include "paged_attend_launch.cuh"

namespace dflash {
template cudaError_t paged_attend_setup_t<PAGED_BF16>();
template cudaError_t launch_paged_attend_t<PAGED_BF16>(const PagedAttendArgs &, const CUtensorMap &, const CUtensorMap &, int,
                                                cudaStream_t);
}  // namespace dflash
