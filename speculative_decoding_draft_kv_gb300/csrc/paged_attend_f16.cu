// The attention and join kernels for f16 queries.
#include "paged_attend_launch.cuh"

namespace dflash {
template cudaError_t paged_attend_setup_t<PAGED_F16>();
template cudaError_t launch_paged_attend_t<PAGED_F16>(const PagedAttendArgs &, const CUtensorMap &, const CUtensorMap &, int,
                                                cudaStream_t);
}  // namespace dflash
