// fx_paged_attend, prompts over bf16 pages whose tables have room for long rows (kernels: paged_attend.cuh; a unit of its own, compiled beside
// the others).
#include "paged_attend.cuh"

namespace fx {

cudaError_t launch_paged_attend_long_bf16(const PagedAttendParams& p, bool pdl, cudaStream_t s)
{
    return launch_attend<false, true>(p, pdl, s);
}

}  // namespace fx
