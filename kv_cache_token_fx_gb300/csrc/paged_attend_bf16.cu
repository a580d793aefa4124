// fx_paged_attend, prompts over bf16 pages (kernels: paged_attend.cuh; a unit of its own, compiled beside
// the others).
#include "paged_attend.cuh"

namespace fx {

cudaError_t launch_paged_attend_bf16(const PagedAttendParams& p, bool pdl, cudaStream_t s)
{
    return launch_attend<false, false>(p, pdl, s);
}

}  // namespace fx
