// fx_paged_attend, prompts over 4-bit pages (kernels: paged_attend.cuh; a unit of its own, compiled beside
// the others).
#include "paged_attend.cuh"

namespace fx {

cudaError_t launch_paged_attend_e2m1(const PagedAttendParams& p, bool pdl, cudaStream_t s)
{
    return launch_attend<true, false>(p, pdl, s);
}

}  // namespace fx
