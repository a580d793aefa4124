// fx_paged_attend over 4-bit pages, without a cap on the scores, where a (sequence, KV head) has few query rows: decode steps
// and drafts, bound by the cache's bytes (kernels: paged_attn.cuh; a unit of its own, compiled beside the others).
#include "paged_attn.cuh"

namespace fx {

cudaError_t launch_paged_attend_few_e2m1_open(const PagedAttnParams& p, int sm_count, bool pdl, cudaStream_t s)
{
    return launch_decode_e2m1<1>(p, sm_count, pdl, s);
}

}  // namespace fx
