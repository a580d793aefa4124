// fx_paged_decode and fx_paged_importance: the launchers of the kernels in paged_attn.cuh.
#include "paged_attn.cuh"

namespace fx {
namespace {

template <bool E2M1>
cudaError_t launch_importance(const PagedAttnParams& p, int sm_count, bool pdl, cudaStream_t s)
{
    constexpr size_t ring = (size_t)kImpWarps * imp_stages(E2M1) * Slot<E2M1, false, E2M1 ? 2 : 1>::kBytes;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(paged_importance_kernel<E2M1>, ring + kMaxRows / 8 * 2048, done);
    if (e != cudaSuccess) return e;
    return launch_kernel(paged_importance_kernel<E2M1>, dim3(imp_ctas(E2M1) * sm_count), dim3(32 * kImpWarps), ring + (p.R + 7) / 8 * 2048, s,
                         pdl, 0u, p);
}

}  // namespace

// The counters' region, then two partials (one of each end of a CTA's stretch) per CTA.
size_t paged_decode_workspace_bytes(int R, int sm_count)
{
    const size_t rows = R <= 4 ? 4 : (R <= 8 ? 8 : 16), ctas = (size_t)(R <= 8 ? 3 : 2) * sm_count;
    return kCounterBytes + ctas * 2 * rows * (kHeadDim + 2) * sizeof(float);
}

cudaError_t launch_paged_decode(const PagedAttnParams& p, bool e2m1, int sm_count, bool pdl, cudaStream_t s)
{
    return e2m1 ? launch_decode_e2m1<0>(p, sm_count, pdl, s) : launch_decode_bf16<0>(p, sm_count, pdl, s);
}

cudaError_t launch_paged_importance(const PagedAttnParams& p, bool e2m1, int sm_count, bool pdl, cudaStream_t s)
{
    return e2m1 ? launch_importance<true>(p, sm_count, pdl, s) : launch_importance<false>(p, sm_count, pdl, s);
}

}  // namespace fx
