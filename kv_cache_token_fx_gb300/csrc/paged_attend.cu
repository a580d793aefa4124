// fx_paged_attend, prompts: how a call is cut, its scratch memory, and which kernel of paged_attend.cuh takes it.
#include "paged_attend.cuh"

namespace fx {

// A call whose blocks leave SMs without work is cut along the cache: one part to a CTA, one CTA to an SM.
PagedAttendCut paged_attend_cut(int B, int Hkv, int G, int64_t max_new, int cap, int sm_count)
{
    PagedAttendCut c;
    const int64_t rows = max_new * G;
    c.blocks = (int)((rows + kBlock - 1) / kBlock);
    c.part_rows = (int)(rows < kBlock ? rows : kBlock);
    const int64_t plan = (int64_t)B * c.blocks;
    c.split = plan <= kMaxPlan && plan * Hkv < sm_count ? sm_count : 0;
    c.slots = !c.split && cap > kFlush * kKeys ? sm_count : 0;   // (a part's own place takes the sums of a call that is cut)
    return c;
}
size_t paged_attend_workspace_bytes(const PagedAttendCut& c)
{
    return kCounterBytes + (c.split ? (size_t)c.split * c.part_rows * (kHeadDim + 2) : (size_t)c.slots * kBlock * kHeadDim) * sizeof(float);
}
// Of every call of up to `rows` query rows a (sequence, KV head), with any table: one of a single block each is cut if any is,
// and a part has no more rows than a block.
size_t paged_attend_workspace_bound(int B, int Hkv, int64_t rows, int sm_count)
{
    PagedAttendCut c;
    c.split = paged_attend_cut(B, Hkv, 1, 1, 0, sm_count).split;
    c.part_rows = (int)(rows < kBlock ? rows : kBlock);
    c.slots = sm_count;
    const size_t cut = paged_attend_workspace_bytes(c);
    c.split = 0;
    const size_t whole = paged_attend_workspace_bytes(c);
    return cut > whole ? cut : whole;
}

cudaError_t launch_paged_attend(const PagedAttendParams& p, bool e2m1, bool pdl, cudaStream_t s)
{
    if (p.c.cap > kFlush * kKeys) return e2m1 ? launch_paged_attend_long_e2m1(p, pdl, s) : launch_paged_attend_long_bf16(p, pdl, s);
    return e2m1 ? launch_paged_attend_e2m1(p, pdl, s) : launch_paged_attend_bf16(p, pdl, s);
}

}  // namespace fx
