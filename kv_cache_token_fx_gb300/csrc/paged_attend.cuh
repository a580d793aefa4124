// Attention of ragged new tokens -- a prompt's, a chunk's, or one of every sequence -- over a paged cache for sm_103a
// (tcgen05, accumulators in tensor memory): fx_paged_attend.
//
// The query rows of a (sequence, KV head) are its new tokens' G heads, token by token: row r is head r % G of token
// r / G.  A CTA takes 256 of them as two subtiles of 128 and walks the tiles of 128 cache rows that any of them sees:
//   S = Q K^T   (M = 128 query rows, N = 128 cache rows, K = 128 dimensions)   shared x shared -> tensor memory
//   O += P V    (M = 128 query rows, N = 128 dimensions, K = 128 cache rows)   tensor memory x shared -> tensor memory
// with an online softmax between them, P in the place of S.  Warps 0-3 and 4-7 are the softmax of the two subtiles, one
// thread a query row, so that no row is shared; one subtile's products run while the other's weights are formed.  Warps
// 8-11 fill a ring of operand slots (K and V tiles in turn) through the page table, warp 12 issues the products.
//
// bf16 pages: rows go to the swizzled slots by cp.async, as they are.  4-bit pages: codes and scales go to a small ring of
// their own and become f16 values there (exact: at most 6 significant bits between 2^-10 and 2688); queries are f16 scaled
// by a power of two per row (largest magnitude in [2^14, 2^15)), so no bit of a bf16 query within 2^-24 of its row's
// largest is lost.
//
// P is rounded once, to the operands' type (bf16: at most 2^-8 of a weight; f16: 2^-11): the output is bf16, whose rounding is as
// large, and a second part would be another product with V for every tile, half as many again as there are.  (The decode, whose
// output is fp32 and whose time is the cache's bytes, holds weights in two or three parts.)  Logits, maxima, sums and O are fp32;
// over long rows O leaves the tensor core for memory (kFlush).
//
// Calls of fewer blocks than SMs are cut along the cache: every block's tiles become parts of nearly equal length by the
// lengths found on the device, and the last CTA of a block to arrive joins its parts in their order.  (Calls of few
// query rows a (sequence, KV head) go to the kernels of paged_attn.cuh, which are bound by the cache's bytes.)
//
// (Template code: paged_attend_*.cu make the kernels of one format each, side by side; paged_attend.cu chooses.)
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include <atomic>

#include "paged.cuh"
#include "tc_ptx.cuh"

namespace fx {
namespace {

constexpr int kThreadsA = 512;
constexpr int kSub = 128;                        // query rows of a subtile: one tensor-memory lane each
constexpr int kBlock = 2 * kSub;                 // query rows of a CTA
constexpr int kKeys = 128;                       // cache rows of a tile
constexpr int kOperand = 128 * 128 * 2;          // bytes of an operand tile
constexpr int kRawTile = kKeys * 64 + kKeys * 8; // codes and scales of a 4-bit tile (K or V)
constexpr int kRaw = 3;                          // such tiles in their ring
// slots of the operand ring: what fits beside Q (and the raw ring)
__host__ __device__ constexpr int slots(bool e2m1) { return e2m1 ? 4 : 5; }
__host__ __device__ constexpr int attend_smem(bool e2m1)
{
    return 2 * kOperand + slots(e2m1) * kOperand + (e2m1 ? kRaw * kRawTile : 0) + 1024;
}
constexpr int kLag = 1;                          // bf16: tiles whose copies are under way
// Registers a thread of the softmax, the fillers and the issuing warp; the launch's 128 a thread cover their sum.
constexpr int kRegsSoftmax = 184, kRegsFill = 88, kRegsIssue = 56;
static_assert(2 * kRegsSoftmax + kRegsFill + kRegsIssue <= 4 * 128, "a split above the launch's registers never starts");
// tensor-memory columns: S (P in its first half) of the subtiles, O of the subtiles
__device__ __forceinline__ uint32_t col_s(int x) { return (uint32_t)(x * 128); }
__device__ __forceinline__ uint32_t col_o(int x) { return (uint32_t)(256 + x * 128); }
constexpr int kRing = 16;                        // tiles whose flags are kept (the fillers are at most 4 ahead, and what
                                                 // they clear lies 8 behind)
// The largest weight so far is 2^kWeightBase when its row's reference moves, and grows by 2^kMaxSlack at most before it
// moves again.  f16: small weights stay normal numbers.  bf16: sums of products with values up to the type's largest
// stay finite, as their mean is.
enum Mode { kPlain, kCap, kBias };   // what is put on the logits: nothing, a cap, a bias by distance (and perhaps a cap)
template <bool E2M1>
constexpr float kWeightBase = E2M1 ? 6.f : -32.f;
// Caps up to which two forms of tanh are mixed: the one that is off by 2^-21 of 1 leaves 2^-15 of a logit at most then, a
// sixteenth of what f16 weights are rounded by (bf16: a 128th).
constexpr float kMixedCap = 64.f;
constexpr float kFarRef = 4194304.f;   // 2^22: beyond it products and their rounded values lie too far apart for one fma

// The tensor core adds P V to O with O's lowest bits cut off: equal bf16 weights over 2^20 rows lost 0.36% of their mean, over
// 2^22 rows 2.2% (2^17 rows: 0.02%, an 18th of the output's rounding).  So over longer rows O leaves for fp32 sums in memory
// every kFlush tiles, 2^17 rows.
constexpr int kFlush = 1024;

constexpr int kMaxPlan = 256;                    // (sequence, block) pairs of a call that is cut along the cache

struct AttendSmem {
    uint64_t full[5], empty[5], q_full, s_full[2], p_full[2], o_done[2];
    uint32_t tmem;
    int4 seen[8];                                // of a warp's query rows: rows that some see, rows that all see
    unsigned skip[kRing];                        // 16-row groups of a tile that lie in bad pages
    float q_factor[kBlock];                      // 4-bit pages: what the f16 queries' logits are multiplied by; then the
                                                 // references of the sums in memory (registers are short)
    unsigned bad_v[kRing][4];                    // rows of a tile whose V is not finite (only where not all see them)
    int slot;                                    // where O's sums lie, in calls that are not cut along the cache; -1: nowhere
    int flags;                                   // kBadV, kSkip: some tile of this CTA has such rows
    int scan[16];
    int plan_i, plan_at, plan_parts, total;
    unsigned last;
};
constexpr int kBadV = 1, kSkip = 2;
static_assert(attend_smem(true) + sizeof(AttendSmem) <= 227 * 1024 && attend_smem(false) + sizeof(AttendSmem) <= 227 * 1024,
              "shared memory of a CTA");

// One wait, given up after kSpinLimit polls; after a first such no later one is waited for.
__device__ __forceinline__ void wait(uint64_t* bar, unsigned parity, unsigned* err, bool& dead)
{
    if (dead) return;
    unsigned spins = 0, done = 0;
    while (!done) {
        asm volatile(
            "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(smem_addr(bar)), "r"(parity)
            : "memory");
        if (!done && ++spins == kSpinLimit) {
            atomicOr(err, FX_DEVERR_TIMEOUT);
            dead = true;
            break;
        }
    }
}
__device__ __forceinline__ void arrive(uint64_t* bar)
{
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void init_barrier(uint64_t* bar, unsigned count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(count));
}
__device__ __forceinline__ void fence_operands() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "mov.b64 rc, {%6, %7};\n\tfma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
template <bool E2M1>
__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    if (E2M1) {
        const __half2 v = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// Instruction descriptor: 16-bit x 16-bit -> fp32, 128 x 128, A K-major, B K-major or MN-major.
template <bool E2M1>
__host__ __device__ constexpr uint32_t idesc(bool b_mn_major)
{
    const uint32_t d = idesc_bf16(128, 128, b_mn_major);
    return E2M1 ? d & ~((1u << 7) | (1u << 10)) : d;   // (both operands f16 instead of bf16)
}

// One lane of the warp, as a predicate that the compiler knows for one: what the products take then stays in uniform
// registers (with lane == 0 in its place each product took 115 cycles to issue, twice its time on the tensor core).
__device__ __forceinline__ bool elect_lane()
{
    uint32_t on;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(on));
    return on != 0;
}
// The low words of an operand's descriptors (their high words are one constant).
__device__ __forceinline__ uint32_t sdesc_low(uint32_t saddr, uint32_t lbo) { return ((saddr & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16); }
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);

// S = Q K^T: eight steps of 16 dimensions.  q, k: the low words of the tiles' first descriptors.
template <bool E2M1>
__device__ __forceinline__ void mma_qk(uint32_t d_tmem, uint32_t q, uint32_t k)
{
    constexpr uint32_t kIdesc = idesc<E2M1>(false);
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
        const uint32_t off = (uint32_t)((ks >> 2) * (kOperand / 2) + (ks & 3) * 32) >> 4;
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tmov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\tsetp.ne.u32 p, %5, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d_tmem),
            "r"(q + off), "r"(k + off), "n"(kDescHigh), "n"(kIdesc), "r"(ks > 0 ? 1u : 0u));
    }
}
// O (+)= P V: eight steps of 16 cache rows.  v: the low word of the tile's first descriptor.
template <bool E2M1>
__device__ __forceinline__ void mma_pv(uint32_t d_tmem, uint32_t p_tmem, uint32_t v, uint32_t accumulate)
{
    constexpr uint32_t kIdesc = idesc<E2M1>(true);
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tmov.b64 b, {%2, %3};\n\tsetp.ne.u32 p, %5, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d_tmem),
            "r"(p_tmem + 8 * ks), "r"(v + (uint32_t)(ks * 2048 >> 4)), "n"(kDescHigh), "n"(kIdesc), "r"(ks > 0 ? 1u : accumulate));
    }
}

// 128 columns of this thread's tensor-memory lane, four loads under way together.
__device__ __forceinline__ void tmem_issue32(uint32_t addr, uint32_t* u)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]),
          "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]),
          "=r"(u[16]), "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]),
          "=r"(u[24]), "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_row(uint32_t addr, float (&s)[128])
{
    uint32_t u[128];
#pragma unroll
    for (int c = 0; c < 4; ++c) tmem_issue32(addr + 32 * c, u + 32 * c);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 128; ++i) {
        asm volatile("" : "+r"(u[i]));   // (used after the wait only)
        s[i] = __uint_as_float(u[i]);
    }
}

// 32 columns of this thread's tensor-memory lane, without waiting for the store.
__device__ __forceinline__ void tmem_put32(uint32_t addr, const uint32_t (&u)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
        "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]),
        "r"(u[9]), "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]), "r"(u[16]), "r"(u[17]),
        "r"(u[18]), "r"(u[19]), "r"(u[20]), "r"(u[21]), "r"(u[22]), "r"(u[23]), "r"(u[24]), "r"(u[25]), "r"(u[26]),
        "r"(u[27]), "r"(u[28]), "r"(u[29]), "r"(u[30]), "r"(u[31])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// ---- the fillers -------------------------------------------------------------------------------------
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool on)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(on ? 16u : 0u) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void* src, bool on)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;\n" ::"r"(dst), "l"(src), "r"(on ? 8u : 0u) : "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void commit_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_copies()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a) : "memory");
    return r;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a)
{
    uint16_t r;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(r) : "r"(a) : "memory");
    return r;
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// The page of 16-row group lane % 8 of a tile: -1 for a group without a row in [lo, hi), -2 for a bad entry.
__device__ __forceinline__ int group_page(const PagedCache& c, const int32_t* table, int tile, int lo, int hi, unsigned* err)
{
    const int row = tile * kKeys + 16 * (threadIdx.x & 7);
    if (row >= hi || row + 16 <= lo) return -1;
    const int pg = table[row >> c.page_shift];
    if ((unsigned)pg < (unsigned)c.n_pages) return pg;
    if ((threadIdx.x & 31) < 8) atomicOr(err, FX_DEVERR_PAGE);
    return -2;
}
__device__ __forceinline__ unsigned bad_groups(int page) { return __ballot_sync(0xffffffffu, page == -2) & 0xffu; }

// Whether 16 bytes of bf16 values hold an infinity or a NaN.
__device__ __forceinline__ bool not_finite(uint4 x)
{
    const uint32_t e = 0x7f807f80u;
    return (__vcmpeq2(x.x & e, e) | __vcmpeq2(x.y & e, e) | __vcmpeq2(x.z & e, e) | __vcmpeq2(x.w & e, e)) != 0;
}

struct FillRange {
    int ta, tb;           // tiles
    int lo, hi;           // rows that some query sees
    int com_lo, com_hi;   // rows that all see
    // whether a tile has rows that only some of the queries see
    __device__ __forceinline__ bool partial(int t) const
    {
        const int a = t * kKeys, b = a + kKeys;
        return max(a, lo) < min(b, com_lo) || max(a, com_hi) < min(b, hi);
    }
};

// Where the rows of a tile lie: lane g (of every eight) holds 16-row group g.
struct Groups {
    int64_t at;      // the group's first row from row 0 of page 0 (of this head), scales too
    int64_t scale;
    unsigned good;   // groups with a page
    bool whole;      // all rows of the tile are copied
};
template <bool E2M1>
__device__ __forceinline__ Groups find_groups(const PagedCache& c, int page, int tile, const FillRange& r)
{
    Groups g;
    const uint32_t in = (uint32_t)((tile * kKeys + 16 * (threadIdx.x & 7)) & c.page_mask), pg = (uint32_t)max(page, 0);
    g.at = (int64_t)((uint64_t)pg * c.sp + (uint64_t)in * c.st);
    g.scale = E2M1 ? (int64_t)((uint64_t)pg * c.ssp + (uint64_t)in * c.sst) : 0;
    g.good = __ballot_sync(0xffffffffu, page >= 0) & 0xffu;
    g.whole = g.good == 0xffu && tile * kKeys >= r.lo && (tile + 1) * kKeys <= r.hi;
    return g;
}
__device__ __forceinline__ int64_t group_at(int64_t mine, int g)
{
    return (int64_t)__shfl_sync(0xffffffffu, (long long)mine, g);
}
// The flags of tile t, for the softmax; clears those of a later one.
__device__ __forceinline__ void put_flags(AttendSmem& sm, int page, int t)
{
    const unsigned bad = bad_groups(page);
    if ((threadIdx.x & 127) == 0) {
        sm.skip[t & (kRing - 1)] = bad;
        if (bad) atomicOr(&sm.flags, kSkip);
#pragma unroll
        for (int w = 0; w < 4; ++w) sm.bad_v[(t + 8) & (kRing - 1)][w] = 0u;   // (the tile that had these is long done)
    }
}

// bf16: a thread copies 16-byte chunk tid % 16 of rows tid / 16 + 8 i of every tile.  A tile whose rows are all copied --
// most are -- takes a copy and an addition for each 16 bytes.
__device__ __forceinline__ void fill_bf16(const PagedAttendParams& p, AttendSmem& sm, uint32_t ring, const int32_t* table, int h,
                                          const FillRange& r)
{
    constexpr int kSlots = slots(false);
    const PagedCache& c = p.c;
    const int tid = threadIdx.x & 127, chunk = tid & 15, row0 = tid >> 4;
    const int n = 2 * (r.tb - r.ta);
    const uint32_t to = sw128(row0, 8 * chunk, kKeys);
    const char* const kb = c.k + (int64_t)h * c.sh + 16 * chunk;
    const int64_t mine = (int64_t)row0 * c.st, eight = 8 * (int64_t)c.st, dv = c.v - c.k;
    bool dead = false;
    auto landed = [&](int m) {   // tile m's copies have landed
        if ((m & 1) && r.partial(r.ta + (m >> 1))) {
            const int t = r.ta + (m >> 1);
            const uint32_t at = ring + (m % kSlots) * kOperand + to;
#pragma unroll 1
            for (int i = 0; i < 16; ++i) {
                if (!not_finite(lds128(at + 1024 * i))) continue;
                sts128(at + 1024 * i, make_uint4(0u, 0u, 0u, 0u));
                const int row = row0 + 8 * i;
                atomicOr(&sm.bad_v[t & (kRing - 1)][row >> 5], 1u << (row & 31));
                atomicOr(&sm.flags, kBadV);
            }
        }
        fence_operands();
        arrive(&sm.full[m % kSlots]);
    };
    int next = group_page(c, table, r.ta, r.lo, r.hi, p.err);
    int slot = 0, turn = 0;
    for (int t = r.ta; t < r.tb; ++t) {
        const int page = next;
        if (t + 1 < r.tb) next = group_page(c, table, t + 1, r.lo, r.hi, p.err);
        put_flags(sm, page, t);
        const Groups g = find_groups<false>(c, page, t, r);
        const char* src[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) src[u] = kb + mine + group_at(g.at, u);
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            if (turn > 0) wait(&sm.empty[slot], (unsigned)(turn - 1) & 1u, p.err, dead);
            const uint32_t dst = ring + slot * kOperand + to;
            if (g.whole) {
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    cp16(dst + 2048 * u, src[u]);
                    cp16(dst + 2048 * u + 1024, src[u] + eight);
                }
            } else {
#pragma unroll
                for (int u = 0; u < 16; ++u) {
                    const int row = t * kKeys + row0 + 8 * u;
                    const bool on = ((g.good >> (u >> 1)) & 1u) && row >= r.lo && row < r.hi;
                    copy16(dst + 1024 * u, on ? src[u >> 1] + (u & 1) * eight : kb, on);
                }
            }
            commit_copies();
            const int m = 2 * (t - r.ta) + which;
            if (m >= kLag) {
                wait_copies<kLag>();
                landed(m - kLag);
            }
            if (++slot == kSlots) {
                slot = 0;
                ++turn;
            }
            if (which == 0) {
#pragma unroll
                for (int u = 0; u < 8; ++u) src[u] += dv;
            }
        }
    }
    wait_copies<0>();
    for (int m = max(n - kLag, 0); m < n; ++m) landed(m);
}

// 4 bits: lane l of a warp takes chunk l / 8 (32 values) of rows 8 warp + l % 8 + 32 i, so that neither the codes' nor the
// values' chunks of eight lanes meet in a bank.
__device__ __forceinline__ void fill_e2m1(const PagedAttendParams& p, AttendSmem& sm, uint32_t ring, uint32_t raw,
                                          const int32_t* table, int h, const FillRange& r)
{
    constexpr int kSlots = slots(true);
    const PagedCache& c = p.c;
    const int tid = threadIdx.x & 127, lane = tid & 31, chunk = lane >> 3, row0 = (tid >> 5) * 8 + (lane & 7);
    const int n = 2 * (r.tb - r.ta), g0 = row0 >> 4;   // the warp's rows lie in groups g0 + 2 i
    const uint32_t from = (uint32_t)(row0 * 64 + ((chunk ^ ((row0 >> 1) & 3)) << 4));
    const char* const kb = c.k + (int64_t)h * c.sh + 16 * chunk + (int64_t)(row0 & 15) * c.st;
    const char* const sb = c.ks + (int64_t)h * c.ssh + (int64_t)(row0 & 15) * c.sst;
    const int64_t dv = c.v - c.k, ds = c.vs - c.ks;
    bool dead = false;
    int next = group_page(c, table, r.ta, r.lo, r.hi, p.err);
    Groups g = {};
    auto feed = [&](int m) {
        if (m < n) {
            const int t = r.ta + (m >> 1);
            if ((m & 1) == 0) {
                const int page = next;
                if (t + 1 < r.tb) next = group_page(c, table, t + 1, r.lo, r.hi, p.err);
                put_flags(sm, page, t);
                g = find_groups<true>(c, page, t, r);
            }
            const uint32_t dst = raw + (m % kRaw) * kRawTile, sdst = dst + kKeys * 64 + row0 * 8;
            const char* const base = m & 1 ? kb + dv : kb;
            const char* const sbase = m & 1 ? sb + ds : sb;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const char* src = base + group_at(g.at, g0 + 2 * i);
                const char* ssrc = sbase + group_at(g.scale, g0 + 2 * i);
                bool on = true;
                if (!g.whole) {
                    const int row = t * kKeys + row0 + 32 * i;
                    on = ((g.good >> (g0 + 2 * i)) & 1u) && row >= r.lo && row < r.hi;
                    if (!on) src = base, ssrc = sbase;
                }
                copy16(dst + from + 2048 * i, src, on);
                if (chunk == 0) copy8(sdst + 256 * i, ssrc, on);
            }
        }
        commit_copies();
    };
    for (int m = 0; m < kRaw - 1; ++m) feed(m);
    int slot = 0, turn = 0;
    for (int m = 0; m < n; ++m) {
        const int t = r.ta + (m >> 1);
        wait_copies<kRaw - 2>();
        __syncwarp();   // (a row's scales were copied by another lane)
        const uint32_t src = raw + (m % kRaw) * kRawTile, dst = ring + slot * kOperand;
        uint4 x[4];
        uint32_t sc[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = lds128(src + from + 2048 * i);
            sc[i] = lds16(src + kKeys * 64 + (row0 + 32 * i) * 8 + 2 * chunk);
        }
        __syncwarp();   // every lane has read the raw tile's neighbour in the ring
        feed(m + kRaw - 1);
        if ((m & 1) && r.partial(t)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = row0 + 32 * i;
                const uint32_t nan = __vcmpeq4(sc[i] & 0x7f7f7f7fu, 0x7f7f7f7fu) & 0xffffu;
                if (nan) {
                    sc[i] &= ~nan;
                    atomicOr(&sm.bad_v[t & (kRing - 1)][row >> 5], 1u << (row & 31));
                    atomicOr(&sm.flags, kBadV);
                }
            }
        }
        if (turn > 0) wait(&sm.empty[slot], (unsigned)(turn - 1) & 1u, p.err, dead);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = row0 + 32 * i;
            const uint32_t z = e4m3x2_to_f16x2(sc[i]);
            const uint32_t s0 = __byte_perm(z, 0, 0x1010), s1 = __byte_perm(z, 0, 0x3232);
            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
            const uint32_t at = dst + (chunk >> 1) * (kOperand / 2) + (row >> 3) * 1024 + (row & 7) * 128;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t f0, f1, f2, f3;
                e2m1x8_to_f16(w[k], f0, f1, f2, f3);
                const uint32_t s = k < 2 ? s0 : s1;
                sts128(at + ((((chunk & 1) * 4 + k) ^ (row & 7)) << 4),
                       make_uint4(hmul2_u32(f0, s), hmul2_u32(f1, s), hmul2_u32(f2, s), hmul2_u32(f3, s)));
            }
        }
        fence_operands();
        arrive(&sm.full[slot]);
        if (++slot == kSlots) {
            slot = 0;
            ++turn;
        }
    }
    wait_copies<0>();
}

// ---- the softmax ---------------------------------------------------------------------------------------
// The queries of sequence b: the first row of q and their number (0 for offsets that are not good).
__device__ __forceinline__ void sequence_queries(const PagedAttendParams& p, int b, bool report, int& q0, int& nb, int& all)
{
    if (!p.start) {
        q0 = b * p.max_new;
        nb = all = p.max_new;
        return;
    }
    q0 = p.start[b];
    const int q1 = p.start[b + 1];
    all = q1 - q0;
    if (q0 < 0 || q1 < q0 || q1 > p.n) {
        q0 = 0;
        all = 0;
        if (report) atomicOr(p.err, FX_DEVERR_OFFSETS);
    } else if (all > p.max_new && report) {
        atomicOr(p.err, FX_DEVERR_OFFSETS);
    }
    nb = min(all, p.max_new);
}
__device__ __forceinline__ int sequence_length(const PagedAttendParams& p, int b, bool report)
{
    const int len = p.c.len[b];
    if (report && (len < 0 || len > p.c.cap)) atomicOr(p.err, FX_DEVERR_LEN);
    return min(max(len, 0), p.c.cap);
}

// What token j of a sequence sees: rows x <= t < y, both within [0, len] (any int may be given: arithmetic on these ends
// must not overflow).
__device__ __forceinline__ int2 token_interval(const PagedAttendParams& p, int q0, int len, int all, int j)
{
    const int pos = len - all + j;
    int2 see = make_int2(p.first ? min(max(p.first[q0 + j], 0), len) : 0, max(min(p.last ? p.last[q0 + j] : pos + 1, len), 0));
    if (p.window > 0) see.x = max(see.x, pos - p.window + 1);
    return see;
}

// A place for the sums of one CTA's O: one of as many as there are SMs, each of which holds one CTA (the registers of a CTA are
// all that an SM has).  The masks of the places taken are the last words of the counters.
__device__ __forceinline__ unsigned* slot_masks(const PagedAttendParams& p) { return p.counters + kCounterBytes / 4 - kSlotWords; }
__device__ __forceinline__ int take_slot(const PagedAttendParams& p)
{
    uint32_t sm;
    asm volatile("mov.u32 %0, %smid;" : "=r"(sm));
    for (int k = 0; k < 2 * p.slots; ++k) {
        const int i = (int)((sm + k) % (unsigned)p.slots);
        const unsigned bit = 1u << (i & 31);
        if ((atomicOr(slot_masks(p) + (i >> 5), bit) & bit) == 0) {
            __threadfence();
            return i;
        }
    }
    atomicOr(p.err, FX_DEVERR_TIMEOUT);
    return -1;
}
__device__ __forceinline__ void leave_slot(const PagedAttendParams& p, int i)
{
    __threadfence();
    atomicAnd(slot_masks(p) + (i >> 5), ~(1u << (i & 31)));
}

constexpr int kMinPart = 4;   // tiles of a part, at least

// Shares the tiles of all blocks among the CTAs: parts of a block of n tiles are ceil(n / share).  Returns false when there
// is nothing for this CTA; else its block (sm.plan_i) and its place among the parts of the block's heads.
__device__ __forceinline__ bool plan(const PagedAttendParams& p, AttendSmem& sm, int* count, int& n_parts, int& at, int& i)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nq = p.c.B * p.blocks;
    for (int k = warp; k < nq; k += kThreadsA / 32) {   // a warp counts a block's tiles: from what its tokens see
        const int b = k / p.blocks, blk = k - b * p.blocks;
        const bool report = blockIdx.x == 0 && blk == 0 && lane == 0;
        int q0, nb, all;
        sequence_queries(p, b, report, q0, nb, all);
        const int len = sequence_length(p, b, report);
        int n = 0;
        if (blk * kBlock < nb * p.G) {
            const int j0 = blk * kBlock / p.G, j1 = min((blk * kBlock + kBlock - 1) / p.G, nb - 1);
            int lo = 0x7fffffff, hi = 0;
            for (int j = j0 + lane; j <= j1; j += 32) {
                const int2 see = token_interval(p, q0, len, all, j);
                if (see.x >= see.y) continue;
                lo = min(lo, see.x);
                hi = max(hi, see.y);
            }
            lo = __reduce_min_sync(0xffffffffu, lo);
            hi = __reduce_max_sync(0xffffffffu, hi);
            n = lo < hi ? (hi + kKeys - 1) / kKeys - lo / kKeys : 1;
        }
        if (lane == 0) count[k] = n;
    }
    __syncthreads();
    const int mine = tid < nq ? count[tid] : 0;
    int total = mine;
#pragma unroll
    for (int d = 16; d; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
    if (lane == 0) sm.scan[warp] = total;
    if (tid == 0) sm.plan_i = -1;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) total += sm.scan[w];
    // lanes try shares of 1 to 3.6 times an even one and no cuts at all (always possible); the shortest longest part wins
    const float even = fmaxf((float)total * p.c.Hkv / (float)gridDim.x, 1.f);
    float inv = lane == 31 ? 0.f : 1.f / fmaxf(even * (1.f + lane / 12.f), (float)kMinPart);
    int sum = 0;
    float longest = 0.f;
    for (int k = 0; k < nq; ++k) {
        const int n = count[k], parts = min((int)((float)n * inv) + 1, n);   // (0 for a block without rows)
        sum += parts;
        longest = fmaxf(longest, __fdividef((float)n, (float)max(parts, 1)));
    }
    if ((int64_t)sum * p.c.Hkv > (int64_t)gridDim.x) longest = 3e38f;
    float best = longest;
#pragma unroll
    for (int d = 16; d; d >>= 1) best = fminf(best, __shfl_xor_sync(0xffffffffu, best, d));
    inv = __shfl_sync(0xffffffffu, inv, __ffs(__ballot_sync(0xffffffffu, longest == best)) - 1);
    const int parts = mine > 0 ? min((int)((float)mine * inv) + 1, mine) : 0;
    int inc = parts;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += o;
    }
    __syncthreads();   // sm.scan is free
    if (lane == 31) sm.scan[warp] = inc;
    __syncthreads();
    int before = inc - parts;
#pragma unroll
    for (int w = 0; w < 16; ++w)
        if (w < warp) before += sm.scan[w];
    const int64_t first = (int64_t)before * p.c.Hkv, here = blockIdx.x;
    if (parts > 0 && here >= first && here < first + (int64_t)parts * p.c.Hkv) {
        sm.plan_i = tid;
        sm.plan_at = (int)(here - first);
        sm.plan_parts = parts;
    }
    __syncthreads();
    i = sm.plan_i;
    at = sm.plan_at;
    n_parts = sm.plan_parts;
    return i >= 0;
}

// WIDE: caps whose logits have to be exact relative to themselves (kMixedCap).  A kernel of its own: with both in one, the
// smaller caps' windowed 4-bit prompt took 413 us instead of 405.
// LONG: rows past kFlush tiles, by the room of the tables (the lengths are on the device).  Kernels of their own, too: sequences
// short all the same take 2% (prompts with pictures 934 us, 955) to 4% longer in them (windowed 4-bit prompts 395, 412).
template <bool E2M1, int MODE, bool WIDE, bool LONG>
__global__ void __launch_bounds__(kThreadsA, 1) paged_attend_kernel(const __grid_constant__ PagedAttendParams p)
{
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    __shared__ __align__(16) AttendSmem sm;
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const uint32_t ring = base + 2 * kOperand, raw = ring + slots(E2M1) * kOperand;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    griddep_wait();
    griddep_launch();
    // ---- which rows, which tiles
    int b, h, blk, part = 0, n_parts = 1, unit = 0;
    if (p.split) {
        int at, i;
        if (!plan(p, sm, reinterpret_cast<int*>(smem_raw), n_parts, at, i)) return;
        b = i / p.blocks;
        blk = i - b * p.blocks;
        h = at / n_parts;
        part = at - h * n_parts;
        unit = i * p.c.Hkv + h;
    } else {
        h = blockIdx.x;
        blk = gridDim.y - 1 - blockIdx.y;   // the longest first, where a query sees what came before it
        b = blockIdx.z;
    }
    int q0, nb, all;
    const bool report = !p.split && h == 0 && blk == 0 && tid == 0;
    sequence_queries(p, b, report, q0, nb, all);
    if (blk * kBlock >= nb * p.G) return;
    const int len = sequence_length(p, b, report);
    const int rows = min(nb * p.G - blk * kBlock, kBlock);
    const bool two = rows > kSub;

    // ---- this thread's row (of the first 256 threads)
    // token (of the sequence) and head of a row; G divides short numbers by a product
    const int j_first = blk * kBlock / p.G, r_first = blk * kBlock - j_first * p.G, g_inv = 65536 / p.G + 1;
    auto row_of = [&](int r, int& head) {
        const int at = r_first + r, j = (at * g_inv) >> 16;   // (at < 256 + 64)
        head = h * p.G + at - j * p.G;
        return j_first + j;
    };
    const int row = tid;
    const bool live = row < rows;
    int lo = 0, hi = 0, pos = 0;
    int64_t qi = 0;   // token
    int g = 0;
    if (live) {
        const int j = row_of(row, g);
        qi = (int64_t)q0 + j;
        pos = len - all + j;
        const int2 see = token_interval(p, q0, len, all, j);
        lo = see.x;
        hi = see.y;
    }
    if (tid < kBlock) {
        const bool sees = live && lo < hi;
        int4 w;
        w.x = __reduce_min_sync(0xffffffffu, sees ? lo : 0x7fffffff);
        w.y = __reduce_max_sync(0xffffffffu, sees ? hi : 0);
        w.z = __reduce_max_sync(0xffffffffu, sees ? lo : 0);
        w.w = __reduce_min_sync(0xffffffffu, sees ? hi : 0x7fffffff);
        if (lane == 0) sm.seen[warp] = w;
    } else if (warp == 12) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sm.tmem)), "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    } else if (warp == 13) {
        if (lane < 2) {
            init_barrier(&sm.s_full[lane], 1);
            init_barrier(&sm.p_full[lane], kSub);
            init_barrier(&sm.o_done[lane], 1);
        }
        if (lane < slots(E2M1)) {
            init_barrier(&sm.full[lane], 128);
            init_barrier(&sm.empty[lane], 1);
        }
        if (lane == 31) init_barrier(&sm.q_full, kBlock);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    } else if (warp == 14) {
        if (lane == 0) {
            sm.flags = 0;
            if (LONG) sm.slot = !p.split && len > kFlush * kKeys ? take_slot(p) : -1;
        }
        for (int i = lane; i < kRing * 4; i += 32) sm.bad_v[i >> 2][i & 3] = 0u;
    }
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = sm.tmem;
    FillRange r;
    r.lo = r.com_hi = 0x7fffffff;
    r.hi = r.com_lo = 0;
#pragma unroll
    for (int w = 0; w < kBlock / 32; ++w) {
        const int4 v = sm.seen[w];
        r.lo = min(r.lo, v.x);
        r.hi = max(r.hi, v.y);
        r.com_lo = max(r.com_lo, v.z);
        r.com_hi = min(r.com_hi, v.w);
    }
    r.ta = r.tb = 0;
    if (r.lo < r.hi) {
        r.ta = r.lo / kKeys;
        r.tb = (r.hi + kKeys - 1) / kKeys;
        if (n_parts > 1) {
            const int64_t n = r.tb - r.ta;
            r.tb = r.ta + (int)(n * (part + 1) / n_parts);
            r.ta += (int)(n * part / n_parts);
        }
    }
    const int nt = r.tb - r.ta;

    if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
        // One lane does it all: a wait that the whole warp takes part in costs some 250 cycles more, which the tensor core
        // stands still (the products' queue is short).
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const int tiles = warp == 12 ? __shfl_sync(0xffffffffu, nt, 0) : 0;
        if (tiles > 0 && elect_lane()) {
            constexpr int kSlots = slots(E2M1);
            bool dead = false;
            const uint32_t q0d = sdesc_low(base, 16);
            auto k_of = [&](int slot) { return sdesc_low(ring + (uint32_t)slot * kOperand, 16); };
            auto v_of = [&](int slot) { return sdesc_low(ring + (uint32_t)slot * kOperand, kOperand / 2); };
            int slot = 0, turn = 0;   // of the next operand tile
            auto wait_full = [&]() { wait(&sm.full[slot], (unsigned)turn & 1u, p.err, dead); };
            auto next = [&]() {
                if (++slot == kSlots) {
                    slot = 0;
                    ++turn;
                }
            };
            wait(&sm.q_full, 0u, p.err, dead);
            wait_full();
            tc_after();
            mma_qk<E2M1>(tm + col_s(0), q0d, k_of(slot));
            mma_commit(&sm.s_full[0]);
            if (two) {
                mma_qk<E2M1>(tm + col_s(1), q0d + (kOperand >> 4), k_of(slot));
                mma_commit(&sm.s_full[1]);
            }
            mma_commit(&sm.empty[slot]);
            next();
            for (int t = 0; t < tiles; ++t) {
                wait_full();   // V
                const int vs = slot;
                next();
                const bool more = t + 1 < tiles;
                if (more) wait_full();   // K of the next tile
                wait(&sm.p_full[0], (unsigned)t & 1u, p.err, dead);
                tc_after();
                mma_pv<E2M1>(tm + col_o(0), tm + col_s(0), v_of(vs), t > 0 ? 1u : 0u);
                if (!two) mma_commit(&sm.empty[vs]);
                if (more) {
                    mma_qk<E2M1>(tm + col_s(0), q0d, k_of(slot));
                    mma_commit(&sm.s_full[0]);
                    if (!two) mma_commit(&sm.empty[slot]);
                } else {
                    mma_commit(&sm.o_done[0]);
                }
                if (two) {
                    wait(&sm.p_full[1], (unsigned)t & 1u, p.err, dead);
                    tc_after();
                    mma_pv<E2M1>(tm + col_o(1), tm + col_s(1), v_of(vs), t > 0 ? 1u : 0u);
                    mma_commit(&sm.empty[vs]);
                    if (more) {
                        mma_qk<E2M1>(tm + col_s(1), q0d + (kOperand >> 4), k_of(slot));
                        mma_commit(&sm.s_full[1]);
                        mma_commit(&sm.empty[slot]);
                    } else {
                        mma_commit(&sm.o_done[1]);
                    }
                }
                if (more) next();
            }
        }
        __syncwarp();
    } else if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsFill));
        if (nt > 0) {
            const int32_t* table = p.c.table + (int64_t)b * p.c.table_stride;
            if constexpr (E2M1)
                fill_e2m1(p, sm, ring, raw, table, h, r);
            else
                fill_bf16(p, sm, ring, table, h, r);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        const int x = warp >> 2;
        const bool on = x == 0 || two;
        float qs = p.scale;   // factor of the row's logits
        {
            // The queries, 16 lanes to a row, so that a load takes whole lines: lanes take 16-byte chunk tid % 16 of rows
            // tid / 16 + 8 i of their subtile.  4-bit pages: as f16 values, whose factor goes to the row's thread.
            const int chunk = lane & 15, first = (warp & 3) * 2 + (lane >> 4);
            const uint32_t tile = base + x * kOperand;
            uint4 q[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                int head;
                const int r = x * kSub + first + 8 * i, j = row_of(r, head);
                q[i] = make_uint4(0u, 0u, 0u, 0u);
                if (r < rows) q[i] = *reinterpret_cast<const uint4*>(p.q + ((int64_t)q0 + j) * p.q_n + (int64_t)head * p.q_h + 8 * chunk);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                uint4 v = make_uint4(q[i].x ^ p.flip, q[i].y ^ p.flip, q[i].z ^ p.flip, q[i].w ^ p.flip);
                if (E2M1) {
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                    uint32_t top = 0;
#pragma unroll
                    for (int e = 0; e < 4; ++e) top = max(top, max((w[e] & 0x7fffu) << 16, w[e] & 0x7fff0000u));
#pragma unroll
                    for (int d = 1; d < 16; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
                    // 2^(14 - exponent of the largest); tiny rows (below 2^-100) are scaled as if they were that large
                    const int ex = min(max((int)(top >> 23) - 127, -100), 127);
                    const float up = __uint_as_float((uint32_t)(127 + 14 - ex) << 23);
                    auto half = [&](uint32_t u) {
                        const uint32_t z = pack2<true>(__uint_as_float(u << 16) * up, __uint_as_float(u & 0xffff0000u) * up);
                        return top < 0x7f800000u ? z : 0x7fff7fffu;   // else the row is NaN
                    };
                    v = make_uint4(half(v.x), half(v.y), half(v.z), half(v.w));
                    if (chunk == 0) sm.q_factor[x * kSub + first + 8 * i] = __uint_as_float((uint32_t)(127 - 14 + ex) << 23);
                }
                sts128(tile + sw128(first + 8 * i, 8 * chunk, kSub), v);
            }
            fence_operands();
            arrive(&sm.q_full);
            // (the subtile's threads; without tiles nothing else orders these stores and those of the outputs)
            if (E2M1 || nt == 0) asm volatile("bar.sync %0, 128;" ::"r"(1 + x) : "memory");
            if (E2M1) qs *= sm.q_factor[row];
        }
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        bool dead = false, poison = false, odd = false;
        float m = -INFINITY, l = 0.f;   // reference and sum (in units of 2^kWeightBase)
        // rows that do not exist see every row of their zeros, so that they ask for no masks
        const int my_lo = live ? lo : -0x40000000, my_hi = live ? hi : 0x7fffffff;
        const float cap = p.cap, icap = cap > 0.f ? 1.f / cap : 0.f;
        const float slope2 = MODE == kBias && live ? p.slope[g] * 1.4426950408889634f : 0.f;
        // A bias that grows along a tile is added from the tile's first key on, 127 slopes long, and taken off again with the
        // reference: 2^-24 of that is lost, so that slopes past 2 (base 2: 2^-16 of a logit there) are taken key by key.
        const int linear_from = !live ? 0x7fffffff : (fabsf(slope2) <= 2.f ? pos : -0x7fffffff);
        if (MODE == kPlain) qs *= 1.4426950408889634f;
        // from s to y of tanh(y); finite with its factors, so that a logit of 0 stays 0
        const float k = fminf(qs * icap, 0x1p126f), k2 = k * 2.885390081777927f;
        auto check = [&](int t) {   // whether the row sees a value of tile t that is not finite (those were left out)
            for (int w = 0; w < 4; ++w) {
                unsigned bits = *(volatile unsigned*)&sm.bad_v[t & (kRing - 1)][w];
                while (bits) {
                    const int at = t * kKeys + 32 * w + __ffs(bits) - 1;
                    bits &= bits - 1;
                    poison |= at >= my_lo && at < my_hi;
                }
            }
        };
        // the row's sums of O in memory, at a reference of their own (-inf: none yet)
        auto sums = [&]() {
            const int64_t at = p.split ? (int64_t)blockIdx.x * p.part_rows : (int64_t)sm.slot * kBlock;
            return reinterpret_cast<float4*>(p.part + (at + row) * kHeadDim);
        };
        auto flushes = [&]() { return LONG && nt > kFlush && (p.split || sm.slot >= 0); };
        if (LONG) sm.q_factor[row] = -INFINITY;
        if (on) {
            for (int t = 0, stop; t < nt; t = stop) {
                // (stretches of tiles, so that what a flush takes of registers is none of the tiles' loop)
                stop = flushes() ? min(t + kFlush, nt) : nt;
                if (LONG && t > 0) {   // O of the tiles before is complete when S of this one is: it was issued after it
                    wait(&sm.s_full[x], (unsigned)t & 1u, p.err, dead);
                    tc_after();
                    const float m_sum = sm.q_factor[row], z = m_sum == -INFINITY ? 0.f : ex2(m_sum - m);
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        float v[32];
                        const uint32_t zero[32] = {};
                        tmem_ld32(lanes + col_o(x) + 32 * c, v);
                        tmem_st32(lanes + col_o(x) + 32 * c, zero);
                        if (live) {
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                float4* const to = sums() + 8 * c + k;
                                float4 o = m_sum == -INFINITY ? make_float4(0.f, 0.f, 0.f, 0.f) : *to;
                                o.x = fmaf(o.x, z, v[4 * k]), o.y = fmaf(o.y, z, v[4 * k + 1]);
                                o.z = fmaf(o.z, z, v[4 * k + 2]), o.w = fmaf(o.w, z, v[4 * k + 3]);
                                *to = o;
                            }
                        }
                    }
                    sm.q_factor[row] = m;
                }
                for (; t < stop; ++t) {
                    wait(&sm.s_full[x], (unsigned)t & 1u, p.err, dead);
                    tc_after();
                    const int flags = *(volatile int*)&sm.flags;
                    float s[128];
                    tmem_row(lanes + col_s(x), s);
                    const int tile = r.ta + t, j0 = tile * kKeys;
                    unsigned skip = 0;
                    if (flags) {
                        if (t > 0 && (flags & kBadV)) check(tile - 1);
                        skip = *(volatile unsigned*)&sm.skip[tile & (kRing - 1)];
                    }
                    const int a = my_lo - j0, e = my_hi - j0;   // the row sees keys a <= k < e of the tile
                    const bool whole = a <= 0 && e >= kKeys;
                    // which keys each row sees, as bits; rows that see all of them take no masks
                    uint32_t see[4];
                    const bool masked = __any_sync(0xffffffffu, !whole) || skip != 0;
                    if (masked) {
                        bool any = false;
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            const int from = min(max(a - 32 * w, 0), 32), to = min(max(e - 32 * w, 0), 32);
                            uint32_t bits = to > from ? (0xffffffffu >> (32 - (to - from))) << from : 0u;
                            if ((skip >> (2 * w)) & 1u) bits &= 0xffff0000u;
                            if ((skip >> (2 * w)) & 2u) bits &= 0x0000ffffu;
                            see[w] = bits;
                            any |= bits != 0;
                        }
                        if (!__any_sync(0xffffffffu, any)) {   // nothing of this tile for any row of the warp
                            uint32_t zero[32] = {};
                            tmem_put32(lanes + col_s(x), zero);
                            tmem_put32(lanes + col_s(x) + 32, zero);
                            tmem_wait_st();
                            tc_before();
                            arrive(&sm.p_full[x]);
                            continue;
                        }
                    }
                    float f = MODE == kPlain ? qs : 1.f, off = 0.f;   // from s to base-2 logits: s * f + off
                    if (MODE != kPlain) {
                        if (cap > 0.f) {
                            float top = 0.f;
#pragma unroll
                            for (int i = 0; i < 128; i += 4) {
                                const float u = max3(fabsf(s[i]), fabsf(s[i + 1]), fabsf(s[i + 2]));
                                top = max3(top, u, fabsf(s[i + 3]));
                            }
                            // tanh(y) = y + y^3 Q(y^2), exact to 2^-22 of itself for y up to 1 (10 steps of the fp32 units for two
                            // values).  Caps up to kMixedCap: beside it tanh(y) = 1 - 2 / (exp(2y) + 1), off by 2^-21 at most (of
                            // 1, not of itself; 3 steps, and 12 of the function unit for one value), so that both units are
                            // busy, and the latter alone where a logit is past the cap.  WIDE: the polynomial alone, and past the
                            // cap each value's own of the two, whose errors are relative to it (the same prompt with a cap of 65:
                            // 426 us; of 64: 391).
                            if (WIDE) {
                                if (!__any_sync(0xffffffffu, !(top * qs * icap <= 1.f))) {
#pragma unroll
                                    for (int i = 0; i < 128; i += 8) {
                                        float2 y[4], u[4], q[4];
#pragma unroll
                                        for (int e = 0; e < 4; ++e) {
                                            y[e] = mul2(mul2(make_float2(s[i + 2 * e], s[i + 2 * e + 1]), make_float2(qs, qs)),
                                                        make_float2(icap, icap));
                                            u[e] = mul2(y[e], y[e]);
                                            q[e] = make_float2(kTanh[6], kTanh[6]);
                                        }
#pragma unroll
                                        for (int c = 5; c >= 0; --c)
#pragma unroll
                                            for (int e = 0; e < 4; ++e) q[e] = fma2(q[e], u[e], make_float2(kTanh[c], kTanh[c]));
#pragma unroll
                                        for (int e = 0; e < 4; ++e) {
                                            const float2 r = fma2(mul2(y[e], u[e]), q[e], y[e]);
                                            s[i + 2 * e] = r.x;
                                            s[i + 2 * e + 1] = r.y;
                                        }
                                    }
                                } else {
#pragma unroll
                                    for (int i = 0; i < 128; ++i) {
                                        const float y = s[i] * qs * icap;
                                        s[i] = fabsf(y) <= 1.f ? tanh_near(y) : tanh_far(y);
                                    }
                                }
                            } else if (!__any_sync(0xffffffffu, !(top * k <= 1.f))) {
#pragma unroll
                                for (int i = 0; i < 128; i += 16) {   // side by side: ten values by one, six by the other
                                    float2 y[5], u[5], q[5];
                                    float z[6];
#pragma unroll
                                    for (int e = 0; e < 5; ++e) {
                                        y[e] = mul2(make_float2(s[i + 2 * e], s[i + 2 * e + 1]), make_float2(k, k));
                                        u[e] = mul2(y[e], y[e]);
                                        q[e] = make_float2(kTanh[6], kTanh[6]);
                                    }
#pragma unroll
                                    for (int e = 0; e < 6; ++e) z[e] = ex2(s[i + 10 + e] * k2) + 1.f;
#pragma unroll
                                    for (int c = 5; c >= 0; --c) {
#pragma unroll
                                        for (int e = 0; e < 5; ++e) q[e] = fma2(q[e], u[e], make_float2(kTanh[c], kTanh[c]));
                                        s[i + 10 + c] = fmaf(-2.f, rcp(z[c]), 1.f);
                                    }
#pragma unroll
                                    for (int e = 0; e < 5; ++e) {
                                        const float2 r = fma2(mul2(y[e], u[e]), q[e], y[e]);
                                        s[i + 2 * e] = r.x;
                                        s[i + 2 * e + 1] = r.y;
                                    }
                                }
                            } else {
#pragma unroll
                                for (int i = 0; i < 128; i += 8) {
                                    float z[8];
#pragma unroll
                                    for (int e = 0; e < 8; ++e) z[e] = ex2(s[i + e] * k2) + 1.f;
#pragma unroll
                                    for (int e = 0; e < 8; ++e) s[i + e] = fmaf(-2.f, rcp(z[e]), 1.f);
                                }
                            }
                        }
                        f = (cap > 0.f ? cap : qs) * 1.4426950408889634f;
                        if (MODE == kBias) {
                            const float d0 = (float)(pos - j0);
                            off = -slope2 * d0;
                            if (!__any_sync(0xffffffffu, linear_from < j0 + kKeys - 1 || fabsf(off) > kFarRef)) {
                                // all keys lie before the queries: their bias grows by slope from one to the next (not where it is
                                // so large that it and the reference, rounded each for itself, lie apart)
#pragma unroll
                                for (int i = 0; i < 64; ++i) {
                                    const float2 y = fma2(make_float2(s[2 * i], s[2 * i + 1]), make_float2(f, f),
                                                          mul2(make_float2(2 * i, 2 * i + 1), make_float2(slope2, slope2)));
                                    s[2 * i] = y.x;
                                    s[2 * i + 1] = y.y;
                                }
                            } else {
#pragma unroll
                                for (int i = 0; i < 128; ++i) s[i] = fmaf(fabsf(d0 - (float)i), -slope2, s[i] * f);
                                off = 0.f;
                            }
                            f = 1.f;
                        }
                    }
                    if (masked) {
#pragma unroll
                        for (int k = 0; k < 128; ++k) s[k] = (see[k >> 5] >> (k & 31)) & 1u ? s[k] : -INFINITY;
                    }
                    // the largest logit that the row sees
                    float mt;
                    {
                        float c[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int k = 0; k < 128; k += 8)
#pragma unroll
                            for (int u = 0; u < 4; ++u) c[u] = max3(c[u], s[k + 2 * u], s[k + 2 * u + 1]);
                        mt = fmaxf(max3(c[0], c[1], c[2]), c[3]);
                    }
                    // (factors are not negative; a hidden logit stays -inf also with a factor of 0)
                    mt = mt == -INFINITY ? mt : __fmul_rn(mt, f);
                    if (MODE == kBias) mt = __fadd_rn(mt, off);
                    const bool grow = mt > m + kMaxSlack;   // also when there is none yet and the row sees something
                    if (__any_sync(0xffffffffu, grow)) {
                        const float mnew = grow ? mt : m;
                        if (t > 0) {   // O of the tiles before is complete: S was issued after it
                            const float z = !grow ? 1.f : (m == -INFINITY ? 0.f : ex2(m - mnew));
#pragma unroll 1
                            for (int c = 0; c < 4; ++c) {
                                float v[32];
                                uint32_t w[32];
                                tmem_ld32(lanes + col_o(x) + 32 * c, v);
#pragma unroll
                                for (int k = 0; k < 32; ++k) w[k] = __float_as_uint(v[k] * z);
                                tmem_st32(lanes + col_o(x) + 32 * c, w);
                            }
                            l *= z;
                        }
                        m = mnew;
                        // a far reference, or hidden logits beside a factor of 0, take rounded products one by one
                        odd = __any_sync(0xffffffffu, fabsf(m) > kFarRef && m != -INFINITY);
                    }
                    const float ref = (m == -INFINITY ? 0.f : -m) + (MODE == kBias ? off : 0.f), bias = ref + kWeightBase<E2M1>;
                    uint32_t w[64];
                    float2 l2 = make_float2(0.f, 0.f), l3 = make_float2(0.f, 0.f);
                    if (!odd && !(masked && f == 0.f)) {
                        const float2 ff = make_float2(f, f), bb = make_float2(bias, bias);
#pragma unroll
                        for (int k0 = 0; k0 < 64; k0 += 4) {   // eight values side by side
                            float2 y[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) y[e] = fma2(make_float2(s[2 * (k0 + e)], s[2 * (k0 + e) + 1]), ff, bb);
#pragma unroll
                            for (int e = 0; e < 4; ++e) y[e] = make_float2(ex2(y[e].x), ex2(y[e].y));
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                if (e & 1)
                                    l3 = add2(l3, y[e]);
                                else
                                    l2 = add2(l2, y[e]);
                                w[k0 + e] = pack2<E2M1>(y[e].x, y[e].y);
                            }
                            if (k0 == 28) tmem_put32(lanes + col_s(x), reinterpret_cast<uint32_t(&)[32]>(w[0]));
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < 64; ++k) {
                            float y[2];
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                const float v = s[2 * k + u];
                                y[u] = v == -INFINITY ? 0.f
                                                      : ex2(__fadd_rn(__fadd_rn(__fmul_rn(v, f), ref), kWeightBase<E2M1>));
                            }
                            l2 = add2(l2, make_float2(y[0], y[1]));
                            w[k] = pack2<E2M1>(y[0], y[1]);
                        }
                        tmem_put32(lanes + col_s(x), reinterpret_cast<uint32_t(&)[32]>(w[0]));
                    }
                    l2 = add2(l2, l3);
                    l += l2.x + l2.y;
                    tmem_put32(lanes + col_s(x) + 32, reinterpret_cast<uint32_t(&)[32]>(w[32]));
                    tmem_wait_st();
                    tc_before();
                    arrive(&sm.p_full[x]);
                }
            }
            if (nt > 0) {
                wait(&sm.o_done[x], 0u, p.err, dead);
                tc_after();
                if (*(volatile int*)&sm.flags & kBadV) check(r.tb - 1);
            }
            const bool none = l == 0.f;
            const bool summed = flushes() && live && sm.q_factor[row] != -INFINITY;   // (else what is there is 0)
            const float z_sum = summed ? ex2(sm.q_factor[row] - m) : 0.f;
            auto add_sums = [&](int c, float (&v)[32]) {     // of dimensions 32 c .. + 31
                if (summed) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float4 o = sums()[8 * c + k];
                        v[4 * k] = fmaf(o.x, z_sum, v[4 * k]), v[4 * k + 1] = fmaf(o.y, z_sum, v[4 * k + 1]);
                        v[4 * k + 2] = fmaf(o.z, z_sum, v[4 * k + 2]), v[4 * k + 3] = fmaf(o.w, z_sum, v[4 * k + 3]);
                    }
                }
            };
            // Rows leave through the query tile, which nothing reads any more, so that a store takes whole lines.
            const uint32_t stage = base + x * kOperand;
            const int chunk = lane & 15, first = (warp & 3) * 32 + (lane >> 4);
            if (n_parts == 1) {
                const float z = none ? 0.f : p.c.v_mul / l;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float v[32];
                    if (nt > 0) tmem_ld32(lanes + col_o(x) + 32 * c, v);
                    add_sums(c, v);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t y[4];
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const float v0 = v[8 * k + 2 * u] * z, v1 = v[8 * k + 2 * u + 1] * z;
                            y[u] = poison ? 0x7fff7fffu : (none ? 0u : pack2<false>(v0, v1));
                        }
                        sts128(stage + sw128(row & 127, 32 * c + 8 * k, kSub), make_uint4(y[0], y[1], y[2], y[3]));
                    }
                }
                if (live && p.lse)
                    p.lse[qi * p.Hq + g] = none ? -INFINITY : ((m == -INFINITY ? 0.f : m) + log2f(l) - kWeightBase<E2M1>) * 0.6931471805599453f;
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    int head;
                    const int r = first + 2 * i, j = row_of(x * kSub + r, head);
                    const uint4 y = lds128(stage + sw128(r, 8 * chunk, kSub));
                    if (x * kSub + r < rows)
                        *reinterpret_cast<uint4*>(p.out + (((int64_t)q0 + j) * p.Hq + head) * kHeadDim + 8 * chunk) = y;
                }
            } else {
                const int64_t at = (int64_t)blockIdx.x * p.part_rows;
#pragma unroll 1
                for (int c = 0; c < 2; ++c) {   // 64 dimensions (256 bytes of a row) at a time
#pragma unroll
                    for (int k2 = 0; k2 < 2; ++k2) {
                        float v[32];
                        if (nt > 0) tmem_ld32(lanes + col_o(x) + 64 * c + 32 * k2, v);
                        add_sums(2 * c + k2, v);
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            uint4 y;
                            y.x = __float_as_uint(v[4 * k]), y.y = __float_as_uint(v[4 * k + 1]);
                            y.z = __float_as_uint(v[4 * k + 2]), y.w = __float_as_uint(v[4 * k + 3]);
                            if (none) y = make_uint4(0u, 0u, 0u, 0u);
                            if (poison) y = make_uint4(0x7fffffffu, 0x7fffffffu, 0x7fffffffu, 0x7fffffffu);
                            sts128(stage + sw128(row & 127, 64 * k2 + 8 * k, kSub), y);
                        }
                    }
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int r = first + 2 * i;
                        const uint4 y = lds128(stage + sw128(r, 8 * chunk, kSub));
                        if (x * kSub + r < rows)
                            *reinterpret_cast<uint4*>(p.part + (at + x * kSub + r) * kHeadDim + 64 * c + 4 * chunk) = y;
                    }
                    __syncwarp();
                }
                if (live) {
                    p.part_ml[2 * (at + row)] = m == -INFINITY && !none ? 0.f : m;   // (NaN logits leave no reference, but show)
                    p.part_ml[2 * (at + row) + 1] = l;
                }
            }
        }
    }
    // ---- the parts of a block meet
    tc_before();
    __syncthreads();
    if (warp == 12) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
    if (LONG && tid == 0 && sm.slot >= 0) leave_slot(p, sm.slot);
    if (n_parts == 1) return;
    if (tid == 0) {
        __threadfence();   // the CTA's part, which the barrier orders before this fence
        sm.last = atomicAdd(p.counters + unit, 1u) == (unsigned)(n_parts - 1) ? 1u : 0u;
        if (sm.last) {
            p.counters[unit] = 0;   // ready for the next call
            __threadfence();
        }
    }
    __syncthreads();
    if (!sm.last) return;
    const int64_t at0 = (int64_t)(blockIdx.x - part) * p.part_rows;
    for (int w = warp; w < rows; w += kThreadsA / 32) {
        float mx = -INFINITY;
        for (int k = lane; k < n_parts; k += 32) mx = fmaxf(mx, __ldcg(p.part_ml + 2 * (at0 + (int64_t)k * p.part_rows + w)));
#pragma unroll
        for (int d = 16; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        float z = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int k = 0; k < n_parts; ++k) {
            const int64_t at = at0 + (int64_t)k * p.part_rows + w;
            const float2 ml = __ldcg(reinterpret_cast<const float2*>(p.part_ml) + at);
            const float4 o = __ldcg(reinterpret_cast<const float4*>(p.part + at * kHeadDim) + lane);
            const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - mx);
            if (ml.y == 0.f) continue;   // that part saw nothing
            z = fmaf(f, ml.y, z);
            acc.x = fmaf(f, o.x, acc.x);
            acc.y = fmaf(f, o.y, acc.y);
            acc.z = fmaf(f, o.z, acc.z);
            acc.w = fmaf(f, o.w, acc.w);
        }
        const bool none = z == 0.f;
        const float y = none ? 0.f : p.c.v_mul / z;
        int head;
        const int j = row_of(w, head);
        const int64_t to = ((int64_t)q0 + j) * p.Hq + head;
        *reinterpret_cast<uint2*>(p.out + to * kHeadDim + 4 * lane) =
            none ? make_uint2(0u, 0u) : make_uint2(pack2<false>(acc.x * y, acc.y * y), pack2<false>(acc.z * y, acc.w * y));
        if (p.lse && lane == 0) p.lse[to] = none ? -INFINITY : (mx + log2f(z) - kWeightBase<E2M1>) * 0.6931471805599453f;
    }
}

template <bool E2M1, int MODE, bool WIDE, bool LONG>
cudaError_t launch(const PagedAttendParams& p, bool pdl, cudaStream_t s)
{
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(done.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(paged_attend_kernel<E2M1, MODE, WIDE, LONG>, cudaFuncAttributeMaxDynamicSharedMemorySize, attend_smem(E2M1));
        if (e != cudaSuccess) return e;
        done.fetch_or(bit, std::memory_order_relaxed);
    }
    const dim3 grid = p.split ? dim3(p.split) : dim3(p.c.Hkv, p.blocks, p.c.B);
    return launch_kernel(paged_attend_kernel<E2M1, MODE, WIDE, LONG>, grid, dim3(kThreadsA), attend_smem(E2M1), s, pdl, 0u, p);
}

// The kernel for what a call puts on its logits.
template <bool E2M1, bool LONG>
cudaError_t launch_attend(const PagedAttendParams& p, bool pdl, cudaStream_t s)
{
    // (a scale so small beside the cap that their quotient is no normal number has to be applied by itself, too)
    const bool wide = p.cap > kMixedCap || (double)p.scale < (double)p.cap * 0x1p-126;
    if (p.slope) return wide ? launch<E2M1, kBias, true, LONG>(p, pdl, s) : launch<E2M1, kBias, false, LONG>(p, pdl, s);
    if (p.cap > 0.f) return wide ? launch<E2M1, kCap, true, LONG>(p, pdl, s) : launch<E2M1, kCap, false, LONG>(p, pdl, s);
    return launch<E2M1, kPlain, false, LONG>(p, pdl, s);
}

}  // namespace
}  // namespace fx
