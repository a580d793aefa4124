// Attention over a paged cache for sm_103a, bf16 or 4-bit: fx_paged_decode and fx_paged_importance.
//
// Work unit of a warp: a tile of 16 cache rows of one (sequence, KV head).  Its K rows go from global memory
// straight into the registers that mma.sync wants as the A operand of S^T = K Q^T (rows of K on M, the query
// rows on N), its V rows into those of O^T += V^T P^T (dimensions on M, cache rows on K).  The dimensions of
// K are permuted inside the product (the queries are laid out the same way), and those of O^T inside M, so that
// a lane reads contiguous bytes: of K 16 bytes (4-bit) or four times 16 (bf16) of two rows, of V 8 bytes or two
// times 16 of four rows.
//
// 4-bit rows: the codes become f16 by cvt.f16x2.e2m1x2, and one multiplication by the block's scale gives
// the value held, exactly (at most 6 significant bits, between 2^-10 and 2688).  The queries are f16 scaled
// by a power of two per row (largest magnitude in [2^14, 2^15)), so no bit of a bf16 query within 2^-24 of its
// row's largest is lost.  P is split into f16 hi + lo (22 bits); bf16 rows take bf16 queries as they are and P
// as bf16 hi + lo (16 bits): outputs are fp32 and one 16-bit P would leave them 2^-9 (bf16) or 2^-12 (f16) off.
//
// Softmax: base-2 logits, one pass.  p = 2^(x - m) with a reference m per row that all lanes of the row share;
// it is set so that the largest logit so far gives 2^kBase and moves only when a p would exceed 2^kTop, so most
// tiles take one vote instead of a reduction; f16 holds such a p to 2^-36 of the row's largest.  Sums are fp32.
#include <cuda_bf16.h>
#include <float.h>
#include <stdint.h>

#include "attn_ptx.cuh"
#include "paged.cuh"

namespace fx {
namespace {

constexpr int kAttnWarps = 8;
constexpr int kAttnThreads = 32 * kAttnWarps;
constexpr int kTileRows = 16;
constexpr int kMinTiles = 2;   // tiles a warp gets at least, before more CTAs share a call
// p is at most 2^kTop (f16 holds up to 2^15.99); a new reference puts the largest logit at 2^kBase.
constexpr float kTop = 15.f;
constexpr float kBase = 11.f;

__device__ __forceinline__ uint4 ld_stream16(const char* p)
{
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p));
    return r;
}
__device__ __forceinline__ uint2 ld_stream8(const char* p)
{
    uint2 r;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
    return r;
}
__device__ __forceinline__ uint32_t ld_u16(const char* p)
{
    uint16_t r;
    asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(r) : "l"(p));
    return r;
}
__device__ __forceinline__ uint32_t ld_u8(const char* p)
{
    uint32_t r;
    asm volatile("ld.global.nc.u8 %0, [%1];" : "=r"(r) : "l"(p));
    return r;
}

template <bool E2M1>
__device__ __forceinline__ void mma16(float d[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1)
{
    if (E2M1) {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    } else {
        mma_bf16(d, a0, a1, a2, a3, b0, b1);
    }
}

// The 16 rows of a tile: lane L < 16 of the warp (and L + 16 again) knows row L.
struct Rows {
    int id;        // pool row (page * page_rows + row in page); 0 when the row is not valid
    int pos;       // cache row (position in the sequence)
    uint32_t vm;   // bit j: row j is valid (uniform over the warp)
};

// A tile's rows as loaded: raw bytes, two K rows and four V rows per lane.
template <bool E2M1>
struct Tile;
template <>
struct Tile<true> {
    uint4 k[2];
    uint2 v[4];
    uint32_t ks;   // two scale bytes of row g, two of row g + 8
    uint32_t vs;   // one scale byte of each of the four V rows
};
template <>
struct Tile<false> {
    uint4 k[2][4];
    uint4 v[4][2];
};

__device__ __forceinline__ int64_t row_offset(const PagedCache& c, int id, int64_t sp, int64_t st)
{
    return (int64_t)(id >> c.page_shift) * sp + (int64_t)(id & c.page_mask) * st;
}

template <bool E2M1>
__device__ __forceinline__ void load_k(const PagedCache& c, int h, const Rows& r, Tile<E2M1>& x)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    if constexpr (E2M1) x.ks = 0;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int id = __shfl_sync(kFull, r.id, g + 8 * u);
        const char* at = c.k + (int64_t)h * c.sh + row_offset(c, id, c.sp, c.st);
        if constexpr (E2M1) {
            x.k[u] = ld_stream16(at + 16 * t);
            x.ks |= ld_u16(c.ks + (int64_t)h * c.ssh + row_offset(c, id, c.ssp, c.sst) + 2 * t) << (16 * u);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) x.k[u][j] = ld_stream16(at + 64 * j + 16 * t);
        }
    }
}

template <bool E2M1>
__device__ __forceinline__ void load_v(const PagedCache& c, int h, const Rows& r, Tile<E2M1>& x)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    if constexpr (E2M1) x.vs = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int id = __shfl_sync(kFull, r.id, 2 * t + (u & 1) + 8 * (u >> 1));
        const char* at = c.v + (int64_t)h * c.sh + row_offset(c, id, c.sp, c.st);
        if constexpr (E2M1) {
            x.v[u] = ld_stream8(at + 8 * g);
            x.vs |= ld_u8(c.vs + (int64_t)h * c.ssh + row_offset(c, id, c.ssp, c.sst) + g) << (8 * u);
        } else {
#pragma unroll
            for (int j = 0; j < 2; ++j) x.v[u][j] = ld_stream16(at + 128 * j + 16 * g);
        }
    }
}

// Calls f(j, a0, a1, a2, a3) with the A fragments of the eight 16-dimension steps of S^T = K Q^T.
template <bool E2M1, typename F>
__device__ __forceinline__ void k_steps(const Tile<E2M1>& x, F&& f)
{
    if constexpr (E2M1) {
        const uint32_t s0 = e4m3x2_to_f16x2(x.ks & 0xffffu), s1 = e4m3x2_to_f16x2(x.ks >> 16);
        const uint32_t sc[2][2] = {{__byte_perm(s0, 0, 0x1010), __byte_perm(s0, 0, 0x3232)},
                                   {__byte_perm(s1, 0, 0x1010), __byte_perm(s1, 0, 0x3232)}};
        const uint32_t w0[4] = {x.k[0].x, x.k[0].y, x.k[0].z, x.k[0].w};
        const uint32_t w1[4] = {x.k[1].x, x.k[1].y, x.k[1].z, x.k[1].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t a[4], b[4];
            e2m1x8_to_f16(w0[j], a[0], a[1], a[2], a[3]);
            e2m1x8_to_f16(w1[j], b[0], b[1], b[2], b[3]);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                a[u] = hmul2_u32(a[u], sc[0][j >> 1]);
                b[u] = hmul2_u32(b[u], sc[1][j >> 1]);
            }
            f(2 * j, a[0], b[0], a[1], b[1]);
            f(2 * j + 1, a[2], b[2], a[3], b[3]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f(2 * j, x.k[0][j].x, x.k[1][j].x, x.k[0][j].y, x.k[1][j].y);
            f(2 * j + 1, x.k[0][j].z, x.k[1][j].z, x.k[0][j].w, x.k[1][j].w);
        }
    }
}

// Calls f(i, a0, a1, a2, a3) with the A fragments of the eight M tiles of O^T += V^T P^T; rows outside `vm`
// count as zero, whatever they hold.
template <bool E2M1, typename F>
__device__ __forceinline__ void v_tiles(const Tile<E2M1>& x, uint32_t vm, F&& f)
{
    const int t = threadIdx.x & 3;
    if constexpr (E2M1) {
        uint32_t vs = x.vs;
        if (vm != 0xffffu) {
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (((vm >> (2 * t + (u & 1) + 8 * (u >> 1))) & 1u) == 0) vs &= ~(0xffu << (8 * u));
        }
        const uint32_t s01 = e4m3x2_to_f16x2(vs & 0xffffu), s23 = e4m3x2_to_f16x2(vs >> 16);
        const uint32_t w[4][2] = {{x.v[0].x, x.v[0].y}, {x.v[1].x, x.v[1].y}, {x.v[2].x, x.v[2].y}, {x.v[3].x, x.v[3].y}};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint32_t a[4][4];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                // neighbouring rows' codes of one dimension side by side, then one conversion a pair
                const uint32_t x0 = w[2 * u][j], x1 = w[2 * u + 1][j];
                const uint32_t even = (x0 & 0x0f0f0f0fu) | ((x1 << 4) & 0xf0f0f0f0u);
                const uint32_t odd = ((x0 >> 4) & 0x0f0f0f0fu) | (x1 & 0xf0f0f0f0u);
                e2m1x8_to_f16(even, a[2 * u][0], a[2 * u][1], a[2 * u][2], a[2 * u][3]);
                e2m1x8_to_f16(odd, a[2 * u + 1][0], a[2 * u + 1][1], a[2 * u + 1][2], a[2 * u + 1][3]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    a[2 * u][i] = hmul2_u32(a[2 * u][i], u ? s23 : s01);
                    a[2 * u + 1][i] = hmul2_u32(a[2 * u + 1][i], u ? s23 : s01);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) f(4 * j + i, a[0][i], a[1][i], a[2][i], a[3][i]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint32_t w[4][4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const bool on = (vm >> (2 * t + (u & 1) + 8 * (u >> 1))) & 1u;
                w[u][0] = on ? x.v[u][j].x : 0u;
                w[u][1] = on ? x.v[u][j].y : 0u;
                w[u][2] = on ? x.v[u][j].z : 0u;
                w[u][3] = on ? x.v[u][j].w : 0u;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                f(4 * j + i, __byte_perm(w[0][i], w[1][i], 0x5410), __byte_perm(w[0][i], w[1][i], 0x7632),
                  __byte_perm(w[2][i], w[3][i], 0x5410), __byte_perm(w[2][i], w[3][i], 0x7632));
        }
    }
}
// First of the two dimensions (the other follows it) that M tile i holds for lane group g.
template <bool E2M1>
__device__ __forceinline__ int v_dim(int i, int g)
{
    return E2M1 ? 16 * g + 2 * i : 64 * (i >> 2) + 8 * g + 2 * (i & 3);
}

// The lane's 32 query values of row g (B fragments of the eight steps), and the factor of the row's logits.
// src: the row, or nullptr for a row that does not exist.  All 32 lanes call it.
template <bool E2M1>
__device__ __forceinline__ float load_query(const uint16_t* src, uint32_t q[8][2])
{
    const int t = threadIdx.x & 3;
    uint32_t w[16];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (src) x = *reinterpret_cast<const uint4*>(src + (E2M1 ? 32 * t + 8 * j : 32 * j + 8 * t));
        w[4 * j] = x.x;
        w[4 * j + 1] = x.y;
        w[4 * j + 2] = x.z;
        w[4 * j + 3] = x.w;
    }
    float factor = 1.f;
    if (E2M1) {
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 16; ++j) top = max(top, max((w[j] & 0x7fffu) << 16, w[j] & 0x7fff0000u));
        top = max(top, __shfl_xor_sync(kFull, top, 1));
        top = max(top, __shfl_xor_sync(kFull, top, 2));
        // 2^(14 - exponent of the largest); tiny rows (below 2^-100) are scaled as if they were that large
        const int ex = min(max((int)(top >> 23) - 127, -100), 127);
        const float up = __uint_as_float((uint32_t)(127 + 14 - ex) << 23);
        factor = __uint_as_float((uint32_t)(127 - 14 + ex) << 23);
        const bool finite = top < 0x7f800000u;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const __half2 v = __floats2half2_rn(__uint_as_float(w[j] << 16) * up, __uint_as_float(w[j] & 0xffff0000u) * up);
            w[j] = finite ? *reinterpret_cast<const uint32_t*>(&v) : 0x7fff7fffu;   // else the row is NaN
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        q[j][0] = w[2 * j];
        q[j][1] = w[2 * j + 1];
    }
    return factor;
}

__device__ __forceinline__ const uint16_t* query_row(const PagedAttnParams& p, int b, int h, int r)
{
    return p.q + (int64_t)b * p.q_b + (int64_t)(h * p.G + r / p.Mq) * p.q_h + (int64_t)(r % p.Mq) * p.q_i;
}

template <bool E2M1>
__device__ __forceinline__ void split_p(float x0, float x1, uint32_t& hi, uint32_t& lo)
{
    if (E2M1) {
        const __half2 a = __floats2half2_rn(x0, x1);
        const __half2 b = __floats2half2_rn(x0 - __low2float(a), x1 - __high2float(a));
        hi = *reinterpret_cast<const uint32_t*>(&a);
        lo = *reinterpret_cast<const uint32_t*>(&b);
    } else {
        split_bf16(x0, x1, hi, lo);
    }
}

// A tile of a sequence in three steps, each needing what the one before loaded: the lane's row (position), its
// page, its place in the pool.  The first nl tiles hold the list, the others the tail, whose tiles start at
// multiples of 16 (so that such a tile lies inside one page).
struct Seq {
    const int32_t* idx;     // the list of (b, h)
    const int32_t* table;   // the pages of b
    int nl, lo, len;        // list tiles, start of the tail, rows
};
__device__ __forceinline__ int tile_pos(const PagedAttnParams& p, const Seq& q, int it)   // -1: no such row
{
    const int j = threadIdx.x & 15;
    if (it < q.nl) {
        const int e = it * kTileRows + j;
        return e < p.kk ? q.idx[e] : -1;
    }
    const int pos = (q.lo & ~(kTileRows - 1)) + (it - q.nl) * kTileRows + j;
    return pos >= q.lo && pos < q.len ? pos : -1;
}
__device__ __forceinline__ int tile_page(const PagedAttnParams& p, const Seq& q, int it, int& pos)
{
    if (it < q.nl && (unsigned)pos >= (unsigned)q.len) {
        if (it * kTileRows + (int)(threadIdx.x & 15) < p.kk) atomicOr(p.err, FX_DEVERR_INDEX);
        pos = -1;
    }
    return pos >= 0 ? q.table[pos >> p.c.page_shift] : 0;
}
__device__ __forceinline__ Rows tile_place(const PagedAttnParams& p, int pos, int page)
{
    Rows r;
    bool ok = pos >= 0;
    if (ok && (unsigned)page >= (unsigned)p.c.n_pages) {
        atomicOr(p.err, FX_DEVERR_PAGE);
        ok = false;
    }
    r.pos = pos;
    r.id = ok ? (page << p.c.page_shift) | (pos & p.c.page_mask) : 0;
    r.vm = __ballot_sync(kFull, ok) & 0xffffu;
    return r;
}

// Joins the warps' partials of one query row in shared memory: the sum over them of dimension d, with the row's
// reference m (-inf: no warp saw anything) and its sum z.
template <int kRows>
__device__ __forceinline__ float join_row(const float* sm_o, const float* sm_m, const float* sm_l, int row, int d,
                                          float& m, float& z)
{
    m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kAttnWarps; ++w) m = fmaxf(m, sm_m[w * kRows + row]);
    z = 0.f;
    float acc = 0.f;
#pragma unroll
    for (int w = 0; w < kAttnWarps; ++w) {
        const float mw = sm_m[w * kRows + row];
        if (mw == -INFINITY) continue;   // that warp saw nothing
        const float f = fast_exp2(mw - m);
        z += f * sm_l[w * kRows + row];
        acc += f * sm_o[(w * kRows + row) * kHeadDim + d];
    }
    return acc;
}

// The query rows of one warp and what it has summed for them.
template <bool E2M1, int NT, bool DUP>
struct Acc {
    uint32_t q[NT][8][2];
    float rs[NT][2];      // factor of the logits of rows 2t, 2t+1 (of each N tile)
    float bias[NT][2];    // minus the reference of those rows; +inf: none yet
    float l[NT][2];
    float o[NT][8][4];
};

// Weights of a tile from its logits s (row g + 8 (e >> 1) of the tile, query row 2t + (e & 1) of N tile n), in
// place; moves the references when one would not fit.  hide: bit 4n + e, that logit does not count.
template <bool E2M1, int NT, bool DUP>
__device__ __forceinline__ void weights(Acc<E2M1, NT, DUP>& a, float (&s)[NT][4], uint32_t hide)
{
    float x2[NT][4];
    bool over = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x2[n][e] = fmaf(s[n][e], a.rs[n][e & 1], a.bias[n][e & 1]);
            if ((hide >> (4 * n + e)) & 1u) x2[n][e] = -INFINITY;
            over |= x2[n][e] > kTop;
        }
    if (__any_sync(kFull, over)) {
        // new references: the largest logit of each row lands on 2^kBase
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float z0 = (hide >> (4 * n + e)) & 1u ? -INFINITY : s[n][e] * a.rs[n][e];
                const float z1 = (hide >> (4 * n + e + 2)) & 1u ? -INFINITY : s[n][e + 2] * a.rs[n][e];
                float m = fmaxf(z0, z1);
                m = fmaxf(m, __shfl_xor_sync(kFull, m, 4));
                m = fmaxf(m, __shfl_xor_sync(kFull, m, 8));
                m = fmaxf(m, __shfl_xor_sync(kFull, m, 16));
                const float nb = fminf(a.bias[n][e], kBase - m);
                if (nb < a.bias[n][e]) {   // never for a row without a visible logit
                    const float f = fast_exp2(nb - a.bias[n][e]);   // 0 for the first reference
                    a.l[n][e] *= f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        a.o[n][i][e] *= f;
                        a.o[n][i][e + 2] *= f;
                    }
                    a.bias[n][e] = nb;
                }
                x2[n][e] = (hide >> (4 * n + e)) & 1u ? -INFINITY : fmaf(s[n][e], a.rs[n][e], nb);
                x2[n][e + 2] = (hide >> (4 * n + e + 2)) & 1u ? -INFINITY : fmaf(s[n][e + 2], a.rs[n][e], nb);
            }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float w = fast_exp2(x2[n][e]);
            if (!E2M1) {
                // to 17 bits, which the two bf16 parts hold exactly: the sum then counts the weights as
                // they are multiplied (one weight far above the others comes out as 1)
                const float c = __fmul_rn(w, 129.f);
                w = __fsub_rn(c, __fsub_rn(c, w));
            }
            s[n][e] = w;
            a.l[n][e & 1] += w;
        }
}

// One tile: logits, weights, O^T += V^T P^T.  after_k and after_v run when the tile's K and V rows are no longer
// needed (the caller loads the next tile into them).
template <bool E2M1, int NT, bool DUP, typename FK, typename FV>
__device__ __forceinline__ void attend_tile(const PagedAttnParams& p, Acc<E2M1, NT, DUP>& a, Tile<E2M1>& x,
                                            const Rows& rows, int r0, int seen, FK&& after_k, FV&& after_v)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    float s[NT][4];
    {
        float s2[NT][2][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 8; ++e) s2[n][e >> 2][e & 3] = 0.f;
        k_steps<E2M1>(x, [&](int j, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16<E2M1>(s2[n][j & 1], a0, a1, a2, a3, a.q[n][j][0], a.q[n][j][1]);
        });
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[n][e] = s2[n][0][e] + s2[n][1][e];
    }
    after_k();
    const bool late = __any_sync(kFull, ((rows.vm >> (lane & 15)) & 1u) && rows.pos > seen);
    uint32_t hide = 0;
    if (late || rows.vm != 0xffffu) {
        const int p0 = __shfl_sync(kFull, rows.pos, g), p1 = __shfl_sync(kFull, rows.pos, g + 8);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = r0 + 8 * n + (DUP ? (2 * t + (e & 1)) & 3 : 2 * t + (e & 1));
                const bool see = ((rows.vm >> (g + 8 * (e >> 1))) & 1u) && (e >> 1 ? p1 : p0) <= seen + r % p.Mq;
                if (!see) hide |= 1u << (4 * n + e);
            }
    }
    weights<E2M1, NT, DUP>(a, s, hide);

    // O^T += V^T P^T with P as a sum of two 16-bit parts.  Each tile's product starts from zero and is added
    // to O by an fp32 addition: the tensor core aligns all products to the accumulator and cuts them off
    // (2^-23 of it), which over a long row costs small weights beside a large one, and drifts.
    uint32_t bh[NT][2], bl[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            uint32_t hi, lo2;
            split_p<E2M1>(s[n][2 * u], s[n][2 * u + 1], hi, lo2);
            if (DUP) {
                bh[n][u] = movmatrix_t(t < 2 ? hi : lo2);
            } else {
                bh[n][u] = movmatrix_t(hi);
                bl[n][u] = movmatrix_t(lo2);
            }
        }
    auto product = [&](uint32_t vm, auto&& adds) {   // adds(n, e): query row 2t + e of N tile n takes it
        v_tiles<E2M1>(x, vm, [&](int i, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float c[4] = {0.f, 0.f, 0.f, 0.f};
                mma16<E2M1>(c, a0, a1, a2, a3, bh[n][0], bh[n][1]);
                if (!DUP) mma16<E2M1>(c, a0, a1, a2, a3, bl[n][0], bl[n][1]);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (adds(n, e & 1)) a.o[n][i][e] += c[e];
            }
        });
    };
    if (!late) {
        product(rows.vm, [](int, int) { return true; });
    } else {
        // rows that only later queries see: one product per query position, over the rows it sees (the
        // others may hold anything, and 0 * NaN is NaN) and for its query rows alone
        for (int i = 0; i < p.Mq; ++i) {
            uint32_t add = 0;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = r0 + 8 * n + (DUP ? (2 * t + e) & 3 : 2 * t + e);
                    if (r % p.Mq == i) add |= 1u << (2 * n + e);
                }
            product(__ballot_sync(kFull, rows.pos <= seen + i) & rows.vm,
                    [&](int n, int e) { return ((add >> (2 * n + e)) & 1u) != 0; });
        }
    }
    after_v();
}

// Query rows of one CTA's pass over a (sequence, KV head).
template <int NT, bool DUP>
__host__ __device__ constexpr int pass_rows() { return DUP ? 4 : 8 * NT; }

// Tiles of sequence b (at least one: an empty sequence's tile holds no valid row, and its output is written).
__device__ __forceinline__ Seq sequence(const PagedAttnParams& p, int b, bool report)
{
    Seq q;
    q.len = p.c.len[b];
    q.lo = p.tail_lo ? p.tail_lo[b] : 0;
    if (report && (q.len < 0 || q.len > p.c.cap || q.lo < 0)) atomicOr(p.err, FX_DEVERR_LEN);
    q.len = min(max(q.len, 0), p.c.cap);
    q.lo = max(q.lo, 0);
    q.nl = (p.kk + kTileRows - 1) / kTileRows;
    q.table = p.c.table + (int64_t)b * p.c.table_stride;
    q.idx = nullptr;
    return q;
}
__device__ __forceinline__ int tile_count(const Seq& q)
{
    const int nt = q.lo < q.len ? (q.len + kTileRows - 1) / kTileRows - q.lo / kTileRows : 0;
    return max(q.nl + nt, 1);
}

// Decode.  The tiles of all (sequence, KV head, group of query rows) form one line, which the CTAs share out
// evenly by the lengths found on the device, so that ragged lengths leave no CTA with more to do than another.
// A CTA walks its stretch of the line piece by piece (one (sequence, head, group) each); its warps take a
// piece's tiles in turn and meet in shared memory.  A piece that spans several CTAs is joined by the last of
// them to arrive, in the order of the CTAs.
//
// DUP: at most 4 query rows; columns 4..7 of the products repeat them, so that one product takes P's high part
// (columns 0..3) and its low part (4..7).
template <bool E2M1, int NT, bool DUP>
__global__ void __launch_bounds__(kAttnThreads, NT == 1 ? 2 : 1) paged_decode_kernel(const PagedAttnParams p)
{
    constexpr int kRows = pass_rows<NT, DUP>();
    extern __shared__ float smem[];
    float* sm_o = smem;                                        // [warp][row][128]
    float* sm_m = smem + kAttnWarps * kRows * kHeadDim;        // [warp][row]
    float* sm_l = sm_m + kAttnWarps * kRows;
    __shared__ long long sm_scan[kAttnWarps];
    __shared__ int sm_b;
    __shared__ long long sm_start;
    __shared__ unsigned sm_last;

    griddep_wait();
    griddep_launch();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int nrg = (p.R + kRows - 1) / kRows;
    const int per_tile = p.c.Hkv * nrg;   // pieces of one sequence

    // total length of the line, then this CTA's stretch of it and the sequence that it starts in
    long long total = 0;
    for (int b = tid; b < p.c.B; b += kAttnThreads) total += tile_count(sequence(p, b, blockIdx.x == 0));
    {
#pragma unroll
        for (int d = 16; d; d >>= 1) total += __shfl_xor_sync(kFull, total, d);
        if (lane == 0) sm_scan[warp] = total;
        __syncthreads();
        total = 0;
        for (int w = 0; w < kAttnWarps; ++w) total += sm_scan[w];
        total *= per_tile;
    }
    const int n_cta = (int)min((long long)gridDim.x, max(1ll, total / (kAttnWarps * kMinTiles)));
    const int cta = blockIdx.x;
    if (cta >= n_cta) return;
    long long at = total * cta / n_cta;                  // next tile of the line
    const long long end = total * (cta + 1) / n_cta;
    long long before = 0;                                // tiles (of one piece each) of the sequences before b
    for (int b0 = 0;; b0 += kAttnThreads) {
        const int b = b0 + tid;
        const int n = b < p.c.B ? tile_count(sequence(p, b, false)) : 0;
        long long inc = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long o = __shfl_up_sync(kFull, inc, d);
            if (lane >= d) inc += o;
        }
        __syncthreads();   // sm_scan is free
        if (tid == 0) sm_b = -1;
        if (lane == 31) sm_scan[warp] = inc;
        __syncthreads();
        long long sum = 0, mine = 0;
        for (int w = 0; w < kAttnWarps; ++w) {
            if (w == warp) mine = sum;
            sum += sm_scan[w];
        }
        const long long first = (before + mine + inc - n) * per_tile;
        if (n > 0 && at >= first && at < first + (long long)n * per_tile) {
            sm_b = b;
            sm_start = first;
        }
        __syncthreads();
        before += sum;
        if (sm_b >= 0) break;   // always found: at < total
    }
    int b = sm_b;
    long long seq_start = sm_start;
    Seq seq = sequence(p, b, false);
    int ntile = tile_count(seq);

    for (bool head = true; at < end; head = false) {
        while (at >= seq_start + (long long)ntile * per_tile) {
            seq_start += (long long)ntile * per_tile;
            seq = sequence(p, ++b, false);
            ntile = tile_count(seq);
        }
        const int piece = (int)((at - seq_start) / ntile);
        const long long piece_start = seq_start + (long long)piece * ntile;
        const int h = piece / nrg, r0 = (piece - h * nrg) * kRows;
        const int s0 = (int)(at - piece_start), s1 = (int)min((long long)ntile, end - piece_start);
        const int seen = seq.len - p.Mq;   // query i sees rows <= seen + i
        seq.idx = p.idx ? p.idx + ((int64_t)b * p.c.Hkv + h) * p.kk : nullptr;

        Acc<E2M1, NT, DUP> a;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = r0 + 8 * n + (DUP ? g & 3 : g);
            const float f = load_query<E2M1>(r < p.R ? query_row(p, b, h, r) : nullptr, a.q[n]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                a.rs[n][e] = p.qscale * __shfl_sync(kFull, f, (2 * t + e) * 4);
                a.bias[n][e] = INFINITY;
                a.l[n][e] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) a.o[n][i][e] = 0.f;
        }

        // the warp's tiles s0 + warp, + 8, ...: the rows of the next one are loaded while one is worked on, its
        // pages one tile earlier, its positions another one earlier
        int it = s0 + warp;
        if (it < s1) {
            int pos = tile_pos(p, seq, it);
            int page = tile_page(p, seq, it, pos);
            Rows rows = tile_place(p, pos, page);
            int pos1 = it + kAttnWarps < s1 ? tile_pos(p, seq, it + kAttnWarps) : -1;
            int page1 = it + kAttnWarps < s1 ? tile_page(p, seq, it + kAttnWarps, pos1) : 0;
            int pos2 = it + 2 * kAttnWarps < s1 ? tile_pos(p, seq, it + 2 * kAttnWarps) : -1;
            Rows next;
            auto advance = [&]() {   // places the next tile, looks the one after it up
                next = tile_place(p, pos1, page1);
                const int i2 = it + 2 * kAttnWarps, i3 = it + 3 * kAttnWarps;
                page1 = i2 < s1 ? tile_page(p, seq, i2, pos2) : 0;
                pos1 = pos2;
                pos2 = i3 < s1 ? tile_pos(p, seq, i3) : -1;
            };
            if constexpr (E2M1) {
                Tile<E2M1> x, y;
                load_k<E2M1>(p.c, h, rows, x);
                load_v<E2M1>(p.c, h, rows, x);
                auto turn = [&](Tile<E2M1>& cur, Tile<E2M1>& nxt) {
                    advance();
                    if (it + kAttnWarps < s1) {
                        load_k<E2M1>(p.c, h, next, nxt);
                        load_v<E2M1>(p.c, h, next, nxt);
                    }
                    attend_tile<E2M1, NT, DUP>(p, a, cur, rows, r0, seen, [] {}, [] {});
                    rows = next;
                    it += kAttnWarps;
                };
                while (true) {
                    turn(x, y);
                    if (it >= s1) break;
                    turn(y, x);
                    if (it >= s1) break;
                }
            } else {
                // bf16 rows fill 64 registers a lane: the next K takes the place of this tile's once the logits
                // are there, the next V that of this one's after the product
                Tile<E2M1> x;
                load_k<E2M1>(p.c, h, rows, x);
                load_v<E2M1>(p.c, h, rows, x);
                for (; it < s1; it += kAttnWarps) {
                    advance();
                    const bool more = it + kAttnWarps < s1;
                    attend_tile<E2M1, NT, DUP>(
                        p, a, x, rows, r0, seen, [&] { if (more) load_k<E2M1>(p.c, h, next, x); },
                        [&] { if (more) load_v<E2M1>(p.c, h, next, x); });
                    rows = next;
                }
            }
        }

        // the warps' partials meet in shared memory
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float z = a.l[n][e];
                z += __shfl_xor_sync(kFull, z, 4);
                z += __shfl_xor_sync(kFull, z, 8);
                z += __shfl_xor_sync(kFull, z, 16);
                const int row = 8 * n + 2 * t + e;
                if (g == 0 && row < kRows) {
                    sm_m[warp * kRows + row] = z != z ? 0.f : -a.bias[n][e];   // a NaN logit leaves no reference but shows
                    sm_l[warp * kRows + row] = z;
                }
            }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (DUP) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) a.o[n][i][e] += __shfl_xor_sync(kFull, a.o[n][i][e], 2);
                }
                if (!DUP || t < 2) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float* to = sm_o + ((warp * kRows + 8 * n + 2 * t + e) * kHeadDim + v_dim<E2M1>(i, g));
                        *reinterpret_cast<float2*>(to) = make_float2(a.o[n][i][e], a.o[n][i][e + 2]);
                    }
                }
            }
        __syncthreads();

        const bool whole = s0 == 0 && s1 == ntile;
        if (!whole) {
            // this CTA's part of the piece goes to its slot; the last CTA to arrive takes all of them over
            const int slot = cta * 2 + (head ? 0 : 1);
            float* part = p.part + (size_t)slot * kRows * (kHeadDim + 2);
            const int d = tid & (kHeadDim - 1);
            for (int row = tid / kHeadDim; row < kRows; row += kAttnThreads / kHeadDim) {
                float z, m;
                const float acc = join_row<kRows>(sm_o, sm_m, sm_l, row, d, m, z);
                part[row * kHeadDim + d] = acc;
                if (d == 0) {
                    part[kRows * kHeadDim + row] = m;
                    part[kRows * kHeadDim + kRows + row] = z;
                }
            }
            // CTA of line tile w: floor(((w + 1) n_cta - 1) / total)
            const int c0 = (int)(((piece_start + 1) * n_cta - 1) / total);
            const int c1 = (int)(((piece_start + ntile) * n_cta - 1) / total);
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const unsigned n = atomicAdd(p.counters + c0, 1u);
                sm_last = n == (unsigned)(c1 - c0);
                if (sm_last) {
                    p.counters[c0] = 0;   // ready for the next call
                    __threadfence();
                }
            }
            __syncthreads();
            if (!sm_last) {
                at = piece_start + s1;
                continue;
            }
            // each warp takes every eighth part, then the warps' sums meet as before.  A CTA's first piece is in
            // its slot 0; the piece starts in c0, as that CTA's first piece only if it starts its stretch
            const int s_first = c0 * 2 + (total * c0 / n_cta == piece_start ? 0 : 1);
            for (int row = 0; row < kRows; ++row) {
                float m = -INFINITY;
                for (int c = c0 + warp + kAttnWarps * lane; c <= c1; c += kAttnWarps * 32) {
                    const int sl = c == c0 ? s_first : c * 2;
                    m = fmaxf(m, __ldcg(p.part + (size_t)sl * kRows * (kHeadDim + 2) + kRows * kHeadDim + row));
                }
#pragma unroll
                for (int d2 = 16; d2; d2 >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, d2));
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                float z = 0.f;
#pragma unroll 4
                for (int c = c0 + warp; c <= c1; c += kAttnWarps) {
                    const int sl = c == c0 ? s_first : c * 2;
                    const float* from = p.part + (size_t)sl * kRows * (kHeadDim + 2);
                    const float mc = __ldcg(from + kRows * kHeadDim + row);
                    const float lc = __ldcg(from + kRows * kHeadDim + kRows + row);
                    const float4 oc = __ldcg(reinterpret_cast<const float4*>(from + row * kHeadDim) + lane);
                    const float f = mc == -INFINITY ? 0.f : fast_exp2(mc - m);
                    z += f * lc;
                    acc.x += f * oc.x;
                    acc.y += f * oc.y;
                    acc.z += f * oc.z;
                    acc.w += f * oc.w;
                }
                *(reinterpret_cast<float4*>(sm_o + (warp * kRows + row) * kHeadDim) + lane) = acc;
                if (lane == 0) {
                    sm_m[warp * kRows + row] = m;
                    sm_l[warp * kRows + row] = z;
                }
            }
            __syncthreads();
        }
        const int d = tid & (kHeadDim - 1);
        for (int row = tid / kHeadDim; row < kRows && r0 + row < p.R; row += kAttnThreads / kHeadDim) {
            float z, m;
            const float acc = join_row<kRows>(sm_o, sm_m, sm_l, row, d, m, z);
            const int r = r0 + row;
            const int64_t to = ((int64_t)b * p.Hq + h * p.G + r / p.Mq) * p.Mq + r % p.Mq;
            const bool none = m == -INFINITY;
            p.out[to * kHeadDim + d] = none ? 0.f : acc / z * p.c.v_mul;
            if (p.lse && d == 0) p.lse[to] = none ? -INFINITY : (m + log2f(z)) * 0.6931471805599453f;
        }
        __syncthreads();   // shared memory is free for the next piece
        at = piece_start + s1;
    }
}

constexpr int kImpTiles = 4;   // tiles of a warp of the importance kernel

// Importance: each warp takes kImpTiles tiles of 16 rows and every query row; the query fragments lie in
// shared memory as the products want them.
template <bool E2M1>
__global__ void __launch_bounds__(kAttnThreads) paged_importance_kernel(const PagedAttnParams p)
{
    __shared__ uint4 sq[kMaxRows / 8][4][32];
    __shared__ float srs[kMaxRows], sls[kMaxRows];
    griddep_wait();
    griddep_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int h = blockIdx.y, b = blockIdx.z;
    Seq seq = sequence(p, b, true);
    const int len = seq.len, seen = len - p.Mq;
    const int ntile = (p.R + 7) / 8;
    for (int n = warp; n < ntile; n += kAttnWarps) {
        const int r = 8 * n + g;
        uint32_t q[8][2];
        const float f = load_query<E2M1>(r < p.R ? query_row(p, b, h, r) : nullptr, q);
#pragma unroll
        for (int j = 0; j < 4; ++j) sq[n][j][lane] = make_uint4(q[2 * j][0], q[2 * j][1], q[2 * j + 1][0], q[2 * j + 1][1]);
        if (t == 0) {
            srs[r] = p.qscale * f;
            float z = -INFINITY;
            if (r < p.R) z = p.lse[((int64_t)b * p.Hq + h * p.G + r / p.Mq) * p.Mq + r % p.Mq];
            sls[r] = z == -INFINITY ? INFINITY : z * 1.4426950408889634f;   // a row that saw nothing adds nothing
        }
    }
    __syncthreads();
    const int first = (p.cand_lo & ~(kTileRows - 1)) + (blockIdx.x * kAttnWarps + warp) * (kImpTiles * kTileRows);
    seq.lo = first;
    float* out = p.scores + ((int64_t)b * p.c.Hkv + h) * (p.cand_hi - p.cand_lo);
    for (int u = 0; u < kImpTiles; ++u) {
        const int base = first + u * kTileRows;
        if (base >= p.cand_hi) break;
        float sum[2] = {0.f, 0.f};
        if (base < len) {
            int pos = tile_pos(p, seq, u);
            const int page = tile_page(p, seq, u, pos);
            const Rows rows = tile_place(p, pos, page);
            Tile<E2M1> x;
            load_k<E2M1>(p.c, h, rows, x);
            uint32_t a[8][4];
            k_steps<E2M1>(x, [&](int j, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
                a[j][0] = a0;
                a[j][1] = a1;
                a[j][2] = a2;
                a[j][3] = a3;
            });
            for (int n = 0; n < ntile; ++n) {
                float s[2][4] = {};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint4 q = sq[n][j][lane];
                    mma16<E2M1>(s[0], a[2 * j][0], a[2 * j][1], a[2 * j][2], a[2 * j][3], q.x, q.y);
                    mma16<E2M1>(s[1], a[2 * j + 1][0], a[2 * j + 1][1], a[2 * j + 1][2], a[2 * j + 1][3], q.z, q.w);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = 8 * n + 2 * t + (e & 1);
                    const int pos = base + g + 8 * (e >> 1);
                    const bool see = ((rows.vm >> (g + 8 * (e >> 1))) & 1u) && r < p.R && pos <= seen + r % p.Mq &&
                                     sls[r] != INFINITY;
                    if (see) sum[e >> 1] += fast_exp2(fmaf(s[0][e] + s[1][e], srs[r], -sls[r]));
                }
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            sum[e] += __shfl_xor_sync(kFull, sum[e], 1);
            sum[e] += __shfl_xor_sync(kFull, sum[e], 2);
        }
        const int pos = base + g + 8 * t;
        if (t < 2 && pos >= p.cand_lo && pos < p.cand_hi) out[pos - p.cand_lo] = t ? sum[1] : sum[0];
    }
}

// CTAs of a decode call: as many as are resident at once (one with more than 8 query rows, else two per SM).
int decode_ctas(int R, int sm_count) { return (R > 8 ? 1 : 2) * sm_count; }

template <bool E2M1, int NT, bool DUP>
cudaError_t launch_decode(const PagedAttnParams& p, int sm_count, bool pdl, cudaStream_t s)
{
    constexpr int kRows = pass_rows<NT, DUP>();
    constexpr size_t smem = sizeof(float) * kAttnWarps * kRows * (kHeadDim + 2);
    cudaError_t e = cudaFuncSetAttribute(paged_decode_kernel<E2M1, NT, DUP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem);
    if (e != cudaSuccess) return e;
    return launch_kernel(paged_decode_kernel<E2M1, NT, DUP>, dim3(decode_ctas(p.R, sm_count)), dim3(kAttnThreads), smem, s,
                         pdl, 0u, p);
}

}  // namespace

// The counters' region, then two partials (one of each end of a CTA's stretch) of up to 16 query rows per CTA.
size_t paged_decode_workspace_bytes(int R, int sm_count)
{
    const size_t rows = R <= 4 ? 4 : (R <= 8 ? 8 : 16);
    return kCounterBytes + (size_t)decode_ctas(R, sm_count) * 2 * rows * (kHeadDim + 2) * sizeof(float);
}

cudaError_t launch_paged_decode(const PagedAttnParams& p, bool e2m1, int sm_count, bool pdl, cudaStream_t s)
{
    if (e2m1) {
        if (p.R <= 4) return launch_decode<true, 1, true>(p, sm_count, pdl, s);
        if (p.R <= 8) return launch_decode<true, 1, false>(p, sm_count, pdl, s);
        return launch_decode<true, 2, false>(p, sm_count, pdl, s);
    }
    if (p.R <= 4) return launch_decode<false, 1, true>(p, sm_count, pdl, s);
    if (p.R <= 8) return launch_decode<false, 1, false>(p, sm_count, pdl, s);
    return launch_decode<false, 2, false>(p, sm_count, pdl, s);
}

cudaError_t launch_paged_importance(const PagedAttnParams& p, bool e2m1, bool pdl, cudaStream_t s)
{
    const int rows = p.cand_hi - (p.cand_lo & ~(kTileRows - 1));
    const int per = kAttnWarps * kImpTiles * kTileRows;
    const dim3 grid((rows + per - 1) / per, p.c.Hkv, p.c.B);
    return e2m1 ? launch_kernel(paged_importance_kernel<true>, grid, dim3(kAttnThreads), 0, s, pdl, 0u, p)
                : launch_kernel(paged_importance_kernel<false>, grid, dim3(kAttnThreads), 0, s, pdl, 0u, p);
}

}  // namespace fx
