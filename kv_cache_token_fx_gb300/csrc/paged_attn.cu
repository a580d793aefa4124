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

// The rows of tile `it` of a sequence: the first nl tiles hold the list, the others the tail, whose tiles start
// at multiples of 16 (so that a tile lies inside one page).
__device__ __forceinline__ Rows tile_rows(const PagedAttnParams& p, int b, int h, int it, int nl, int lo, int len)
{
    const int j = threadIdx.x & 15;
    Rows r;
    bool ok;
    if (it < nl) {
        const int e = it * kTileRows + j;
        ok = e < p.kk;
        r.pos = ok ? p.idx[((int64_t)b * p.c.Hkv + h) * p.kk + e] : 0;
        if (ok && (r.pos < 0 || r.pos >= len)) {
            ok = false;
            atomicOr(p.err, FX_DEVERR_INDEX);
        }
    } else {
        r.pos = (lo & ~(kTileRows - 1)) + (it - nl) * kTileRows + j;
        ok = r.pos >= lo && r.pos < len;
    }
    r.id = 0;
    if (ok) {
        const int pg = paged_page(p.c, b, r.pos, p.err);
        ok = pg >= 0;
        if (ok) r.id = (pg << p.c.page_shift) | (r.pos & p.c.page_mask);
    }
    r.vm = __ballot_sync(kFull, ok) & 0xffffu;
    return r;
}

// One CTA attends NT * 8 query rows (4 with DUP) of one (sequence, KV head) over all its tiles.
// DUP: at most 4 query rows; columns 4..7 repeat them, so that one product takes P's high part (columns
// 0..3) and its low part (4..7).
template <bool E2M1, int NT, bool DUP>
__global__ void __launch_bounds__(kAttnThreads, NT == 1 ? 2 : 1) paged_decode_kernel(const PagedAttnParams p)
{
    constexpr int kRows = DUP ? 4 : 8 * NT;   // query rows of the CTA
    extern __shared__ float smem[];
    float* sm_o = smem;                                        // [warp][row][128]
    float* sm_m = smem + kAttnWarps * kRows * kHeadDim;        // [warp][row]
    float* sm_l = sm_m + kAttnWarps * kRows;

    griddep_wait();
    griddep_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int nrg = (p.R + kRows - 1) / kRows;
    const int rg = blockIdx.x % nrg;
    const int h = (blockIdx.x / nrg) % p.c.Hkv;
    const int b = blockIdx.x / (nrg * p.c.Hkv);
    const int r0 = rg * kRows;
    const int len = paged_len(p.c, b, p.err);
    int lo = 0;
    if (p.tail_lo) {
        lo = p.tail_lo[b];
        if (lo < 0) {
            atomicOr(p.err, FX_DEVERR_LEN);
            lo = 0;
        }
    }
    const int nl = (p.kk + kTileRows - 1) / kTileRows;
    const int nt = lo < len ? (len + kTileRows - 1) / kTileRows - lo / kTileRows : 0;
    const int seen = len - p.Mq;   // query i sees rows <= seen + i

    uint32_t q[NT][8][2];
    float rs[NT][2];               // factor of the logits of rows 2t, 2t+1 (of each N tile)
    float bias[NT][2];             // minus the reference of those rows; +inf: none yet
    float l[NT][2];
    float o[NT][8][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int r = r0 + 8 * n + (DUP ? g & 3 : g);
        const float f = load_query<E2M1>(r < p.R ? query_row(p, b, h, r) : nullptr, q[n]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            rs[n][e] = p.qscale * __shfl_sync(kFull, f, (2 * t + e) * 4);
            bias[n][e] = INFINITY;
            l[n][e] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][i][e] = 0.f;
    }

    for (int it = warp; it < nl + nt; it += kAttnWarps) {
        const Rows rows = tile_rows(p, b, h, it, nl, lo, len);
        Tile<E2M1> x;
        load_k<E2M1>(p.c, h, rows, x);
        load_v<E2M1>(p.c, h, rows, x);

        float s[NT][4];
        {
            float s2[NT][2][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 8; ++e) s2[n][e >> 2][e & 3] = 0.f;
            k_steps<E2M1>(x, [&](int j, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
                for (int n = 0; n < NT; ++n) mma16<E2M1>(s2[n][j & 1], a0, a1, a2, a3, q[n][j][0], q[n][j][1]);
            });
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[n][e] = s2[n][0][e] + s2[n][1][e];
        }
        // logits of rows g, g + 8 of the tile (e >> 1) and query rows 2t, 2t + 1 (e & 1)
        const bool late = __any_sync(kFull, ((rows.vm >> (lane & 15)) & 1u) && rows.pos > seen);
        const bool edge = late || rows.vm != 0xffffu;
        uint32_t hide = 0;   // bit 4n + e: that logit does not count
        if (edge) {
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
        float x2[NT][4];
        bool over = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x2[n][e] = fmaf(s[n][e], rs[n][e & 1], bias[n][e & 1]);
                if ((hide >> (4 * n + e)) & 1u) x2[n][e] = -INFINITY;
                over |= x2[n][e] > kTop;
            }
        if (__any_sync(kFull, over)) {
            // new references: the largest logit of each row lands on 2^kBase
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float z0 = (hide >> (4 * n + e)) & 1u ? -INFINITY : s[n][e] * rs[n][e];
                    const float z1 = (hide >> (4 * n + e + 2)) & 1u ? -INFINITY : s[n][e + 2] * rs[n][e];
                    float m = fmaxf(z0, z1);
                    m = fmaxf(m, __shfl_xor_sync(kFull, m, 4));
                    m = fmaxf(m, __shfl_xor_sync(kFull, m, 8));
                    m = fmaxf(m, __shfl_xor_sync(kFull, m, 16));
                    const float nb = fminf(bias[n][e], kBase - m);
                    if (nb < bias[n][e]) {   // never for a row without a visible logit
                        const float f = fast_exp2(nb - bias[n][e]);   // 0 for the first reference
                        l[n][e] *= f;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            o[n][i][e] *= f;
                            o[n][i][e + 2] *= f;
                        }
                        bias[n][e] = nb;
                    }
                    x2[n][e] = (hide >> (4 * n + e)) & 1u ? -INFINITY : fmaf(s[n][e], rs[n][e], nb);
                    x2[n][e + 2] = (hide >> (4 * n + e + 2)) & 1u ? -INFINITY : fmaf(s[n][e + 2], rs[n][e], nb);
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
                l[n][e & 1] += w;
            }

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
        auto product = [&](uint32_t vm, uint32_t add) {   // bit 2n + e of add: row 2t + e of N tile n takes it
            v_tiles<E2M1>(x, vm, [&](int i, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float c[4] = {0.f, 0.f, 0.f, 0.f};
                    mma16<E2M1>(c, a0, a1, a2, a3, bh[n][0], bh[n][1]);
                    if (!DUP) mma16<E2M1>(c, a0, a1, a2, a3, bl[n][0], bl[n][1]);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if ((add >> (2 * n + (e & 1))) & 1u) o[n][i][e] += c[e];
                }
            });
        };
        if (!late) {
            product(rows.vm, 0xffffu);
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
                product(__ballot_sync(kFull, rows.pos <= seen + i) & rows.vm, add);
            }
        }
    }

    // the warps' partials meet in shared memory
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float z = l[n][e];
            z += __shfl_xor_sync(kFull, z, 4);
            z += __shfl_xor_sync(kFull, z, 8);
            z += __shfl_xor_sync(kFull, z, 16);
            const int row = 8 * n + 2 * t + e;
            if (g == 0 && row < kRows) {
                sm_m[warp * kRows + row] = z != z ? 0.f : -bias[n][e];   // a NaN logit leaves no reference but shows
                sm_l[warp * kRows + row] = z;
            }
        }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (DUP) {
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][i][e] += __shfl_xor_sync(kFull, o[n][i][e], 2);
            }
            if (!DUP || t < 2) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float* at = sm_o + ((warp * kRows + 8 * n + 2 * t + e) * kHeadDim + v_dim<E2M1>(i, g));
                    *reinterpret_cast<float2*>(at) = make_float2(o[n][i][e], o[n][i][e + 2]);
                }
            }
        }
    __syncthreads();
    const int d = threadIdx.x & (kHeadDim - 1);
    for (int row = threadIdx.x / kHeadDim; row < kRows && r0 + row < p.R; row += kAttnThreads / kHeadDim) {
        float m = -INFINITY;
        for (int w = 0; w < kAttnWarps; ++w) m = fmaxf(m, sm_m[w * kRows + row]);
        float z = 0.f, acc = 0.f;
        for (int w = 0; w < kAttnWarps; ++w) {
            const float mw = sm_m[w * kRows + row];
            if (mw == -INFINITY) continue;   // that warp saw nothing
            const float f = fast_exp2(mw - m);
            z += f * sm_l[w * kRows + row];
            acc += f * sm_o[(w * kRows + row) * kHeadDim + d];
        }
        const int r = r0 + row;
        const int64_t at = ((int64_t)b * p.Hq + h * p.G + r / p.Mq) * p.Mq + r % p.Mq;
        const bool none = m == -INFINITY;
        p.out[at * kHeadDim + d] = none ? 0.f : acc / z * p.c.v_mul;
        if (p.lse && d == 0) p.lse[at] = none ? -INFINITY : (m + log2f(z)) * 0.6931471805599453f;
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
    const int len = paged_len(p.c, b, p.err);
    const int seen = len - p.Mq;
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
    float* out = p.scores + ((int64_t)b * p.c.Hkv + h) * (p.cand_hi - p.cand_lo);
    for (int u = 0; u < kImpTiles; ++u) {
        const int base = first + u * kTileRows;
        if (base >= p.cand_hi) break;
        float sum[2] = {0.f, 0.f};
        if (base < len) {
            const Rows rows = tile_rows(p, b, h, u, 0, first, len);
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

template <bool E2M1, int NT, bool DUP>
cudaError_t launch_decode(const PagedAttnParams& p, bool pdl, cudaStream_t s)
{
    constexpr int kRows = DUP ? 4 : 8 * NT;
    constexpr size_t smem = sizeof(float) * kAttnWarps * kRows * (kHeadDim + 2);
    cudaError_t e = cudaFuncSetAttribute(paged_decode_kernel<E2M1, NT, DUP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem);
    if (e != cudaSuccess) return e;
    const int64_t grid = (int64_t)p.c.B * p.c.Hkv * ((p.R + kRows - 1) / kRows);
    return launch_kernel(paged_decode_kernel<E2M1, NT, DUP>, dim3((unsigned)grid), dim3(kAttnThreads), smem, s, pdl, 0u, p);
}

}  // namespace

size_t paged_decode_workspace_bytes(int B, int Hkv, int R, int sm_count)
{
    (void)B, (void)Hkv, (void)R, (void)sm_count;
    return kCounterBytes;
}

cudaError_t launch_paged_decode(const PagedAttnParams& p, bool e2m1, int sm_count, bool pdl, cudaStream_t s)
{
    (void)sm_count;
    if (e2m1) {
        if (p.R <= 4) return launch_decode<true, 1, true>(p, pdl, s);
        if (p.R <= 8) return launch_decode<true, 1, false>(p, pdl, s);
        return launch_decode<true, 2, false>(p, pdl, s);
    }
    if (p.R <= 4) return launch_decode<false, 1, true>(p, pdl, s);
    if (p.R <= 8) return launch_decode<false, 1, false>(p, pdl, s);
    return launch_decode<false, 2, false>(p, pdl, s);
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
