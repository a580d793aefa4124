// Rows into, out of and about a paged cache for sm_103a: the append with the position rotation (and, for the 4-bit
// format, the quantisation) on the way, the gather back to contiguous bf16 rows, compaction into other pages and copies of
// pages.
//
// Both move rows of 128 values and compute a few operations a value.  Bytes bound the long gather (4 x 32768 4-bit rows
// to bf16, 447 MB: 70 us, 0.94 of the copy bandwidth); the quantisation's instructions and bytes together the long
// append (24 K tokens, 4 bits, with 32 query heads: 77 us, 0.88 of the copy bandwidth; bf16 79 us, 0.97); start-up the
// decode step's few rows (2.0 us for one token of each of 8 sequences, 2.5 us of 64 in 4 bits).
#include <cuda_bf16.h>
#include <stdint.h>

#include "paged.cuh"

namespace fx {
namespace {

constexpr int kThreadsRows = 128;
constexpr int kCopyRows = kThreadsRows / 16;
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// x' = x c - y s and y' = y c + x s of the pairs in two words of bf16 values, every product and sum rounded to fp32
// (no contraction: the plain statement of the rotation then gives the same bits, and a 4-bit code never depends
// on how a compiler fused it).
__device__ __forceinline__ float turn_first(float x, float y, float c, float s) { return __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s)); }
__device__ __forceinline__ float turn_second(float x, float y, float c, float s) { return __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s)); }

// fp32 values to the nearest f16 and back.
__device__ __forceinline__ float2 snap(float x, float y) { return __half22float2(__floats2half2_rn(x, y)); }

// The codes (8 of them, 4 bytes) and the scale byte of the lane's half of a block of 16 values; the two lanes
// of a block (neighbours) agree on the scale.  All 32 lanes call it.
//
// Both quotients, max|y| / 6 and y / scale, are products with a rounded reciprocal: off by less than 2^-22 of
// themselves.  Their borders fall as in exact arithmetic all the same.  y is m 2^a with m < 256, an e4m3 border
// times 6 is 3 odd 2^b with odd < 32, an e2m1 border times the scale is c n 2^b with c n <= 300: a quotient that
// is not a border exactly is at least 1/300 of itself away from it.  Rounding to f16 (2^-11 of the value) puts
// the product of one that is a border exactly on it -- the borders are f16 values -- and moves no other across.
__device__ __forceinline__ uint32_t quantize_chunk(uint4 x, float inv, uint32_t& scale_byte)
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t top2 = 0;   // largest magnitudes as bits (ordered like the magnitudes; NaN above infinity)
#pragma unroll
    for (int j = 0; j < 4; ++j) top2 = __vmaxu2(top2, w[j] & 0x7fff7fffu);
    top2 = __vmaxu2(top2, __shfl_xor_sync(kAll, top2, 1));
    const uint32_t top = max(top2 << 16, top2 & 0xffff0000u);
    const bool finite = top < 0x7f800000u;
    const float a = __uint_as_float(top) * inv * (1.f / 6.f);
    scale_byte = e4m3_from_f32(snap(fminf(fmaxf(a, 0.001953125f), 480.f), 0.f).x);   // 2^-9 to 448
    const float s = __half2float(__ushort_as_half((unsigned short)(e4m3x2_to_f16x2(scale_byte) & 0xffffu)));
    const float f = inv * __frcp_rn(s);
    uint32_t codes = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 v = snap(bf16_lo(w[j]) * f, bf16_hi(w[j]) * f);
        codes |= e2m1x2_from_f32(v.x, v.y) << (8 * j);
    }
    if (!finite) {
        scale_byte = 0x7fu;
        codes = 0;
    }
    return codes;
}

// Cosines and sines of pairs j .. j + 3 (j a multiple of 4), each at the position of its axis.
__device__ __forceinline__ void pairs_of_axes(const PagedAppendParams& p, const int (&ax)[kMaxAxes], int j, float4& c, float4& s)
{
    const int half = p.rot >> 1;
    auto at = [&](int a) { return a == 0 ? ax[0] : (a == 1 ? ax[1] : (a == 2 ? ax[2] : ax[3])); };
    const uchar4 w = *reinterpret_cast<const uchar4*>(p.axis + j);
    if (w.x == w.y && w.x == w.z && w.x == w.w) {
        const float* cs = p.cos_sin + (int64_t)at(w.x) * p.rot + j;
        c = __ldg(reinterpret_cast<const float4*>(cs));
        s = __ldg(reinterpret_cast<const float4*>(cs + half));
    } else {
        const float* cs = p.cos_sin + j;
        const int64_t a0 = (int64_t)at(w.x) * p.rot, a1 = (int64_t)at(w.y) * p.rot + 1, a2 = (int64_t)at(w.z) * p.rot + 2,
                      a3 = (int64_t)at(w.w) * p.rot + 3;
        c = make_float4(__ldg(cs + a0), __ldg(cs + a1), __ldg(cs + a2), __ldg(cs + a3));
        s = make_float4(__ldg(cs + half + a0), __ldg(cs + half + a1), __ldg(cs + half + a2), __ldg(cs + half + a3));
    }
}

// 8 lanes take R rows of one token -- K heads, V heads or query heads -- and of each row two chunks of 8 values:
// chunks c0 and c1, which are the two sides of 8 rotated pairs in the half-split form.  The rows' loads need
// neither the token's place nor its position and go out first, and the rows share its cosines and sines.
// 8 CTAs of 128 threads an SM (64 registers), and queries and new rows that pass by L2's older contents when there are
// many: a prompt of 24 K tokens, 4 bits, with its read-back 91 us, against 95 without the latter, 100 without either and
// 105 with 10 CTAs.
//
// AXES: a pair's cosine and sine are of its own axis' position.  Four neighbouring pairs of one axis are loaded as one.
template <bool E2M1, int R, bool INTERLEAVED, bool AXES>
__global__ void __launch_bounds__(kThreadsRows, AXES ? 10 : 8) paged_append_kernel(const PagedAppendParams p)
{
    griddep_wait();
    griddep_launch();
    const unsigned gk = (p.c.Hkv + R - 1) / R, groups = 2 * gk + (p.Hq + R - 1) / R;   // groups of one token
    const unsigned u = blockIdx.x * (unsigned)(kThreadsRows / 8) + (threadIdx.x >> 3);
    const int l = threadIdx.x & 7, half = p.rot >> 1, hc = p.rot >> 4;
    const int i = (int)(u / groups);
    const unsigned in = u - i * groups;
    const int kind = in < gk ? 0 : (in < 2 * gk ? 1 : 2);          // K, V, queries
    const int h0 = (int)(in - (kind == 0 ? 0 : (kind == 1 ? gk : 2 * gk))) * R;
    // (hc is even, so chunk ^ 1 is the same chunk of lane ^ 1: the other half of its block of 16)
    const int c0 = INTERLEAVED || l < hc ? l : l + hc, c1 = INTERLEAVED || l >= hc ? l + 8 : l + hc;
    bool live = i < p.n;
    const int rows = live ? min(R, (kind == 2 ? p.Hq : p.c.Hkv) - h0) : 0;
    uint4 x[R][2];
    {
        const uint16_t* src = kind == 2 ? p.q + i * p.q_n + h0 * p.q_h : (kind ? p.v : p.k) + i * p.n_stride + h0 * p.h_stride;
        const int64_t step = kind == 2 ? p.q_h : p.h_stride;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            x[r][0] = x[r][1] = make_uint4(0, 0, 0, 0);
            if (r < rows) {
                // (q_out may be q: not read-only loads)
                x[r][0] = R > 1 ? __ldcs(reinterpret_cast<const uint4*>(src + 8 * c0)) : *reinterpret_cast<const uint4*>(src + 8 * c0);
                x[r][1] = R > 1 ? __ldcs(reinterpret_cast<const uint4*>(src + 8 * c1)) : *reinterpret_cast<const uint4*>(src + 8 * c1);
            }
            src += step;
        }
    }
    int seq = -1, pos = 0, at = 0, page = -1;
    int ax[kMaxAxes] = {};
    if (live) {
        seq = __ldg(p.seq + i);
        pos = __ldg(p.pos + i);
        at = p.rope_pos ? __ldg(p.rope_pos + i) : pos;
        // Neighbours: tested before the chain below (prompts of up to 8191 tokens in 4 bits 71.2 us for 73.5).  Halves: within it
        // (bf16 79.3 for 81.0); with axes, axis by axis (bf16 81.7 for 87.0).
        bool at_bad = INTERLEAVED && p.rot > 0 && (at < 0 || at >= p.n_pos);
        if (AXES) {
#pragma unroll
            for (int a = 0; a < kMaxAxes; ++a) {
                ax[a] = a < p.n_axes ? __ldg(p.rope_pos + (int64_t)a * p.n + i) : 0;
                at_bad |= ax[a] < 0 || ax[a] >= p.n_pos;
            }
        }
        unsigned bad = 0;
        if (seq < 0 || seq >= p.c.B)
            bad = seq == -1 ? 0u : FX_DEVERR_INDEX;
        else if (pos < 0 || pos >= p.c.cap)
            bad = FX_DEVERR_LEN;
        else if (INTERLEAVED || AXES ? at_bad : p.rot > 0 && (at < 0 || at >= p.n_pos))
            bad = FX_DEVERR_INDEX;
        live = seq >= 0 && bad == 0;
        if (bad && in == 0 && l == 0) atomicOr(p.err, bad);
        if (live && kind != 2) page = paged_page(p.c, seq, pos, p.err);
    }
    if (live && kind != 1 && p.rot > 0) {
        const float* cs = p.cos_sin + (int64_t)at * p.rot;
        float c[8], s[8];
        if (!INTERLEAVED) {
            if (l < hc) {   // pairs (8 l + j, 8 l + j + half)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float4 a, b;
                    if (AXES) {
                        pairs_of_axes(p, ax, 8 * l + 4 * j, a, b);
                    } else {
                        a = __ldg(reinterpret_cast<const float4*>(cs + 8 * l) + j);
                        b = __ldg(reinterpret_cast<const float4*>(cs + half + 8 * l) + j);
                    }
                    c[4 * j] = a.x, c[4 * j + 1] = a.y, c[4 * j + 2] = a.z, c[4 * j + 3] = a.w;
                    s[4 * j] = b.x, s[4 * j + 1] = b.y, s[4 * j + 2] = b.z, s[4 * j + 3] = b.w;
                }
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const uint32_t a[4] = {x[r][0].x, x[r][0].y, x[r][0].z, x[r][0].w};
                    const uint32_t b[4] = {x[r][1].x, x[r][1].y, x[r][1].z, x[r][1].w};
                    uint32_t y[4], z[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float a0 = bf16_lo(a[j]), a1 = bf16_hi(a[j]), b0 = bf16_lo(b[j]), b1 = bf16_hi(b[j]);
                        y[j] = pack_bf16x2(turn_first(a0, b0, c[2 * j], s[2 * j]), turn_first(a1, b1, c[2 * j + 1], s[2 * j + 1]));
                        z[j] = pack_bf16x2(turn_second(a0, b0, c[2 * j], s[2 * j]), turn_second(a1, b1, c[2 * j + 1], s[2 * j + 1]));
                    }
                    x[r][0] = make_uint4(y[0], y[1], y[2], y[3]);
                    x[r][1] = make_uint4(z[0], z[1], z[2], z[3]);
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int chunk = k ? c1 : c0;
                if (chunk >= 2 * hc) continue;
                float4 a, b;
                if (AXES) {
                    pairs_of_axes(p, ax, 4 * chunk, a, b);
                } else {
                    a = __ldg(reinterpret_cast<const float4*>(cs + 4 * chunk));
                    b = __ldg(reinterpret_cast<const float4*>(cs + half + 4 * chunk));
                }
                c[0] = a.x, c[1] = a.y, c[2] = a.z, c[3] = a.w;
                s[0] = b.x, s[1] = b.y, s[2] = b.z, s[3] = b.w;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const uint32_t w[4] = {x[r][k].x, x[r][k].y, x[r][k].z, x[r][k].w};
                    uint32_t y[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        y[j] = pack_bf16x2(turn_first(bf16_lo(w[j]), bf16_hi(w[j]), c[j], s[j]),
                                           turn_second(bf16_lo(w[j]), bf16_hi(w[j]), c[j], s[j]));
                    x[r][k] = make_uint4(y[0], y[1], y[2], y[3]);
                }
            }
        }
    }
    const int64_t row = pos & p.c.page_mask;
    if (kind == 2 && live) {
        uint16_t* to = p.q_out + i * p.qo_n + h0 * p.qo_h;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (r < rows) {
                if (R > 1) {
                    __stcs(reinterpret_cast<uint4*>(to + 8 * c0), x[r][0]);
                    __stcs(reinterpret_cast<uint4*>(to + 8 * c1), x[r][1]);
                } else {
                    *reinterpret_cast<uint4*>(to + 8 * c0) = x[r][0];
                    *reinterpret_cast<uint4*>(to + 8 * c1) = x[r][1];
                }
            }
            to += p.qo_h;
        }
    }
    const bool keep = page >= 0;   // K or V rows with a place in the pool
    if (!__any_sync(kAll, keep)) return;
    char* dst = (kind ? p.c.v : p.c.k) + (int64_t)max(page, 0) * p.c.sp + h0 * p.c.sh + row * p.c.st;
    char* sd = (kind ? p.c.vs : p.c.ks) + (int64_t)max(page, 0) * p.c.ssp + h0 * p.c.ssh + row * p.c.sst;
    const float inv = kind ? p.c.v_inv : p.c.k_inv;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (E2M1) {
            uint32_t b0, b1;
            const uint32_t z0 = quantize_chunk(x[r][0], inv, b0), z1 = quantize_chunk(x[r][1], inv, b1);
            if (keep && r < rows) {
                *reinterpret_cast<uint32_t*>(dst + 4 * c0) = z0;
                *reinterpret_cast<uint32_t*>(dst + 4 * c1) = z1;
                if ((l & 1) == 0) {
                    sd[c0 >> 1] = (char)b0;
                    sd[c1 >> 1] = (char)b1;
                }
            }
        } else if (keep && r < rows) {
            *reinterpret_cast<uint4*>(dst + 16 * c0) = x[r][0];
            *reinterpret_cast<uint4*>(dst + 16 * c1) = x[r][1];
        }
        dst += p.c.sh;
        sd += p.c.ssh;
    }
}

// 16 lanes take R rows, 16 apart, of one (sequence, KV head): the loads of all go out before the first store.
template <bool E2M1, int R>
__global__ void __launch_bounds__(kThreadsRows) paged_gather_kernel(const PagedGatherParams p)
{
    griddep_wait();
    griddep_launch();
    const int c = threadIdx.x & 15;
    const int h = blockIdx.y, b = blockIdx.z;
    const int i0 = blockIdx.x * (kCopyRows * R) + (threadIdx.x >> 4);
    const int64_t out0 = ((int64_t)b * p.c.Hkv + h) * p.n;
    int len = p.c.len[b], lo = p.lo ? p.lo[b] : 0;
    if (len < 0 || len > p.c.cap || lo < 0) {
        if (threadIdx.x == 0) atomicOr(p.err, FX_DEVERR_LEN);
        len = len < 0 ? 0 : min(len, p.c.cap);
        lo = max(lo, 0);
    }
    int t[R], page[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int i = i0 + r * kCopyRows;
        t[r] = -1;
        if (i < p.n) {
            if (p.idx) {
                t[r] = p.idx[out0 + i];
                if (t[r] < 0 || t[r] >= len) {
                    if (c == 0) atomicOr(p.err, FX_DEVERR_INDEX);
                    t[r] = -1;
                }
            } else if ((int64_t)lo + i < len) {
                t[r] = lo + i;
            }
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) page[r] = t[r] >= 0 ? paged_page(p.c, b, t[r], p.err) : -1;
    uint4 x[R][2];
    uint32_t sb[R][2];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (page[r] < 0) continue;
        const int64_t row = t[r] & p.c.page_mask;
        const int64_t at = (int64_t)page[r] * p.c.sp + h * p.c.sh + row * p.c.st;
        const int64_t sat = (int64_t)page[r] * p.c.ssp + h * p.c.ssh + row * p.c.sst + (c >> 1);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const char* src = (w ? p.c.v : p.c.k) + at;
            if (E2M1) {
                x[r][w].x = __ldcs(reinterpret_cast<const uint32_t*>(src + 4 * c));
                sb[r][w] = (uint8_t)(w ? p.c.vs : p.c.ks)[sat];
            } else {
                x[r][w] = __ldcs(reinterpret_cast<const uint4*>(src + 16 * c));
            }
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (page[r] < 0) continue;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            uint4 o = x[r][w];
            if (E2M1) {
                const float s = __half2float(__ushort_as_half((unsigned short)(e4m3x2_to_f16x2(sb[r][w]) & 0xffffu))) *
                                (w ? p.c.v_mul : p.c.k_mul);
                uint32_t f[4], z[4];
                e2m1x8_to_f16(o.x, f[0], f[1], f[2], f[3]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 v = __half22float2(*reinterpret_cast<__half2*>(&f[j]));
                    z[j] = pack_bf16x2(v.x * s, v.y * s);
                }
                o = make_uint4(z[0], z[1], z[2], z[3]);
            }
            __stcs(reinterpret_cast<uint4*>((w ? p.v_out : p.k_out) + (out0 + i0 + r * kCopyRows) * kHeadDim + 8 * c), o);
        }
    }
}

// Rows of K and V as they are stored, 16 bytes (and a 4-bit row's 8 bytes of scales) at a time.
//
// Compaction: kLanes lanes take R rows, a CTA's rows apart, of one (sequence, KV head): the loads of all go out before the
// first store.
template <bool E2M1, int R>
__global__ void __launch_bounds__(kThreadsRows) paged_compact_kernel(const PagedCompactParams p)
{
    griddep_wait();
    griddep_launch();
    constexpr int kLanes = E2M1 ? 4 : 16, kRows = kThreadsRows / kLanes;
    const int c = threadIdx.x % kLanes, h = blockIdx.y, b = blockIdx.z;
    const int64_t first = (int64_t)blockIdx.x * (kRows * R);
    int len = p.src.len[b], lo = p.tail_lo ? p.tail_lo[b] : 0;
    const bool report = blockIdx.x == 0 && h == 0 && threadIdx.x == 0;
    if (report && (len < 0 || len > p.src.cap || lo < 0)) atomicOr(p.err, FX_DEVERR_LEN);
    len = min(max(len, 0), p.src.cap);
    lo = max(lo, 0);
    const int64_t total = (int64_t)p.k + (p.tail_lo ? max(len - lo, 0) : 0);
    const int rows = (int)(total < p.dst.cap ? total : p.dst.cap);
    if (report) {
        if (total > rows) atomicOr(p.err, FX_DEVERR_CAPACITY);
        const_cast<int32_t*>(p.dst.len)[b] = rows;
    }
    if (first >= rows) return;
    const int32_t* idx = p.idx + ((int64_t)b * p.src.Hkv + h) * p.k;
    int t[R], from[R], to[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int64_t i = first + r * kRows + threadIdx.x / kLanes;
        t[r] = -1;
        if (i < rows) {
            t[r] = i < p.k ? idx[i] : lo + (int)(i - p.k);
            if (t[r] < 0 || t[r] >= len) {
                if (c == 0) atomicOr(p.err, FX_DEVERR_INDEX);
                t[r] = -1;
            }
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int i = (int)(first + r * kRows) + threadIdx.x / kLanes;
        from[r] = t[r] >= 0 ? paged_page(p.src, b, t[r], p.err) : -1;
        to[r] = t[r] >= 0 ? paged_page(p.dst, b, i, p.err) : -1;
    }
    uint4 x[R][2];
    uint2 z[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (from[r] < 0 || to[r] < 0) continue;
        const int64_t row = t[r] & p.src.page_mask;
        const int64_t at = (int64_t)from[r] * p.src.sp + h * p.src.sh + row * p.src.st + 16 * c;
        x[r][0] = __ldcs(reinterpret_cast<const uint4*>(p.src.k + at));
        x[r][1] = __ldcs(reinterpret_cast<const uint4*>(p.src.v + at));
        if (E2M1 && c < 2)
            z[r] = __ldcs(reinterpret_cast<const uint2*>((c ? p.src.vs : p.src.ks) + (int64_t)from[r] * p.src.ssp + h * p.src.ssh +
                                                            row * p.src.sst));
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (from[r] < 0 || to[r] < 0) continue;
        const int64_t row = ((int)(first + r * kRows) + threadIdx.x / kLanes) & p.dst.page_mask;
        const int64_t at = (int64_t)to[r] * p.dst.sp + h * p.dst.sh + row * p.dst.st + 16 * c;
        __stcs(reinterpret_cast<uint4*>(p.dst.k + at), x[r][0]);
        __stcs(reinterpret_cast<uint4*>(p.dst.v + at), x[r][1]);
        if (E2M1 && c < 2)
            __stcs(reinterpret_cast<uint2*>((c ? p.dst.vs : p.dst.ks) + (int64_t)to[r] * p.dst.ssp + h * p.dst.ssh + row * p.dst.sst),
                   z[r]);
    }
}

// Copies of pages: a CTA takes the rows of one (page, KV head), R pieces of 16 bytes of K and of V a thread at a time.
template <bool E2M1, int R>
__global__ void __launch_bounds__(kThreadsRows) paged_copy_kernel(const PagedCopyParams p)
{
    griddep_wait();
    griddep_launch();
    constexpr int kLanes = E2M1 ? 4 : 16, kRows = kThreadsRows / kLanes;
    const int h = blockIdx.y;
    const int from = p.from[blockIdx.x], to = p.to[blockIdx.x];
    if (from == -1 || to == -1) return;
    if ((unsigned)from >= (unsigned)p.c.n_pages || (unsigned)to >= (unsigned)p.c.n_pages) {
        if (h == 0 && threadIdx.x == 0) atomicOr(p.err, FX_DEVERR_PAGE);
        return;
    }
    const int64_t in = h * p.c.sh + 16 * (threadIdx.x % kLanes);
    const char* const src = p.c.k + (int64_t)from * p.c.sp + in;
    char* const dst = p.c.k + (int64_t)to * p.c.sp + in;
    const int64_t dv = p.c.v - p.c.k;
    const int page_rows = p.c.page_mask + 1;
    for (int row0 = threadIdx.x / kLanes; row0 < page_rows; row0 += R * kRows) {
        uint4 x[R][2];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t at = (int64_t)(row0 + r * kRows) * p.c.st;
            if (row0 + r * kRows < page_rows) {
                x[r][0] = __ldcs(reinterpret_cast<const uint4*>(src + at));
                x[r][1] = __ldcs(reinterpret_cast<const uint4*>(src + dv + at));
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t at = (int64_t)(row0 + r * kRows) * p.c.st;
            if (row0 + r * kRows < page_rows) {
                __stcs(reinterpret_cast<uint4*>(dst + at), x[r][0]);
                __stcs(reinterpret_cast<uint4*>(dst + dv + at), x[r][1]);
            }
        }
    }
    if (E2M1) {
        const int64_t ds = p.c.vs - p.c.ks;
        for (int row = threadIdx.x; row < page_rows; row += kThreadsRows) {
            const int64_t at = h * p.c.ssh + (int64_t)row * p.c.sst;
            const char* s = p.c.ks + (int64_t)from * p.c.ssp + at;
            char* d = p.c.ks + (int64_t)to * p.c.ssp + at;
            const uint2 a = __ldcs(reinterpret_cast<const uint2*>(s)), b = __ldcs(reinterpret_cast<const uint2*>(s + ds));
            __stcs(reinterpret_cast<uint2*>(d), a);
            __stcs(reinterpret_cast<uint2*>(d + ds), b);
        }
    }
}

template <bool E2M1, bool INTERLEAVED, bool AXES>
cudaError_t append(const PagedAppendParams& p, int sm_count, bool pdl, cudaStream_t s)
{
    // A decode step's few rows: one row each, for the shortest way through (a step of 64 sequences with its read-back
    // 4.6 us, against 5.6 with four).  More rows than the machine has groups of 8 lanes: four rows each, for their shared
    // cosines and more loads in flight (a prompt of 24 K tokens with its read-back 92 us, against 124 with one).
    const bool many = (int64_t)p.n * (2 * p.c.Hkv + p.Hq) > sm_count * 2048 / 8;
    // With axes two rows each and 10 CTAs an SM: the angles are more loads, which more warps wait for.  Four prompts of up to
    // 8191 tokens, us with axes in sections and in turns:
    //   rows, CTAs    bf16 halves    bf16 neighbours    4 bits halves    4 bits neighbours   (halves: 5 us less in the first
    //                                                                                        line since, as noted in the kernel)
    //   2, 10           82,  86         84,  92            76,  88           76,  88
    //   4, 8            97, 102         98, 105            85,  87           84,  88
    //   2, 8            91,  98         95, 105            80,  94           81,  96
    //   4, 10          102, 111        103, 109            99, 106           87,  92
    //   1, 10          116, 131        124, 153           115, 138          123, 154
    constexpr int kMany = AXES ? 2 : 4;
    const int R = many ? kMany : 1;
    const int64_t groups = (int64_t)p.n * (2 * ((p.c.Hkv + R - 1) / R) + (p.Hq + R - 1) / R);
    const dim3 grid((unsigned)((groups + kThreadsRows / 8 - 1) / (kThreadsRows / 8)));
    return many ? launch_kernel(paged_append_kernel<E2M1, kMany, INTERLEAVED, AXES>, grid, dim3(kThreadsRows), 0, s, pdl, 0u, p)
                : launch_kernel(paged_append_kernel<E2M1, 1, INTERLEAVED, AXES>, grid, dim3(kThreadsRows), 0, s, pdl, 0u, p);
}

template <bool E2M1>
cudaError_t gather(const PagedGatherParams& p, int sm_count, bool pdl, cudaStream_t s)
{
    // few rows: one each (205 listed rows of 64 heads: bf16 4.2 us, against 5.1 with four, 4 bits 3.5 against 4.4); many:
    // four in flight (4 x 32768 4-bit rows 70 us, against 133 with one)
    const bool many = (int64_t)p.n * p.c.Hkv * p.c.B > 2 * sm_count * 2048 / 16;
    const int rows = kCopyRows * (many ? 4 : 1);
    const dim3 grid((p.n + rows - 1) / rows, p.c.Hkv, p.c.B);
    return many ? launch_kernel(paged_gather_kernel<E2M1, 4>, grid, dim3(kThreadsRows), 0, s, pdl, 0u, p)
                : launch_kernel(paged_gather_kernel<E2M1, 1>, grid, dim3(kThreadsRows), 0, s, pdl, 0u, p);
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendParams& p, bool e2m1, int sm_count, bool pdl, cudaStream_t s)
{
    if (p.n_axes) {
        if (p.interleaved) return e2m1 ? append<true, true, true>(p, sm_count, pdl, s) : append<false, true, true>(p, sm_count, pdl, s);
        return e2m1 ? append<true, false, true>(p, sm_count, pdl, s) : append<false, false, true>(p, sm_count, pdl, s);
    }
    if (p.interleaved) return e2m1 ? append<true, true, false>(p, sm_count, pdl, s) : append<false, true, false>(p, sm_count, pdl, s);
    return e2m1 ? append<true, false, false>(p, sm_count, pdl, s) : append<false, false, false>(p, sm_count, pdl, s);
}

cudaError_t launch_paged_compact(const PagedCompactParams& p, bool e2m1, int sm_count, bool pdl, cudaStream_t s)
{
    const int rows = kThreadsRows / (e2m1 ? 4 : 16) * 4;
    const dim3 grid((unsigned)((p.rows + (int64_t)rows - 1) / rows), p.src.Hkv, p.src.B);
    return e2m1 ? launch_kernel(paged_compact_kernel<true, 4>, grid, dim3(kThreadsRows), 0, s, pdl, 0u, p)
                : launch_kernel(paged_compact_kernel<false, 4>, grid, dim3(kThreadsRows), 0, s, pdl, 0u, p);
}

cudaError_t launch_paged_copy(const PagedCopyParams& p, bool e2m1, bool pdl, cudaStream_t s)
{
    const dim3 grid(p.n, p.c.Hkv);
    return e2m1 ? launch_kernel(paged_copy_kernel<true, 2>, grid, dim3(kThreadsRows), 0, s, pdl, 0u, p)
                : launch_kernel(paged_copy_kernel<false, 4>, grid, dim3(kThreadsRows), 0, s, pdl, 0u, p);
}

cudaError_t launch_paged_gather(const PagedGatherParams& p, bool e2m1, int sm_count, bool pdl, cudaStream_t s)
{
    return e2m1 ? gather<true>(p, sm_count, pdl, s) : gather<false>(p, sm_count, pdl, s);
}

}  // namespace fx
