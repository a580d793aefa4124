// Rows into and out of a paged cache for sm_103a: the append with the position rotation (and, for the 4-bit
// format, the quantisation) on the way, and the gather back to contiguous bf16 rows.
//
// Both move rows of 128 values and compute a few operations a value: bytes bound them (a long append or
// gather), or start-up (a decode step's few rows).  16 lanes take one row, 8 values (16 bytes of bf16, 4 bytes
// of codes) a lane.
#include <cuda_bf16.h>
#include <stdint.h>

#include "paged.cuh"

namespace fx {
namespace {

constexpr int kThreadsRows = 256;
constexpr int kCopyRows = kThreadsRows / 16;
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// One member of a rotated pair: own * c -+ other * s, every product and the sum rounded to fp32 (no
// contraction: the plain statement of the rotation then gives the same bits, and a 4-bit code never depends on
// how a compiler fused it).
__device__ __forceinline__ float turn(float own, float other, float c, float s, bool second)
{
    const float a = __fmul_rn(own, c), b = __fmul_rn(other, s);
    return second ? __fadd_rn(a, b) : __fsub_rn(a, b);
}

// Cosines and sines of the lane's 8 dimensions at one position (only c[0..3], s[0..3] when pairs are neighbours).
struct Turn {
    float c[8], s[8];
};
__device__ __forceinline__ void load_turn(Turn& w, const float* cs, int c, int rot, bool interleaved)
{
    const int half = rot >> 1, hc = rot >> 4;
    const float* at = cs + (interleaved ? 4 * c : 8 * (c >= hc ? c - hc : c));
    const float4 c0 = __ldg(reinterpret_cast<const float4*>(at)), s0 = __ldg(reinterpret_cast<const float4*>(at + half));
    w.c[0] = c0.x, w.c[1] = c0.y, w.c[2] = c0.z, w.c[3] = c0.w;
    w.s[0] = s0.x, w.s[1] = s0.y, w.s[2] = s0.z, w.s[3] = s0.w;
    if (!interleaved) {
        const float4 c1 = __ldg(reinterpret_cast<const float4*>(at + 4)), s1 = __ldg(reinterpret_cast<const float4*>(at + half + 4));
        w.c[4] = c1.x, w.c[5] = c1.y, w.c[6] = c1.z, w.c[7] = c1.w;
        w.s[4] = s1.x, w.s[5] = s1.y, w.s[6] = s1.z, w.s[7] = s1.w;
    }
}

// The lane's 8 values of a row, rotated (`on`: this row is).  Lane c of the 16 holds dimensions 8c .. 8c+7.  All
// 32 lanes call it (the half-split form exchanges values between lanes).
__device__ __forceinline__ uint4 rotate_chunk(uint4 x, int c, const Turn& w, int rot, bool interleaved, bool on)
{
    const int nc = rot >> 3, hc = rot >> 4;   // rotated chunks, chunks of one half
    uint4 o = x;
    if (!interleaved) {
        const int partner = c < hc ? c + hc : (c < nc ? c - hc : c);
        const int src = (threadIdx.x & 16) | partner;
        o.x = __shfl_sync(kAll, x.x, src);
        o.y = __shfl_sync(kAll, x.y, src);
        o.z = __shfl_sync(kAll, x.z, src);
        o.w = __shfl_sync(kAll, x.w, src);
    }
    if (c >= nc || !on) return x;
    const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
    const uint32_t os[4] = {o.x, o.y, o.z, o.w};
    uint32_t r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float a = bf16_lo(xs[j]), b = bf16_hi(xs[j]);
        if (interleaved)
            r[j] = pack_bf16x2(turn(a, b, w.c[j], w.s[j], false), turn(b, a, w.c[j], w.s[j], true));
        else
            r[j] = pack_bf16x2(turn(a, bf16_lo(os[j]), w.c[2 * j], w.s[2 * j], c >= hc),
                               turn(b, bf16_hi(os[j]), w.c[2 * j + 1], w.s[2 * j + 1], c >= hc));
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// fp32 values to the nearest f16 and back.
__device__ __forceinline__ float2 snap(float x, float y) { return __half22float2(__floats2half2_rn(x, y)); }

// The codes (8 of them, 4 bytes) and the scale byte of the lane's half of a block of 16 values; the two lanes
// of a block agree on the scale.  All 32 lanes call it.
//
// Both quotients, max|y| / 6 and y / scale, are products with a rounded reciprocal: off by less than 2^-22 of
// themselves.  Their borders fall as in exact arithmetic all the same.  y is m 2^a with m < 256, an e4m3 border
// times 6 is 3 odd 2^b with odd < 32, an e2m1 border times the scale is c n 2^b with c n <= 300: a quotient that
// is not a border exactly is at least 1/300 of itself away from it.  Rounding to f16 (2^-11 of the value) puts
// the product of one that is a border exactly on it -- the borders are f16 values -- and moves no other across.
__device__ __forceinline__ uint32_t quantize_chunk(uint4 x, float inv, uint32_t& scale_byte)
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t top = 0;   // largest magnitude as bits (ordered like the magnitudes; NaN above infinity)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        top = max(top, (w[j] & 0x7fffu) << 16);
        top = max(top, w[j] & 0x7fff0000u);
    }
    top = max(top, __shfl_xor_sync(kAll, top, 1));
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

// 16 lanes take R rows (K heads, V heads, then query heads) of one token: their loads need neither the token's
// place nor its position and go out first, and the rows share its cosines and sines.
template <bool E2M1, int R>
__global__ void __launch_bounds__(kThreadsRows) paged_append_kernel(const PagedAppendParams p)
{
    griddep_wait();
    griddep_launch();
    const int per = 2 * p.c.Hkv + p.Hq;                            // rows of one token
    const unsigned groups = (per + R - 1) / R;
    const unsigned u = blockIdx.x * (unsigned)kCopyRows + (threadIdx.x >> 4);
    const int c = threadIdx.x & 15;
    const int i = (int)(u / groups);
    const int j0 = (int)(u - i * groups) * R;
    bool live = i < p.n;
    uint4 x[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int j = j0 + r;
        x[r] = make_uint4(0, 0, 0, 0);
        if (live && j < per) {
            const uint16_t* src = j >= 2 * p.c.Hkv ? p.q + i * p.q_n + (j - 2 * p.c.Hkv) * p.q_h
                                                   : (j >= p.c.Hkv ? p.v + i * p.n_stride + (j - p.c.Hkv) * p.h_stride
                                                                   : p.k + i * p.n_stride + j * p.h_stride);
            x[r] = *reinterpret_cast<const uint4*>(src + 8 * c);   // q_out may be q: not a read-only load
        }
    }
    int seq = -1, pos = 0;
    if (live) {
        seq = __ldg(p.seq + i);
        pos = __ldg(p.pos + i);
        const int t = p.rope_pos ? __ldg(p.rope_pos + i) : pos;
        unsigned bad = 0;
        if (seq < 0 || seq >= p.c.B)
            bad = seq == -1 ? 0u : FX_DEVERR_INDEX;
        else if (pos < 0 || pos >= p.c.cap)
            bad = FX_DEVERR_LEN;
        else if (p.rot > 0 && (t < 0 || t >= p.n_pos))
            bad = FX_DEVERR_INDEX;
        live = seq >= 0 && bad == 0;
        if (bad && j0 == 0 && c == 0) atomicOr(p.err, bad);
    }
    int page = -1;
    if (live && j0 < 2 * p.c.Hkv) page = paged_page(p.c, seq, pos, p.err);
    if (p.rot > 0) {
        Turn w = {};
        const bool turned = live && c < (p.rot >> 3);
        if (turned) load_turn(w, p.cos_sin + (int64_t)(p.rope_pos ? __ldg(p.rope_pos + i) : pos) * p.rot, c, p.rot, p.interleaved != 0);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int j = j0 + r;
            const bool is_v = j >= p.c.Hkv && j < 2 * p.c.Hkv;
            x[r] = rotate_chunk(x[r], c, w, p.rot, p.interleaved != 0, turned && !is_v);
        }
    }
    const int64_t row = pos & p.c.page_mask;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int j = j0 + r;
        const bool is_v = j >= p.c.Hkv;
        const bool keep = page >= 0 && j < 2 * p.c.Hkv;   // a K or V row with a place in the pool
        if (live && j >= 2 * p.c.Hkv && j < per)
            *reinterpret_cast<uint4*>(p.q_out + i * p.qo_n + (j - 2 * p.c.Hkv) * p.qo_h + 8 * c) = x[r];
        const int h = is_v ? j - p.c.Hkv : j;
        char* dst = (is_v ? p.c.v : p.c.k) + (int64_t)page * p.c.sp + h * p.c.sh + row * p.c.st;
        if (E2M1) {
            if (!__any_sync(kAll, keep)) continue;
            uint32_t sb;
            const uint32_t codes = quantize_chunk(x[r], is_v ? p.c.v_inv : p.c.k_inv, sb);
            if (keep) {
                *reinterpret_cast<uint32_t*>(dst + 4 * c) = codes;
                char* sd = (is_v ? p.c.vs : p.c.ks) + (int64_t)page * p.c.ssp + h * p.c.ssh + row * p.c.sst;
                if ((c & 1) == 0) sd[c >> 1] = (char)sb;
            }
        } else if (keep) {
            *reinterpret_cast<uint4*>(dst + 16 * c) = x[r];
        }
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

template <bool E2M1>
cudaError_t append(const PagedAppendParams& p, bool pdl, cudaStream_t s)
{
    // A decode step's few rows: one row each, for the shortest way through.  More than two rounds of the
    // machine's 16-lane groups: four rows each, for their shared cosines and more loads in flight.
    const int per = 2 * p.c.Hkv + p.Hq;
    const bool many = (int64_t)p.n * per > 2 * 152 * 2048 / 16;
    const int64_t groups = (int64_t)p.n * (many ? (per + 3) / 4 : per);
    const dim3 grid((unsigned)((groups + kCopyRows - 1) / kCopyRows));
    return many ? launch_kernel(paged_append_kernel<E2M1, 4>, grid, dim3(kThreadsRows), 0, s, pdl, 0u, p)
                : launch_kernel(paged_append_kernel<E2M1, 1>, grid, dim3(kThreadsRows), 0, s, pdl, 0u, p);
}

template <bool E2M1>
cudaError_t gather(const PagedGatherParams& p, bool pdl, cudaStream_t s)
{
    const bool many = (int64_t)p.n * p.c.Hkv * p.c.B > 2 * 152 * 2048 / 16;
    const int rows = kCopyRows * (many ? 4 : 1);
    const dim3 grid((p.n + rows - 1) / rows, p.c.Hkv, p.c.B);
    return many ? launch_kernel(paged_gather_kernel<E2M1, 4>, grid, dim3(kThreadsRows), 0, s, pdl, 0u, p)
                : launch_kernel(paged_gather_kernel<E2M1, 1>, grid, dim3(kThreadsRows), 0, s, pdl, 0u, p);
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendParams& p, bool e2m1, bool pdl, cudaStream_t s)
{
    return e2m1 ? append<true>(p, pdl, s) : append<false>(p, pdl, s);
}

cudaError_t launch_paged_gather(const PagedGatherParams& p, bool e2m1, bool pdl, cudaStream_t s)
{
    return e2m1 ? gather<true>(p, pdl, s) : gather<false>(p, pdl, s);
}

}  // namespace fx
