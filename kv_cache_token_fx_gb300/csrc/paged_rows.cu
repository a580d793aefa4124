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

// The lane's 8 values of a row, rotated.  Lane c of the 16 holds dimensions 8c .. 8c+7; `cs` is the position's
// row of cosines and sines.  All 32 lanes call it (the half-split form exchanges values between lanes).
__device__ __forceinline__ uint4 rotate_chunk(uint4 x, int c, const float* cs, int rot, bool interleaved)
{
    const int half = rot >> 1;
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
    if (c >= nc || cs == nullptr) return x;
    const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
    const uint32_t os[4] = {o.x, o.y, o.z, o.w};
    uint32_t r[4];
    if (interleaved) {
        const float4 co = *reinterpret_cast<const float4*>(cs + 4 * c);
        const float4 si = *reinterpret_cast<const float4*>(cs + half + 4 * c);
        const float cv[4] = {co.x, co.y, co.z, co.w}, sv[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float a = bf16_lo(xs[j]), b = bf16_hi(xs[j]);
            r[j] = pack_bf16x2(turn(a, b, cv[j], sv[j], false), turn(b, a, cv[j], sv[j], true));
        }
    } else {
        const bool second = c >= hc;
        const float* at = cs + 8 * (second ? c - hc : c);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float4 co = *reinterpret_cast<const float4*>(at + 4 * j);
            const float4 si = *reinterpret_cast<const float4*>(at + half + 4 * j);
            r[2 * j] = pack_bf16x2(turn(bf16_lo(xs[2 * j]), bf16_lo(os[2 * j]), co.x, si.x, second),
                                   turn(bf16_hi(xs[2 * j]), bf16_hi(os[2 * j]), co.y, si.y, second));
            r[2 * j + 1] = pack_bf16x2(turn(bf16_lo(xs[2 * j + 1]), bf16_lo(os[2 * j + 1]), co.z, si.z, second),
                                       turn(bf16_hi(xs[2 * j + 1]), bf16_hi(os[2 * j + 1]), co.w, si.w, second));
        }
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// The codes (8 of them, 4 bytes) and the scale byte of the lane's half of a block of 16 values; the two lanes
// of a block agree on the scale.  All 32 lanes call it.
//
// scale = e4m3(max|y|/6): the quotient is correctly rounded, and a value with 8 significant bits over 6 is
// either an e4m3 border exactly or at least 2^-9 of itself away from one, so the border falls as in exact
// arithmetic.  code = e2m1(y/scale) likewise: y has 8 significant bits, the scale 4, so y/scale is a border
// exactly or at least 2^-10 of itself away, far more than the quotient's rounding.
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
    const float a = __fdiv_rn(__uint_as_float(top) * inv, 6.f);
    scale_byte = e4m3_from_f32(fmaxf(a, 0.001953125f));   // at least 2^-9, the smallest e4m3 value
    const float s = __half2float(__ushort_as_half((unsigned short)(e4m3x2_to_f16x2(scale_byte) & 0xffffu)));
    uint32_t codes = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        codes |= e2m1x2_from_f32(__fdiv_rn(bf16_lo(w[j]) * inv, s), __fdiv_rn(bf16_hi(w[j]) * inv, s)) << (8 * j);
    if (!finite) {
        scale_byte = 0x7fu;
        codes = 0;
    }
    return codes;
}

template <bool E2M1>
__global__ void __launch_bounds__(kThreadsRows) paged_append_kernel(const PagedAppendParams p)
{
    griddep_wait();
    griddep_launch();
    const int per = 2 * p.c.Hkv + p.Hq;   // rows of one token: K, V, then q heads
    const int64_t u = (int64_t)blockIdx.x * kCopyRows + (threadIdx.x >> 4);
    const int c = threadIdx.x & 15;
    const int64_t i = u / per;
    const int j = (int)(u - i * per);
    bool live = i < p.n;
    const bool is_q = j >= 2 * p.c.Hkv, is_v = !is_q && j >= p.c.Hkv;
    const int h = is_q ? j - 2 * p.c.Hkv : (is_v ? j - p.c.Hkv : j);
    int seq = -1, pos = 0, page = 0;
    const float* cs = nullptr;
    if (live) {
        seq = p.seq[i];
        live = seq >= 0 && seq < p.c.B;
        if (!live && seq != -1 && j == 0 && c == 0) atomicOr(p.err, FX_DEVERR_INDEX);
    }
    if (live) {
        pos = p.pos[i];
        if (pos < 0 || pos >= p.c.cap) {
            live = false;
            if (j == 0 && c == 0) atomicOr(p.err, FX_DEVERR_LEN);
        }
    }
    if (live && p.rot > 0) {
        const int t = p.rope_pos ? p.rope_pos[i] : pos;
        if (t < 0 || t >= p.n_pos) {
            live = false;
            if (j == 0 && c == 0) atomicOr(p.err, FX_DEVERR_INDEX);
        } else if (!is_v) {
            cs = p.cos_sin + (int64_t)t * p.rot;
        }
    }
    if (live && !is_q) {
        page = paged_page(p.c, seq, pos, p.err);
        live = page >= 0;
    }
    uint4 x = make_uint4(0, 0, 0, 0);
    if (live) {
        const uint16_t* src = is_q ? p.q + i * p.q_n + h * p.q_h : (is_v ? p.v : p.k) + i * p.n_stride + h * p.h_stride;
        x = *reinterpret_cast<const uint4*>(src + 8 * c);
    }
    if (p.rot > 0) x = rotate_chunk(x, c, cs, p.rot, p.interleaved != 0);
    if (is_q && live) *reinterpret_cast<uint4*>(p.q_out + i * p.qo_n + h * p.qo_h + 8 * c) = x;
    const int64_t row = pos & p.c.page_mask;
    char* dst = (is_v ? p.c.v : p.c.k) + (int64_t)page * p.c.sp + h * p.c.sh + row * p.c.st;
    if (E2M1) {
        uint32_t sb;
        const uint32_t codes = quantize_chunk(x, is_v ? p.c.v_inv : p.c.k_inv, sb);
        if (live && !is_q) {
            *reinterpret_cast<uint32_t*>(dst + 4 * c) = codes;
            char* sd = (is_v ? p.c.vs : p.c.ks) + (int64_t)page * p.c.ssp + h * p.c.ssh + row * p.c.sst;
            if ((c & 1) == 0) sd[c >> 1] = (char)sb;
        }
    } else if (live && !is_q) {
        *reinterpret_cast<uint4*>(dst + 16 * c) = x;
    }
}

template <bool E2M1>
__global__ void __launch_bounds__(kThreadsRows) paged_gather_kernel(const PagedGatherParams p)
{
    griddep_wait();
    griddep_launch();
    const int i = blockIdx.x * kCopyRows + (threadIdx.x >> 4);
    const int c = threadIdx.x & 15;
    const int h = blockIdx.y, b = blockIdx.z;
    if (i >= p.n) return;
    const int len = paged_len(p.c, b, p.err);
    const int64_t out_row = ((int64_t)b * p.c.Hkv + h) * p.n + i;
    int64_t t;
    if (p.idx) {
        t = p.idx[out_row];
        if (t < 0 || t >= len) {
            if (c == 0) atomicOr(p.err, FX_DEVERR_INDEX);
            return;
        }
    } else {
        int lo = p.lo ? p.lo[b] : 0;
        if (lo < 0) {
            if (c == 0) atomicOr(p.err, FX_DEVERR_LEN);
            lo = 0;
        }
        t = (int64_t)lo + i;
        if (t >= len) return;
    }
    const int page = paged_page(p.c, b, (int)t, p.err);
    if (page < 0) return;
    const int64_t row = t & p.c.page_mask;
    const int64_t at = (int64_t)page * p.c.sp + h * p.c.sh + row * p.c.st;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const char* src = (w ? p.c.v : p.c.k) + at;
        uint4 x;
        if (E2M1) {
            const uint32_t codes = *reinterpret_cast<const uint32_t*>(src + 4 * c);
            const char* ss = (w ? p.c.vs : p.c.ks) + (int64_t)page * p.c.ssp + h * p.c.ssh + row * p.c.sst;
            const uint32_t sb = (uint8_t)ss[c >> 1];
            const float s = __half2float(__ushort_as_half((unsigned short)(e4m3x2_to_f16x2(sb) & 0xffffu))) *
                            (w ? p.c.v_mul : p.c.k_mul);
            uint32_t f[4];
            e2m1x8_to_f16(codes, f[0], f[1], f[2], f[3]);
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 v = __half22float2(*reinterpret_cast<__half2*>(&f[j]));
                o[j] = pack_bf16x2(v.x * s, v.y * s);
            }
            x = make_uint4(o[0], o[1], o[2], o[3]);
        } else {
            x = *reinterpret_cast<const uint4*>(src + 16 * c);
        }
        *reinterpret_cast<uint4*>((w ? p.v_out : p.k_out) + out_row * kHeadDim + 8 * c) = x;
    }
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendParams& p, bool e2m1, bool pdl, cudaStream_t s)
{
    const int64_t rows = (int64_t)p.n * (2 * p.c.Hkv + p.Hq);
    const dim3 grid((unsigned)((rows + kCopyRows - 1) / kCopyRows));
    return e2m1 ? launch_kernel(paged_append_kernel<true>, grid, dim3(kThreadsRows), 0, s, pdl, 0u, p)
                : launch_kernel(paged_append_kernel<false>, grid, dim3(kThreadsRows), 0, s, pdl, 0u, p);
}

cudaError_t launch_paged_gather(const PagedGatherParams& p, bool e2m1, bool pdl, cudaStream_t s)
{
    const dim3 grid((p.n + kCopyRows - 1) / kCopyRows, p.c.Hkv, p.c.B);
    return e2m1 ? launch_kernel(paged_gather_kernel<true>, grid, dim3(kThreadsRows), 0, s, pdl, 0u, p)
                : launch_kernel(paged_gather_kernel<false>, grid, dim3(kThreadsRows), 0, s, pdl, 0u, p);
}

}  // namespace fx
