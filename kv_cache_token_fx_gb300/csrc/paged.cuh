// Paged KV cache: what the kernels of paged_rows.cu and paged_attn.cu share -- row addresses through the
// page table and the 4-bit (e2m1 codes, e4m3 block scales) conversions.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "fx_internal.h"

namespace fx {
namespace {

// The four bytes of a word of codes, each (low half = first value) to a pair of f16 values, exact.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3)
{
    asm("{\n\t.reg .b8 c0, c1, c2, c3;\n\tmov.b32 {c0, c1, c2, c3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, c0;\n\tcvt.rn.f16x2.e2m1x2 %1, c1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c2;\n\tcvt.rn.f16x2.e2m1x2 %3, c3;\n\t}"
        : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
        : "r"(w));
}
// Byte k (a constant) of a word of codes to a pair of f16 values.
__device__ __forceinline__ uint32_t e2m1x2_to_f16(uint32_t w, int k)
{
    uint32_t r;
    switch (k) {
    case 0: asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(r) : "r"(w)); break;
    case 1: asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(r) : "r"(w)); break;
    case 2: asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}" : "=r"(r) : "r"(w)); break;
    default: asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, d;\n\t}" : "=r"(r) : "r"(w)); break;
    }
    return r;
}
// Two e4m3 bytes to two f16 values, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two)
{
    uint32_t r;
    asm("{\n\t.reg .b16 c;\n\tcvt.u16.u32 c, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}" : "=r"(r) : "r"(two));
    return r;
}
// Two fp32 values to two e2m1 codes (first value in the low half), nearest, ties to the even code, at most 6.
__device__ __forceinline__ uint32_t e2m1x2_from_f32(float first, float second)
{
    uint32_t r;
    asm("{\n\t.reg .b8 c;\n\tcvt.rn.satfinite.e2m1x2.f32 c, %2, %1;\n\tcvt.u32.u8 %0, c;\n\t}"
        : "=r"(r)
        : "f"(first), "f"(second));
    return r;
}
// fp32 to an e4m3 byte, nearest even, at most 448.
__device__ __forceinline__ uint32_t e4m3_from_f32(float x)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
    return r;
}

__device__ __forceinline__ uint32_t hmul2_u32(uint32_t a, uint32_t b)
{
    const __half2 r = __hmul2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// Page number of row t of sequence b (0 <= t < cap), or -1 (flagged) for a bad table entry.
__device__ __forceinline__ int paged_page(const PagedCache& c, int b, int t, unsigned* err)
{
    const int pg = c.table[(int64_t)b * c.table_stride + (t >> c.page_shift)];
    if (pg < 0 || pg >= c.n_pages) {
        atomicOr(err, FX_DEVERR_PAGE);
        return -1;
    }
    return pg;
}

}  // namespace
}  // namespace fx
