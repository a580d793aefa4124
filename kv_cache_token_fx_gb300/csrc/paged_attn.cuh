// Attention over a paged cache for sm_103a, bf16 or 4-bit: the kernels of fx_paged_decode and fx_paged_importance
// (paged_attn.cu), and of fx_paged_attend where a (sequence, KV head) has few query rows (paged_attn_shaped_*.cu).
//
// Work unit of a warp: a tile of 16 cache rows of one (sequence, KV head); two tiles at a time in 4 bits.  Every
// warp owns a ring of slots in shared memory and fills it with cp.async ahead of its work; no warp waits for
// another until their results meet.  S^T = K Q^T has the cache rows on M and the query rows on N (mma.sync
// m16n8k16), O^T += V^T P^T the dimensions on M and the cache rows on K.
//
// 4-bit rows: a lane's K fragments are 16 bytes of codes of two rows (the dimensions are permuted inside the
// product, the queries are laid out the same way), its V fragments 8 bytes of four rows (the dimensions of O^T
// are permuted inside M).  The codes become f16 by cvt.f16x2.e2m1x2, and one multiplication by the block's scale
// gives the value held, exactly (at most 6 significant bits, between 2^-10 and 2688).  The queries are f16
// scaled by a power of two per row (largest magnitude in [2^14, 2^15)), so no bit of a bf16 query within 2^-24
// of its row's largest is lost.  bf16 rows take bf16 queries as they are.  P enters as a sum of 16-bit parts, two
// f16 or three bf16: outputs are fp32, and one part would leave them 2^-12 (f16) or 2^-9 (bf16) off.
//
// Why mma.sync and not tcgen05: the codes must be unpacked by the threads in either case.  A version with 128-row tiles
// unpacked into swizzled shared memory, S^T and O^T by tcgen05.mma and one cache row to a thread gave the same outputs,
// but took 52 M warp instructions instead of 36 M for 64 x 3335 rows and 14 query rows (139 us against 94 then): the
// stores of the operands and of P cost more than the products it saves.  That was timed for 14 query rows of a decode and
// 32 of an importance.  At most 64 query rows share a cache row here; a decode of more than 16 takes a pass over the cache
// for every 16 (64 x 3335 4-bit rows: 16 query rows 79 us, 32 146, 64 280), where one unpacking might yet pay.
//
// Softmax: base-2 logits, one pass.  p = 2^(x - m) with a reference m per row that all lanes of the row share;
// it is set so that the largest logit so far gives 2^kBase and moves only when a p would exceed 2^kTop, so most
// tiles take one vote instead of a reduction; f16 holds such a p to 2^-36 of the row's largest.  Sums are fp32.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include <atomic>

#include "attn_ptx.cuh"
#include "paged.cuh"

namespace fx {
namespace {

constexpr int kTileRows = 16;
constexpr int kMinTiles = 2;    // tiles a warp gets at least, before more CTAs share a call (decode of one head's 1024 4-bit
                                // rows: 7.3 us with 1, 7.7 with 2, 8.6 with 4; of 8 x 4864 rows: 14.7, 14.4 and 14.7)
constexpr int kMaxParts = 128;  // CTAs that share one (sequence, KV head, row group) on average, at most: the last
                                // of them joins all their parts
// 4 bits, up to 8 query rows: tiles a warp may get at most for units of one tile instead of two (512 heads' 40 rows, a
// tile: 9.4 us against 11.6; 833 rows, 15 tiles: 23.3 against 22.3; 1667 rows, 29 tiles: 34.1 against 30.4; 128 heads'
// 32768 rows, 144 tiles: 105 against 84).  Pages of 16 rows hold no pair of neighbours: always one (64 heads' 4864 rows
// 14.4 us against 15.4, 38912 rows 76 against 74).
// The host knows no lengths: it counts the rows that the table has room for, and the list.  Where a table has far more room
// than its sequences use, short work runs in units of two: 64 heads' 1024 rows 9.9 us against 9.5, 4864 rows 13.9 both, 2048
// listed rows and a tail of 512 14.7 against 14.2.
constexpr int kShort = 16;
// What a piece costs a CTA besides its tiles -- its first rows and queries, its join: 5 to 10 us -- counted in tiles.
struct LineCost {
    int second;   // parts this much longer than an even share are better than a second piece for some CTAs
    int start;    // the start of a piece in a line
    int near;     // between a cut and an end of a piece, at least
};
// Decode, 4 bits (a tile of a CTA takes 0.2 us).  second: 8 x 4864 rows 14.4 us against 17.9 with 0; 16 x 32768 rows 84 us
// with 0, 32 or 48.  start: 64 sequences of up to 3335 rows, 14 query rows: 79 us against 84 with 16, 89 without; of up to 40
// rows: 17 us against 29 without.  near: those 3335 rows 78.7 us, 79.1 with 8, 81.8 with 32, 79.3 with 1.
// bf16 (a tile is 3.5 times the bytes): 64 sequences of up to 1000 rows, 14 query rows: 48 us against 53 with a start of 32
// and near of 16, 49 with 8 and 4; 1667 rows, 2 query rows: 51.8 us against 52.3 and 53.0.
__host__ __device__ constexpr LineCost decode_cost(bool e2m1) { return e2m1 ? LineCost{48, 32, 16} : LineCost{48, 16, 8}; }
// Importance has no join, so cuts may fall anywhere (64 x 2000 4-bit rows: 21.3 us against 22.3 with near = 16; bf16:
// 34.5 us against 35.4 with near = 16, 36.1 with a start of 32 as well).
__host__ __device__ constexpr LineCost importance_cost(bool e2m1) { return LineCost{32, e2m1 ? 32 : 8, 1}; }
static_assert(decode_cost(true).start <= kPieceStart && decode_cost(false).start <= kPieceStart &&
                  importance_cost(true).start <= kPieceStart && importance_cost(false).start <= kPieceStart,
              "lines are counted in 32 bits");
// p is at most 2^kTop (f16 holds up to 2^15.99); a new reference puts the largest logit at 2^kBase.
constexpr float kTop = 15.f;
constexpr float kBase = 11.f;
// bf16 rows: a weight is taken 2^-46 of that large (at most 2^-31, a change of its exponent alone), so that sums of up to
// 2^31 products with values up to bf16's largest stay finite, as their weighted mean is.  The price is at the other end:
// products below fp32's normal range lose bits, which values below some 2^-90 meet.  (4-bit values are at most 2688 here.)
template <bool E2M1>
constexpr float kWeightUnit = E2M1 ? 1.f : 1.f / (float)(1ull << 46);
// A reference further than this from 0 comes of logits that fp32 holds to 1/2 at best.  It is taken from the rounded
// product of a logit and its factor, an fma has the exact one, and what lies between them is then more than a weight has
// room for (the largest might come out as 0 or as 2^1000).  So the tiles that ask for such a reference take the rounded
// products as well, and weights of 2^kTop at most; later tiles come back here when theirs are larger.
constexpr float kFarRef = 4194304.f;   // 2^22
// Minus the reference of a row without one: any finite logit then asks for a reference, and a logit of -inf gives a
// weight of 0 (beside +inf it would give NaN).
constexpr float kNoRef = 3.402823466e38f;

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

// The same from zero.
template <bool E2M1>
__device__ __forceinline__ void mma16_zero(float d[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                           uint32_t b1)
{
    if (E2M1) {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %10, %10, %10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
    } else {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %10, %10, %10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
    }
}

__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;\n" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t a)
{
    uint32_t r;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(a));
    return r;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a)
{
    uint16_t r;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(r) : "r"(a));
    return r;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a)
{
    uint32_t r;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(a));
    return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
    return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t a)
{
    uint2 r;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a));
    return r;
}

// ---- rows of a sequence -----------------------------------------------------------------------------
struct Seq {
    const int32_t* idx;     // the list of (b, h)
    const int32_t* table;   // the pages of b
    int nl, lo, len;        // list tiles, start of the tail, rows
    // SHAPED: a sequence's rows are those that some of its queries see, [lo, len)
    int pos0, q0, nb;       // position of its first query, its place in q, the queries' number
    int com_lo, com_hi;     // rows that every query sees
    int rows;               // rows of the cache
};
// What query i of a sequence sees: rows x <= t < y, both within [0, rows] (any int may be given: arithmetic on these ends
// must not overflow).
__device__ __forceinline__ int2 shaped_interval(const PagedAttnParams& p, const Seq& q, int i)
{
    const int pos = q.pos0 + i;
    int2 see = make_int2(p.first ? min(max(p.first[q.q0 + i], 0), q.rows) : 0,
                         max(min(p.last ? p.last[q.q0 + i] : pos + 1, q.rows), 0));
    if (p.window > 0) see.x = max(see.x, pos - p.window + 1);
    return see;
}
__device__ __forceinline__ void shaped_sequence(const PagedAttnParams& p, int b, bool report, Seq& q)
{
    q.rows = p.c.len[b];
    if (report && (q.rows < 0 || q.rows > p.c.cap)) atomicOr(p.err, FX_DEVERR_LEN);
    q.rows = min(max(q.rows, 0), p.c.cap);
    int all = p.Mq;
    q.q0 = b * p.Mq;
    if (p.start) {
        q.q0 = p.start[b];
        const int q1 = p.start[b + 1];
        all = q1 - q.q0;
        if (q.q0 < 0 || q1 < q.q0 || q1 > p.n) {
            q.q0 = all = 0;
            if (report) atomicOr(p.err, FX_DEVERR_OFFSETS);
        } else if (all > p.Mq && report) {
            atomicOr(p.err, FX_DEVERR_OFFSETS);
        }
    }
    q.nb = min(all, p.Mq);
    q.pos0 = q.rows - all;
    q.lo = 0x7fffffff;
    q.len = 0;
    q.com_lo = 0;
    q.com_hi = 0x7fffffff;
    if (!p.first && !p.last && q.nb > 0) {   // the ends grow by one from query to query
        const int lo = p.window > 0 ? p.window - 1 : 0x3fffffff, end = q.pos0 + q.nb;   // (end = rows, or max_new of them)
        q.com_hi = q.pos0 + 1;
        q.len = max(end, 0);
        q.lo = max(max(q.pos0, 0) - lo, 0);
        q.com_lo = max(end - 1 - lo, 0);
    } else for (int i = 0; i < q.nb; ++i) {
        const int2 see = shaped_interval(p, q, i);
        q.com_lo = max(q.com_lo, see.x);
        q.com_hi = min(q.com_hi, see.y);
        if (see.x < see.y) {
            q.lo = min(q.lo, see.x);
            q.len = max(q.len, see.y);
        }
    }
    q.lo = min(q.lo, q.len);
    q.nl = 0;
    q.table = p.c.table + (int64_t)b * p.c.table_stride;
    q.idx = nullptr;
}
// Tiles of sequence b (at least one: an empty sequence's tile holds no valid row, and its output is written).
template <int SHAPED>
__device__ __forceinline__ Seq sequence(const PagedAttnParams& p, int b, bool report)
{
    Seq q;
    if (SHAPED) {
        shaped_sequence(p, b, report, q);
        return q;
    }
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


__device__ __forceinline__ int64_t row_offset(const PagedCache& c, int id, uint32_t sp, uint32_t st)
{
    return (uint64_t)(uint32_t)(id >> c.page_shift) * sp + (uint64_t)(uint32_t)(id & c.page_mask) * st;
}

// ---- slots in shared memory ---------------------------------------------------------------------------
// A slot holds a unit of U tiles.  4-bit: K codes (rows of 64 bytes), V codes, K scales (rows of 8 bytes), V
// scales; of bf16: K rows (256 bytes), V rows; then the rows' positions (-1: not valid), present only for tiles
// with an edge.  The importance takes K alone.
// Codes: two rows share a 128-byte line, whose eight 16-byte chunks are permuted by chunk ^ 2 (line % 4), so
// that neither the 16-byte reads of K (8 rows side by side) nor the 8-byte reads of V (rows 2t, the halves g of
// them) meet in a bank.  bf16 rows are permuted as kv_off() has it.
template <bool E2M1, bool WITH_V, int U>
struct Slot {
    static constexpr int kTile = E2M1 ? 1024 : 4096;     // K (or V) of one tile
    static constexpr int kV = U * kTile;
    static constexpr int kScale = (WITH_V ? 2 : 1) * U * kTile;
    static constexpr int kScaleV = kScale + U * 128;
    static constexpr int kPos = kScale + (E2M1 ? (WITH_V ? 2 : 1) * U * 128 : 0);
    static constexpr int kBytes = kPos + U * 64;
};

// Fills slots with the tiles [it, end) of a sequence in order.  The first nl tiles hold the list, the others the
// tail, whose tiles start at multiples of 16, so that such a tile lies inside one page; the tail's pairs start
// at multiples of 32.  All lanes call it.
//
// Tail: the lanes hold the next 32 page numbers, and inside a page the lane's addresses only advance; a pair of
// whole tiles of one page is ten copies and a few additions.  List: the lanes hold the rows of two tiles (lane
// L: entry L of them), looked up a batch ahead, their positions another batch ahead.
template <bool E2M1, bool WITH_V, int U, int SHAPED = 0>
struct Feeder {
    using S = Slot<E2M1, WITH_V, U>;
    const PagedAttnParams& p;
    const Seq& q;
    const char* k0;   // the lane's places relative to row 0 of page 0: K codes or rows, K scales (V and its scales
    const char* s0;   // lie c.v - c.k and c.vs - c.ks further on: their strides are K's)
    uint32_t to;      // the lane's place in a tile (codes or rows)
    int it, end;
    int plain0, plain1;   // tail tiles whose rows all count for every query, in pages without gaps between rows
    int clear0, clear;   // rows [clear0, clear) are seen by every query
    // tail
    int pos;          // first row of the next tail tile
    int pages, page_base;
    bool enter, ok;   // it starts a page (or the feeder); its page is good
    const char* ka;   // the lane's K place of that row (scales: of the lane-th row from it on)
    const char* sa;
    // list
    int id, at;       // the lane's pool row (-1: not valid) and position in the current two tiles
    int at1, page1, at2;
    int parity = 0;   // 16: the second of the two tiles is next

    __device__ __forceinline__ Feeder(const PagedAttnParams& p_, const Seq& q_, int h, int it_, int end_)
        : p(p_), q(q_), it(it_), end(end_), clear0(SHAPED ? q_.com_lo : q_.lo), clear(SHAPED ? q_.com_hi : q_.len - p_.Mq + 1)
    {
        const PagedCache& c = p.c;
        const int lane = threadIdx.x & 31;
        const int chunk = E2M1 ? lane & 3 : lane & 15, row = E2M1 ? lane >> 2 : lane >> 4;
        k0 = c.k + (int64_t)h * c.sh + row * (int64_t)c.st + 16 * chunk;
        s0 = c.ks + (int64_t)h * c.ssh + lane * (int64_t)c.sst;
        to = E2M1 ? (row >> 1) * 128 + ((((row & 1) * 4 + chunk) ^ (2 * ((row >> 1) & 3))) << 4)
                  : row * 256 + ((chunk ^ row) << 4);
        if (it < q.nl && it < end) {
            at = list_pos(it * kTileRows + lane);
            at1 = list_pos((it + 2) * kTileRows + lane);
            const int page = list_page(at, it * kTileRows + lane);
            page1 = list_page(at1, (it + 2) * kTileRows + lane);
            at2 = list_pos((it + 4) * kTileRows + lane);
            id = place(at, page);
        }
        const int tail0 = q.lo & ~(kTileRows - 1);
        pos = tail0 + (max(it, q.nl) - q.nl) * kTileRows;
        plain0 = q.nl + (SHAPED ? max(clear0 - tail0 + kTileRows - 1, 0) / kTileRows : (tail0 < q.lo ? 1 : 0));
        plain1 = c.st == (E2M1 ? 64 : 256) && (!E2M1 || c.sst == 8) ? min(end, q.nl + max(clear - tail0, 0) / kTileRows) : 0;
        ok = false;
        ka = k0;
        sa = s0;
        enter = true;
        if (end > q.nl) load_pages();
    }

    __device__ __forceinline__ int list_pos(int e) const { return e < min(p.kk, end * kTileRows) ? q.idx[e] : -1; }
    __device__ __forceinline__ int list_page(int& t, int e) const
    {
        if ((unsigned)t >= (unsigned)q.len) {
            if (e < min(p.kk, end * kTileRows)) atomicOr(p.err, FX_DEVERR_INDEX);
            t = -1;
        }
        return t >= 0 ? q.table[t >> p.c.page_shift] : 0;
    }
    __device__ __forceinline__ int place(int t, int page) const
    {
        if (t < 0) return -1;
        if ((unsigned)page >= (unsigned)p.c.n_pages) {
            atomicOr(p.err, FX_DEVERR_PAGE);
            return -1;
        }
        return (page << p.c.page_shift) | (t & p.c.page_mask);
    }
    __device__ __forceinline__ void load_pages()
    {
        page_base = pos >> p.c.page_shift;
        const int64_t first = (int64_t)(page_base + (int)(threadIdx.x & 31)) << p.c.page_shift;
        pages = first < q.len ? q.table[page_base + (threadIdx.x & 31)] : -1;
    }
    __device__ __forceinline__ bool enter_page()
    {
        const PagedCache& c = p.c;
        if ((pos >> c.page_shift) - page_base >= 32) load_pages();
        const int page = __shfl_sync(kFull, pages, (pos >> c.page_shift) - page_base);
        ok = (unsigned)page < (unsigned)c.n_pages;
        if (!ok && pos < q.len) atomicOr(p.err, FX_DEVERR_PAGE);
        const int pg = ok ? page : 0, row = pos & c.page_mask;
        ka = k0 + (uint64_t)(uint32_t)pg * c.sp + (uint64_t)(uint32_t)row * c.st;
        if (E2M1) sa = s0 + (uint64_t)(uint32_t)pg * c.ssp + (uint64_t)(uint32_t)row * c.sst;
        enter = false;
        return true;
    }
    // Feeds the next unit.  Bit U - 1 - u of the result: tile u has a row that is not valid or not seen by every
    // query (or there is no tile u); bit U: there is a tile at all.
    __device__ __forceinline__ uint32_t feed(uint32_t slot)
    {
        const PagedCache& c = p.c;
        uint32_t flags = 0;
        if (E2M1 && U == 2 && it >= plain0 && it + 2 <= plain1 && (pos & c.page_mask) + 32 <= c.page_mask + 1 &&
            (!enter || enter_page()) && ok) {
            feed_pair(slot);
            advance(2);
            flags = 1u << U;
        } else {
#pragma unroll 1
            for (int u = 0; u < U; ++u) {
                bool edge = true;
                if (it >= end || (u > 0 && it >= q.nl && (pos & kTileRows) == 0)) {
                    put_pos(slot, u, -1);
                } else {
                    flags |= 1u << U;
                    if (it < q.nl) {
                        edge = feed_list(slot, u);
                        ++it;
                    } else {
                        if (enter) enter_page();
                        edge = feed_tail(slot, u);
                        advance(1);
                    }
                }
                if (edge) flags |= 1u << (U - 1 - u);
            }
        }
        cp_async_commit();
        return flags;
    }
    __device__ __forceinline__ void advance(int n)
    {
        it += n;
        pos += n * kTileRows;
        ka += (uint64_t)(uint32_t)(n * kTileRows) * p.c.st;
        if (E2M1) sa += (uint64_t)(uint32_t)(n * kTileRows) * p.c.sst;
        enter = (pos & p.c.page_mask) == 0;
    }

    __device__ __forceinline__ void feed_pair(uint32_t slot)
    {
        const PagedCache& c = p.c;
        const uint32_t dst = slot + to, sdst = slot + S::kScale + 8 * (threadIdx.x & 31);
        const char* va = ka + (c.v - c.k);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            cp_async16(dst + 512 * u, ka + 512 * u);
            if (WITH_V) cp_async16(dst + S::kV + 512 * u, va + 512 * u);
        }
        cp_async8(sdst, sa);
        if (WITH_V) cp_async8(sdst + U * 128, sa + (c.vs - c.ks));
    }

    __device__ __forceinline__ void put_pos(uint32_t slot, int u, int t)
    {
        const int lane = threadIdx.x & 31;
        if (lane < 16) asm volatile("st.shared.s32 [%0], %1;" ::"r"(slot + S::kPos + 64 * u + 4 * lane), "r"(t) : "memory");
    }

    __device__ __forceinline__ bool feed_tail(uint32_t slot, int u)
    {
        const PagedCache& c = p.c;
        const int lane = threadIdx.x & 31, j = lane & 15;
        const bool edge = !ok || pos < clear0 || pos + kTileRows > clear;
        if (edge) {
            const int t = pos + j;
            put_pos(slot, u, ok && t >= q.lo && t < q.len ? t : -1);
        }
        const int64_t dv = c.v - c.k;
        if (E2M1) {
            const uint32_t dst = slot + to + u * S::kTile;
            const char* kb = ka + 8 * (int64_t)c.st;
            cp_async16(dst, ka);
            cp_async16(dst + 512, kb);
            if (WITH_V) {
                cp_async16(dst + S::kV, ka + dv);
                cp_async16(dst + S::kV + 512, kb + dv);
            }
            if (lane < 16)
                cp_async8(slot + S::kScale + u * 128 + 8 * lane, sa);
            else if (WITH_V)
                cp_async8(slot + S::kScaleV + u * 128 + 8 * j, sa + (c.vs - c.ks) - 16 * (int64_t)c.sst);
        } else {
#pragma unroll
            for (int w = 0; w < 8; ++w) {
                const uint32_t d = slot + u * S::kTile + w * 512 + (to ^ ((2 * w & 6) << 4));
                const char* from = ka + 2 * w * (int64_t)c.st;
                cp_async16(d, from);
                if (WITH_V) cp_async16(d + S::kV, from + dv);
            }
        }
        return edge;
    }

    __device__ __forceinline__ bool feed_list(uint32_t slot, int u)
    {
        const PagedCache& c = p.c;
        const int lane = threadIdx.x & 31, j = lane & 15;
        const int half = parity;
        const int mine = __shfl_sync(kFull, id, half + j), t = __shfl_sync(kFull, at, half + j);
        const bool edge = __any_sync(kFull, mine < 0 || t >= clear);
        if (edge) put_pos(slot, u, mine >= 0 ? t : -1);
        constexpr int kCopies = E2M1 ? 2 : 8;   // rows of K (and V) that a lane copies 16 bytes of
        const int lane_row = E2M1 ? lane >> 2 : lane >> 4;
        const char* base = k0 - lane_row * (int64_t)c.st;
#pragma unroll
        for (int w = 0; w < kCopies; ++w) {
            const int row = max(__shfl_sync(kFull, id, half + (E2M1 ? lane_row + 8 * w : lane_row + 2 * w)), 0);
            const char* from = base + row_offset(c, row, c.sp, c.st);
            const uint32_t dst = slot + u * S::kTile + 512 * w + (E2M1 ? to : to ^ ((2 * w & 6) << 4));
            cp_async16(dst, from);
            if (WITH_V) cp_async16(dst + S::kV, from + (c.v - c.k));
        }
        if (E2M1 && (WITH_V || lane < 16)) {
            const char* from = s0 - lane * (int64_t)c.sst + row_offset(c, max(mine, 0), c.ssp, c.sst);
            cp_async8(slot + (lane < 16 ? S::kScale : S::kScaleV) + u * 128 + 8 * j, lane < 16 ? from : from + (c.vs - c.ks));
        }
        parity ^= 16;
        if (parity == 0) {   // the next two tiles
            at = at1;
            id = place(at, page1);
            at1 = at2;
            page1 = list_page(at1, (it + 3) * kTileRows + lane);
            at2 = list_pos((it + 5) * kTileRows + lane);
        }
        return edge;
    }
};

// A tile's K rows: pair(j) gives the A fragments of the 16-dimension steps 2j and 2j + 1 of S^T = K Q^T.
template <bool E2M1>
struct KTile;
template <>
struct KTile<true> {
    uint32_t w[2][4];    // 32 dimensions from 32t on of rows g and g + 8
    uint32_t sc[2][2];   // [row][block of 16 of them]: the scale, twice

    template <typename S>
    __device__ __forceinline__ void load(uint32_t slot, int u)
    {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        const uint32_t at = slot + u * S::kTile + (g >> 1) * 128 + ((((g & 1) * 4 + t) ^ (2 * ((g >> 1) & 3))) << 4);
        const uint32_t sa = slot + S::kScale + u * 128 + 8 * g + 2 * t;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const uint4 x = lds128(at + 512 * r);
            w[r][0] = x.x, w[r][1] = x.y, w[r][2] = x.z, w[r][3] = x.w;
            const uint32_t z = e4m3x2_to_f16x2(lds16(sa + 64 * r));
            sc[r][0] = __byte_perm(z, 0, 0x1010);
            sc[r][1] = __byte_perm(z, 0, 0x3232);
        }
    }
    __device__ __forceinline__ void pair(int j, uint32_t (&x)[2][4]) const
    {
        uint32_t a[4], b[4];
        e2m1x8_to_f16(w[0][j], a[0], a[1], a[2], a[3]);
        e2m1x8_to_f16(w[1][j], b[0], b[1], b[2], b[3]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i >> 1][2 * (i & 1)] = hmul2_u32(a[i], sc[0][j >> 1]);
            x[i >> 1][2 * (i & 1) + 1] = hmul2_u32(b[i], sc[1][j >> 1]);
        }
    }
};
template <>
struct KTile<false> {
    uint32_t at;

    template <typename S>
    __device__ __forceinline__ void load(uint32_t slot, int u) { at = slot + u * S::kTile; }
    __device__ __forceinline__ void pair(int j, uint32_t (&x)[2][4]) const
    {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            ldsm_x4(at + kv_off(lane & 15, 2 * (2 * j + i) + (lane >> 4)), x[i][0], x[i][1], x[i][2], x[i][3]);
    }
};

// A tile's V rows: get(i) gives the A fragment of M tile i of O^T += V^T P^T.  MASKED: rows outside `vm` count as
// zero, whatever they hold.
template <bool E2M1>
struct VTile;
template <>
struct VTile<true> {
    uint32_t code[2][4];   // [dimensions 16g .. + 7, + 8 .. + 15][rows 2t, 2t + 1: even, odd dimensions; 2t + 8, + 9]
    uint32_t s01, s23;     // scales of rows 2t, 2t + 1 and 2t + 8, 2t + 9

    template <bool MASKED, typename S>
    __device__ __forceinline__ void load(uint32_t slot, int tile, uint32_t vm)
    {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        const uint32_t sa = slot + S::kScaleV + tile * 128 + 16 * t + g;
        uint32_t vs01 = lds8(sa) | (lds8(sa + 8) << 8), vs23 = lds8(sa + 64) | (lds8(sa + 72) << 8);
        if (MASKED) {
            const uint32_t on = vm >> (2 * t);   // bits 0, 1, 8, 9
            vs01 &= (on & 1u ? 0xffu : 0u) | (on & 2u ? 0xff00u : 0u);
            vs23 &= (on & 0x100u ? 0xffu : 0u) | (on & 0x200u ? 0xff00u : 0u);
        }
        s01 = e4m3x2_to_f16x2(vs01);
        s23 = e4m3x2_to_f16x2(vs23);
        const uint32_t in = t * 128 + (((g >> 1) ^ (2 * t)) << 4) + (g & 1) * 8;
        const uint32_t va = slot + S::kV + tile * S::kTile + in, vb = slot + S::kV + tile * S::kTile + (in ^ 64u);
        const uint2 x[4] = {lds64(va), lds64(vb), lds64(va + 512), lds64(vb + 512)};
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                // neighbouring rows' codes of one dimension side by side, so that one conversion takes the pair
                const uint32_t x0 = j ? x[2 * u].y : x[2 * u].x, x1 = j ? x[2 * u + 1].y : x[2 * u + 1].x;
                code[j][2 * u] = (x0 & 0x0f0f0f0fu) | ((x1 << 4) & 0xf0f0f0f0u);
                code[j][2 * u + 1] = ((x0 >> 4) & 0x0f0f0f0fu) | (x1 & 0xf0f0f0f0u);
            }
    }
    template <bool MASKED>
    __device__ __forceinline__ void get(int i, uint32_t (&x)[4])
    {
#pragma unroll
        for (int u = 0; u < 4; ++u) x[u] = hmul2_u32(e2m1x2_to_f16(code[i >> 2][u], i & 3), u < 2 ? s01 : s23);
    }
};
template <>
struct VTile<false> {
    uint32_t at;
    uint32_t m01, m23;

    template <bool MASKED, typename S>
    __device__ __forceinline__ void load(uint32_t slot, int tile, uint32_t vm)
    {
        at = slot + S::kV + tile * S::kTile;
        if (MASKED) {
            const uint32_t on = vm >> (2 * (threadIdx.x & 3));   // bits 0, 1, 8, 9: rows 2t, 2t + 1, 2t + 8, 2t + 9
            m01 = (on & 1u ? 0xffffu : 0u) | (on & 2u ? 0xffff0000u : 0u);
            m23 = (on & 0x100u ? 0xffffu : 0u) | (on & 0x200u ? 0xffff0000u : 0u);
        }
    }
    template <bool MASKED>
    __device__ __forceinline__ void get(int i, uint32_t (&x)[4])
    {
        const int lane = threadIdx.x & 31;
        ldsm_x4_t(at + kv_off((lane & 7) + 8 * (lane >> 4), 2 * i + ((lane >> 3) & 1)), x[0], x[1], x[2], x[3]);
        if (MASKED) {
            x[0] &= m01;
            x[1] &= m01;
            x[2] &= m23;
            x[3] &= m23;
        }
    }
};
// The two dimensions that rows g and g + 8 of M tile i hold.
template <bool E2M1>
__device__ __forceinline__ int v_dim(int i, int g, int half)
{
    return E2M1 ? 16 * g + 2 * i + half : 16 * i + g + 8 * half;
}

// The lane's 32 query values of row g as they lie in memory, in the order of the eight steps' B fragments.
// src: the row, or nullptr for a row that does not exist.
template <bool E2M1>
__device__ __forceinline__ void fetch_query(const uint16_t* src, uint32_t (&w)[16])
{
    const int t = threadIdx.x & 3;
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j] = 0;
    if (src) {
        if (E2M1) {   // step j: dimensions 32t + 4j .. + 3, as a lane's 16 bytes of codes have them
#pragma unroll
            for (int j = 0; j < 4; ++j)
                asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(w[4 * j]), "=r"(w[4 * j + 1]), "=r"(w[4 * j + 2]), "=r"(w[4 * j + 3])
                             : "l"(src + 32 * t + 8 * j));
        } else {      // step j: dimensions 16j + 2t, + 1 and 16j + 8 + 2t, + 1
#pragma unroll
            for (int j = 0; j < 16; ++j) asm volatile("ld.global.u32 %0, [%1];" : "=r"(w[j]) : "l"(src + 8 * j + 2 * t));
        }
    }
}
// Turns them into the B fragments; returns the factor of the row's logits.  All 32 lanes call it.
template <bool E2M1>
__device__ __forceinline__ float make_query(uint32_t (&w)[16])
{
    if (!E2M1) return 1.f;
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 16; ++j) top = max(top, max((w[j] & 0x7fffu) << 16, w[j] & 0x7fff0000u));
    top = max(top, __shfl_xor_sync(kFull, top, 1));
    top = max(top, __shfl_xor_sync(kFull, top, 2));
    // 2^(14 - exponent of the largest); tiny rows (below 2^-100) are scaled as if they were that large
    const int ex = min(max((int)(top >> 23) - 127, -100), 127);
    const float up = __uint_as_float((uint32_t)(127 + 14 - ex) << 23);
    const bool finite = top < 0x7f800000u;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const __half2 v = __floats2half2_rn(__uint_as_float(w[j] << 16) * up, __uint_as_float(w[j] & 0xffff0000u) * up);
        w[j] = finite ? *reinterpret_cast<const uint32_t*>(&v) : 0x7fff7fffu;   // else the row is NaN
    }
    return __uint_as_float((uint32_t)(127 - 14 + ex) << 23);
}

__device__ __forceinline__ const uint16_t* query_row(const PagedAttnParams& p, int b, int h, int r)
{
    return p.q + (int64_t)b * p.q_b + (int64_t)(h * p.G + r / p.Mq) * p.q_h + (int64_t)(r % p.Mq) * p.q_i;
}

// A pair of weights as a sum of 16-bit parts: two f16 beside 4-bit rows (23 bits: what is dropped is below 2^-23 of a
// weight, or 2^-25 where a weight is below 2^-3: the largest of a row lies between 2^11 and 2^15), three bf16 beside
// bf16 rows (all 24 bits of a weight above 2^-103, which is 2^-68 of a row's largest at least; two would leave 17, and
// outputs 1.8 times as far off as fp32 arithmetic has them).
template <bool E2M1>
constexpr int kWeightParts = E2M1 ? 2 : 3;
template <bool E2M1>
__device__ __forceinline__ void split_p(float x0, float x1, uint32_t (&part)[kWeightParts<E2M1>])
{
    if constexpr (E2M1) {
        const __half2 a = __floats2half2_rn(x0, x1);
        const __half2 b = __floats2half2_rn(x0 - __low2float(a), x1 - __high2float(a));
        part[0] = *reinterpret_cast<const uint32_t*>(&a);
        part[1] = *reinterpret_cast<const uint32_t*>(&b);
    } else {
        split_bf16(x0, x1, part[0], part[1]);
        const float r0 = (x0 - __uint_as_float(part[0] << 16)) - __uint_as_float(part[1] << 16);   // exact
        const float r1 = (x1 - __uint_as_float(part[0] & 0xffff0000u)) - __uint_as_float(part[1] & 0xffff0000u);
        part[2] = pack_bf16(r0, r1);
    }
}

// Joins the W warps' partials of one query row in shared memory (partial w: its O at sm_o + w * pitch, rows kOPitch
// apart, m and z in sm_m and sm_l): the sum over them of the lane's dimensions 4 lane .. + 3, with the row's
// reference m (-inf: nothing was seen) and its sum z.
constexpr int kOPitch = kHeadDim + 4;   // floats; the pad spreads the rows 2t over the banks
template <int kRows, int W>
__device__ __forceinline__ float4 join_row(const float* sm_o, int pitch, const float* sm_m, const float* sm_l, int row,
                                           float& m, float& z)
{
    const int lane = threadIdx.x & 31;
    m = -INFINITY;
#pragma unroll
    for (int w = 0; w < W; ++w) m = fmaxf(m, sm_m[w * kRows + row]);
    z = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < W; ++w) {
        const float mw = sm_m[w * kRows + row];
        if (mw == -INFINITY) continue;   // that warp saw nothing
        const float f = fast_exp2(mw - m);
        const float4 o = *(reinterpret_cast<const float4*>(sm_o + w * pitch + row * kOPitch) + lane);
        z += f * sm_l[w * kRows + row];
        acc.x += f * o.x;
        acc.y += f * o.y;
        acc.z += f * o.z;
        acc.w += f * o.w;
    }
    return acc;
}

// Writes one query row's output (the lane's dimensions 4 lane .. + 3) and its lse.
template <bool E2M1, int SHAPED>
__device__ __forceinline__ void write_row(const PagedAttnParams& p, const Seq& q, int b, int h, int r, float4 acc, float m, float z)
{
    const int lane = threadIdx.x & 31;
    if (SHAPED) {
        const int i = r % p.Mq;
        if (i >= q.nb) return;
        const int64_t to = (int64_t)(q.q0 + i) * p.Hq + h * p.G + r / p.Mq;
        const bool none = m == -INFINITY;
        const float f = p.c.v_mul;
        reinterpret_cast<uint2*>(p.out16 + to * kHeadDim)[lane] =
            none ? make_uint2(0u, 0u) : make_uint2(pack_bf16(acc.x / z * f, acc.y / z * f), pack_bf16(acc.z / z * f, acc.w / z * f));
        if (p.lse && lane == 0) p.lse[to] = none ? -INFINITY : (m + log2f(z / kWeightUnit<E2M1>)) * 0.6931471805599453f;
        return;
    }
    const int64_t to = ((int64_t)b * p.Hq + h * p.G + r / p.Mq) * p.Mq + r % p.Mq;
    const bool none = m == -INFINITY;
    const float f = p.c.v_mul;
    reinterpret_cast<float4*>(p.out + to * kHeadDim)[lane] =
        none ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(acc.x / z * f, acc.y / z * f, acc.z / z * f, acc.w / z * f);
    if (p.lse && lane == 0) p.lse[to] = none ? -INFINITY : (m + log2f(z / kWeightUnit<E2M1>)) * 0.6931471805599453f;
}

// The query rows of one warp and what it has summed for them.
// SHAPED: what fx_paged_attend puts on the logits.  It lies in shared memory and is read for every unit: registers are what
// 4-bit rows have least of.
struct Shaping {
    const int2* see;      // what the query positions see
    uint32_t rows;        // of rows 2t, 2t + 1 of each N tile (64 bytes a tile): their positions from the first query's on,
                          // their slopes (base 2)
    uint32_t factors;     // of the rows' logits (32 bytes a tile), or 0: one factor for all
};
__device__ __forceinline__ float4 lds_float4(uint32_t a)
{
    const uint4 v = lds128(a);
    return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
}
// Logits of U tiles whose first row is `first`, as logits() gives them: under the cap, and with their bias by distance as
// base-2 logits (without one, the factor of a capped logit, p.cap2, is left to weights()).  Rows and queries are counted from
// the first query's position on: near rows then have their exact distances at any length of the cache, which positions past
// 2^24 by themselves do not have in fp32.
template <bool CAP, int U, int NT>
__device__ __forceinline__ void shape_logits(const PagedAttnParams& p, const Shaping& sh, float (&s)[U * NT][4], int first)
{
    const float unit = CAP ? p.cap_unit : p.qscale * 1.4426950408889634f;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        float f0 = unit, f1 = unit;
        if (sh.factors) {
            const uint2 w = lds64(sh.factors + 32 * n);
            f0 *= __uint_as_float(w.x);
            f1 *= __uint_as_float(w.y);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[u * NT + n][e] *= e & 1 ? f1 : f0;
    }
    if (CAP) {
        if (p.cap_apart) {
#pragma unroll
            for (int m = 0; m < U * NT; ++m)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[m][e] *= p.icap;
        }
        float top = 0.f;
#pragma unroll
        for (int m = 0; m < U * NT; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) top = fmaxf(top, fabsf(s[m][e]));
        if (!__any_sync(kFull, top > 1.f)) {   // (a NaN stays one)
#pragma unroll
            for (int m = 0; m < U * NT; ++m)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[m][e] = tanh_near(s[m][e]);
        } else {
#pragma unroll
            for (int m = 0; m < U * NT; ++m)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[m][e] = fabsf(s[m][e]) <= 1.f ? tanh_near(s[m][e]) : tanh_far(s[m][e]);
        }
    }
    if (p.slope) {
        const float row = (float)(first + (int)((threadIdx.x & 31) >> 2));
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float4 w = lds_float4(sh.rows + 64 * n);
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float far = (e & 1 ? w.z : w.x) - row;   // of the unit's first row
                    float& x = s[u * NT + n][e];
                    x = fmaf(fabsf(far - (float)(16 * u + 8 * (e >> 1))), -(e & 1 ? w.w : w.y), CAP ? x * p.cap2 : x);
                }
        }
    }
}

template <bool E2M1, int NT, bool DUP>
struct Acc {
    static constexpr bool kSharedQ = E2M1 || NT > 1;   // the queries' fragments lie in shared memory (not in 16
                                                       // registers an N tile)
    uint32_t q[kSharedQ ? 1 : NT][16];         // B fragments: registers 2j, 2j + 1 of step j
    uint32_t sq;                               // or the lane's place in [N tile][pair of steps][32] of 16 bytes
    float rs[NT][2];      // factor of the logits of rows 2t, 2t+1 (of each N tile)
    float bias[NT][2];    // minus the reference of those rows; kNoRef: none yet
    float l[NT][2];
    float o[NT][8][4];
};

// Weights of U tiles from their logits s[u * NT + n][e] (row g + 8 (e >> 1) of tile u, query row 2t + (e & 1) of
// N tile n), in place; moves the references when one would not fit.  With HIDE, bit 4 (u * NT + n) + e of hide:
// that logit does not count.
template <bool HIDE, int U, bool E2M1, int NT, bool DUP>
__device__ __forceinline__ void weights(Acc<E2M1, NT, DUP>& a, float (&s)[U * NT][4], uint32_t hide)
{
    auto hidden = [&](int m, int e) { return HIDE && ((hide >> (4 * m + e)) & 1u) != 0; };
    float x2[U * NT][4];
    bool over = false;
#pragma unroll
    for (int m = 0; m < U * NT; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x2[m][e] = hidden(m, e) ? -INFINITY : fmaf(s[m][e], a.rs[m % NT][e & 1], a.bias[m % NT][e & 1]);
            over |= x2[m][e] > kTop;
        }
    if (__any_sync(kFull, over)) {
        // new references: the largest logit of each row lands on 2^kBase
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float m = -INFINITY;
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int z = e; z < 4; z += 2)
                        if (!hidden(u * NT + n, z)) m = fmaxf(m, __fmul_rn(s[u * NT + n][z], a.rs[n][e]));
                m = fmaxf(m, __shfl_xor_sync(kFull, m, 4));
                m = fmaxf(m, __shfl_xor_sync(kFull, m, 8));
                m = fmaxf(m, __shfl_xor_sync(kFull, m, 16));
                const float nb = fminf(a.bias[n][e], kBase - m);
                if (nb < a.bias[n][e]) {   // never for a row without a visible logit above -inf
                    const float f = fast_exp2(nb - a.bias[n][e]);   // 0 for the first reference
                    a.l[n][e] *= f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        a.o[n][i][e] *= f;
                        a.o[n][i][e + 2] *= f;
                    }
                    a.bias[n][e] = nb;
                }
                const bool far = fabsf(nb) > kFarRef;
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int z = e; z < 4; z += 2) {
                        float x = fmaf(s[u * NT + n][z], a.rs[n][e], nb);
                        if (far) {
                            x = __fadd_rn(__fmul_rn(s[u * NT + n][z], a.rs[n][e]), nb);
                            x = x > kTop ? kTop : x;   // (a NaN stays)
                        }
                        x2[u * NT + n][z] = hidden(u * NT + n, z) ? -INFINITY : x;
                    }
            }
    }
#pragma unroll
    for (int m = 0; m < U * NT; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            s[m][e] = fast_exp2(x2[m][e]) * kWeightUnit<E2M1>;
            a.l[m % NT][e & 1] += s[m][e];
        }
}

// Logits of U tiles from tile u0 of a slot on: s[u * NT + n][e] of row g + 8 (e >> 1) and query row 2t + (e & 1) of
// N tile n.
template <int U, typename S, bool E2M1, int NT, bool DUP>
__device__ __forceinline__ void logits(const Acc<E2M1, NT, DUP>& a, uint32_t slot, int u0, float (&s)[U * NT][4])
{
    float s2[U * NT][2][4];   // two chains of products, for their latency
    KTile<E2M1> k[U];
#pragma unroll
    for (int u = 0; u < U; ++u) k[u].template load<S>(slot, u0 + u);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t x[U][2][4];
#pragma unroll
        for (int u = 0; u < U; ++u) k[u].pair(j, x[u]);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            uint4 q;
            if (Acc<E2M1, NT, DUP>::kSharedQ)
                q = lds128(a.sq + (n * 4 + j) * 512);
            else
                q = make_uint4(a.q[n][4 * j], a.q[n][4 * j + 1], a.q[n][4 * j + 2], a.q[n][4 * j + 3]);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float(&c)[2][4] = s2[u * NT + n];
                if (j == 0) {
                    mma16_zero<E2M1>(c[0], x[u][0][0], x[u][0][1], x[u][0][2], x[u][0][3], q.x, q.y);
                    mma16_zero<E2M1>(c[1], x[u][1][0], x[u][1][1], x[u][1][2], x[u][1][3], q.z, q.w);
                } else {
                    mma16<E2M1>(c[0], x[u][0][0], x[u][0][1], x[u][0][2], x[u][0][3], q.x, q.y);
                    mma16<E2M1>(c[1], x[u][1][0], x[u][1][1], x[u][1][2], x[u][1][3], q.z, q.w);
                }
            }
        }
    }
#pragma unroll
    for (int m = 0; m < U * NT; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[m][e] = s2[m][0][e] + s2[m][1][e];
}

// A tile's weights as B fragments, one for each product that its V takes part in: one for each part of the weights.
// With DUP a fragment has two parts: one in columns 0..3, the next in columns 4..7.
template <bool E2M1, int NT, bool DUP>
struct Weights {
    static constexpr int kTerms = DUP ? (kWeightParts<E2M1> + 1) / 2 : kWeightParts<E2M1>;
    uint32_t x[kTerms][NT][2];
};
template <bool E2M1, int NT, bool DUP>
__device__ __forceinline__ void fragments(const float (&s)[NT][4], Weights<E2M1, NT, DUP>& w)
{
    const int t = threadIdx.x & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            uint32_t part[kWeightParts<E2M1>];
            split_p<E2M1>(s[n][2 * u], s[n][2 * u + 1], part);
#pragma unroll
            for (int k = 0; k < w.kTerms; ++k) {
                if (DUP) {
                    const uint32_t next = 2 * k + 1 < kWeightParts<E2M1> ? part[(2 * k + 1) % kWeightParts<E2M1>] : 0u;
                    w.x[k][n][u] = movmatrix_t(t < 2 ? part[2 * k % kWeightParts<E2M1>] : next);
                } else {
                    w.x[k][n][u] = movmatrix_t(part[k % kWeightParts<E2M1>]);
                }
            }
        }
}
template <bool E2M1, int NT, bool DUP>
__device__ __forceinline__ void term(float (&c)[4], const Weights<E2M1, NT, DUP>& w, int n, const uint32_t (&v)[4], bool first)
{
#pragma unroll
    for (int k = 0; k < w.kTerms; ++k) {
        if (first && k == 0)
            mma16_zero<E2M1>(c, v[0], v[1], v[2], v[3], w.x[k][n][0], w.x[k][n][1]);
        else
            mma16<E2M1>(c, v[0], v[1], v[2], v[3], w.x[k][n][0], w.x[k][n][1]);
    }
}

// r % Mq of a query row (r < 64).
__device__ __forceinline__ int query_pos(const PagedAttnParams& p, int r) { return r - ((r * p.mq_inv) >> 16) * p.Mq; }

// A unit of U tiles.  EDGE: the tiles whose bit is set in `edge` (tile u: bit U - 1 - u) have rows that do not count
// for every query: not valid, or past what some query sees.  Rows that are not valid may hold anything, and 0 *
// NaN is NaN: their V counts as zeros.
//
// O^T += V^T P^T: the tiles' product starts from zero and is added to O by an fp32 addition.  The tensor core
// aligns all products to the accumulator and cuts them off (2^-23 of it): accumulated over a long row that costs
// small weights beside a large one, and drifts.
template <int U, bool EDGE, typename S, int SHAPED, bool E2M1, int NT, bool DUP>
__device__ __forceinline__ void attend(const PagedAttnParams& p, Acc<E2M1, NT, DUP>& a, uint32_t slot, uint32_t edge, int r0,
                                       int seen, const Shaping& sh, int first)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    float s[U * NT][4];
    logits<U, S, E2M1, NT, DUP>(a, slot, 0, s);
    if (SHAPED) shape_logits<SHAPED == 2, U, NT>(p, sh, s, first);
    uint32_t hide = 0, vm[U];
    if (EDGE) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            int pos = 0;   // of a whole tile: seen by all
            if ((edge >> (U - 1 - u)) & 1u) pos = (int)lds32(slot + S::kPos + 64 * u + 4 * (lane & 15));
            vm[u] = __ballot_sync(kFull, pos >= 0) & 0xffffu;   // the valid rows
            const int p0 = __shfl_sync(kFull, pos, g), p1 = __shfl_sync(kFull, pos, g + 8);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int at = e >> 1 ? p1 : p0;
                    const int r = r0 + 8 * n + (DUP ? (2 * t + (e & 1)) & 3 : 2 * t + (e & 1));
                    if (SHAPED) {
                        // (a whole tile beside one with an edge has no positions: all of it is seen)
                        const int2 see = sh.see[query_pos(p, r)];
                        if (((edge >> (U - 1 - u)) & 1u) && (at < see.x || at >= see.y)) hide |= 1u << (4 * (u * NT + n) + e);
                    } else if (at < 0 || at > seen + query_pos(p, r)) {
                        hide |= 1u << (4 * (u * NT + n) + e);
                    }
                }
        }
    }
    weights<EDGE, U, E2M1, NT, DUP>(a, s, hide);
    Weights<E2M1, NT, DUP> w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) fragments<E2M1, NT, DUP>(reinterpret_cast<float(&)[NT][4]>(s[u * NT]), w[u]);
    VTile<E2M1> v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u].template load<EDGE, S>(slot, u, EDGE ? vm[u] : 0u);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float c[NT][4];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            uint32_t x[4];
            v[u].template get<EDGE>(i, x);
#pragma unroll
            for (int n = 0; n < NT; ++n) term<E2M1, NT, DUP>(c[n], w[u], n, x, u == 0);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) a.o[n][i][e] += c[n][e];
    }
}

// Whether a valid row of tile u outside [from, to), which every query sees, holds an infinity or a NaN in V.
template <typename S, bool E2M1>
__device__ __forceinline__ bool not_all_finite(uint32_t slot, int u, int from, int to)
{
    const int lane = threadIdx.x & 31;
    const int pos = (int)lds32(slot + S::kPos + 64 * u + 4 * (lane & 15));
    auto outside = [&](int t) { return t >= to || (t >= 0 && t < from); };
    const bool some = outside(pos);
    if (!__any_sync(kFull, some)) return false;
    bool bad = false;
    if (E2M1) {   // a NaN scale (the lane looks at half the scales of row lane / 2)
        const uint32_t z = lds32(slot + S::kScaleV + 128 * u + 4 * lane) & 0x7f7f7f7fu;
        bad = outside(__shfl_sync(kFull, pos, lane >> 1)) && __vcmpeq4(z, 0x7f7f7f7fu) != 0;
    } else {      // an all-ones exponent
        for (int j = 0; j < 16; ++j) {
            const uint2 z = lds64(slot + S::kV + u * S::kTile + 256 * j + 8 * lane);
            const uint32_t x = __vcmpeq2(z.x & 0x7f807f80u, 0x7f807f80u) | __vcmpeq2(z.y & 0x7f807f80u, 0x7f807f80u);
            bad |= __shfl_sync(kFull, some, j) && x != 0;
        }
    }
    return __any_sync(kFull, bad);
}

// A tile where rows that only later queries see hold an infinity or a NaN: one product per query position, over
// the rows that it sees, taken by its query rows alone.  whole: a tile without an edge beside such a one.
template <typename S, int SHAPED, bool E2M1, int NT, bool DUP>
__device__ __forceinline__ void attend_apart(const PagedAttnParams& p, Acc<E2M1, NT, DUP>& a, uint32_t slot, int u, int r0,
                                             int seen, bool whole, const Shaping& sh, int first)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    int pos = 0;   // of a whole tile: seen by all
    if (!whole) pos = (int)lds32(slot + S::kPos + 64 * u + 4 * (lane & 15));
    const uint32_t vm = __ballot_sync(kFull, pos >= 0) & 0xffffu;   // the valid rows
    if (vm == 0) return;
    float s[NT][4];
    logits<1, S, E2M1, NT, DUP>(a, slot, u, s);
    if (SHAPED) shape_logits<SHAPED == 2, 1, NT>(p, sh, s, first);
    uint32_t hide = 0;
    const int p0 = __shfl_sync(kFull, pos, g), p1 = __shfl_sync(kFull, pos, g + 8);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = r0 + 8 * n + (DUP ? (2 * t + (e & 1)) & 3 : 2 * t + (e & 1));
            const int at = e >> 1 ? p1 : p0;
            if (SHAPED) {
                const int2 see = sh.see[query_pos(p, r)];
                if (!whole && (at < see.x || at >= see.y)) hide |= 1u << (4 * n + e);
            } else if (at < 0 || at > seen + query_pos(p, r)) {
                hide |= 1u << (4 * n + e);
            }
        }
    weights<true, 1, E2M1, NT, DUP>(a, s, hide);
    Weights<E2M1, NT, DUP> w;
    fragments<E2M1, NT, DUP>(s, w);
#pragma unroll 1
    for (int i = 0; i < p.Mq; ++i) {
        uint32_t add = 0;   // bit 2n + e: query row 2t + e of N tile n
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (query_pos(p, r0 + 8 * n + (DUP ? (2 * t + e) & 3 : 2 * t + e)) == i) add |= 1u << (2 * n + e);
        VTile<E2M1> v;
        bool sees = pos <= seen + i;
        if (SHAPED) sees = whole || (pos >= sh.see[i].x && pos < sh.see[i].y);
        v.template load<true, S>(slot, u, __ballot_sync(kFull, sees) & vm);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint32_t x[4];
            v.template get<true>(j, x);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float c[4];
                term<E2M1, NT, DUP>(c, w, n, x, true);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if ((add >> (2 * n + (e & 1))) & 1u) a.o[n][j][e] += c[e];
            }
        }
    }
}

// How the CTAs of a kernel share its work.  A piece is one (sequence, KV head, group of query rows).  By the
// lengths found on the device, the tiles of all pieces are shared in one of two ways.  Short work: every piece is
// cut into equal parts, one to a CTA, so that no CTA starts twice.  Long work, or more pieces than CTAs: the tiles
// of all pieces form one line, of which every CTA walks an equal stretch piece by piece, so that ragged lengths
// leave no CTA with more to do than another.
template <int W>
struct LineSmem {
    int scan[W], start, b, len, lo, cnt[32 * W];
};
template <int W, typename Count, int SHAPED = 0>
struct Line {
    const PagedAttnParams& p;
    const Count count;         // tiles of a sequence's piece, at least 1
    const int per_seq;         // pieces of one sequence
    const LineCost cost;
    Seq seq;
    int b, ntile;              // the sequence, tiles of its pieces
    int piece, s0, s1;         // the piece of the sequence, this CTA's tiles of it
    int c0, n_part, slot0;     // the CTAs that share it: c0 .. c0 + n_part - 1; the partial slot of the first
    int part;                  // which of them this is
    int slot;                  // this CTA's partial slot

    __device__ __forceinline__ Line(const PagedAttnParams& p_, Count count_, int per_seq_, LineCost cost_)
        : p(p_), count(count_), per_seq(per_seq_), cost(cost_)
    {
    }

    // Parts that a piece of n tiles is cut into (at most n of them).
    __device__ __forceinline__ int parts(int n) const { return min((int)((float)n * inv) + 1, n); }

    // Chooses how the work is shared from its length (total) and the tiles of every sequence's piece (get(i), i < B):
    // the lanes try shares of 1 to 2 times the ideal one and agree on the one with the shortest longest part.
    template <typename Get>
    __device__ __forceinline__ void choose(int B, const Get& get)
    {
        cta = blockIdx.x;
        const int most = (int)gridDim.x;
        const bool many = B >= most || B * per_seq >= most;   // (of one tile at least)
        const int grid = many ? most : min(most, kMaxParts * B * per_seq);
        n_cta = many ? grid : min(grid, max(1, total / (W * kMinTiles)));
        inv = 0.f;
        if (B < grid && B * per_seq <= grid) {
            const float ideal = fmaxf((float)total / (float)grid, (float)(W * kMinTiles));
            inv = 1.f / (ideal * (1.f + (float)(threadIdx.x & 31) / 32.f));
            int sum = 0;
            float longest = 0.f;
            for (int i = 0; i < B; ++i) {
                const int n = get(i), k = parts(n);
                sum += k;
                longest = fmaxf(longest, __fdividef((float)n, (float)k));
            }
            if (sum > grid || sum * per_seq > grid) longest = INFINITY;
            float best = longest;
#pragma unroll
            for (int d = 16; d; d >>= 1) best = fminf(best, __shfl_xor_sync(kFull, best, d));
            const unsigned who = __ballot_sync(kFull, longest == best);
            inv = __shfl_sync(kFull, inv, __ffs(who) - 1);
            if (!(best <= ideal + cost.second)) inv = 0.f;
        }
        at = cta;
        end = cta + 1;
        if (inv == 0.f) {
            total += p.c.B * per_seq * cost.start;
            quota = total / n_cta;
            extra = total - quota * n_cta;
            at = place(cta);
            end = place(cta + 1);
        }
    }
    // Stretches of the line: quota tiles to a CTA, one more to each of the first `extra`.
    __device__ __forceinline__ int place(int c) const { return quota * c + min(c, extra); }
    __device__ __forceinline__ int owner(int tile) const
    {
        const int big = extra * (quota + 1);
        return tile < big ? tile / (quota + 1) : extra + (tile - big) / quota;
    }

    // False: nothing for this CTA.  All threads call it.
    __device__ __forceinline__ bool start(LineSmem<W>& sm)
    {
        constexpr int kThreadsL = 32 * W;
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
        const int B = p.c.B;
        if (B <= 32) {
            // every warp finds the CTA's place by itself: lane i holds sequence i
            seq = sequence<SHAPED>(p, min(lane, B - 1), blockIdx.x == 0 && tid < B);
            const int mine = lane < B ? count(seq) : 0;
            total = mine;
#pragma unroll
            for (int d = 16; d; d >>= 1) total += __shfl_xor_sync(kFull, total, d);
            total *= per_seq;
            choose(B, [&](int i) { return __shfl_sync(kFull, mine, i); });
            if (inv == 0.f && cta >= n_cta) return false;
            const int n = lane < B ? (inv == 0.f ? mine + cost.start : parts(mine)) : 0;
            int inc = n;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(kFull, inc, d);
                if (lane >= d) inc += o;
            }
            const int first = (inc - n) * per_seq;
            const unsigned who = __ballot_sync(kFull, n > 0 && at >= first && at < first + n * per_seq);
            if (who == 0) return false;   // more CTAs than parts
            b = __ffs(who) - 1;
            seq_start = __shfl_sync(kFull, first, b);
            seq.len = __shfl_sync(kFull, seq.len, b);
            seq.lo = __shfl_sync(kFull, seq.lo, b);
        } else {
            // Up to as many sequences as threads take one scan; more take one pass for the line's length and a
            // scan of blocks of them.
            seq = sequence<SHAPED>(p, min(tid, B - 1), blockIdx.x == 0 && tid < B);
            const bool one_scan = B <= kThreadsL;
            const int n_first = tid < B ? count(seq) : 0;
            total = n_first;
            for (int i = tid + kThreadsL; i < B; i += kThreadsL) total += count(sequence<SHAPED>(p, i, blockIdx.x == 0));
#pragma unroll
            for (int d = 16; d; d >>= 1) total += __shfl_xor_sync(kFull, total, d);
            if (lane == 0) sm.scan[warp] = total;
            sm.cnt[tid] = n_first;
            if (tid == 0) sm.b = -1;
            __syncthreads();
            total = 0;
#pragma unroll
            for (int w = 0; w < W; ++w) total += sm.scan[w];
            total *= per_seq;
            if (one_scan) {
                choose(B, [&](int i) { return sm.cnt[i]; });
            } else {
                choose(0x7fffffff, [](int) { return 0; });   // (always stretches: equal parts are looked for among the
                                                             // lengths of one scan)
            }
            if (inv == 0.f && cta >= n_cta) return false;
            int before = 0;   // units (of one piece each) of the sequences before this block
            for (int b0 = 0; b0 < B; b0 += kThreadsL) {
                const int i = b0 + tid;
                if (b0 > 0 && i < B) seq = sequence<SHAPED>(p, i, false);
                const int c = b0 == 0 ? n_first : (i < B ? count(seq) : 0);
                const int n = i < B ? (inv == 0.f ? c + cost.start : parts(c)) : 0;
                int inc = n;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int o = __shfl_up_sync(kFull, inc, d);
                    if (lane >= d) inc += o;
                }
                __syncthreads();   // sm.scan is free
                if (lane == 31) sm.scan[warp] = inc;
                __syncthreads();
                int sum = 0, mine = 0;
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    if (w == warp) mine = sum;
                    sum += sm.scan[w];
                }
                const int first = (before + mine + inc - n) * per_seq;
                if (n > 0 && at >= first && at < first + n * per_seq) {
                    sm.b = i;
                    sm.start = first;
                    sm.len = seq.len;
                    sm.lo = seq.lo;
                }
                __syncthreads();
                before += sum;
                if (sm.b >= 0) break;
            }
            b = sm.b;
            if (b < 0) return false;   // more CTAs than parts
            seq_start = sm.start;
            seq.len = sm.len;
            seq.lo = sm.lo;
        }
        seq.table = p.c.table + (int64_t)b * p.c.table_stride;
        if (SHAPED) seq = sequence<SHAPED>(p, b, false);   // (the rest of it: what it reads is near by now)
        ntile = count(seq);
        if (inv == 0.f) at -= (at - seq_start) % (ntile + cost.start);   // the start of its first piece
        return true;
    }

    // The next piece of this CTA; false: there is none.
    __device__ __forceinline__ bool next()
    {
        if (inv == 0.f) {
            for (;;) {
                if (at >= end) return false;
                while (at >= seq_start + (ntile + cost.start) * per_seq) {
                    seq_start += (ntile + cost.start) * per_seq;
                    if (++b >= p.c.B) return false;   // (lengths that change during the call)
                    seq = sequence<SHAPED>(p, b, false);
                    ntile = count(seq);
                }
                // a cut near an end of the piece moves there, all cuts of a short piece do: no CTA comes for a few
                // tiles, and a piece of one CTA has no parts to join
                const int near = min(cost.near, ntile / 2), from = at + cost.start;
                c0 = owner(from + near);
                n_part = owner(max(from + ntile - near - 1, from + near)) - c0 + 1;
                piece = (at - seq_start) / (ntile + cost.start);
                at += ntile + cost.start;
                part = cta - c0;
                if (part < 0 || part >= n_part) continue;
                s0 = part == 0 ? 0 : place(cta) - from;
                s1 = part == n_part - 1 ? ntile : place(cta + 1) - from;
                break;
            }
        } else {
            if (at >= end) return false;
            n_part = parts(ntile);
            piece = (at - seq_start) / n_part;
            part = at - seq_start - piece * n_part;
            const int least = ntile / n_part, more = ntile - least * n_part;
            s0 = least * part + min(part, more);
            s1 = s0 + least + (part < more ? 1 : 0);
            c0 = cta - part;
            at = end;
        }
        // a CTA is the first of one shared piece at most, and comes later in one other at most
        slot = cta * 2 + (part == 0 ? 1 : 0);
        slot0 = c0 * 2 + 1;
        return true;
    }

private:
    int cta, n_cta, quota, extra;
    float inv;                 // 1 / tiles of a part where every CTA takes one part of one piece; 0: stretches
    int total, at, end;        // length of the line (tiles); the next piece's start and the CTA's end (tiles, or parts)
    int seq_start;             // place where the sequence starts
};

// Start of warp w's stretch of the tiles [s0, s1) of a sequence: nearly equal ones; where tiles are taken in pairs,
// the tail's start at multiples of 32 rows.
template <int U, int W>
__device__ __forceinline__ int warp_start(const Seq& q, int s0, int s1, int w)
{
    static_assert((W & (W - 1)) == 0, "");
    const int x = s0 + (int)((unsigned)((s1 - s0) * w) / W);   // (fewer than 2^28 tiles)
    return w == W ? s1 : (w == 0 || U == 1 || x < q.nl ? x : min(x + (((q.lo >> 4) + x - q.nl) & 1), s1));
}

// Shape of the decode kernel for a format and up to 4 (DUP), 8 or 16 query rows a pass.
//
// bf16: bound by bytes.  A tile is 8 KB, and the rings of two CTAs fill the shared memory of an SM (8 x 32768 rows,
// 755 MB: 117 us, 0.95 of the copy bandwidth; rings of 4 units instead of 3, with one CTA an SM: 117 us).
// 4 bits: a tile is 2.3 KB and takes 310 instructions of a warp, of which 64 are conversions of codes and 64 their
// scaling (the conversion issues every second cycle).  Bytes are the floor (8 x 32768 rows: 32 us; to issue their 30 M
// instructions 29), latency is the bound: the 3 warps of a scheduler issue in 54% of the cycles, and wait for the results
// of chains of conversions, products and exponentials (1.0 cycle an instruction) and for instructions themselves (0.6).  As
// many warps as the registers allow: 3 CTAs an SM for up to 8 rows (16 x 32768 rows, 411 MB: 84 us, 0.72 of the copy
// bandwidth; 2 CTAs: 91 us), 2 CTAs for 16 rows (3 spilled 400 to 600 bytes, and gained nothing).  As it is, 16 rows spill
// 32 to 40 bytes, and 8 rows in units of two tiles 60.  Two tiles at a time share the loads of the queries and the additions
// to O; where a warp gets few tiles, one at a time is sooner done (kShort).  DUP: 84 us against 94 for up to 4 rows.  One
// pass of 16 rows instead of two of 8: 79 us against 96 (64 x 3335 rows, 14 query rows).
template <bool E2M1, int NT, bool DUP, int U>
struct Shape {
    static constexpr int kRows = DUP ? 4 : 8 * NT;       // query rows of a pass over a (sequence, KV head)
    static constexpr int kWarps = 4;                  // few, so that other CTAs of the SM work while one starts or joins
    static constexpr int kCtas = E2M1 && NT == 1 ? 3 : 2;       // per SM
    static constexpr int kStages = U == 2 ? 2 : 3;       // units (of U tiles that a warp attends at a time) in its ring
    using Unit = Slot<E2M1, true, U>;
    static constexpr int kRing = kStages * Unit::kBytes;   // bytes of a warp; its partial O later takes them
    static constexpr size_t kSmem = (size_t)kWarps * kRing;
    static_assert(kRows * kOPitch * 4 <= kRing, "a warp's partial O lies in its ring");
};

// Decode.  A CTA's warps take a stretch each of its tiles of a piece and meet in shared memory; a piece that several
// CTAs share is joined by the last of them to arrive, in the order of the CTAs.
//
// DUP: at most 4 query rows; columns 4..7 of the products repeat them, so that one product takes P's high part
// (columns 0..3) and its low part (4..7).
//
// SHAPED: fx_paged_attend -- new tokens of ragged sequences, a cap and a bias on the logits, an interval of rows for each
// query position; the positions of a unit's rows follow from its place.
template <bool E2M1, int NT, bool DUP, int U, int SHAPED>
__global__ void __launch_bounds__(32 * Shape<E2M1, NT, DUP, U>::kWarps, Shape<E2M1, NT, DUP, U>::kCtas)
    paged_decode_kernel(const PagedAttnParams p)
{
    using S = Shape<E2M1, NT, DUP, U>;
    constexpr int kRows = S::kRows, W = S::kWarps, kStages = S::kStages, kSlot = S::Unit::kBytes;
    constexpr int kPitch = S::kRing / 4;   // floats between the warps' partial O
    extern __shared__ __align__(128) float smem[];
    float* const sm_o = smem;
    constexpr bool kSharedQ = Acc<E2M1, NT, DUP>::kSharedQ;
    __shared__ float sm_m[W * kRows], sm_l[W * kRows];
    __shared__ uint4 sm_q[kSharedQ ? NT * 128 : 1];   // the queries' fragments, the factors of their logits
    __shared__ __align__(8) float sm_f[8 * NT];
    __shared__ LineSmem<W> sm_line;
    __shared__ int2 sm_see[SHAPED ? kMaxRows : 1];
    __shared__ __align__(16) float2 sm_row[SHAPED ? 8 * NT : 1];   // positions and slopes
    __shared__ unsigned sm_last;

    griddep_wait();
    griddep_launch();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const uint32_t ring = smem_addr(smem) + warp * S::kRing;
    const int nrg = (p.R + kRows - 1) / kRows;
    auto tiles = [](const Seq& q) { return tile_count(q); };
    Line<W, decltype(tiles), SHAPED> line(p, tiles, p.c.Hkv * nrg, decode_cost(E2M1));
    if (!line.start(sm_line)) return;

    while (line.next()) {
        const int b = line.b, s0 = line.s0, s1 = line.s1, n_part = line.n_part;
        const int h = line.piece / nrg, r0 = (line.piece - h * nrg) * kRows;
        Seq seq = line.seq;
        const int seen = seq.len - p.Mq;   // query i sees rows <= seen + i
        seq.idx = p.idx ? p.idx + ((int64_t)b * p.c.Hkv + h) * p.kk : nullptr;
        const int base = SHAPED ? (seq.lo & ~(kTileRows - 1)) - seq.pos0 : 0;   // first row of the first tile, from the first query on
        if (SHAPED) {
            for (int i = tid; i < p.Mq; i += 32 * W) sm_see[i] = i < seq.nb ? shaped_interval(p, seq, i) : make_int2(0, 0);
            if (tid < 8 * NT) {
                const int r = r0 + (DUP ? tid & 3 : tid);
                sm_row[tid] = make_float2((float)query_pos(p, r),
                                          p.slope && r < p.R ? p.slope[h * p.G + r / p.Mq] * 1.4426950408889634f : 0.f);
            }
        }

        // the queries, the pages and the first rows are under way together
        Acc<E2M1, NT, DUP> a;
        if (!kSharedQ || warp < NT) {   // shared: a warp prepares one N tile
            const int r = r0 + (DUP ? g & 3 : (kSharedQ ? 8 * warp + g : g));
            if (SHAPED)
                fetch_query<E2M1>(r < p.R && r % p.Mq < seq.nb ? p.q + (int64_t)(seq.q0 + r % p.Mq) * p.q_i + (int64_t)(h * p.G + r / p.Mq) * p.q_h
                                                             : nullptr,
                                  a.q[0]);
            else
                fetch_query<E2M1>(r < p.R ? query_row(p, b, h, r) : nullptr, a.q[0]);
        }
        // a warp's share of the tiles is a stretch of them (in one page the next tile is 16 rows further on; pairs
        // start at multiples of 32); the ring's first units go on their way, then each turn feeds the unit
        // kStages - 1 turns ahead
        Feeder<E2M1, true, U, SHAPED> feeder(p, seq, h, warp_start<U, W>(seq, s0, s1, warp), warp_start<U, W>(seq, s0, s1, warp + 1));
        uint32_t flags[kStages];   // of the units in the ring, oldest first
        int first[kStages];        // SHAPED: their first rows, from the first query on
#pragma unroll
        for (int k = 0; k < kStages - 1; ++k) {
            if (SHAPED) first[k] = base + feeder.it * kTileRows;
            flags[k] = feeder.feed(ring + k * kSlot);
        }
        if (!kSharedQ || warp < NT) {
            const float f = make_query<E2M1>(a.q[0]);
            if (kSharedQ) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    sm_q[(warp * 4 + j) * 32 + lane] = make_uint4(a.q[0][4 * j], a.q[0][4 * j + 1], a.q[0][4 * j + 2], a.q[0][4 * j + 3]);
                if (t == 0) sm_f[8 * warp + g] = f;
            } else {
#pragma unroll
                for (int e = 0; e < 2; ++e) a.rs[0][e] = p.qscale * __shfl_sync(kFull, f, (2 * t + e) * 4);
            }
        }
        if (kSharedQ || SHAPED) __syncthreads();
        const Shaping sh{sm_see, smem_addr(sm_row) + 16 * t, kSharedQ ? smem_addr(sm_f) + 8 * t : 0u};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (kSharedQ) a.rs[n][e] = p.qscale * sm_f[8 * n + 2 * t + e];
                if (SHAPED) a.rs[n][e] = SHAPED == 2 && !p.slope ? p.cap2 : 1.f;
                a.bias[n][e] = kNoRef;
                a.l[n][e] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) a.o[n][i][e] = 0.f;
        }
        a.sq = smem_addr(sm_q) + 16 * lane;

        uint32_t slot = ring, into = ring + (kStages - 1) * kSlot;
        while (flags[0] >> U) {
            cp_async_wait_stages<kStages - 1>();   // this lane's copies; the barrier covers the others'
            __syncwarp();
            if (SHAPED) first[kStages - 1] = base + feeder.it * kTileRows;
            flags[kStages - 1] = feeder.feed(into);
            const uint32_t edge = flags[0] & ((1u << U) - 1);
            const int row0 = SHAPED ? first[0] : 0;
            if (edge == 0) {
                attend<U, false, typename S::Unit, SHAPED>(p, a, slot, 0, r0, seen, sh, row0);
            } else {
                bool apart = false;
#pragma unroll 1
                for (int u = 0; u < U && p.Mq > 1; ++u)
                    if ((edge >> (U - 1 - u)) & 1u)
                        apart |= not_all_finite<typename S::Unit, E2M1>(slot, u, SHAPED ? seq.com_lo : 0, SHAPED ? seq.com_hi : seen + 1);
                if (!apart) {
                    attend<U, true, typename S::Unit, SHAPED>(p, a, slot, edge, r0, seen, sh, row0);
                } else {
#pragma unroll 1
                    for (int u = 0; u < U; ++u)
                        attend_apart<typename S::Unit, SHAPED>(p, a, slot, u, r0, seen, ((edge >> (U - 1 - u)) & 1u) == 0, sh, row0 + 16 * u);
                }
            }
            into = slot;
            slot = slot + kSlot == ring + S::kRing ? ring : slot + kSlot;
#pragma unroll
            for (int k = 0; k < kStages - 1; ++k) {
                flags[k] = flags[k + 1];
                if (SHAPED) first[k] = first[k + 1];
            }
        }
        cp_async_wait_all_groups();
        __syncwarp();   // every lane is done with the ring

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
                    // a NaN logit leaves no reference but shows
                    sm_m[warp * kRows + row] = z != z ? 0.f : (a.bias[n][e] == kNoRef ? -INFINITY : -a.bias[n][e]);
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
                if (!E2M1) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (!DUP || t < 2)
                            sm_o[warp * kPitch + (8 * n + 2 * t + (e & 1)) * kOPitch + v_dim<E2M1>(i, g, e >> 1)] = a.o[n][i][e];
                } else if ((i & 1) && (!DUP || t < 2)) {   // M tiles i - 1, i: four neighbouring dimensions
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        *reinterpret_cast<float4*>(sm_o + warp * kPitch + (8 * n + 2 * t + e) * kOPitch + v_dim<E2M1>(i - 1, g, 0)) =
                            make_float4(a.o[n][i - 1][e], a.o[n][i - 1][e + 2], a.o[n][i][e], a.o[n][i][e + 2]);
                }
            }
        __syncthreads();

        if (n_part == 1) {
            for (int row = warp; row < kRows && r0 + row < p.R; row += W) {
                float z, m;
                const float4 acc = join_row<kRows, W>(sm_o, kPitch, sm_m, sm_l, row, m, z);
                write_row<E2M1, SHAPED>(p, seq, b, h, r0 + row, acc, m, z);
            }
        } else {
            // this CTA's part of the piece goes to its slot; the last CTA to arrive joins all of them
            constexpr int kPart = kRows * (kHeadDim + 2);
            float* part = p.part + (size_t)line.slot * kPart;
#pragma unroll
            for (int row = warp; row < kRows; row += W) {
                float z, m;
                reinterpret_cast<float4*>(part + row * kHeadDim)[lane] = join_row<kRows, W>(sm_o, kPitch, sm_m, sm_l, row, m, z);
                if (lane == 0) {
                    part[kRows * kHeadDim + row] = m;
                    part[kRows * kHeadDim + kRows + row] = z;
                }
            }
            __syncthreads();
            if (tid == 0) {
                __threadfence();   // the CTA's part, which the barrier orders before this fence
                sm_last = atomicAdd(p.counters + line.c0, 1u) == (unsigned)(n_part - 1);
                if (sm_last) {
                    p.counters[line.c0] = 0;   // ready for the next call
                    __threadfence();
                }
            }
            __syncthreads();
            if (sm_last) {
                // a warp takes every W-th row; 32 parts at a time, whose references and sums the lanes hold
                constexpr int kMine = kRows / W;   // rows of a warp
                float m[kMine], z[kMine];
                float4 acc[kMine];
#pragma unroll
                for (int k = 0; k < kMine; ++k) {
                    m[k] = -INFINITY;
                    z[k] = 0.f;
                    acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                }
                for (int c1 = 0; c1 < n_part; c1 += 32) {
                    const int mine = c1 + lane;
                    const float* ref = p.part + (size_t)(mine == 0 ? line.slot0 : (line.c0 + mine) * 2) * kPart + kRows * kHeadDim;
                    float f[kMine];
#pragma unroll
                    for (int k = 0; k < kMine; ++k) {
                        const int row = warp + k * W;
                        const float mp = mine < n_part ? __ldcg(ref + row) : -INFINITY;
                        const float zp = mine < n_part ? __ldcg(ref + kRows + row) : 0.f;
                        float mx = mp;
#pragma unroll
                        for (int d = 16; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, d));
                        mx = fmaxf(mx, m[k]);
                        const float old = m[k] == -INFINITY ? 0.f : fast_exp2(m[k] - mx);
                        f[k] = mp == -INFINITY ? 0.f : fast_exp2(mp - mx);
                        float zs = f[k] * zp;
#pragma unroll
                        for (int d = 16; d; d >>= 1) zs += __shfl_xor_sync(kFull, zs, d);
                        z[k] = z[k] * old + zs;
                        acc[k] = make_float4(acc[k].x * old, acc[k].y * old, acc[k].z * old, acc[k].w * old);
                        m[k] = mx;
                    }
                    const int n = min(32, n_part - c1);
                    constexpr int kBatch = 16 / kMine;   // parts under way together (a divisor of 32)
#pragma unroll 1
                    for (int c = 0; c < n; c += kBatch) {
                        float4 o[kBatch][kMine];
#pragma unroll
                        for (int u = 0; u < kBatch; ++u) {
                            const int at = c1 + c + u;
                            const float* from = p.part + (size_t)(at == 0 ? line.slot0 : (line.c0 + at) * 2) * kPart;
#pragma unroll
                            for (int k = 0; k < kMine; ++k)
                                o[u][k] = c + u < n ? __ldcg(reinterpret_cast<const float4*>(from + (warp + k * W) * kHeadDim) + lane)
                                                    : make_float4(0.f, 0.f, 0.f, 0.f);
                        }
#pragma unroll
                        for (int u = 0; u < kBatch; ++u)
#pragma unroll
                            for (int k = 0; k < kMine; ++k) {
                                const float w = __shfl_sync(kFull, f[k], c + u);   // (0 past the last part)
                                acc[k].x += w * o[u][k].x;
                                acc[k].y += w * o[u][k].y;
                                acc[k].z += w * o[u][k].z;
                                acc[k].w += w * o[u][k].w;
                            }
                    }
                }
#pragma unroll
                for (int k = 0; k < kMine; ++k)
                    if (r0 + warp + k * W < p.R) write_row<E2M1, SHAPED>(p, seq, b, h, r0 + warp + k * W, acc[k], m[k], z[k]);
            }
        }
        __syncthreads();   // shared memory is free for the next piece
    }
}

template <bool B>
struct Flag {
    static constexpr bool value = B;
};
constexpr int kImpWarps = 4;
__host__ __device__ constexpr int imp_stages(bool e2m1) { return e2m1 ? 2 : 3; }   // units in a warp's ring
__host__ __device__ constexpr int imp_ctas(bool e2m1) { return e2m1 ? 3 : 4; }   // per SM (registers)

// Importance.  4 bits: bound by latency, 3 warps a scheduler issuing in 43% of the cycles (4 x 32768 rows, 49 MB, 32 query
// rows: 28.8 us, whose 13 M instructions would issue in 13.5; 4 query rows: 18.0; 2 CTAs an SM instead of 3: 28.8 and 21.2).
// bf16: by bytes and the start (8 x 4864 rows, 2 query rows: 11.7 us for 46 MB; rings of 2 units instead of 3: 11.9 us, of 4,
// with fewer CTAs: 15.8 us).  Pieces are (sequence, KV head)s; the
// query fragments of a piece lie in shared memory as the products want them, and each of them serves a unit of tiles
// at a time.  Rows of the fragments that add nothing -- beyond the last query row, or with an lse of -inf, whatever the
// query holds -- are zeros with a factor of 2^-inf.  Beside finite keys that is enough; tiles with an edge, and those whose
// sums come out as NaN, leave such rows out one by one.
template <bool E2M1>
__global__ void __launch_bounds__(32 * kImpWarps, imp_ctas(E2M1)) paged_importance_kernel(const PagedAttnParams p)
{
    constexpr int U = E2M1 ? 2 : 1, W = kImpWarps, kImpStages = imp_stages(E2M1);
    using S = Slot<E2M1, false, U>;
    extern __shared__ __align__(128) uint4 sq[];     // [8-row tile][4][32], then the warps' rings
    __shared__ float4 sf[kMaxRows / 2];              // of two rows each: factor of the logits, minus the lse (base 2)
    static_assert(alignof(decltype(sf)) == 16, "two rows are read at a time");
    __shared__ LineSmem<W> sm_line;
    griddep_wait();
    griddep_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int nq = (p.R + 7) / 8, n_cand = p.cand_hi - p.cand_lo;
    const uint32_t ring = smem_addr(sq + nq * 128) + warp * kImpStages * S::kBytes, ring_end = ring + kImpStages * S::kBytes;
    const int base = p.cand_lo & ~(2 * kTileRows - 1);                       // first row of the first tile
    auto tiles = [&](const Seq& q) { return max((min(q.len, p.cand_hi) - base + kTileRows - 1) / kTileRows, 1); };
    Line<W, decltype(tiles)> line(p, tiles, p.c.Hkv, importance_cost(E2M1));
    if (!line.start(sm_line)) return;

    while (line.next()) {
        const int b = line.b, h = line.piece;
        Seq seq = line.seq;
        seq.lo = base;
        const int seen = seq.len - p.Mq, stop = min(seq.len, p.cand_hi);
        Feeder<E2M1, false, U> feeder(p, seq, h, warp_start<U, W>(seq, line.s0, line.s1, warp),
                                      warp_start<U, W>(seq, line.s0, line.s1, warp + 1));
        // the ring's first units go on their way, then each turn feeds the unit kImpStages - 1 turns ahead
        uint32_t flags[kImpStages];      // of the units in the ring, oldest first, and their first rows
        int first[kImpStages + 1];
#pragma unroll
        for (int k = 0; k < kImpStages - 1; ++k) {
            first[k] = base + feeder.it * kTileRows;
            flags[k] = feeder.feed(ring + k * S::kBytes);
        }
        first[kImpStages - 1] = base + feeder.it * kTileRows;
        for (int n = warp; n < nq; n += W) {
            const int r = 8 * n + g;
            uint32_t q[16];
            fetch_query<E2M1>(r < p.R ? query_row(p, b, h, r) : nullptr, q);
            const float z = r < p.R ? p.lse[((int64_t)b * p.Hq + h * p.G + r / p.Mq) * p.Mq + r % p.Mq] : -INFINITY;
            if (z == -INFINITY) {
#pragma unroll
                for (int j = 0; j < 16; ++j) q[j] = 0;
            }
            const float f = make_query<E2M1>(q);
#pragma unroll
            for (int j = 0; j < 4; ++j) sq[(n * 4 + j) * 32 + lane] = make_uint4(q[4 * j], q[4 * j + 1], q[4 * j + 2], q[4 * j + 3]);
            if (t == 0) reinterpret_cast<float2*>(sf)[r] = make_float2(p.qscale * f, z == -INFINITY ? z : z * -1.4426950408889634f);
        }
        __syncthreads();
        float* out = p.scores + ((int64_t)b * p.c.Hkv + h) * n_cand - p.cand_lo;
        uint32_t slot = ring, into = ring + (kImpStages - 1) * S::kBytes;
        while (flags[0] >> U) {
            cp_async_wait_stages<kImpStages - 1>();   // this lane's copies of the unit; the barrier covers the others'
            __syncwarp();
            flags[kImpStages - 1] = feeder.feed(into);
            first[kImpStages] = base + feeder.it * kTileRows;
            const uint32_t edges = flags[0] & ((1u << U) - 1);
            uint32_t a[U][4][2][4];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                KTile<E2M1> k;
                k.template load<S>(slot, u);
#pragma unroll
                for (int j = 0; j < 4; ++j) k.pair(j, a[u][j]);
            }
            int pos[U][2];   // of the tile's rows g, g + 8
#pragma unroll
            for (int u = 0; u < U; ++u) {
                pos[u][0] = pos[u][1] = 0;
                if ((edges >> (U - 1 - u)) & 1u) {
                    pos[u][0] = (int)lds32(slot + S::kPos + 64 * u + 4 * g);
                    pos[u][1] = (int)lds32(slot + S::kPos + 64 * u + 32 + 4 * g);
                }
            }
            float sum[U][2] = {};
            auto add = [&](auto masked) {
                constexpr bool MASKED = decltype(masked)::value;
#pragma unroll 1
                for (int n = 0; n < nq; ++n) {
                    float s[U][2][4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint4 q = sq[(n * 4 + j) * 32 + lane];
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            const uint32_t(&x)[4] = a[u][j][0], (&y)[4] = a[u][j][1];
                            if (j == 0) {
                                mma16_zero<E2M1>(s[u][0], x[0], x[1], x[2], x[3], q.x, q.y);
                                mma16_zero<E2M1>(s[u][1], y[0], y[1], y[2], y[3], q.z, q.w);
                            } else {
                                mma16<E2M1>(s[u][0], x[0], x[1], x[2], x[3], q.x, q.y);
                                mma16<E2M1>(s[u][1], y[0], y[1], y[2], y[3], q.z, q.w);
                            }
                        }
                    }
                    const float4 f = sf[4 * n + t];   // rows 2t, 2t + 1
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float x = fmaf(s[u][0][e] + s[u][1][e], e & 1 ? f.z : f.x, e & 1 ? f.w : f.y);
                            if (MASKED) {
                                const int row = pos[u][e >> 1];
                                if (row < 0 || row > seen + query_pos(p, 8 * n + 2 * t + (e & 1)) || (e & 1 ? f.w : f.y) == -INFINITY)
                                    x = -INFINITY;
                            }
                            sum[u][e >> 1] += fast_exp2(x);
                        }
                }
            };
            bool apart = edges != 0;
            if (!apart) {
                add(Flag<false>());
                // 0 times a key's infinity or NaN is NaN: such a sum is formed again from the query rows that count
                bool bad = false;
#pragma unroll
                for (int u = 0; u < U; ++u) bad |= sum[u][0] != sum[u][0] || sum[u][1] != sum[u][1];
                apart = __any_sync(kFull, bad);
                if (apart) {
#pragma unroll
                    for (int u = 0; u < U; ++u) sum[u][0] = sum[u][1] = 0.f;
                }
            }
            if (apart) add(Flag<true>());
#pragma unroll
            for (int u = 0; u < U; ++u) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    sum[u][e] += __shfl_xor_sync(kFull, sum[u][e], 1);
                    sum[u][e] += __shfl_xor_sync(kFull, sum[u][e], 2);
                }
                // (a tile of the unit that does not exist starts at or past `stop`, or the next unit writes it)
                const int row = first[0] + u * kTileRows + g + 8 * t;
                const bool mine = u == 0 || !((edges >> (U - 1 - u)) & 1u) || first[0] + u * kTileRows < first[1];
                if (t < 2 && mine && row >= p.cand_lo && row < stop) out[row] = t ? sum[u][1] : sum[u][0];
            }
            into = slot;
            slot = slot + S::kBytes == ring_end ? ring : slot + S::kBytes;
#pragma unroll
            for (int k = 0; k < kImpStages; ++k) first[k] = first[k + 1];
#pragma unroll
            for (int k = 0; k < kImpStages - 1; ++k) flags[k] = flags[k + 1];
        }
        cp_async_wait_all_groups();
        // the candidates past the end: the piece's CTAs share them
        for (int64_t r = (int64_t)max(seq.len, p.cand_lo) + line.part * (32 * W) + threadIdx.x; r < p.cand_hi; r += line.n_part * (32 * W))
            out[r] = 0.f;
        __syncthreads();   // the query fragments and the rings are free for the next piece
    }
}

// Raises a kernel's dynamic shared memory limit, once a device (a runtime call of about a microsecond).
template <typename K>
cudaError_t allow_smem(K* kernel, size_t bytes, std::atomic<uint64_t>& done)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

template <bool E2M1, int NT, bool DUP, int U, int SHAPED>
cudaError_t launch_decode(const PagedAttnParams& p, int sm_count, bool pdl, cudaStream_t s)
{
    using S = Shape<E2M1, NT, DUP, U>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(paged_decode_kernel<E2M1, NT, DUP, U, SHAPED>, S::kSmem, done);
    if (e != cudaSuccess) return e;
    return launch_kernel(paged_decode_kernel<E2M1, NT, DUP, U, SHAPED>, dim3(S::kCtas * sm_count), dim3(32 * S::kWarps), S::kSmem, s,
                         pdl, 0u, p);
}

// The kernel for a call's query rows.
template <int SHAPED>
cudaError_t launch_decode_bf16(const PagedAttnParams& p, int sm_count, bool pdl, cudaStream_t s)
{
    if (p.R <= 4) return launch_decode<false, 1, true, 1, SHAPED>(p, sm_count, pdl, s);
    if (p.R <= 8) return launch_decode<false, 1, false, 1, SHAPED>(p, sm_count, pdl, s);
    return launch_decode<false, 2, false, 1, SHAPED>(p, sm_count, pdl, s);
}
template <int SHAPED>
cudaError_t launch_decode_e2m1(const PagedAttnParams& p, int sm_count, bool pdl, cudaStream_t s)
{
    if (p.R > 8) return launch_decode<true, 2, false, 2, SHAPED>(p, sm_count, pdl, s);
    // tiles a warp may get, if every sequence fills its pages
    const int64_t most = (int64_t)p.c.B * p.c.Hkv * ((p.c.cap + p.kk) / kTileRows) / (12 * sm_count);
    if (most <= kShort || p.c.page_mask < 2 * kTileRows - 1)
        return p.R <= 4 ? launch_decode<true, 1, true, 1, SHAPED>(p, sm_count, pdl, s)
                        : launch_decode<true, 1, false, 1, SHAPED>(p, sm_count, pdl, s);
    return p.R <= 4 ? launch_decode<true, 1, true, 2, SHAPED>(p, sm_count, pdl, s)
                    : launch_decode<true, 1, false, 2, SHAPED>(p, sm_count, pdl, s);
}

}  // namespace
}  // namespace fx
