// The 4-bit K/V pool: its layout, its number formats, and the page-table reads of the
// attention calls over it.
//
// A block of 16 head dims of one row is 16 e2m1 codes and one e4m3 scale s; with the kv
// head's fp32 scale g its values are code * s * g.  code * s has at most 2 + 4 significant
// bits and lies within 2^-10 .. 2688, so it is exact in fp16 and in bf16: attention
// multiplies it on the 16-bit tensor cores without rounding and applies g in fp32 (K's to
// the scores, V's to the output).
//
// A tile is t = min(page_size, 64) consecutive slots of one kv head, laid out as K codes
// [t][D/2], V codes [t][D/2], K scales [t][D/16], V scales [t][D/16] and rounded up to 16
// bytes (only t = 1, D = 64 needs it): everything attention reads of a page is one
// contiguous, 16-byte aligned piece that one bulk copy fetches (9216 bytes for 64 keys of
// 128 dims), and DRAM sees whole runs of it instead of 64-byte rows.
#pragma once

#include <cuda_fp16.h>

#include "pkv_internal.cuh"

namespace pkv {
namespace quant {

constexpr int kBlock = 16;      // head dims that share a scale
constexpr int kMaxTile = 64;    // slots per tile at most
constexpr uint8_t kMostScale = 0x7e;  // e4m3 448: the largest, and what larger ones saturate to
constexpr uint8_t kNanScale = 0x7f;   // e4m3 NaN: a block that held an infinity or a NaN

constexpr int tile_bytes(int t, int d) { return (t * d * 9 / 8 + 15) / 16 * 16; }

// ---------------------------------------------------------------- formats
// Eight e2m1 codes (one 32-bit word, the even element of a pair in the low half of its
// byte) as four fp16 pairs.
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
        " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
        " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}
// Two e4m3 scales (low byte first) as an fp16 pair.
__device__ __forceinline__ uint32_t scales_to_f16(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
    return h;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ float2 f16x2_to_f32(uint32_t h) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}
// e2m1 codes of two floats (to nearest, ties to even, at most 6), `lo` in the low half.
__device__ __forceinline__ uint32_t pair_to_codes(float lo, float hi) {
    uint32_t r;
    asm("{\n .reg .b8 b;\n cvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n cvt.u32.u8 %0, b;\n}\n"
        : "=r"(r)
        : "f"(hi), "f"(lo));
    return r;
}
// e4m3 of a non-negative float (to nearest, ties to even, at most 448).
__device__ __forceinline__ uint32_t float_to_scale(float x) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(0.f), "f"(x));
    return r;
}
// 32 bytes in one access (a whole sector per thread).
__device__ __forceinline__ void load_32(const void *p, uint32_t (&w)[8]) {
    asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
}
__device__ __forceinline__ void store_32(void *p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// A head scale is a positive finite number.
__device__ __forceinline__ bool good_scale(float g) { return g > 0.f && g <= 3.402823466e38f; }

// ---------------------------------------------------------------- page tables
// Where a request's keys are: the fields of the three layouts (see pkv_layout).
struct Table {
    int32_t layout, ps_shift, ps_mask, bt_width, max_len;
    int64_t num_pages, kv_indices_len;
    const int32_t *kv_indptr, *kv_indices, *kv_last, *block_table, *seq_lens;
    const int32_t *r2t, *req_pool_idx, *kv_start;
    int64_t r2t_rows, r2t_stride, r2t_width;
};

// Keys of request b (0 for malformed inputs) and the base its slot_of() takes; the
// flags are raised only with `report`.
__device__ __forceinline__ int key_count(const Table &p, int b, int64_t &base, int32_t *err, bool report) {
    int64_t L, cap;
    if (p.layout == PKV_LAYOUT_CSR) {
        const int64_t lo = p.kv_indptr[b], hi = p.kv_indptr[b + 1], n = hi - lo;
        const int last = n > 0 && lo >= 0 && hi <= p.kv_indices_len ? p.kv_last[b] : 0;
        base = lo;
        if (lo < 0 || n < 0 || hi > p.kv_indices_len || (n > 0 && (last < 1 || last > p.ps_mask + 1))) {
            if (report) raise_flag(err, PKV_DEVERR_RANGE);
            base = 0;
            return 0;
        }
        L = n > 0 ? ((n - 1) << p.ps_shift) + last : 0;
        cap = L;
    } else if (p.layout == PKV_LAYOUT_REQ_TO_TOKEN) {
        const int64_t row = p.req_pool_idx[b], st = p.kv_start ? p.kv_start[b] : 0;
        L = p.seq_lens[b];
        if (row < 0 || row >= p.r2t_rows || st < 0 || (st & p.ps_mask) || L < 0 || st + L > p.r2t_width) {
            if (report) raise_flag(err, PKV_DEVERR_RANGE);
            base = 0;
            return 0;
        }
        base = row * p.r2t_stride + st;
        cap = L;
    } else {
        base = static_cast<int64_t>(b) * p.bt_width;
        L = p.seq_lens[b];
        cap = static_cast<int64_t>(p.bt_width) << p.ps_shift;
    }
    const int64_t limit = min(cap, static_cast<int64_t>(p.max_len));
    if (L < 0 || L > limit) {
        if (report) raise_flag(err, L < 0 ? PKV_DEVERR_RANGE : PKV_DEVERR_CAPACITY);
        L = L < 0 ? 0 : limit;
    }
    return static_cast<int>(L);
}

// Pool slot of key t: -1 when its page lies outside the pool, -2 when the token table
// gives a page start that is not a multiple of the page size.
__device__ __forceinline__ int64_t slot_of(const Table &p, int64_t base, int t) {
    if (p.layout == PKV_LAYOUT_REQ_TO_TOKEN) {
        const int64_t first = __ldg(p.r2t + base + (t & ~p.ps_mask));
        if (first < 0 || first >= (p.num_pages << p.ps_shift)) return -1;
        if (first & p.ps_mask) return -2;
        return first + (t & p.ps_mask);
    }
    const int32_t *tab = p.layout == PKV_LAYOUT_CSR ? p.kv_indices : p.block_table;
    const int64_t page = __ldg(tab + base + (t >> p.ps_shift));
    if (page < 0 || page >= p.num_pages) return -1;
    return (page << p.ps_shift) + (t & p.ps_mask);
}

}  // namespace quant
}  // namespace pkv
