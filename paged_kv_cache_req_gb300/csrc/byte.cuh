// The 8-bit K/V pool: its layout and number formats.
//
// A tile is t = min(page_size, 64) consecutive slots: for each kv head K codes [t][D] and V
// codes [t][D] (e4m3), then for each kv head the bytes E of K and of V; their scales are
// 2^(E - 127).  The codes of a kv head are one piece of whole lines that one bulk copy
// fetches, and the scale bytes lie behind all of them so that they shift none.
//
// The scale is a power of two: e4m3 keeps its four bits over 15 octaves, so a finer scale
// gains nothing, and a scale that grows when a larger row joins the block changes the codes
// that are there in their exponent only.
#pragma once

#include "quant.cuh"

namespace pkv {
namespace byte {

__host__ __device__ constexpr int64_t codes_bytes(int t, int d, int64_t hkv) { return hkv * 2 * t * d; }
__host__ __device__ constexpr int64_t tile_bytes(int t, int d, int64_t hkv) {
    const int pad = t >= 16 ? 128 : 32;
    return codes_bytes(t, d, hkv) + (2 * hkv + pad - 1) / pad * pad;
}

// Two e4m3 codes (low byte first) as an fp16 pair; the low and the high half of a word.
__device__ __forceinline__ uint32_t lo_to_f16(uint32_t w) { return quant::scales_to_f16(w & 0xffff); }
__device__ __forceinline__ uint32_t hi_to_f16(uint32_t w) { return quant::scales_to_f16(w >> 16); }
// e4m3 codes of two floats (to nearest, ties to even, at most 448; NaN stays), `lo` in the low byte.
__device__ __forceinline__ uint32_t pair_to_codes(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// Bytes of a word that are NaN codes, as a mask.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu); }
// E of a block whose largest finite magnitude has the bf16 bits `top` (sign bit clear): 448 = 1.75 x 2^8,
// so the exponent less 8, one more where the fraction is above 1.75.
__device__ __forceinline__ uint32_t scale_of(uint32_t top) { return max(1, static_cast<int>((top + 0x1f) >> 7) - 8); }
__device__ __forceinline__ float scale_value(uint32_t e) { return __uint_as_float(e << 23); }   // 2^(E - 127)

}  // namespace byte
}  // namespace pkv
