// Rows of the 4-bit pool: pkv_quant_store (quantise new K/V rows into their slots) and
// pkv_quant_gather (read a batch's rows back as bf16).
#include "gather.cuh"

namespace pkv {
namespace quant {
namespace {

// 16 bf16 elements at p as 8 packed words.
template <bool kVec>
__device__ __forceinline__ void load_block(const uint16_t *__restrict__ p, uint32_t (&w)[8]) {
    if (kVec) {
        load_32(p, w);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i] = static_cast<uint32_t>(p[2 * i]) | (static_cast<uint32_t>(p[2 * i + 1]) << 16);
    }
}

// One block of 16 elements: s = e4m3(amax / (6 g)), codes e2m1(x / (s g)) with quotients
// rounded to nearest in fp32, so that one on a border between two codes is decided by the
// tie rule and not by a reciprocal's rounding.  With y = RN(1 / d), q = RN(x y) and the exact
// remainder r = x - q d, RN(q + r y) is the correctly rounded x / d as long as nothing leaves
// the normal range (Markstein 1990): two FMAs for an element instead of a division.  The
// largest magnitude is found on the bf16 bits (they order like the numbers, infinities and
// NaN last).
__device__ __forceinline__ uint2 quantise(const uint32_t (&w)[8], float g, uint32_t &scale) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
    const uint32_t top = max(m & 0xffffu, m >> 16);
    if (top >= 0x7f80u) {
        scale = kNanScale;
        return make_uint2(0, 0);
    }
    scale = float_to_scale(__fdiv_rn(__uint_as_float(top << 16), __fmul_rn(6.f, g)));
    const float den = __fmul_rn(f16x2_to_f32(scales_to_f16(scale)).x, g);
    if (!(den > 0.f)) return make_uint2(0, 0);
    uint32_t c[8];
    if (scale != kMostScale && den > 0x1p-90f && den < 0x1p90f) {
        // (no quotient is above 9 where the scale did not saturate, and an element below 2^-30 den
        // has code 0 whatever its quotient's last bit)
        const float y = __frcp_rn(den);
        auto quotient = [&](float x) {
            const float q = __fmul_rn(x, y);
            return __fmaf_rn(__fmaf_rn(-q, den, x), y, q);
        };
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = pair_to_codes(quotient(bf16_lo(w[i])), quotient(bf16_hi(w[i])));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = pair_to_codes(__fdiv_rn(bf16_lo(w[i]), den), __fdiv_rn(bf16_hi(w[i]), den));
    }
    return make_uint2(c[0] | (c[1] << 8) | (c[2] << 16) | (c[3] << 24), c[4] | (c[5] << 8) | (c[6] << 16) | (c[7] << 24));
}

template <int D, bool kVec>
__global__ void __launch_bounds__(kThreads)
store_kernel(uint8_t *__restrict__ pool, int64_t num_slots, int64_t tile_stride, int t_shift, int32_t hkv,
             const float *__restrict__ k_scale, const float *__restrict__ v_scale,
             const uint16_t *__restrict__ k_new, const uint16_t *__restrict__ v_new, int64_t k_stride,
             int64_t v_stride, const int32_t *__restrict__ slot_mapping, uint32_t n, uint32_t parts, int pack,
             int32_t *__restrict__ err) {
    pdl_wait();          // inputs may come from the previous kernel of the stream
    pdl_launch_next();
    constexpr int kPerRow = D / kBlock;
    const uint32_t item = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), token = item / parts;
    const int part = static_cast<int>(item - token * parts), lane = threadIdx.x & (31 >> pack), j = lane % kPerRow;
    const uint32_t i = (token << pack) + ((threadIdx.x & 31) >> (5 - pack));
    if (i >= n) return;
    const int64_t slot = slot_mapping[i];
    if (slot < 0) return;   // a padded token
    if (slot >= num_slots) {
        if (lane == 0 && part == 0) raise_flag(err, PKV_DEVERR_RANGE);
        return;
    }
    const int t = 1 << t_shift, at = static_cast<int>(slot & (t - 1));
    uint8_t *tile = pool + (slot >> t_shift) * tile_stride;
    const int iters = (2 * hkv * kPerRow + 31) / 32, each = (iters + static_cast<int>(parts) - 1) / static_cast<int>(parts);
    const int end = min(2 * hkv, (part + 1) * each * (32 / kPerRow));
    for (int h = part * each * (32 / kPerRow) + lane / kPerRow; h < end; h += 32 / kPerRow) {
        const bool is_v = h >= hkv;
        const int kh = is_v ? h - hkv : h;
        const float *scales = is_v ? v_scale : k_scale;
        uint32_t w[8];
        load_block<kVec>((is_v ? v_new + i * v_stride : k_new + i * k_stride) + static_cast<int64_t>(kh) * D + j * kBlock, w);
        const float g = scales ? __ldg(scales + kh) : 1.f;
        if (!good_scale(g)) {
            if (j == 0) raise_flag(err, PKV_DEVERR_RANGE);
            continue;
        }
        uint32_t scale;
        const uint2 codes = quantise(w, g, scale);
        uint8_t *piece = tile + static_cast<int64_t>(kh) * tile_bytes(t, D);
        *reinterpret_cast<uint2 *>(piece + (is_v ? t * (D / 2) : 0) + at * (D / 2) + j * 8) = codes;
        piece[t * D + (is_v ? t * kPerRow : 0) + at * kPerRow + j] = static_cast<uint8_t>(scale);
    }
}

// Writes 16 bf16 elements: codes x scale x g, rounded to nearest even.
template <bool kVec>
__device__ __forceinline__ void write_block(uint16_t *__restrict__ dst, uint2 codes, uint32_t scale, float g) {
    const float s = __fmul_rn(f16x2_to_f32(scales_to_f16(scale)).x, g);
    uint32_t h[8], o[8];
    codes_to_f16(codes.x, *reinterpret_cast<uint32_t(*)[4]>(h));
    codes_to_f16(codes.y, *reinterpret_cast<uint32_t(*)[4]>(h + 4));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 c = f16x2_to_f32(h[i]);
        o[i] = pack_bf16x2(c.x * s, c.y * s);
    }
    if (kVec) {
        store_32(dst, o);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            dst[2 * i] = static_cast<uint16_t>(o[i]);
            dst[2 * i + 1] = static_cast<uint16_t>(o[i] >> 16);
        }
    }
}

template <int D>
struct Rows4 {
    static constexpr int kDim = D;
    struct Block {
        uint2 codes;
        uint32_t scale;
    };
    struct Place {
        const uint8_t *code_at, *scale_at;
    };
    __device__ __forceinline__ static Place place(const GatherParams &, const uint8_t *base, int t, int at, int j) {
        return {base + at * (D / 2) + j * 8, base + t * D + at * (D / kBlock) + j};
    }
    __device__ __forceinline__ static Block load(const Place &x, int t, int kh, bool is_v) {
        const int64_t piece = static_cast<int64_t>(kh) * tile_bytes(t, D);
        Block b;
        b.codes = __ldg(reinterpret_cast<const uint2 *>(x.code_at + piece + (is_v ? t * (D / 2) : 0)));
        b.scale = __ldg(x.scale_at + piece + (is_v ? t * (D / kBlock) : 0));
        return b;
    }
    template <bool kVec>
    __device__ __forceinline__ static void write(uint16_t *__restrict__ dst, const Block &b, float g) {
        write_block<kVec>(dst, b.codes, b.scale, g);
    }
};

// The checks that store and gather share.
pkv_status check_pool(const char *who, const void *pool, int64_t num_tiles, int64_t tile_stride, int32_t kv_heads,
                      int32_t head_dim, int32_t page_size) {
    if (num_tiles < 0 || kv_heads < 1) return fail(PKV_ERR_INVALID_ARG, "%s: bad sizes", who);
    if (head_dim != 64 && head_dim != 128) return fail(PKV_ERR_UNSUPPORTED, "%s: head_dim 64 or 128", who);
    if (!is_pow2(page_size) || page_size > 1024)
        return fail(PKV_ERR_UNSUPPORTED, "%s: page_size must be a power of two in [1, 1024]", who);
    const int t = std::min(page_size, kMaxTile);
    if (tile_stride % 16 || tile_stride < static_cast<int64_t>(kv_heads) * tile_bytes(t, head_dim))
        return fail(PKV_ERR_INVALID_ARG, "%s: the tile stride must hold all kv heads and be a multiple of 16 bytes", who);
    if (!aligned(pool, 16)) return fail(PKV_ERR_INVALID_ARG, "%s: the pool must be 16-byte aligned", who);
    return PKV_OK;
}

template <int D>
pkv_status launch_store(uint8_t *pool, int64_t num_slots, int64_t tile_stride, int t_shift, int32_t hkv,
                        const float *ks, const float *vs, const uint16_t *kn, const uint16_t *vn, int64_t k_stride,
                        int64_t v_stride, const int32_t *slots, int32_t n, int32_t *err, cudaStream_t s) {
    const bool vec = aligned(kn, 32) && aligned(vn, 32) && k_stride % 16 == 0 && v_stride % 16 == 0;
    const int pack = row_pack(D, hkv);
    const int64_t parts = row_parts(n, row_iters(D, hkv)), items = ((n + (int64_t{1} << pack) - 1) >> pack) * parts;
    if (items > INT32_MAX) return fail(PKV_ERR_UNSUPPORTED, "pkv_quant_store: too many rows for one call");
    const int64_t grid = (items + kThreads / 32 - 1) / (kThreads / 32);
    auto kern = vec ? store_kernel<D, true> : store_kernel<D, false>;
    return launch_status(launch_chained(kern, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, s, pool, num_slots,
                                        tile_stride, t_shift, hkv, ks, vs, kn, vn, k_stride, v_stride, slots,
                                        static_cast<uint32_t>(n), static_cast<uint32_t>(parts), pack, err),
                         "pkv_quant_store");
}

}  // namespace
}  // namespace quant
}  // namespace pkv

extern "C" size_t pkv_quant_tile_bytes(int32_t page_size, int32_t head_dim) {
    using namespace pkv;
    if (!is_pow2(page_size) || page_size > 1024 || (head_dim != 64 && head_dim != 128)) return 0;
    return static_cast<size_t>(quant::tile_bytes(std::min(page_size, quant::kMaxTile), head_dim));
}

extern "C" pkv_status pkv_quant_store(void *pool, int64_t num_tiles, int64_t tile_stride, int32_t kv_heads,
                                      int32_t head_dim, int32_t page_size, const float *k_scale,
                                      const float *v_scale, const void *k_new, const void *v_new,
                                      int64_t k_token_stride, int64_t v_token_stride, const int32_t *slot_mapping,
                                      int32_t n_tokens, int32_t *err_flags, pkv_stream_t stream) {
    using namespace pkv;
    using namespace pkv::quant;
    if (!err_flags) return fail(PKV_ERR_INVALID_ARG, "pkv_quant_store: err_flags is required");
    if (n_tokens < 0) return fail(PKV_ERR_INVALID_ARG, "pkv_quant_store: bad sizes");
    const pkv_status st = check_pool("pkv_quant_store", pool, num_tiles, tile_stride, kv_heads, head_dim, page_size);
    if (st != PKV_OK) return st;
    const int64_t row = static_cast<int64_t>(kv_heads) * head_dim;
    if (k_token_stride < row || v_token_stride < row)
        return fail(PKV_ERR_INVALID_ARG, "pkv_quant_store: token stride smaller than a token's rows");
    if (n_tokens == 0) return ok();
    if (!pool || !k_new || !v_new || !slot_mapping) return fail(PKV_ERR_INVALID_ARG, "pkv_quant_store: null pointer");
    const int t_shift = ilog2(std::min(page_size, kMaxTile));
    auto *launch = head_dim == 128 ? launch_store<128> : launch_store<64>;
    return launch(static_cast<uint8_t *>(pool), num_tiles << t_shift, tile_stride, t_shift, kv_heads, k_scale, v_scale,
                  static_cast<const uint16_t *>(k_new), static_cast<const uint16_t *>(v_new), k_token_stride,
                  v_token_stride, slot_mapping, n_tokens, err_flags, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" pkv_status pkv_quant_gather(const void *pool, int64_t num_tiles, int64_t tile_stride, int32_t kv_heads,
                                       int32_t head_dim, int32_t page_size, const float *k_scale,
                                       const float *v_scale, const int32_t *req_to_token, int64_t r2t_rows,
                                       int64_t r2t_row_stride, int64_t r2t_width, const int32_t *req_pool_idx,
                                       const int32_t *kv_start, const int32_t *seq_lens, int32_t batch,
                                       int32_t max_seq_len, void *k_out, void *v_out, int64_t out_rows_cap,
                                       int32_t *cu_seqlens, int32_t *err_flags, pkv_stream_t stream) {
    using namespace pkv;
    using namespace pkv::quant;
    if (!err_flags || !cu_seqlens) return fail(PKV_ERR_INVALID_ARG, "pkv_quant_gather: null err_flags/cu_seqlens");
    if (batch < 0 || r2t_rows < 0 || r2t_width < 0 || r2t_row_stride < r2t_width || out_rows_cap < 0 || max_seq_len < 0)
        return fail(PKV_ERR_INVALID_ARG, "pkv_quant_gather: bad sizes");
    const pkv_status st = check_pool("pkv_quant_gather", pool, num_tiles, tile_stride, kv_heads, head_dim, page_size);
    if (st != PKV_OK) return st;
    if (batch > 0 && (!pool || !k_out || !v_out || !req_to_token || !req_pool_idx || !seq_lens))
        return fail(PKV_ERR_INVALID_ARG, "pkv_quant_gather: null pointer");
    GatherParams p{};
    p.pool = static_cast<const uint8_t *>(pool);
    p.t_shift = ilog2(std::min(page_size, kMaxTile));
    p.num_slots = num_tiles << p.t_shift;
    p.tile_stride = tile_stride;
    p.hkv = kv_heads;
    p.batch = batch;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.r2t = req_to_token;
    p.req_pool_idx = req_pool_idx;
    p.kv_start = kv_start;
    p.seq_lens = seq_lens;
    p.r2t_rows = r2t_rows;
    p.r2t_stride = r2t_row_stride;
    p.r2t_width = r2t_width;
    p.cap = out_rows_cap;
    p.k_out = static_cast<uint16_t *>(k_out);
    p.v_out = static_cast<uint16_t *>(v_out);
    p.cu_seqlens = cu_seqlens;
    p.err = err_flags;
    return gather<Rows4>("pkv_quant_gather", p, head_dim, max_seq_len, reinterpret_cast<cudaStream_t>(stream));
}
