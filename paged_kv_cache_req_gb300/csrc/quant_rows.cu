// Rows of the 4-bit pool: pkv_quant_store (quantise new K/V rows into their slots) and
// pkv_quant_gather (read a batch's rows back as bf16).
#include <algorithm>

#include "quant.cuh"

namespace pkv {
namespace quant {
namespace {

constexpr int kThreads = 256;

// 16 bf16 elements at p as 8 packed words.
template <bool kVec>
__device__ __forceinline__ void load_block(const uint16_t *__restrict__ p, uint32_t (&w)[8]) {
    if (kVec) {
        const uint4 a = ld_stream_16(p), b = ld_stream_16(p + 8);
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i] = static_cast<uint32_t>(p[2 * i]) | (static_cast<uint32_t>(p[2 * i + 1]) << 16);
    }
}

// One block of 16 elements: s = e4m3(amax / (6 g)), codes e2m1(x / (s g)), in fp32 with
// IEEE division, so that a quotient on a border between two codes is decided by the tie
// rule and not by a reciprocal's rounding.  The largest magnitude is found on the bf16
// bits (they order like the numbers, infinities and NaN last).
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
    uint32_t c[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        c[i >> 2] |= pair_to_codes(__fdiv_rn(bf16_lo(w[i]), den), __fdiv_rn(bf16_hi(w[i]), den)) << (8 * (i & 3));
    return make_uint2(c[0], c[1]);
}

// One thread per block of 16 dims of a K or V row.
template <int D, bool kVec>
__global__ void __launch_bounds__(kThreads)
store_kernel(uint8_t *__restrict__ pool, int64_t num_slots, int64_t tile_stride, int t_shift, int32_t hkv,
             const float *__restrict__ k_scale, const float *__restrict__ v_scale,
             const uint16_t *__restrict__ k_new, const uint16_t *__restrict__ v_new, int64_t k_stride,
             int64_t v_stride, const int32_t *__restrict__ slot_mapping, int64_t blocks, int32_t *__restrict__ err) {
    pdl_wait();          // inputs may come from the previous kernel of the stream
    pdl_launch_next();
    constexpr int kPerRow = D / kBlock;
    const int64_t e = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (e >= blocks) return;
    const int j = static_cast<int>(e % kPerRow);
    const int64_t r = e / kPerRow;
    const int kh = static_cast<int>(r % hkv);
    const bool is_v = (r / hkv) & 1;
    const int64_t i = r / hkv / 2;
    const int64_t slot = slot_mapping[i];
    if (slot < 0) return;   // padded token
    const float *scales = is_v ? v_scale : k_scale;
    const float g = scales ? scales[kh] : 1.f;
    if (slot >= num_slots || !good_scale(g)) {
        if (j == 0) raise_flag(err, PKV_DEVERR_RANGE);
        return;
    }
    uint32_t w[8];
    load_block<kVec>((is_v ? v_new + i * v_stride : k_new + i * k_stride) + static_cast<int64_t>(kh) * D + j * kBlock, w);
    uint32_t scale;
    const uint2 codes = quantise(w, g, scale);
    const int t = 1 << t_shift, at = static_cast<int>(slot & (t - 1));
    uint8_t *tile = pool + (slot >> t_shift) * tile_stride + static_cast<int64_t>(kh) * tile_bytes(t, D);
    *reinterpret_cast<uint2 *>(tile + (is_v ? t * (D / 2) : 0) + at * (D / 2) + j * 8) = codes;
    tile[t * D + (is_v ? t * (D / kBlock) : 0) + at * (D / kBlock) + j] = static_cast<uint8_t>(scale);
}

constexpr int kGatherChunk = kThreads * 8;   // requests per step of the offset scan

// Exclusive block-wide prefix of one value per thread; *total gets the sum.
__device__ __forceinline__ long long block_scan(long long v, long long *warp_sums, long long *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long incl = v;
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    long long before = 0, all = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        const long long x = warp_sums[w];
        if (w < warp) before += x;
        all += x;
    }
    *total = all;
    __syncthreads();
    return before + incl - v;
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
        st_stream_16(dst, make_uint4(o[0], o[1], o[2], o[3]));
        st_stream_16(dst + 8, make_uint4(o[4], o[5], o[6], o[7]));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            dst[2 * i] = static_cast<uint16_t>(o[i]);
            dst[2 * i + 1] = static_cast<uint16_t>(o[i] >> 16);
        }
    }
}

struct GatherParams {
    const uint8_t *pool;
    int64_t num_slots, tile_stride;
    int t_shift;
    int32_t hkv, batch;
    const float *k_scale, *v_scale;
    const int32_t *r2t, *req_pool_idx, *kv_start, *seq_lens;
    int64_t r2t_rows, r2t_stride, r2t_width, splits, cap;
    uint16_t *k_out, *v_out;
    int32_t *cu_seqlens, *err;
};

// Work items (request, split), dealt to a persistent grid in request order; every CTA
// scans the lengths once for its offsets (as pkv_ragged_gather does).  A warp takes a
// token: its lanes the blocks of 16 dims of the token's K and V rows.
template <int D, bool kVec>
__global__ void __launch_bounds__(kThreads) gather_kernel(const GatherParams p) {
    pdl_wait();          // inputs may come from the previous kernel of the stream
    pdl_launch_next();
    __shared__ long long warp_sums[kThreads / 32];
    __shared__ long long off_s[kGatherChunk];
    constexpr int W = kThreads / 32, kPerRow = D / kBlock;
    if (blockIdx.x == 0 && threadIdx.x == 0) p.cu_seqlens[0] = 0;
    if (blockIdx.x == 0 && threadIdx.x < 2) {   // unusable head scales
        const float *g = threadIdx.x ? p.v_scale : p.k_scale;
        for (int h = 0; g && h < p.hkv; ++h)
            if (!good_scale(g[h])) raise_flag(p.err, PKV_DEVERR_RANGE);
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = 1 << p.t_shift;
    const int64_t items = static_cast<int64_t>(p.batch) * p.splits;
    int64_t w = blockIdx.x;
    long long carry = 0;
    for (int c0 = 0; c0 < p.batch && w < items; c0 += kGatherChunk) {
        long long n8[8], mine = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int j = c0 + threadIdx.x * 8 + k;
            n8[k] = j < p.batch ? max(p.seq_lens[j], 0) : 0;
            mine += n8[k];
        }
        long long total = 0;
        long long run = carry + block_scan(mine, warp_sums, &total);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            off_s[threadIdx.x * 8 + k] = run;
            run += n8[k];
        }
        carry += total;
        __syncthreads();
        for (; w < items && w / p.splits < c0 + kGatherChunk; w += gridDim.x) {
            const int b = static_cast<int>(w / p.splits);
            const int64_t y = w % p.splits;
            const long long before = off_s[b - c0];
            const int64_t row = p.req_pool_idx[b], s = p.kv_start ? p.kv_start[b] : 0;
            int64_t L = max(p.seq_lens[b], 0);
            const bool valid = row >= 0 && row < p.r2t_rows && s >= 0 && s + L <= p.r2t_width && p.seq_lens[b] >= 0;
            if (y == 0 && threadIdx.x == 0) {
                p.cu_seqlens[b + 1] = static_cast<int32_t>(before + L);
                if (before + L > p.cap) raise_flag(p.err, PKV_DEVERR_CAPACITY);
                if (!valid) raise_flag(p.err, PKV_DEVERR_RANGE);
            }
            if (before + L > p.cap) L = p.cap > before ? p.cap - before : 0;
            for (int64_t i = y * W + warp; i < L; i += p.splits * W) {
                const int64_t o = before + i;
                int64_t slot = valid ? __ldg(p.r2t + row * p.r2t_stride + s + i) : -1;
                if (slot < 0 || slot >= p.num_slots) {
                    if (valid && lane == 0) raise_flag(p.err, PKV_DEVERR_RANGE);
                    slot = -1;
                }
                const int at = static_cast<int>(slot & (t - 1));
                const uint8_t *base = p.pool + (slot < 0 ? 0 : slot >> p.t_shift) * p.tile_stride;
                for (int e = lane; e < 2 * p.hkv * kPerRow; e += 32) {
                    const int j = e % kPerRow, kh = (e / kPerRow) % p.hkv;
                    const bool is_v = e >= p.hkv * kPerRow;
                    const float *scales = is_v ? p.v_scale : p.k_scale;
                    uint2 codes = make_uint2(0, 0);
                    uint32_t scale = 0;
                    if (slot >= 0) {
                        const uint8_t *tile = base + static_cast<int64_t>(kh) * tile_bytes(t, D);
                        codes = __ldg(reinterpret_cast<const uint2 *>(tile + (is_v ? t * (D / 2) : 0) + at * (D / 2) + j * 8));
                        scale = __ldg(tile + t * D + (is_v ? t * kPerRow : 0) + at * kPerRow + j);
                    }
                    uint16_t *dst = (is_v ? p.v_out : p.k_out) + (o * p.hkv + kh) * D + j * kBlock;
                    write_block<kVec>(dst, codes, scale, scales ? scales[kh] : 1.f);
                }
            }
        }
        __syncthreads();   // off_s is rewritten by the next chunk
    }
}

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
    const bool vec = aligned(kn, 16) && aligned(vn, 16) && k_stride % 8 == 0 && v_stride % 8 == 0;
    const int64_t blocks = static_cast<int64_t>(n) * 2 * hkv * (D / kBlock);
    const int64_t grid = (blocks + kThreads - 1) / kThreads;
    if (grid > INT32_MAX) return fail(PKV_ERR_UNSUPPORTED, "pkv_quant_store: too many rows for one call");
    auto kern = vec ? store_kernel<D, true> : store_kernel<D, false>;
    return launch_status(launch_chained(kern, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, s, pool, num_slots,
                                        tile_stride, t_shift, hkv, ks, vs, kn, vn, k_stride, v_stride, slots, blocks, err),
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
    // enough items for two waves of the device even for a handful of long requests
    const int64_t sms = std::max(1, sm_count()), W = kThreads / 32;
    const int64_t want = 2 * sms * (2048 / kThreads);
    p.splits = (static_cast<int64_t>(max_seq_len) + W * 4 - 1) / (W * 4);
    if (batch > 0) p.splits = std::min<int64_t>(p.splits, std::max<int64_t>(1, (want + batch - 1) / batch));
    p.splits = std::max<int64_t>(1, p.splits);
    const int64_t items = static_cast<int64_t>(std::max(batch, 1)) * p.splits;
    const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(items, 8 * sms));
    const bool vec = aligned(k_out, 16) && aligned(v_out, 16);
    auto *kern = head_dim == 128 ? (vec ? gather_kernel<128, true> : gather_kernel<128, false>)
                                 : (vec ? gather_kernel<64, true> : gather_kernel<64, false>);
    return launch_status(launch_chained(kern, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0,
                                        reinterpret_cast<cudaStream_t>(stream), p),
                         "pkv_quant_gather");
}
