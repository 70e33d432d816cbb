// Rows of the 4-bit pool: pkv_quant_store (quantise new K/V rows into their slots) and
// pkv_quant_gather (read a batch's rows back as bf16).
#include <algorithm>
#include <type_traits>

#include "quant.cuh"

namespace pkv {
namespace quant {
namespace {

constexpr int kThreads = 256;

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

// Both kernels give a lane one block of 16 dims and a warp 32 neighbouring blocks of one token
// (its K rows head by head, then its V rows): 1 KB of bf16 in one run, which is where most of
// the bytes are.  (A warp that takes the same row of 4 or 8 tokens instead has the pool's
// codes in one run and bf16 in pieces of 128 or 256 bytes: 3 to 7 % slower.)  A token is
// `iters` such steps; few tokens are cut into `parts` of them so that every SM has some.
//
// Both are bound by memory, the conversions next (ALU half busy).  Stored and read back: 86,000
// tokens x 20 heads of 64 (1.13 GB in all) 210 us, 5.4 TB/s; 8192 x 8 heads of 128 (86 MB) 24 us.
__host__ __device__ inline int row_iters(int head_dim, int hkv) { return (2 * hkv * (head_dim / kBlock) + 31) / 32; }
// log2 of the tokens that share a warp, where a token has half a warp's blocks or fewer (one kv
// head, or two of 64 dims): 262,144 tokens of one head of 128 read back 77 us with one to a
// warp, 44 with two; of 64, 77 and 24 us with four.
inline int row_pack(int head_dim, int hkv) {
    const int blocks = 2 * hkv * (head_dim / kBlock);
    return blocks < 32 && is_pow2(blocks) ? 5 - ilog2(blocks) : 0;
}
inline int64_t row_parts(int64_t tokens, int iters) {
    const int64_t want = 48ll * std::max(1, sm_count());   // warps that the device holds
    return std::max<int64_t>(1, std::min<int64_t>(iters, want / std::max<int64_t>(1, tokens)));
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
        store_32(dst, o);
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
    int64_t r2t_rows, r2t_stride, r2t_width, cap;
    int32_t parts, pack;
    uint16_t *k_out, *v_out;
    int32_t *cu_seqlens, *err;
};

// The batch's tokens (and parts), in order, are dealt to the warps of a persistent grid,
// whatever the requests' lengths; every CTA scans the lengths for the offsets (2048 requests
// at a time, as pkv_ragged_gather does) and a warp finds its token's request in them.  The
// writes of bf16 bound it: 3.6 times the bytes that it reads, at the 4.0 TB/s at which plain fills
// of memory ran (copies: 6.8).  96,000 tokens x 20 heads of 64 (492 MB written) 120 us, 4.1 TB/s of
// writes; 15,700 x 8 heads of 128 (65 MB of 82) 21 us.
constexpr int kGatherCtas = 5;   // per SM

// kTokens: a warp takes two whole tokens in turn (neighbours share the sectors of their scales);
// kPacked: so do the lanes of it that a small token needs; kParts: one part of one token.
enum { kParts, kTokens, kPacked };
template <int D, bool kVec, int kMode>
__global__ void __launch_bounds__(kThreads, kGatherCtas) gather_kernel(const GatherParams p) {
    pdl_wait();          // inputs may come from the previous kernel of the stream
    pdl_launch_next();
    __shared__ long long warp_sums[kThreads / 32];
    __shared__ long long off_s[kGatherChunk + 1];
    __shared__ long long row_s[kGatherChunk];   // offset of the request's first column in the table; -1: malformed
    constexpr int kPerRow = D / kBlock;
    constexpr bool kWhole = kMode != kParts;
    const int pack = kMode == kPacked ? p.pack : 0;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & (31 >> pack);   // (of those that share a token)
    const bool first = blockIdx.x == 0;
    if (first && threadIdx.x == 0) p.cu_seqlens[0] = 0;
    if (first && warp < 2) {   // unusable head scales
        const float *g = warp ? p.v_scale : p.k_scale;
        for (int h = threadIdx.x & 31; g && h < p.hkv; h += 32)
            if (!good_scale(g[h])) raise_flag(p.err, PKV_DEVERR_RANGE);
    }
    const int t = 1 << p.t_shift;
    long long carry = 0;
    for (int c0 = 0; c0 < p.batch; c0 += kGatherChunk) {
        const int nreq = min(kGatherChunk, p.batch - c0);
        const int per = (nreq + kThreads - 1) / kThreads, j0 = min(nreq, static_cast<int>(threadIdx.x) * per);
        const int j1 = min(nreq, j0 + per);
        long long mine = 0;
        for (int j = j0; j < j1; ++j) {
            const int b = c0 + j;
            const int64_t n = p.seq_lens[b], row = p.req_pool_idx[b], s = p.kv_start ? p.kv_start[b] : 0;
            const bool ok = n >= 0 && row >= 0 && row < p.r2t_rows && s >= 0 && s + n <= p.r2t_width;
            if (first && !ok) raise_flag(p.err, PKV_DEVERR_RANGE);
            row_s[j] = ok ? row * p.r2t_stride + s : -1;
            off_s[j + 1] = max(n, static_cast<int64_t>(0));
            mine += off_s[j + 1];
        }
        long long total = 0;
        long long run = block_scan(mine, warp_sums, &total);
        for (int j = j0; j < j1; ++j) {   // (entry j0 belongs to the thread before)
            run += off_s[j + 1];
            off_s[j + 1] = run;
            if (first) {
                p.cu_seqlens[c0 + j + 1] = static_cast<int32_t>(carry + run);
                if (carry + run > p.cap) raise_flag(p.err, PKV_DEVERR_CAPACITY);
            }
        }
        if (threadIdx.x == 0) off_s[0] = 0;
        __syncthreads();
        // (row numbers fit cu_seqlens' int32)
        const int tokens = static_cast<int>(min(min(total, max(p.cap - carry, 0ll)), static_cast<long long>(INT32_MAX)));
        const int j = lane % kPerRow, each = (row_iters(D, p.hkv) + p.parts - 1) / p.parts * (32 / kPerRow);
        const int sub = (threadIdx.x & 31) >> (5 - pack);
        const int mine0 = blockIdx.x * (kThreads / 32) + warp, warps = gridDim.x * (kThreads / 32);
        for (int64_t w = mine0; w < (kWhole ? ((static_cast<int64_t>(tokens) + 1) / 2 + (1 << pack) - 1) >> pack : static_cast<int64_t>(tokens) * p.parts);
             w += warps) {
            const int g0 = static_cast<int>(kWhole ? 2 * ((w << pack) + sub) : w / p.parts);
            const int h0 = kWhole ? 0 : static_cast<int>(w - static_cast<int64_t>(g0) * p.parts) * each;
            const int h1 = kWhole ? 2 * p.hkv : min(2 * p.hkv, h0 + each);
            int b = 0;
            for (int hi = nreq; hi - b > 1;) {   // the last request that starts at or before the token
                const int mid = (b + hi) >> 1;
                if (off_s[mid] <= g0) b = mid; else hi = mid;
            }
            for (int g = g0; g < (kWhole ? min(tokens, g0 + 2) : g0 + 1); ++g) {
                while (off_s[b + 1] <= g) ++b;
                const int64_t row = row_s[b], o = carry + g;
                int64_t slot = row >= 0 ? __ldg(p.r2t + row + (g - off_s[b])) : -1;
                if (slot < 0 || slot >= p.num_slots) {
                    if (row >= 0 && lane == 0) raise_flag(p.err, PKV_DEVERR_RANGE);
                    slot = -1;
                }
                const int at = static_cast<int>(slot & (t - 1));
                const uint8_t *base = p.pool + (slot < 0 ? 0 : slot >> p.t_shift) * p.tile_stride;
                const uint8_t *code_at = base + at * (D / 2) + j * 8, *scale_at = base + t * D + at * kPerRow + j;
#pragma unroll 4
                for (int h = h0 + lane / kPerRow; h < h1; h += 32 / kPerRow) {
                    const bool is_v = h >= p.hkv;
                    const int kh = is_v ? h - p.hkv : h;
                    const float *scales = is_v ? p.v_scale : p.k_scale;
                    const int64_t piece = static_cast<int64_t>(kh) * tile_bytes(t, D);
                    uint2 codes = make_uint2(0, 0);
                    uint32_t scale = 0;
                    if (slot >= 0) {
                        codes = __ldg(reinterpret_cast<const uint2 *>(code_at + piece + (is_v ? t * (D / 2) : 0)));
                        scale = __ldg(scale_at + piece + (is_v ? t * kPerRow : 0));
                    }
                    uint16_t *dst = (is_v ? p.v_out : p.k_out) + (o * p.hkv + kh) * D + j * kBlock;
                    write_block<kVec>(dst, codes, scale, scales ? __ldg(scales + kh) : 1.f);
                }
            }
        }
        carry += total;
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
    // as many blocks as fit at once, or as the tokens (at most batch x max_seq_len) need
    const int64_t most = static_cast<int64_t>(batch) * max_seq_len;
    p.parts = static_cast<int32_t>(row_parts(most, row_iters(head_dim, kv_heads)));
    p.pack = row_pack(head_dim, kv_heads);   // (then a token is one step, and parts 1)
    const int64_t grid = std::max<int64_t>(1, std::min<int64_t>((most * p.parts + kThreads / 32 - 1) / (kThreads / 32),
                                                                static_cast<int64_t>(kGatherCtas) * std::max(1, sm_count())));
    const bool vec = aligned(k_out, 32) && aligned(v_out, 32);
    auto pick = [&](auto d, auto v) {
        constexpr int D = decltype(d)::value;
        constexpr bool V = decltype(v)::value;
        return p.pack ? gather_kernel<D, V, kPacked> : p.parts == 1 ? gather_kernel<D, V, kTokens> : gather_kernel<D, V, kParts>;
    };
    using D128 = std::integral_constant<int, 128>;
    using D64 = std::integral_constant<int, 64>;
    auto *kern = head_dim == 128 ? (vec ? pick(D128{}, std::true_type{}) : pick(D128{}, std::false_type{}))
                                 : (vec ? pick(D64{}, std::true_type{}) : pick(D64{}, std::false_type{}));
    return launch_status(launch_chained(kern, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0,
                                        reinterpret_cast<cudaStream_t>(stream), p),
                         "pkv_quant_gather");
}
