// Reading the rows of a quantised pool back as bf16: what pkv_quant_gather and pkv_byte_gather share.
//
// A format F gives kDim, the place of a token's blocks of 16 dims in its tile (place), the
// read of one (load) and its bf16 values (write).
#pragma once

#include <algorithm>
#include <type_traits>

#include "quant.cuh"

namespace pkv {
namespace quant {

constexpr int kThreads = 256;

// Reading back, and the 4-bit store, give a lane one block of 16 dims and a warp 32 neighbouring blocks of one token
// (its K rows head by head, then its V rows): 1 KB of bf16 in one run, which is where most of
// the bytes are.  (A warp that takes the same row of 4 or 8 tokens instead has the pool's
// codes in one run and bf16 in pieces of 128 or 256 bytes: 3 to 7 % slower.)  A token is
// `iters` such steps; few tokens are cut into `parts` of them so that every SM has some.
//
// Both are bound by memory, the conversions next (ALU half busy).  Stored in 4 bits and read back: 86,000
// tokens x 20 heads of 64 (1.13 GB in all) 210 us, 5.4 TB/s; 8192 x 8 heads of 128 (86 MB) 24 us.  (From the
// 8-bit pool the latter are read back in 13.5 us, 50 MB.)
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
template <class F, bool kVec, int kMode>
__global__ void __launch_bounds__(kThreads, kGatherCtas) gather_kernel(const GatherParams p) {
    pdl_wait();          // inputs may come from the previous kernel of the stream
    pdl_launch_next();
    __shared__ long long warp_sums[kThreads / 32];
    __shared__ long long off_s[kGatherChunk + 1];
    __shared__ long long row_s[kGatherChunk];   // offset of the request's first column in the table; -1: malformed
    constexpr int D = F::kDim, kPerRow = D / kBlock;
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
                const auto place = F::place(p, base, t, at, j);
#pragma unroll 4
                for (int h = h0 + lane / kPerRow; h < h1; h += 32 / kPerRow) {
                    const bool is_v = h >= p.hkv;
                    const int kh = is_v ? h - p.hkv : h;
                    const float *scales = is_v ? p.v_scale : p.k_scale;
                    typename F::Block block{};
                    if (slot >= 0) block = F::load(place, t, kh, is_v);
                    uint16_t *dst = (is_v ? p.v_out : p.k_out) + (o * p.hkv + kh) * D + j * kBlock;
                    F::template write<kVec>(dst, block, scales ? __ldg(scales + kh) : 1.f);
                }
            }
        }
        carry += total;
        __syncthreads();   // off_s is rewritten by the next chunk
    }
}

// The launch, of checked arguments.
template <template <int> class Fm>
pkv_status gather(const char *who, GatherParams p, int head_dim, int64_t max_seq_len, cudaStream_t s) {
    // as many blocks as fit at once, or as the tokens (at most batch x max_seq_len) need
    const int64_t most = static_cast<int64_t>(p.batch) * max_seq_len;
    p.parts = static_cast<int32_t>(row_parts(most, row_iters(head_dim, p.hkv)));
    p.pack = row_pack(head_dim, p.hkv);   // (then a token is one step, and parts 1)
    const int64_t grid = std::max<int64_t>(1, std::min<int64_t>((most * p.parts + kThreads / 32 - 1) / (kThreads / 32),
                                                                static_cast<int64_t>(kGatherCtas) * std::max(1, sm_count())));
    const bool vec = aligned(p.k_out, 32) && aligned(p.v_out, 32);
    auto pick = [&](auto d, auto v) {
        using F = Fm<decltype(d)::value>;
        constexpr bool V = decltype(v)::value;
        return p.pack ? gather_kernel<F, V, kPacked> : p.parts == 1 ? gather_kernel<F, V, kTokens> : gather_kernel<F, V, kParts>;
    };
    using D128 = std::integral_constant<int, 128>;
    using D64 = std::integral_constant<int, 64>;
    auto *kern = head_dim == 128 ? (vec ? pick(D128{}, std::true_type{}) : pick(D128{}, std::false_type{}))
                                 : (vec ? pick(D64{}, std::true_type{}) : pick(D64{}, std::false_type{}));
    return launch_status(launch_chained(kern, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, s, p), who);
}

}  // namespace quant
}  // namespace pkv
