// Rows of the 8-bit pool: pkv_byte_store (quantise new K/V rows into their slots) and
// pkv_byte_gather (read a batch's rows back as bf16).
//
// A store has to know which of a call's rows fall into one tile, whatever their order.  The
// first kernel writes each token's number to who[slot].  Nothing clears that array: an entry
// counts when the token that it names is one of the call's and has that slot.  The second
// kernel gives each tile to one owner, the token of the tile's first named slot, which finds
// the others in who, takes the maximum over all of them, and writes scales and codes.  For few tokens (a
// decode step) one kernel does both: each of its blocks looks at all of the call's slots.
//
// Rows stay in registers between the maximum and the codes, so each is read once.  8192 tokens of 8 heads of 128 take
// 12.5 us (50 MB: 4.0 TB/s, from and into L2), 22.6 cold; a block waits for its slots, then its owners, then its rows.
#include "gather.cuh"
#include "byte.cuh"

namespace pkv {
namespace byte {
namespace {

using quant::kThreads;

constexpr int kWarps = kThreads / 32;
constexpr int kMaxTile = quant::kMaxTile;
constexpr int kMaxChunk = 64;   // tokens that a block looks at
constexpr uint32_t kMostScale = 247;

struct StoreParams {
    uint8_t *pool;
    int64_t num_slots, tile_stride;
    int32_t t_shift, hkv, n, chunk;
    const uint16_t *k_new, *v_new;
    int64_t k_stride, v_stride;
    const int32_t *slots;
    int32_t *who, *err;
};

__global__ void __launch_bounds__(kThreads) claim_kernel(const StoreParams p) {
    pdl_wait();          // inputs may come from the previous kernel of the stream
    pdl_launch_next();
    const int i = blockIdx.x * kThreads + threadIdx.x;
    if (i >= p.n) return;
    const int64_t slot = p.slots[i];
    if (slot < 0) return;   // a padded token
    if (slot >= p.num_slots) {
        raise_flag(p.err, PKV_DEVERR_RANGE);
        return;
    }
    p.who[slot] = i;
}

template <bool kVec>
__device__ __forceinline__ void load_block(const uint16_t *__restrict__ a, uint32_t (&w)[8]) {
    if (kVec) {
        quant::load_32(a, w);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = static_cast<uint32_t>(a[2 * i]) | (static_cast<uint32_t>(a[2 * i + 1]) << 16);
    }
}

// The call's rows in a tile, by their entries in ascending order.
struct Members {
    int ent[kMaxTile], tok[kMaxTile];
};

// Stores the m rows of a tile's kv head by a group of threads: a warp (few rows) or the block.  A
// thread takes 16 dims of a K or V row; all rows are read once, into registers.
template <int D, bool kVec, int kGroup>
__device__ __forceinline__ void store_tile(const StoreParams &p, int64_t tile, int kh, const Members &mem, uint64_t mask, int m,
                                           uint32_t (&red)[kWarps][2]) {
    constexpr int kPer = D / 16, kRowThreads = 2 * kPer, kRows = kGroup / kRowThreads;
    constexpr int kPasses = kGroup == 32 ? 2 : kMaxTile / kRows;
    const int g = kGroup == 32 ? threadIdx.x & 31 : threadIdx.x;
    const int j = g % kPer, row = g / kRowThreads;
    const bool is_v = (g / kPer) & 1;
    const int t = 1 << p.t_shift;
    uint8_t *base = p.pool + tile * p.tile_stride;
    uint8_t *codes = base + (static_cast<int64_t>(kh) * 2 * D << p.t_shift) + (is_v ? t * D : 0) + j * 16;
    uint8_t *scale = base + codes_bytes(t, D, p.hkv) + 2 * kh + is_v;
    const uint32_t old = *scale;
    const uint16_t *src = (is_v ? p.v_new : p.k_new) + static_cast<int64_t>(kh) * D + j * 16;
    const int64_t stride = is_v ? p.v_stride : p.k_stride;
    uint32_t w[kPasses][8], top = 0;
#pragma unroll
    for (int i = 0; i < kPasses; ++i)
        if (i * kRows + row < m) load_block<kVec>(src + mem.tok[i * kRows + row] * stride, w[i]);
#pragma unroll
    for (int i = 0; i < kPasses; ++i)
        if (i * kRows + row < m) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t a = w[i][e] & 0x7fff7fffu, bad = __vcmpgeu2(a, 0x7f807f80u);
                top = __vmaxu2(top, a & ~bad);
                w[i][e] = (w[i][e] & ~bad) | (bad & 0x7fc07fc0u);   // an infinity becomes NaN
            }
        }
    top = max(top & 0xffffu, top >> 16);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
        if (o != kPer) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (kGroup == 32) {
        __syncwarp();   // every lane has read the old scale
    } else {
        if ((threadIdx.x & 31) % kRowThreads % kPer == 0 && (threadIdx.x & 31) < kRowThreads) red[threadIdx.x >> 5][is_v] = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kWarps; ++i) top = max(top, red[i][is_v]);
    }
    const bool fresh = mem.ent[0] == 0;
    uint32_t e = scale_of(top);
    if (!fresh) e = max(e, min(old, kMostScale));
    const float inv = scale_value(254 - e);   // 2^(127 - E)
#pragma unroll
    for (int i = 0; i < kPasses; ++i)
        if (i * kRows + row < m) {
            uint32_t c[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                c[k] = pair_to_codes(bf16_lo(w[i][2 * k]) * inv, bf16_hi(w[i][2 * k]) * inv) |
                       (pair_to_codes(bf16_lo(w[i][2 * k + 1]) * inv, bf16_hi(w[i][2 * k + 1]) * inv) << 16);
            *reinterpret_cast<uint4 *>(codes + mem.ent[i * kRows + row] * D) = make_uint4(c[0], c[1], c[2], c[3]);
        }
    if (j == 0 && row == 0) *scale = static_cast<uint8_t>(e);
    if (fresh || e <= old) return;
    // the scale grew: the codes of the tile's other slots follow
    const float by = e - old < 127 ? scale_value(127 - (e - old)) : 0.f;
    for (int at = row; at < t; at += kRows) {
        if ((mask >> at) & 1) continue;
        uint4 *a = reinterpret_cast<uint4 *>(codes + at * D);
        const uint4 x = *a;
        uint32_t c[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 lo = quant::f16x2_to_f32(lo_to_f16(c[k])), hi = quant::f16x2_to_f32(hi_to_f16(c[k]));
            c[k] = pair_to_codes(lo.x * by, lo.y * by) | (pair_to_codes(hi.x * by, hi.y * by) << 16);
        }
        *a = make_uint4(c[0], c[1], c[2], c[3]);
    }
}

// Tokens up to which every block looks at all of them.  (Stores of one token per tile, 8 kv heads of 128, one after
// another: 32 tokens 1.9 us so and 3.8 with two kernels, 128 3.2 and 5.9, 256 5.1 and 5.8.)
constexpr int kFewTokens = kThreads;

// A block per token and kv head: the tile, if the token owns it.
template <int D, bool kVec>
__global__ void __launch_bounds__(kThreads) store_few_kernel(const StoreParams p) {
    __shared__ Members mem;
    __shared__ int who[kMaxTile];
    __shared__ uint32_t red[kWarps][2];
    pdl_wait();          // inputs may come from the previous kernel of the stream
    pdl_launch_next();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, i = blockIdx.x, kh = blockIdx.y, t = 1 << p.t_shift;
    const int64_t mine = tid < p.n ? p.slots[tid] : -1, slot = p.slots[i];
    if (slot < 0) return;   // a padded token
    if (slot >= p.num_slots) {
        if (tid == 0 && kh == 0) raise_flag(p.err, PKV_DEVERR_RANGE);
        return;
    }
    if (tid < kMaxTile) who[tid] = -1;
    __syncthreads();
    if (mine >= 0 && mine >> p.t_shift == slot >> p.t_shift) atomicMax(&who[mine & (t - 1)], tid);   // (the last of equal ones)
    __syncthreads();
    // every warp for itself: the named slots of the tile, which of them is the first, and the list
    const int w0 = who[lane], w1 = who[lane + 32];
    const uint32_t h0 = __ballot_sync(0xffffffffu, w0 >= 0), h1 = __ballot_sync(0xffffffffu, w1 >= 0);
    const uint64_t mask = h0 | (static_cast<uint64_t>(h1) << 32);
    const int first = __ffsll(static_cast<long long>(mask)) - 1;
    if (who[first] != i) return;   // another token owns the tile
    if (warp == 0 && w0 >= 0) {
        const int at = __popc(h0 & ((1u << lane) - 1));
        mem.ent[at] = lane;
        mem.tok[at] = w0;
    }
    if (warp == 1 && w1 >= 0) {
        const int at = __popc(h0) + __popc(h1 & ((1u << lane) - 1));
        mem.ent[at] = lane + 32;
        mem.tok[at] = w1;
    }
    __syncthreads();
    const int m = __popcll(mask);
    constexpr int kFew = 2 * (32 / (2 * D / 16));
    if (m > kFew)
        store_tile<D, kVec, kThreads>(p, slot >> p.t_shift, kh, mem, mask, m, red);
    else if (warp == 0)
        store_tile<D, kVec, 32>(p, slot >> p.t_shift, kh, mem, mask, m, red);
}

// A block looks at a chunk of tokens and stores the tiles that they own, of one kv head: tiles
// of few rows a warp each, the others by all its threads.
constexpr int kLists = 4;   // tiles of many rows whose members are listed where they are found
template <int D, bool kVec>
__global__ void __launch_bounds__(kThreads, 3) store_kernel(const StoreParams p) {
    __shared__ Members many[kLists], few[kWarps];
    __shared__ int64_t seen[kMaxChunk], big[kMaxChunk];
    __shared__ uint32_t red[kWarps][2];
    __shared__ int n_seen, n_big;
    __shared__ uint32_t mask_s[2];
    __shared__ uint64_t masks[kLists];
    __shared__ int32_t chunk_s[kMaxChunk];
    pdl_wait();          // who comes from the kernel before
    pdl_launch_next();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, kh = blockIdx.y, t = 1 << p.t_shift;
    if (tid == 0) n_seen = n_big = 0;
    const int i0 = static_cast<int>(blockIdx.x) * p.chunk, i = i0 + tid;
    if (tid < p.chunk) chunk_s[tid] = tid < p.n - i0 ? p.slots[i] : -1;
    __syncthreads();
    // The token that the call stores at `slot`, or -1 (one of the chunk is not looked at in memory again).
    auto owner_of = [&](int64_t slot) {
        const int w = p.who[slot];
        if (w < 0 || w >= p.n) return -1;
        return (w >= i0 && w - i0 < p.chunk ? chunk_s[w - i0] : p.slots[w]) == slot ? w : -1;
    };
    if (tid < p.chunk) {
        const int64_t slot = chunk_s[tid];
        // (the slot before it is mostly the token before it: then that, or one further back, owns the tile)
        if (slot >= 0 && slot < p.num_slots) {
            const bool head = !(slot & (t - 1));
            const int w = p.who[slot], before = head ? -1 : owner_of(slot - 1);
            if (w == i && before < 0) seen[atomicAdd(&n_seen, 1)] = slot;
        }
    }
    __syncthreads();
    constexpr int kFew = 2 * (32 / (2 * D / 16));
    for (int s = warp; s < n_seen; s += kWarps) {
        const int64_t slot = seen[s], tile = slot >> p.t_shift;
        int w[2];
        uint32_t have[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int e = 32 * h + lane;
            w[h] = e < t ? owner_of((tile << p.t_shift) + e) : -1;
            have[h] = __ballot_sync(0xffffffffu, w[h] >= 0);
        }
        const uint64_t mask = have[0] | (static_cast<uint64_t>(have[1]) << 32);
        if (mask & ((1ull << (slot & (t - 1))) - 1)) continue;   // an earlier slot's token owns the tile
        const int m = __popcll(mask);
        int place = -1;
        if (m > kFew) {
            if (lane == 0) {
                place = atomicAdd(&n_big, 1);
                big[place] = tile;
                if (place < kLists) masks[place] = mask;
            }
            place = __shfl_sync(0xffffffffu, place, 0);
            if (place >= kLists) continue;
        }
        Members &list = place >= 0 ? many[place] : few[warp];
        __syncwarp();
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (w[h] >= 0) {
                const int at = (h ? __popc(have[0]) : 0) + __popc(have[h] & ((1u << lane) - 1));
                list.ent[at] = 32 * h + lane;
                list.tok[at] = w[h];
            }
        __syncwarp();
        if (place >= 0) continue;
        store_tile<D, kVec, 32>(p, tile, kh, few[warp], mask, m, red);
    }
    __syncthreads();
    const int all = n_big;
    for (int s = 0; s < all; ++s) {
        if (s >= kLists) {   // (rows in no order: the list again, over the last one)
            int w = -1;
            uint32_t have = 0;
            Members &list = many[kLists - 1];
            if (warp < 2) {
                w = tid < t ? owner_of((big[s] << p.t_shift) + tid) : -1;
                have = __ballot_sync(0xffffffffu, w >= 0);
                if (lane == 0) mask_s[warp] = have;
            }
            __syncthreads();
            if (w >= 0) {
                const int at = (warp ? __popc(mask_s[0]) : 0) + __popc(have & ((1u << lane) - 1));
                list.ent[at] = tid;
                list.tok[at] = w;
            }
            if (tid == 0) masks[kLists - 1] = mask_s[0] | (static_cast<uint64_t>(mask_s[1]) << 32);
            __syncthreads();
        }
        const int at = min(s, kLists - 1);
        store_tile<D, kVec, kThreads>(p, big[s], kh, many[at], masks[at], __popcll(masks[at]), red);
        __syncthreads();
    }
}

template <int D>
struct Rows8 {
    static constexpr int kDim = D;
    struct Block {
        uint4 codes;
        uint32_t scale;
    };
    struct Place {
        const uint8_t *code_at, *scale_at;
    };
    __device__ __forceinline__ static Place place(const quant::GatherParams &p, const uint8_t *base, int t, int at, int j) {
        return {base + at * D + j * 16, base + codes_bytes(t, D, p.hkv)};
    }
    __device__ __forceinline__ static Block load(const Place &x, int t, int kh, bool is_v) {
        Block b;
        b.codes = __ldg(reinterpret_cast<const uint4 *>(x.code_at + (static_cast<int64_t>(2 * kh) + is_v) * t * D));
        b.scale = __ldg(x.scale_at + 2 * kh + is_v);
        return b;
    }
    template <bool kVec>
    __device__ __forceinline__ static void write(uint16_t *__restrict__ dst, const Block &b, float) {
        const float s = scale_value(b.scale);
        const uint32_t w[4] = {b.codes.x, b.codes.y, b.codes.z, b.codes.w};
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 c = quant::f16x2_to_f32(i % 2 ? hi_to_f16(w[i / 2]) : lo_to_f16(w[i / 2]));
            o[i] = pack_bf16x2(c.x * s, c.y * s);
        }
        if (kVec) {
            quant::store_32(dst, o);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                dst[2 * i] = static_cast<uint16_t>(o[i]);
                dst[2 * i + 1] = static_cast<uint16_t>(o[i] >> 16);
            }
        }
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
    if (num_tiles > INT32_MAX / t) return fail(PKV_ERR_UNSUPPORTED, "%s: more than 2^31 pool slots", who);
    if (tile_stride % 16 || tile_stride < tile_bytes(t, head_dim, kv_heads))
        return fail(PKV_ERR_INVALID_ARG, "%s: the tile stride must hold all kv heads and be a multiple of 16 bytes", who);
    if (!aligned(pool, 16)) return fail(PKV_ERR_INVALID_ARG, "%s: the pool must be 16-byte aligned", who);
    return PKV_OK;
}

}  // namespace
}  // namespace byte
}  // namespace pkv

extern "C" size_t pkv_byte_tile_bytes(int32_t page_size, int32_t head_dim, int32_t kv_heads) {
    using namespace pkv;
    if (!is_pow2(page_size) || page_size > 1024 || (head_dim != 64 && head_dim != 128) || kv_heads < 1) return 0;
    return static_cast<size_t>(byte::tile_bytes(std::min(page_size, quant::kMaxTile), head_dim, kv_heads));
}

extern "C" size_t pkv_byte_store_workspace_size(int64_t num_tiles, int32_t page_size) {
    using namespace pkv;
    if (!is_pow2(page_size) || page_size > 1024 || num_tiles < 0) return 0;
    const int t = std::min(page_size, quant::kMaxTile);
    if (num_tiles > INT32_MAX / t) return 0;
    return std::max<size_t>(256, (static_cast<size_t>(num_tiles) * t * 4 + 255) / 256 * 256);
}

extern "C" pkv_status pkv_byte_store(void *pool, int64_t num_tiles, int64_t tile_stride, int32_t kv_heads, int32_t head_dim,
                                   int32_t page_size, const void *k_new, const void *v_new, int64_t k_token_stride,
                                   int64_t v_token_stride, const int32_t *slot_mapping, int32_t n_tokens,
                                   void *workspace, size_t workspace_bytes, int32_t *err_flags, pkv_stream_t stream) {
    using namespace pkv;
    using namespace pkv::byte;
    if (!err_flags) return fail(PKV_ERR_INVALID_ARG, "pkv_byte_store: err_flags is required");
    if (n_tokens < 0) return fail(PKV_ERR_INVALID_ARG, "pkv_byte_store: bad sizes");
    const pkv_status st = check_pool("pkv_byte_store", pool, num_tiles, tile_stride, kv_heads, head_dim, page_size);
    if (st != PKV_OK) return st;
    const int64_t row = static_cast<int64_t>(kv_heads) * head_dim;
    if (k_token_stride < row || v_token_stride < row)
        return fail(PKV_ERR_INVALID_ARG, "pkv_byte_store: token stride smaller than a token's rows");
    if (kv_heads > 65535) return fail(PKV_ERR_UNSUPPORTED, "pkv_byte_store: more than 65535 kv heads");
    if (n_tokens == 0) return ok();
    if (!pool || !k_new || !v_new || !slot_mapping) return fail(PKV_ERR_INVALID_ARG, "pkv_byte_store: null pointer");
    const size_t need = pkv_byte_store_workspace_size(num_tiles, page_size);
    if (workspace_bytes < need) return fail(PKV_ERR_CAPACITY, "pkv_byte_store: workspace of %zu bytes, %zu needed", workspace_bytes, need);
    if (!workspace || !aligned(workspace, 256))
        return fail(PKV_ERR_INVALID_ARG, "pkv_byte_store: workspace must be non-null and 256-byte aligned");
    StoreParams p{};
    p.pool = static_cast<uint8_t *>(pool);
    p.t_shift = ilog2(std::min(page_size, kMaxTile));
    p.num_slots = num_tiles << p.t_shift;
    p.tile_stride = tile_stride;
    p.hkv = kv_heads;
    p.n = n_tokens;
    p.k_new = static_cast<const uint16_t *>(k_new);
    p.v_new = static_cast<const uint16_t *>(v_new);
    p.k_stride = k_token_stride;
    p.v_stride = v_token_stride;
    p.slots = slot_mapping;
    p.who = static_cast<int32_t *>(workspace);
    p.err = err_flags;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool vec = aligned(k_new, 32) && aligned(v_new, 32) && k_token_stride % 16 == 0 && v_token_stride % 16 == 0;
    if (n_tokens <= kFewTokens) {
        auto *few = head_dim == 128 ? (vec ? store_few_kernel<128, true> : store_few_kernel<128, false>)
                                    : (vec ? store_few_kernel<64, true> : store_few_kernel<64, false>);
        return launch_status(launch_chained(few, dim3(static_cast<unsigned>(n_tokens), static_cast<unsigned>(kv_heads)), dim3(kThreads), 0, s, p),
                             "pkv_byte_store");
    }
    // as many tokens to a block as leave two blocks for each SM
    const int64_t blocks = 2ll * std::max(1, sm_count());
    p.chunk = 1;
    while (p.chunk < kMaxChunk && static_cast<int64_t>(n_tokens) * kv_heads / (2 * p.chunk) >= blocks) p.chunk *= 2;
    const pkv_status c = launch_status(launch_chained(claim_kernel, dim3((static_cast<unsigned>(n_tokens) + kThreads - 1) / kThreads),
                                                      dim3(kThreads), 0, s, p), "pkv_byte_store");
    if (c != PKV_OK) return c;
    auto *kern = head_dim == 128 ? (vec ? store_kernel<128, true> : store_kernel<128, false>)
                                 : (vec ? store_kernel<64, true> : store_kernel<64, false>);
    return launch_status(launch_chained(kern, dim3((static_cast<unsigned>(n_tokens) + p.chunk - 1) / p.chunk, static_cast<unsigned>(kv_heads)),
                                        dim3(kThreads), 0, s, p), "pkv_byte_store");
}

extern "C" pkv_status pkv_byte_gather(const void *pool, int64_t num_tiles, int64_t tile_stride, int32_t kv_heads,
                                    int32_t head_dim, int32_t page_size, const int32_t *req_to_token, int64_t r2t_rows,
                                    int64_t r2t_row_stride, int64_t r2t_width, const int32_t *req_pool_idx,
                                    const int32_t *kv_start, const int32_t *seq_lens, int32_t batch,
                                    int32_t max_seq_len, void *k_out, void *v_out, int64_t out_rows_cap,
                                    int32_t *cu_seqlens, int32_t *err_flags, pkv_stream_t stream) {
    using namespace pkv;
    using namespace pkv::byte;
    if (!err_flags || !cu_seqlens) return fail(PKV_ERR_INVALID_ARG, "pkv_byte_gather: null err_flags/cu_seqlens");
    if (batch < 0 || r2t_rows < 0 || r2t_width < 0 || r2t_row_stride < r2t_width || out_rows_cap < 0 || max_seq_len < 0)
        return fail(PKV_ERR_INVALID_ARG, "pkv_byte_gather: bad sizes");
    const pkv_status st = check_pool("pkv_byte_gather", pool, num_tiles, tile_stride, kv_heads, head_dim, page_size);
    if (st != PKV_OK) return st;
    if (batch > 0 && (!pool || !k_out || !v_out || !req_to_token || !req_pool_idx || !seq_lens))
        return fail(PKV_ERR_INVALID_ARG, "pkv_byte_gather: null pointer");
    quant::GatherParams p{};
    p.pool = static_cast<const uint8_t *>(pool);
    p.t_shift = ilog2(std::min(page_size, kMaxTile));
    p.num_slots = num_tiles << p.t_shift;
    p.tile_stride = tile_stride;
    p.hkv = kv_heads;
    p.batch = batch;
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
    return quant::gather<Rows8>("pkv_byte_gather", p, head_dim, max_seq_len, reinterpret_cast<cudaStream_t>(stream));
}
