// What keys receive: sum over query rows of 2^(logit - lse2), for pkv_byte_weights and for pkv_byte_decode
// with acc_out.
#include "byte_weigh.cuh"
#include "tc05.cuh"

namespace pkv {
namespace qattn {
namespace {

// ---------------------------------------------------------------- few rows
// What keys receive from given rows: a block takes 512 keys of one request and kv head, its warps 64
// each, over all the request's rows, 128 at a time in shared memory as fp16.  With lse known a
// weight is one exponential: w = 2^(logit - lse2).  Partial sums, one per kv head, are added up
// by add_kernel in a fixed order.
constexpr int kWeighWarps = 8, kWeighKeys = 64 * kWeighWarps, kWeighRows = 128;

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Place in its row of the k-th 16 bytes of lane (r, c)'s dims: the four c of two rows lie in eight bank groups.
__device__ __forceinline__ int q_chunk(int row, int c, int k) { return (4 * k + c) ^ ((row & 1) << 2); }
template <int D>
struct WeighSmem {
    uint4 q[kWeighRows * D / 8];                        // fp16, 16 bytes of a row at a time (see q_chunk)
    float f[kWeighRows], minus_lse[kWeighRows];         // score -> base-2 logit without K's scale; -lse2
    int end[kWeighRows], low[kWeighRows / 8];           // key bounds; the least of each eight
};

template <int D>
__global__ void __launch_bounds__(kWeighWarps * 32, 2) weigh_kernel(const Params p, const WeighParams wp) {
    __shared__ __align__(16) WeighSmem<D> sm;
    pdl_wait();          // inputs may come from the previous kernel of the stream
    pdl_launch_next();
    const int b = blockIdx.z, kh = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    const Req req = load_req(p, b, blockIdx.x == 0 && kh == 0 && threadIdx.x == 0);
    const int k0 = blockIdx.x * kWeighKeys + warp * 64;
    if (static_cast<int>(blockIdx.x) * kWeighKeys >= req.L) return;
    const int rows = req.n * p.g;
    constexpr int KS = D / 16;
    float sum[2][2][2] = {};   // [half][16-key group][u] of keys k0 + 32 h + 16 kt + r + 8 u
    for (int r0 = 0; r0 < rows; r0 += kWeighRows) {
        const int live = min(kWeighRows, rows - r0), blocks = (live + 7) / 8;
        __syncthreads();
        // eight lanes per row
        for (int row = threadIdx.x >> 3; row < blocks * 8; row += kWeighWarps * 4) {
            const int rr = r0 + row, tok = token_of(p, rr), j = threadIdx.x & 7;
            uint32_t w[D / 16];
            uint32_t top = 0;
            const bool in = row < live;
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                uint4 x = make_uint4(0, 0, 0, 0);
                if (in) x = __ldg(reinterpret_cast<const uint4 *>(p.q + static_cast<int64_t>(req.qo0 + tok) * p.q_stride +
                                                                  (kh * p.g + rr - tok * p.g) * D + j * (D / 8)) + i);
                w[4 * i] = x.x; w[4 * i + 1] = x.y; w[4 * i + 2] = x.z; w[4 * i + 3] = x.w;
            }
#pragma unroll
            for (int i = 0; i < D / 16; ++i) top = __vmaxu2(top, w[i] & 0x7fff7fffu);
            top = max(top & 0xffffu, top >> 16);
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            int e = min(126, 6 + 127 - static_cast<int>(top >> 7));   // (see start_segment)
            if (top == 0 || top >= 0x7f80u) e = 0;
            const float up = __int_as_float((e + 127) << 23), down = __int_as_float((127 - e) << 23);
#pragma unroll
            for (int i = 0; i < D / 16; ++i) w[i] = pack_f16x2(bf16_lo(w[i]) * up, bf16_hi(w[i]) * up);
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                const int chunk = j * (D / 64) + i;
                sm.q[row * (D / 8) + q_chunk(row, chunk / (D / 32), chunk % (D / 32))] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
            }
            int end = 0;
            float minus_lse = 0.f;
            if (in && j == 0) {
                const float lse = wp.lse[static_cast<int64_t>(req.qo0 + tok) * p.hq + kh * p.g + rr - tok * p.g] * kLog2e;
                end = !p.qo_indptr ? req.L : p.kv_end ? p.kv_end[req.qo0 + tok] : req.L - req.n + tok + 1;
                if (end < 0 || end > req.L) {
                    if (blockIdx.x == 0 && kh == 0) raise_flag(p.err, PKV_DEVERR_RANGE);
                    end = 0;
                }
                if (lse == -INFINITY) end = 0;
                minus_lse = -lse;
            }
            if (j == 0) {   // (rows past the last have bound 0: nothing of them counts)
                sm.f[row] = p.scale_log2 * down;
                sm.minus_lse[row] = minus_lse;
                sm.end[row] = end;
            }
        }
        __syncthreads();
        if (threadIdx.x < blocks) {
            int low = INT32_MAX;
#pragma unroll
            for (int i = 0; i < 8; ++i) low = min(low, sm.end[threadIdx.x * 8 + i]);
            sm.low[threadIdx.x] = low;
        }
        __syncthreads();
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
            const int key0 = k0 + h * 32;
            if (key0 >= req.L) break;
            uint32_t a[2][2][KS][2];   // [16-key group][u][step][lo / hi]
            uint64_t ks[2][2];
#pragma unroll
            for (int kt = 0; kt < 2; ++kt)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int key = key0 + kt * 16 + r + 8 * u;
                    const int64_t slot = key < req.L ? quant::slot_of(p.tab, req.base, key) : -3;
                    if (slot == -1 || slot == -2) raise_flag(p.err, slot == -1 ? PKV_DEVERR_RANGE : PKV_DEVERR_CONTIG);
                    uint32_t w[KS];
                    uint32_t e = 1;
#pragma unroll
                    for (int i = 0; i < KS; ++i) w[i] = 0;
                    if (slot >= 0) {
                        const int t = 1 << p.t_shift;
                        const uint8_t *base = piece_at<D>(p, slot, kh);
                        const uint4 *cp = reinterpret_cast<const uint4 *>(base + (slot & (t - 1)) * D + c * (D / 4));
#pragma unroll
                        for (int i = 0; i < D / 64; ++i) {
                            const uint4 x = ld_stream_16(cp + i);
                            w[4 * i] = x.x; w[4 * i + 1] = x.y; w[4 * i + 2] = x.z; w[4 * i + 3] = x.w;
                        }
                        e = __ldg(scales_at<D>(p, base, kh));
                    }
                    ks[kt][u] = pair(byte::scale_value(e), byte::scale_value(e));
#pragma unroll
                    for (int i = 0; i < KS; ++i) {
                        a[kt][u][i][0] = byte::lo_to_f16(w[i]);
                        a[kt][u][i][1] = byte::hi_to_f16(w[i]);
                    }
                }
            uint64_t part[2][2] = {};   // of rows 2 c and 2 c + 1
#pragma unroll 1
            for (int n = 0; n < blocks; ++n) {
                float s[2][4] = {};
                const uint4 *qp = sm.q + (n * 8 + r) * (D / 8);
#pragma unroll
                for (int i = 0; i < KS; i += 2) {
                    const uint4 x = qp[q_chunk(r, c, i / 2)];
#pragma unroll
                    for (int kt = 0; kt < 2; ++kt) mma_f16(s[kt], a[kt][0][i][0], a[kt][1][i][0], a[kt][0][i][1], a[kt][1][i][1], x.x, x.y);
#pragma unroll
                    for (int kt = 0; kt < 2; ++kt)
                        mma_f16(s[kt], a[kt][0][i + 1][0], a[kt][1][i + 1][0], a[kt][0][i + 1][1], a[kt][1][i + 1][1], x.z, x.w);
                }
                const int row = n * 8 + 2 * c;
                const uint64_t f = *reinterpret_cast<const uint64_t *>(&sm.f[row]), lse = *reinterpret_cast<const uint64_t *>(&sm.minus_lse[row]);
                const bool whole = key0 + 32 <= sm.low[n];
                int2 end = make_int2(0, 0);
                if (!whole) end = *reinterpret_cast<const int2 *>(&sm.end[row]);
#pragma unroll
                for (int kt = 0; kt < 2; ++kt)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const float2 y = unpair(fma2(mul2(pair(s[kt][2 * u], s[kt][2 * u + 1]), f), ks[kt][u], lse));
                        float x0 = ex2(y.x), x1 = ex2(y.y);
                        if (!whole) {
                            const int key = key0 + kt * 16 + r + 8 * u;
                            x0 = key < end.x ? x0 : 0.f;
                            x1 = key < end.y ? x1 : 0.f;
                        }
                        part[kt][u] = add2(part[kt][u], pair(x0, x1));
                    }
            }
#pragma unroll
            for (int kt = 0; kt < 2; ++kt)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float2 x = unpair(part[kt][u]);
#pragma unroll
                    for (int i = 0; i < 2; ++i) sum[i][kt][u] += h == i ? x.x + x.y : 0.f;
                }
        }
    }
    float *part = wp.part + (static_cast<int64_t>(kh) * p.batch + b) * p.tab.max_len;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int kt = 0; kt < 2; ++kt)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float x = sum[h][kt][u];
                x += __shfl_xor_sync(0xffffffffu, x, 1);
                x += __shfl_xor_sync(0xffffffffu, x, 2);
                const int key = k0 + h * 32 + kt * 16 + r + 8 * u;
                if (c == 0 && key < req.L) part[key] = x;
            }
}

// ---------------------------------------------------------------- many rows
// The same on the 5th-generation tensor cores: S = K q^T with 128 keys as MMA rows and up to 128 query
// rows as columns, fp16 in shared memory, fp32 in tensor memory.  Four warps take codes out of the
// pool into fp16 lines (a tile of 128 keys ahead of its use), one thread issues the MMAs, and four warps have a
// key per thread: its row of scores becomes weights and their sum.  Per score that is one
// exponential, which bounds it: 16 of them per cycle and SM.
constexpr int kTcKeys = 128, kTcTiles = 8, kTcRows = 128;   // keys of a tile, tiles of a block, query rows at a time
constexpr int kTcThreads = 288;                             // warps 0-3 copy, 4-7 weigh, 8 issues

template <int D>
struct TcSmem {
    static constexpr int kSlab = 128 * 128;                 // 128 rows of 64 dims
    static constexpr int kQ = 0, kK = D / 64 * kSlab;       // q, then two tiles of keys
    static constexpr int kBytes = 3 * (D / 64) * kSlab;
};

// Bounded wait; once one ran out, all of the block's later ones give up at once.
__device__ __forceinline__ bool wait_or_leave(uint64_t *bar, uint32_t parity, volatile int *left, int32_t *err, uint64_t limit_ns) {
    if (*left) return false;
    if (wait_for(bar, parity, limit_ns)) return true;
    *left = 1;
    raise_flag(err, PKV_DEVERR_TIMEOUT);
    return false;
}
// 16 dims (32 bytes) of a row of 64 into swapped lines of 128 bytes: chunk x ^ (row % 8).
__device__ __forceinline__ void put_16(uint8_t *slab, int row, int at, const uint32_t (&h)[8]) {
    uint8_t *line = slab + row * 128;
    *reinterpret_cast<uint4 *>(line + (((2 * at) ^ (row & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4 *>(line + (((2 * at + 1) ^ (row & 7)) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
}

template <int D>
__global__ void __launch_bounds__(kTcThreads, 2) weigh_many_kernel(const Params p, const WeighParams wp) {
    using C = TcSmem<D>;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    __shared__ __align__(16) float f_s[kTcRows], minus_lse_s[kTcRows];   // score -> base-2 logit without K's scale; -lse2
    __shared__ __align__(16) int end_s[kTcRows];
    __shared__ float scale_s[2][kTcKeys], acc_s[kTcTiles * kTcKeys];
    __shared__ __align__(8) uint64_t bars[6];                // full, scored, free: two each
    __shared__ uint32_t tmem_slot;
    __shared__ int left_s, low_s;
    uint8_t *smem = aligned_smem<1024>(smem_raw);
    uint64_t *full = bars, *scored = bars + 2, *freed = bars + 4;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.z, kh = blockIdx.y, k0 = blockIdx.x * (kTcTiles * kTcKeys);
    pdl_wait();          // inputs may come from the previous kernel of the stream
    const Req req = load_req(p, b, blockIdx.x == 0 && kh == 0 && threadIdx.x == 0);
    if (k0 >= req.L) return;
    const int tiles = min(kTcTiles, (req.L - k0 + kTcKeys - 1) / kTcKeys), rows = req.n * p.g;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&full[i], 128);
            mbar_init(&scored[i], 1);
            mbar_init(&freed[i], 4);
        }
        mbar_init_fence();
        left_s = 0;
    }
    if (warp == 8) {
        tc05::tmem_alloc(&tmem_slot, 256);
        tc05::tmem_relinquish();
    }
    for (int i = threadIdx.x; i < kTcTiles * kTcKeys; i += kTcThreads) acc_s[i] = 0.f;
    tc05::fence_before_sync();
    __syncthreads();
    tc05::fence_after_sync();
    pdl_launch_next();   // (no sooner: a kernel that takes tensor memory must not come between)
    const uint32_t tbase = tmem_slot;
    volatile int *left = &left_s;
    uint32_t n = 0;          // tiles so far
    for (int r0 = 0; r0 < rows; r0 += kTcRows) {
        const int live = min(kTcRows, rows - r0), cols = (live + 15) / 16 * 16;
        // ---- the rows of q, D/16 lanes each
        if (threadIdx.x == 0) low_s = INT32_MAX;
        __syncthreads();
        if (warp < 8) {
            constexpr int kPer = D / 16, kRows = 256 / kPer;
            const int j = threadIdx.x % kPer;
            int low = INT32_MAX;
#pragma unroll
            for (int i = 0; i < kTcRows / kRows; ++i) {
                const int row = i * kRows + threadIdx.x / kPer, rr = r0 + row, tok = token_of(p, rr);
                if (row >= cols) break;              // (a warp's rows are whole sixteens or none, or it has one row group)
                const bool in = row < live;
                uint32_t w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = 0;
                if (in) {
                    const uint4 *src = reinterpret_cast<const uint4 *>(p.q + static_cast<int64_t>(req.qo0 + tok) * p.q_stride +
                                                                       (kh * p.g + rr - tok * p.g) * D + j * 16);
                    const uint4 x = __ldg(src), y = __ldg(src + 1);
                    w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
                    w[4] = y.x; w[5] = y.y; w[6] = y.z; w[7] = y.w;
                }
                uint32_t top = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) top = __vmaxu2(top, w[e] & 0x7fff7fffu);
                top = max(top & 0xffffu, top >> 16);
#pragma unroll
                for (int o = 1; o < kPer; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                int e2 = min(126, 6 + 127 - static_cast<int>(top >> 7));   // (see start_segment)
                if (top == 0 || top >= 0x7f80u) e2 = 0;
                const float up = __int_as_float((e2 + 127) << 23), down = __int_as_float((127 - e2) << 23);
                uint32_t h[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) h[e] = pack_f16x2(bf16_lo(w[e]) * up, bf16_hi(w[e]) * up);
                put_16(smem + C::kQ + j / 4 * C::kSlab, row, j % 4, h);
                if (j == 0) {
                    int end = 0;                     // (rows past the last have bound 0: nothing of them counts)
                    float lse = 0.f;
                    if (in) {
                        lse = wp.lse[static_cast<int64_t>(req.qo0 + tok) * p.hq + kh * p.g + rr - tok * p.g] * kLog2e;
                        end = !p.qo_indptr ? req.L : p.kv_end ? p.kv_end[req.qo0 + tok] : req.L - req.n + tok + 1;
                        if (end < 0 || end > req.L) {
                            if (blockIdx.x == 0 && kh == 0) raise_flag(p.err, PKV_DEVERR_RANGE);
                            end = 0;
                        }
                        if (lse == -INFINITY) end = 0;
                    }
                    f_s[row] = p.scale_log2 * down;
                    minus_lse_s[row] = -lse;
                    end_s[row] = end;
                    low = min(low, end);
                }
            }
            low = __reduce_min_sync(0xffffffffu, low);
            if (lane == 0) atomicMin(&low_s, low);
            fence_proxy_async_smem();                // before the tensor cores read it
        }
        __syncthreads();
        const int low = low_s;
        if (warp < 4) {
            // ------------------------------------------------------------ keys: 32 of a tile to a warp
            constexpr int kPer = D / 16, kAtOnce = 32 / kPer, kRounds = 32 / kAtOnce;   // lanes of a key, keys at a time
            const int j = lane % kPer;
            bool ok = true;
            uint4 code[kRounds];
            float scale;
            auto load = [&](int t) {
                const int key = k0 + t * kTcKeys + warp * 32 + lane;
                const int64_t slot = key < req.L ? quant::slot_of(p.tab, req.base, key) : -3;
                if (r0 == 0 && kh == 0 && (slot == -1 || slot == -2)) raise_flag(p.err, slot == -1 ? PKV_DEVERR_RANGE : PKV_DEVERR_CONTIG);
                const uint8_t *piece = slot >= 0 ? piece_at<D>(p, slot, kh) : nullptr;
                const uint8_t *row = piece ? piece + (slot & ((1 << p.t_shift) - 1)) * D : nullptr;
                scale = piece ? byte::scale_value(__ldg(scales_at<D>(p, piece, kh))) : 1.f;
#pragma unroll
                for (int i = 0; i < kRounds; ++i) {
                    const uint8_t *a = from_lane(row, i * kAtOnce + lane / kPer);
                    code[i] = a ? ld_stream_16(a + j * 16) : make_uint4(0, 0, 0, 0);
                }
            };
            load(0);
            for (int t = 0; t < tiles; ++t) {
                const uint32_t m = n + t, s = m & 1;
                if (m >= 2) ok = __all_sync(0xffffffffu, ok && wait_or_leave(&freed[s], ((m >> 1) & 1) ^ 1, left, p.err, p.wait_ns));
                if (!ok) break;
                uint8_t *tile = smem + C::kK + s * (D / 64) * C::kSlab;
#pragma unroll
                for (int i = 0; i < kRounds; ++i) {
                    const uint32_t w[4] = {code[i].x, code[i].y, code[i].z, code[i].w};
                    uint32_t h[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) h[e] = e % 2 ? byte::hi_to_f16(w[e / 2]) : byte::lo_to_f16(w[e / 2]);
                    put_16(tile + j / 4 * C::kSlab, warp * 32 + i * kAtOnce + lane / kPer, j % 4, h);
                }
                scale_s[s][warp * 32 + lane] = scale;
                fence_proxy_async_smem();
                mbar_arrive(&full[s]);
                if (t + 1 < tiles) load(t + 1);
            }
        } else if (warp == 8) {
            // ------------------------------------------------------------ S = K q^T
            const uint32_t idesc = tc05::idesc_f16_f32(kTcKeys, cols, false, false);
            bool ok = true;
            for (int t = 0; t < tiles; ++t) {
                const uint32_t m = n + t, s = m & 1;
                ok = __all_sync(0xffffffffu, ok && wait_or_leave(&full[s], (m >> 1) & 1, left, p.err, p.wait_ns));
                if (!ok) break;
                tc05::fence_after_sync();
                if (lane == 0) {
                    const uint64_t kd = tc05::smem_desc(smem + C::kK + s * (D / 64) * C::kSlab, 16, 1024);
                    const uint64_t qd = tc05::smem_desc(smem + C::kQ, 16, 1024);
#pragma unroll
                    for (int sl = 0; sl < D / 64; ++sl)
#pragma unroll
                        for (int k = 0; k < 4; ++k)   // 16 dims: +32 bytes
                            tc05::mma_ss(tbase + s * kTcRows, kd + static_cast<uint64_t>((sl * C::kSlab + k * 32) >> 4),
                                         qd + static_cast<uint64_t>((sl * C::kSlab + k * 32) >> 4), idesc, (sl | k) ? 1u : 0u);
                    tc05::commit(&scored[s]);
                }
                __syncwarp();
            }
        } else {
            // ------------------------------------------------------------ weights: a key per thread
            const int quarter = warp & 3, row = quarter * 32 + lane;
            bool ok = true;
            for (int t = 0; t < tiles; ++t) {
                const uint32_t m = n + t, s = m & 1;
                // (full: the scales; it stays in this phase until `freed` says that they were read)
                ok = __all_sync(0xffffffffu, ok && wait_or_leave(&full[s], (m >> 1) & 1, left, p.err, p.wait_ns) &&
                                                 wait_or_leave(&scored[s], (m >> 1) & 1, left, p.err, p.wait_ns));
                if (!ok) break;
                tc05::fence_after_sync();
                const float ks1 = scale_s[s][row];
                const uint64_t ks = pair(ks1, ks1);
                const int key = k0 + t * kTcKeys + row;
                const bool whole = k0 + (t + 1) * kTcKeys <= low;
                const uint32_t from = tc05::taddr(tbase, quarter * 32, s * kTcRows);
                uint64_t sum0 = 0, sum1 = 0;
                for (int c0 = 0; c0 < cols; c0 += 16) {
                    float x[16];
                    tc05::ld_x16(from + c0, x);
                    tc05::wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; e += 4) {
                        const ulonglong2 f = *reinterpret_cast<const ulonglong2 *>(&f_s[c0 + e]);
                        const ulonglong2 l = *reinterpret_cast<const ulonglong2 *>(&minus_lse_s[c0 + e]);
                        const float2 y0 = unpair(fma2(mul2(pair(x[e], x[e + 1]), f.x), ks, l.x));
                        const float2 y1 = unpair(fma2(mul2(pair(x[e + 2], x[e + 3]), f.y), ks, l.y));
                        float w0 = ex2(y0.x), w1 = ex2(y0.y), w2 = ex2(y1.x), w3 = ex2(y1.y);
                        if (!whole) {
                            const int4 end = *reinterpret_cast<const int4 *>(&end_s[c0 + e]);
                            w0 = key < end.x ? w0 : 0.f;
                            w1 = key < end.y ? w1 : 0.f;
                            w2 = key < end.z ? w2 : 0.f;
                            w3 = key < end.w ? w3 : 0.f;
                        }
                        sum0 = add2(sum0, pair(w0, w1));
                        sum1 = add2(sum1, pair(w2, w3));
                    }
                }
                const float2 a = unpair(add2(sum0, sum1));
                acc_s[t * kTcKeys + row] += a.x + a.y;
                tc05::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&freed[s]);
            }
        }
        n += tiles;
        tc05::fence_before_sync();
        __syncthreads();
        tc05::fence_after_sync();
        if (*left) break;
    }
    if (warp == 8) {
        if (*left) {   // MMAs that nobody waited for end before their memory is given back
            __shared__ uint64_t last;
            if (lane == 0) {
                mbar_init(&last, 1);
                mbar_init_fence();
                tc05::commit(&last);
                mbar_wait(&last, 0);
            }
            __syncwarp();
        }
        tc05::tmem_dealloc(tbase, 256);
    }
    float *part = wp.part + (static_cast<int64_t>(kh) * p.batch + b) * p.tab.max_len;
    for (int i = threadIdx.x; i < min(kTcTiles * kTcKeys, req.L - k0); i += kTcThreads) part[k0 + i] = acc_s[i];
}

__global__ void __launch_bounds__(256) add_kernel(const Params p, const WeighParams wp) {
    pdl_wait();          // inputs may come from the previous kernel of the stream
    pdl_launch_next();
    const int b = blockIdx.y, key = blockIdx.x * 256 + threadIdx.x;
    int64_t base;
    const int L = quant::key_count(p.tab, b, base, p.err, false);
    if (key >= L) return;
    const int64_t row = p.tab.req_pool_idx[b], at = row * wp.acc_stride + (p.tab.kv_start ? p.tab.kv_start[b] : 0) + key;
    float x = 0.f;
    for (int kh = 0; kh < p.hkv; ++kh) x += wp.part[(static_cast<int64_t>(kh) * p.batch + b) * p.tab.max_len + key];
    wp.acc_out[at] = wp.acc_in ? wp.acc_in[at] + x : x;
}

// The same from a decode's logits: acc_out = acc_in + sum over heads of 2^(logit - lse2).  A thread
// has four keys and every fourth head, whose loads are all on their way before the first is used.
constexpr int kFinishKeys = 256;
__global__ void __launch_bounds__(256) finish_kernel(const Params p, const WeighParams wp) {
    __shared__ float4 sums[4][kFinishKeys / 4];
    pdl_wait();          // the logits
    pdl_launch_next();
    const int b = blockIdx.y, quad = threadIdx.x & 63, group = threadIdx.x >> 6, key0 = blockIdx.x * kFinishKeys;
    int64_t base;
    const int L = quant::key_count(p.tab, b, base, p.err, false);
    if (key0 >= L) return;
    const int64_t row = p.tab.req_pool_idx[b], first = row * wp.acc_stride + (p.tab.kv_start ? p.tab.kv_start[b] : 0);
    const int mine = key0 + threadIdx.x;
    const float before = wp.acc_in && mine < L ? wp.acc_in[first + mine] : 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (key0 + 4 * quad < L) {   // (a row of logits is whole 8 floats; what lies behind L is dropped below)
        const float *y = p.logits + static_cast<int64_t>(b) * p.hq * p.logit_stride + key0 + 4 * quad;
        const float *lse = wp.lse + static_cast<int64_t>(b) * p.hq;
        for (int h0 = group; h0 < p.hq; h0 += 32) {
            float4 v[8];
            float l[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int h = h0 + 4 * i;
                v[i] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
                l[i] = 0.f;
                if (h < p.hq) {
                    v[i] = __ldcs(reinterpret_cast<const float4 *>(y + h * p.logit_stride));
                    l[i] = __ldg(lse + h);
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float m = l[i] * kLog2e;
                x.x += ex2(v[i].x - m);
                x.y += ex2(v[i].y - m);
                x.z += ex2(v[i].z - m);
                x.w += ex2(v[i].w - m);
            }
        }
    }
    sums[group][quad] = x;
    __syncthreads();
    if (mine >= L) return;
    const float *s = reinterpret_cast<const float *>(sums) + threadIdx.x;
    wp.acc_out[first + mine] = before + ((s[0] + s[kFinishKeys]) + (s[2 * kFinishKeys] + s[3 * kFinishKeys]));
}

// Rows of a request and kv head from which the tensor cores' tiles of 128 keys pay.
constexpr int kManyRows = 32;

}  // namespace

pkv_status launch_weigh(const char *who, const Params &p, const WeighParams &wp, int head_dim, int64_t rows, cudaStream_t s) {
    const unsigned L = static_cast<unsigned>(p.tab.max_len), B = static_cast<unsigned>(p.batch), H = static_cast<unsigned>(p.hkv);
    if (L == 0) return ok();
    pkv_status st;
    if (rows >= kManyRows) {
        auto *kern = head_dim == 128 ? weigh_many_kernel<128> : weigh_many_kernel<64>;
        const size_t smem = (head_dim == 128 ? TcSmem<128>::kBytes : TcSmem<64>::kBytes) + 1024;
        if (raise_smem_limit(reinterpret_cast<const void *>(kern)) < smem)
            return fail(PKV_ERR_CUDA, "%s: cannot raise the shared-memory limit", who);
        st = launch_status(launch_chained(kern, dim3((L + kTcTiles * kTcKeys - 1) / (kTcTiles * kTcKeys), H, B), dim3(kTcThreads), smem, s, p, wp), who);
    } else {
        auto *kern = head_dim == 128 ? weigh_kernel<128> : weigh_kernel<64>;
        st = launch_status(launch_chained(kern, dim3((L + kWeighKeys - 1) / kWeighKeys, H, B), dim3(kWeighWarps * 32), 0, s, p, wp), who);
    }
    if (st != PKV_OK) return st;
    return launch_status(launch_chained(add_kernel, dim3((L + 255) / 256, B), dim3(256), 0, s, p, wp), who);
}

pkv_status launch_finish(const char *who, const Params &p, const WeighParams &wp, cudaStream_t s) {
    return launch_status(launch_chained(finish_kernel, dim3((static_cast<unsigned>(p.tab.max_len) + kFinishKeys - 1) / kFinishKeys,
                                                            static_cast<unsigned>(p.batch)), dim3(256), 0, s, p, wp), who);
}

}  // namespace qattn
}  // namespace pkv
