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
// by add_kernel in a fixed order.  Up to 16 rows the loads' latency bounds it (8 requests x 16384 keys, 8 heads of
// 128: 70 us for 134 MB of K), above that the MMAs and exponentials (128 rows: 154).
constexpr int kWeighWarps = 8, kWeighKeys = 64 * kWeighWarps, kWeighRows = 128;

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Factors from scores to base-2 logits of two rows and a key's scale.  The two are joined before the score: a score times
// a row's factor alone may be past fp32 (queries near 2^123 over keys near 2^-123).  Finite, so that a score of 0 stays 0.
__device__ __forceinline__ uint64_t factors(uint64_t f, uint64_t ks) {
    const float2 x = unpair(mul2(f, ks));
    return pair(fminf(x.x, 3.4e38f), fminf(x.y, 3.4e38f));
}

// Given bounds of a request without keys are 0 (the block's threads look at them).
__device__ __forceinline__ void check_bounds_of_none(const Params &p, const Req &req) {
    if (req.L > 0 || !p.qo_indptr || !p.kv_end) return;
    for (int tok = threadIdx.x; tok < req.n; tok += blockDim.x)
        if (__ldg(p.kv_end + req.qo0 + tok) != 0) raise_flag(p.err, PKV_DEVERR_RANGE);
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
    if (blockIdx.x == 0 && kh == 0) check_bounds_of_none(p, req);
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
                        const float2 y = unpair(fma2(pair(s[kt][2 * u], s[kt][2 * u + 1]), factors(f, ks[kt][u]), lse));
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
// rows as columns, q as fp16 in shared memory, K as fp16 and S as fp32 in tensor memory.  The tiles of 128
// keys of all requests and kv heads form one sequence that is cut into equal spans, one per SM.  One
// warp brings the codes of a tile into shared memory (tensor boxes of whole pool tiles, or 16 bytes per lane
// for small ones); four warps make them fp16, a key per thread, in its lane of tensor memory.
// (Loaded a key per thread, without the detour: 64 us at 8 x 32 rows of 32 heads over up to 32768 keys.  As
// fp16 in shared memory, with the fence that the tensor cores then need and that waits for the next
// tiles' loads too: 107.)  One thread issues the MMAs, and two groups of four warps take the tiles' scores in
// turn, a key per thread: its row becomes weights and their sum.
// 8 requests x 32 rows of 32 heads over up to 32768 keys take 47 us with add_kernel's 5.  A tile of 128 keys takes an SM
// 0.77 us, the chain from codes to weights (no pipe is more than a third busy), and the start of a run of keys of one
// request and kv head 4 to 5: its rows, then their factors.  A span of several runs has fewer tiles for that (53.5 us without).
constexpr int kTcKeys = 128, kTcRows = 128;   // keys of a tile, query rows at a time
constexpr int kTcThreads = 448;               // warps 0-3 convert, 4-11 weigh, 12 issues, 13 copies
constexpr int kTcStart = 6;                   // stand-in tiles before a run's first: what starting it takes
constexpr int kTcBatch = 1024;                // requests whose tiles are numbered in shared memory
constexpr int kTcRaw = 4, kTcK = 2, kTcS = 3; // tiles of codes in shared memory; of keys, and of scores, in tensor memory

// Pools whose tiles' K rows of a head are 1 KB or more are copied as boxes.
__host__ __device__ constexpr bool boxes(int t_shift, int d) { return (d << t_shift) >= 1024; }

template <int D>
struct TcSmem {
    static constexpr int kSlab = 128 * 128;   // q: 128 rows of 64 dims
    static constexpr int kRaw = D / 64 * kSlab, kRawBytes = kTcKeys * D;
    static constexpr int kReq = kRaw + kTcRaw * kRawBytes;  // [B] the requests
    static constexpr int kOff = kReq + kTcBatch * static_cast<int>(sizeof(Req));   // [B + 1] first tile of each
    static constexpr int kBytes = kOff + (kTcBatch + 1) * 4;
    static constexpr int kColS = kTcK * D / 2;              // tensor memory: keys, then scores
};

// Bounded wait; once one ran out, all of the block's later ones give up at once.
__device__ __forceinline__ bool wait_or_leave(uint64_t *bar, uint32_t parity, volatile int *left, int32_t *err, uint64_t limit_ns) {
    if (*left) return false;
    if (limit_ns >= 1000 && mbar_try_wait(bar, parity)) return true;   // (mostly; the clock is slow to read)
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
__global__ void __launch_bounds__(kTcThreads, 1) weigh_many_kernel(const __grid_constant__ Params p, const WeighParams wp) {
    using C = TcSmem<D>;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    __shared__ __align__(16) float f_s[kTcRows], minus_lse_s[kTcRows];   // score -> base-2 logit without K's scale; -lse2
    __shared__ __align__(16) int end_s[kTcRows];
    __shared__ __align__(8) uint64_t bars[2 * kTcRaw + 2 * kTcK + 2 * kTcS + 1];
    __shared__ int scan_s[kTcThreads / 32];
    __shared__ uint32_t tmem_slot;
    __shared__ int left_s, low_s, exp_lo_s, exp_hi_s, stop_s[2];
    uint8_t *smem = aligned_smem<1024>(smem_raw);
    int *off = reinterpret_cast<int *>(smem + C::kOff);
    Req *reqs = reinterpret_cast<Req *>(smem + C::kReq);
    uint64_t *full = bars, *used = bars + kTcK, *scored = used + kTcK, *freed = scored + kTcS, *brought = freed + kTcS,
             *taken = brought + kTcRaw, *last = taken + kTcRaw;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kTcK; ++i) {
            mbar_init(&full[i], 128);
            mbar_init(&used[i], 1);
        }
        for (int i = 0; i < kTcS; ++i) {
            mbar_init(&scored[i], 1);
            mbar_init(&freed[i], 4);
        }
        for (int i = 0; i < kTcRaw; ++i) {
            mbar_init(&brought[i], boxes(p.t_shift, D) ? 1 : 32);
            mbar_init(&taken[i], 4);
        }
        mbar_init(last, 1);
        mbar_init_fence();
        left_s = 0;
        off[0] = 0;
    }
    pdl_wait();          // inputs may come from the previous kernel of the stream
    if (warp == 12) {
        tc05::tmem_alloc(&tmem_slot, 512);
        tc05::tmem_relinquish();
    }
    // ---- the sequence: off[b] = tiles of one kv head before request b, stand-ins among them
    for (int b0 = 0, before = 0; b0 < p.batch; b0 += kTcThreads) {
        const int b = b0 + threadIdx.x;
        int v = 0;
        if (b < p.batch) {
            const Req r = load_req(p, b, blockIdx.x == 0);
            reqs[b] = r;
            v = r.L > 0 ? (r.L + kTcKeys - 1) / kTcKeys + kTcStart : 0;
        }
        int incl = v;
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        __syncthreads();
        if (lane == 31) scan_s[warp] = incl;
        __syncthreads();
        int all = 0;
        for (int w = 0; w < kTcThreads / 32; ++w) {
            if (w == warp) incl += all;
            all += scan_s[w];
        }
        if (b < p.batch) off[b + 1] = before + incl;
        before += all;
    }
    tc05::fence_before_sync();
    __syncthreads();
    tc05::fence_after_sync();
    pdl_launch_next();   // (no sooner: a kernel that takes tensor memory must not come between)
    for (int b = blockIdx.x; b < p.batch; b += gridDim.x) check_bounds_of_none(p, reqs[b]);
    const uint32_t tbase = tmem_slot;
    volatile int *left = &left_s;
    const int64_t all = static_cast<int64_t>(off[p.batch]) * p.hkv, per = (all + gridDim.x - 1) / gridDim.x;
    int64_t pos = blockIdx.x * per;
    const int64_t pos_end = min(all, pos + per);
    constexpr int kPerRow = D / 16;   // lanes of a row of q
    const int kj = lane % kPerRow;
    uint32_t n = 0, issued = 0;   // tiles so far; of which the copies were issued
    uint32_t pass = 0;
    int b = 0;
    // The roles go through the same runs and passes, each as far ahead as the barriers of the tiles let it: a run's
    // first keys are in tensor memory before the last one's weights are done.  The warps that weigh stage the rows and
    // meet the issuing one before each pass; those leave together, the others by themselves.
    const bool weighs = warp >= 4 && warp < 12;
    bool ok = true, stop = false;
    while (pos < pos_end && ok && !stop) {
        // ---- the next run of tiles of one request and kv head
        for (int hi = p.batch; hi - b > 1;) {
            const int mid = (b + hi) >> 1;
            if (static_cast<int64_t>(off[mid]) * p.hkv <= pos) b = mid; else hi = mid;
        }
        const Req req = reqs[b];
        const int of_b = off[b + 1] - off[b], in_b = static_cast<int>(pos - static_cast<int64_t>(off[b]) * p.hkv);
        const int kh = in_b / of_b, at_b = in_b - kh * of_b, k0 = max(0, at_b - kTcStart) * kTcKeys;
        const int part_of = static_cast<int>(min(static_cast<int64_t>(of_b - at_b), pos_end - pos));
        const int tiles = part_of - max(0, kTcStart - at_b);
        pos += part_of;
        if (tiles <= 0) continue;
        const int rows = req.n * p.g;
        const bool report = kh == 0;
        float *part = wp.part + (static_cast<int64_t>(kh) * p.batch + b) * p.tab.max_len;
        if (rows == 0 && weighs)
            for (int i = threadIdx.x - 128; i < min(tiles * kTcKeys, req.L - k0); i += 256) part[k0 + i] = 0.f;
        // a converting or weighing thread's key in each tile
        const int mine = (warp & 3) * 32 + lane;
        // (a warp stops where it first uses what it loaded: an entry of the table is looked at, and a scale
        // converted, a tile after their loads)
        auto entry = [&](int t) {
            const int key = k0 + t * kTcKeys + mine;
            int32_t first = -4;
            if (t < tiles && key < req.L) first = __ldg(p.tab.r2t + req.base + (key & ~p.tab.ps_mask));
            return first;
        };
        auto slot_at = [&](int32_t first, int t) -> int32_t {   // (see slot_of; -3: no key)
            if (first == -4 && !(t < tiles && k0 + t * kTcKeys + mine < req.L)) return -3;
            if (first < 0 || first >= (p.tab.num_pages << p.tab.ps_shift)) return -1;
            if (first & p.tab.ps_mask) return -2;
            return first + ((k0 + t * kTcKeys + mine) & p.tab.ps_mask);
        };
        auto scale_byte = [&](int32_t from) {
            uint32_t e = 1;
            if (from >= 0) e = __ldg(scales_at<D>(p, piece_at<D>(p, from, kh), kh));
            return e;
        };
        for (int r0 = 0; r0 < rows; r0 += kTcRows) {
            const int live = min(kTcRows, rows - r0), cols = (live + 31) / 32 * 32;
            if (weighs) {
                named_bar_sync(2, 256);              // the last pass is done: its rows may be overwritten
                if (threadIdx.x == 128) {
                    low_s = exp_lo_s = INT32_MAX;
                    exp_hi_s = INT32_MIN;
                    stop_s[pass & 1] = *left;        // (two in turn: the issuing warp may still look at the one before)
                }
                named_bar_sync(2, 256);
                // ---- the rows of q, D/16 lanes each
                constexpr int kRows = 256 / kPerRow;
                const int tid = threadIdx.x - 128;
                int low = INT32_MAX;
                uint32_t w[kTcRows / kRows][8];
                float lse_of[kTcRows / kRows];       // with the rows: all loads are on their way at once
                int end_of[kTcRows / kRows];
#pragma unroll
                for (int i = 0; i < kTcRows / kRows; ++i) {
                    const int row = i * kRows + tid / kPerRow, rr = r0 + row, tok = token_of(p, rr);
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[i][e] = 0;
                    lse_of[i] = 0.f;
                    end_of[i] = 0;                   // (rows past the last have bound 0: nothing of them counts)
                    if (row < live) {
                        if (kj == 0) {
                            lse_of[i] = __ldg(wp.lse + static_cast<int64_t>(req.qo0 + tok) * p.hq + kh * p.g + rr - tok * p.g);
                            end_of[i] = !p.qo_indptr ? req.L : p.kv_end ? __ldg(p.kv_end + req.qo0 + tok) : req.L - req.n + tok + 1;
                        }
                        const uint4 *src = reinterpret_cast<const uint4 *>(p.q + static_cast<int64_t>(req.qo0 + tok) * p.q_stride +
                                                                           (kh * p.g + rr - tok * p.g) * D + kj * 16);
                        const uint4 x = __ldg(src), y = __ldg(src + 1);
                        w[i][0] = x.x; w[i][1] = x.y; w[i][2] = x.z; w[i][3] = x.w;
                        w[i][4] = y.x; w[i][5] = y.y; w[i][6] = y.z; w[i][7] = y.w;
                    }
                }
                int up_by[kTcRows / kRows], lo = INT32_MAX, hi = INT32_MIN;
#pragma unroll
                for (int i = 0; i < kTcRows / kRows; ++i) {
                    uint32_t top = 0;
#pragma unroll
                    for (int e = 0; e < 8; ++e) top = __vmaxu2(top, w[i][e] & 0x7fff7fffu);
                    top = max(top & 0xffffu, top >> 16);
#pragma unroll
                    for (int o = 1; o < kPerRow; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                    up_by[i] = min(126, 6 + 127 - static_cast<int>(top >> 7));   // (see start_segment)
                    if (top >= 0x7f80u) up_by[i] = 0;
                    if (top != 0) {
                        lo = min(lo, up_by[i]);
                        hi = max(hi, up_by[i]);
                    }
                }
                lo = __reduce_min_sync(0xffffffffu, lo);
                hi = __reduce_max_sync(0xffffffffu, hi);
                if (lane == 0) {
                    atomicMin(&exp_lo_s, lo);
                    atomicMax(&exp_hi_s, hi);
                }
                named_bar_sync(2, 256);
                // one power of two for all rows, the largest's, where it is at most 2^8 from the others'
                const bool same = exp_hi_s - exp_lo_s <= 8;
#pragma unroll
                for (int i = 0; i < kTcRows / kRows; ++i) {
                    const int row = i * kRows + tid / kPerRow;
                    const int e2 = exp_hi_s == INT32_MIN ? 0 : same ? exp_lo_s : up_by[i];   // (no row but zeros: any)
                    const float up = __int_as_float((e2 + 127) << 23), down = __int_as_float((127 - e2) << 23);
                    uint32_t h[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) h[e] = pack_f16x2(bf16_lo(w[i][e]) * up, bf16_hi(w[i][e]) * up);
                    put_16(smem + kj / 4 * C::kSlab, row, kj % 4, h);
                    if (kj == 0 && row < cols) {
                        const float lse = lse_of[i] * kLog2e;
                        int end = end_of[i];
                        if (end < 0 || end > req.L) {
                            if (report) raise_flag(p.err, PKV_DEVERR_RANGE);
                            end = 0;
                        }
                        if (lse == -INFINITY) end = 0;
                        f_s[row] = p.scale_log2 * down;
                        minus_lse_s[row] = -lse;
                        end_s[row] = end;
                        low = min(low, end);
                    }
                }
                low = __reduce_min_sync(0xffffffffu, low);
                if (lane == 0) atomicMin(&low_s, low);
                fence_proxy_async_smem();            // before the tensor cores read it
            }
            if (weighs || warp == 12) {
                named_bar_sync(1, 288);              // (the others go ahead)
                stop = stop_s[pass & 1] != 0;
                if (stop) break;
            }
            ++pass;
            if (warp < 4) {
                // -------------------------------------------------------- codes to fp16
                // (the warps that weigh load the rows when they have done the last pass: these are ahead of them)
                for (int i = threadIdx.x; i < live * (D / 64); i += 128) {   // lines of 128 bytes
                    const int rr = r0 + i / (D / 64), tok = token_of(p, rr);
                    prefetch_l2(p.q + static_cast<int64_t>(req.qo0 + tok) * p.q_stride + (kh * p.g + rr - tok * p.g) * D + i % (D / 64) * 64);
                }
                for (int t = 0; t < tiles; ++t) {
                    const uint32_t m = n + t, a = m % kTcK, raw = m % kTcRaw;
                    ok = __all_sync(0xffffffffu, ok && wait_or_leave(&brought[raw], (m / kTcRaw) & 1, left, p.err, p.wait_ns));
                    if (!ok) break;
                    const uint8_t *from = smem + C::kRaw + raw * C::kRawBytes;
                    uint32_t c[D / 4];
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        const int at = mine * D + 16 * i;
                        const uint4 x = *reinterpret_cast<const uint4 *>(from + (at ^ ((at >> 3) & 0x70)));
                        c[4 * i] = x.x; c[4 * i + 1] = x.y; c[4 * i + 2] = x.z; c[4 * i + 3] = x.w;
                    }
                    if (m >= kTcK) ok = __all_sync(0xffffffffu, ok && wait_or_leave(&used[a], ((m / kTcK) & 1) ^ 1, left, p.err, p.wait_ns));
                    if (!ok) break;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&taken[raw]);
                    tc05::fence_after_sync();
                    const uint32_t to = tc05::taddr(tbase, warp * 32, a * (D / 2));
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) {
                        uint32_t h[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) h[e] = e % 2 ? byte::hi_to_f16(c[8 * i + e / 2]) : byte::lo_to_f16(c[8 * i + e / 2]);
                        tc05::st_x16_u32(to + 16 * i, h);
                    }
                    tc05::wait_st();
                    tc05::fence_before_sync();
                    mbar_arrive(&full[a]);
                }
            } else if (warp == 13) {
                // -------------------------------------------------------- the tiles' codes
                // lane j: the table's entry of the tile's piece j (boxes), or of its keys j, + 32 ...
                const bool box = boxes(p.t_shift, D);
                const int pieces = kTcKeys >> p.t_shift;   // (boxes: at most 16)
                auto entry_of = [&](int key) {
                    int32_t first = -4;
                    if (key < req.L) first = __ldg(p.tab.r2t + req.base + (key & ~p.tab.ps_mask));
                    return first;
                };
                auto slot_of_key = [&](int32_t first, int key) -> int32_t {   // (see slot_of; -3: no key)
                    if (key >= req.L) return -3;
                    if (first < 0 || first >= (p.tab.num_pages << p.tab.ps_shift)) return -1;
                    if (first & p.tab.ps_mask) return -2;
                    return first + (key & p.tab.ps_mask);
                };
                const int past = max(1, static_cast<int>(p.tab.num_pages << p.tab.ps_shift >> p.t_shift));   // the map's tiles
                int32_t ahead[2][4];                       // of this tile and the next
                auto look_up = [&](int t, int32_t (&e)[4]) {
                    const int key0 = k0 + t * kTcKeys;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (box && i > 0) break;
                        const int key = key0 + (box ? lane << p.t_shift : 32 * i + lane);
                        e[i] = t < tiles && (!box || lane < pieces) ? entry_of(key) : -4;
                    }
                };
                auto bring = [&](int t, int32_t (&e)[4]) {
                    const uint32_t m = n + t, raw = m % kTcRaw;
                    if (m >= kTcRaw) ok = __all_sync(0xffffffffu, ok && wait_or_leave(&taken[raw], ((m / kTcRaw) & 1) ^ 1, left, p.err, p.wait_ns));
                    if (!ok) return;
                    issued = m + 1;
                    const int key0 = k0 + t * kTcKeys;
                    uint8_t *to = smem + C::kRaw + raw * C::kRawBytes;
                    int flags = 0;
                    if (box) {
                        if (lane == 0) mbar_arrive_expect_tx(&brought[raw], C::kRawBytes);
                        __syncwarp();
                        if (lane < pieces) {               // (a bad page, or none: a box past the pool's last tile, zeros)
                            const int32_t slot = slot_of_key(e[0], key0 + (lane << p.t_shift));
                            if (slot == -1 || slot == -2) flags = slot == -1 ? PKV_DEVERR_RANGE : PKV_DEVERR_CONTIG;
                            const int tile = slot >= 0 ? slot >> p.t_shift : past;
                            tma_load_3d(to + (lane << p.t_shift) * D, &p.map, 0, kh * ((2 * D << p.t_shift) / 128), tile, &brought[raw]);
                        }
                    } else {
                        constexpr int kRow = D / 16;       // lanes of a key
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int32_t slot = slot_of_key(e[i], key0 + 32 * i + lane);
                            if (slot == -1 || slot == -2) flags |= slot == -1 ? PKV_DEVERR_RANGE : PKV_DEVERR_CONTIG;
                            const uint8_t *row = slot >= 0 ? piece_at<D>(p, slot, kh) + (slot & ((1 << p.t_shift) - 1)) * D : nullptr;
                            for (int k = 0; k < kRow; ++k) {
                                const int key = k * (32 / kRow) + lane / kRow, at = (32 * i + key) * D + lane % kRow * 16;
                                const uint8_t *a = from_lane(row, key);
                                cp_async_16(to + (at ^ ((at >> 3) & 0x70)), a ? a + lane % kRow * 16 : p.pool, a ? 16 : 0);
                            }
                        }
                        arrive_with_copies(&brought[raw]);
                    }
                    if (report && r0 == 0 && flags) raise_flag(p.err, flags);
                    look_up(t + 2, e);
                };
                look_up(0, ahead[0]);
                look_up(1, ahead[1]);
                for (int t = 0; t < tiles && ok; t += 2) {
                    bring(t, ahead[0]);
                    if (t + 1 < tiles && ok) bring(t + 1, ahead[1]);
                }
            } else if (warp == 12) {
                // -------------------------------------------------------- S = K q^T
                const uint32_t idesc = tc05::idesc_f16_f32(kTcKeys, cols, false, false);
                bool on = true;
                for (int t = 0; t < tiles; ++t) {
                    const uint32_t m = n + t, a = m % kTcK, s = m % kTcS;
                    on = __all_sync(0xffffffffu, wait_or_leave(&full[a], (m / kTcK) & 1, left, p.err, p.wait_ns) &&
                                                     (m < kTcS || wait_or_leave(&freed[s], ((m / kTcS) & 1) ^ 1, left, p.err, p.wait_ns)));
                    if (!on) break;
                    tc05::fence_after_sync();
                    if (lane == 0) {
                        const uint64_t qd = tc05::smem_desc(smem, 16, 1024);
#pragma unroll
                        for (int sl = 0; sl < D / 64; ++sl)
#pragma unroll
                            for (int k = 0; k < 4; ++k)   // 16 dims: 8 columns of K, 32 bytes of q
                                tc05::mma_ts(tbase + C::kColS + s * kTcRows, tbase + a * (D / 2) + (sl * 4 + k) * 8,
                                             qd + static_cast<uint64_t>((sl * C::kSlab + k * 32) >> 4), idesc, (sl | k) ? 1u : 0u);
                        tc05::commit(&scored[s]);
                        tc05::commit(&used[a]);
                    }
                    __syncwarp();
                }
            } else {
                // -------------------------------------------------------- weights: a key per thread
                bool on = true;
                const int turn = static_cast<int>(((warp >> 2) + 1 + n) & 1);   // the group's tiles: t % 2 = turn
                const int low = low_s;
                const bool same = exp_hi_s - exp_lo_s <= 8;
                const int32_t first = entry(turn);
                int32_t next = entry(turn + 2);
                uint32_t e_next = scale_byte(slot_at(first, turn));   // K's scale of the next tile's key
                for (int t = turn; t < tiles; t += 2) {
                    const uint32_t m = n + t, s = m % kTcS;
                    const float scale = byte::scale_value(e_next);
                    const uint64_t ks = pair(scale, scale);
                    e_next = scale_byte(slot_at(next, t + 2));
                    next = entry(t + 4);
                    on = __all_sync(0xffffffffu, wait_or_leave(&scored[s], (m / kTcS) & 1, left, p.err, p.wait_ns));
                    if (!on) break;
                    tc05::fence_after_sync();
                    const int key = k0 + t * kTcKeys + mine;
                    const bool whole = k0 + (t + 1) * kTcKeys <= low;
                    const uint32_t from = tc05::taddr(tbase, (warp & 3) * 32, C::kColS + s * kTcRows);
                    uint64_t sum0 = 0, sum1 = 0;
                    const float one = fminf(f_s[0] * scale, 3.4e38f);   // (where the rows share a factor; finite, so that 0 stays 0)
                    const uint64_t fks = pair(one, one);
                    for (int c0 = 0; c0 < cols; c0 += 64) {
                        float x[64];         // (columns behind `cols` may hold anything: they are not looked at)
                        tc05::ld_x64(from + c0, x);
#pragma unroll
                        for (int h = 0; h < 64; h += 32) {
                            if (c0 + h >= cols) break;
                            if (whole && same) {
#pragma unroll
                                for (int e = h; e < h + 32; e += 4) {
                                    const ulonglong2 l = *reinterpret_cast<const ulonglong2 *>(&minus_lse_s[c0 + e]);
                                    const float2 y0 = unpair(fma2(pair(x[e], x[e + 1]), fks, l.x));
                                    const float2 y1 = unpair(fma2(pair(x[e + 2], x[e + 3]), fks, l.y));
                                    sum0 = add2(sum0, pair(ex2(y0.x), ex2(y0.y)));
                                    sum1 = add2(sum1, pair(ex2(y1.x), ex2(y1.y)));
                                }
                                continue;
                            }
#pragma unroll
                            for (int e = h; e < h + 32; e += 4) {
                                const ulonglong2 f = *reinterpret_cast<const ulonglong2 *>(&f_s[c0 + e]);
                                const ulonglong2 l = *reinterpret_cast<const ulonglong2 *>(&minus_lse_s[c0 + e]);
                                const int4 end = *reinterpret_cast<const int4 *>(&end_s[c0 + e]);
                                const float2 y0 = unpair(fma2(pair(x[e], x[e + 1]), factors(f.x, ks), l.x));
                                const float2 y1 = unpair(fma2(pair(x[e + 2], x[e + 3]), factors(f.y, ks), l.y));
                                sum0 = add2(sum0, pair(key < end.x ? ex2(y0.x) : 0.f, key < end.y ? ex2(y0.y) : 0.f));
                                sum1 = add2(sum1, pair(key < end.z ? ex2(y1.x) : 0.f, key < end.w ? ex2(y1.y) : 0.f));
                            }
                        }
                    }
                    tc05::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&freed[s]);
                    const float2 a = unpair(add2(sum0, sum1));
                    if (key < req.L) part[key] = r0 == 0 ? a.x + a.y : part[key] + (a.x + a.y);
                }
            }
            n += tiles;
            if (!ok) break;
        }
    }
    tc05::fence_before_sync();
    __syncthreads();
    tc05::fence_after_sync();
    if (warp == 13 && *left)   // copies that nobody waited for land before the block's memory is given back
        for (uint32_t m = issued > kTcRaw ? issued - kTcRaw : 0; m < issued; ++m) mbar_wait(&brought[m % kTcRaw], (m / kTcRaw) & 1);
    if (warp == 12) {
        if (*left) {   // MMAs that nobody waited for end before their memory is given back
            if (lane == 0) {
                tc05::commit(last);
                mbar_wait(last, 0);
            }
            __syncwarp();
        }
        tc05::tmem_dealloc(tbase, 512);
    }
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
// has four keys and every fourth head, whose loads are all on their way before the first is used: the logits are
// still in L2 (32 requests of up to 8192 keys, 32 heads: 12 MB in 7.9 us cold), and latency bounds it.
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

// The tensor cores' tiles cost the same for few rows as for many, and a run of keys of one request and kv head starts
// slowly; the other kernel's blocks are short, but take each row's time.  So the first is taken for many rows, or
// where an SM has many tiles.  Measured (8 kv heads of 128, us; tensor cores / not): 16 requests x 4096 keys (27 tiles
// per SM), 4 rows per kv head 36.9 / 39.0, 32 rows 36.8 / 47.1, 128 rows 39 / 84; 8 x 16384 (54 tiles), 4 rows 55 / 70; 16 x
// 2048 (13 tiles), 4 rows 24.7 / 20.6, 32 rows 24.7 / 24.6, 64 rows 26.7 / 32.7; 64 x 512, 32 rows 33.2 / 24.9, 64 rows
// 34.9 / 33.3, 128 rows 41 / 47; 4 x 4096, 32 rows 18.5 / 14.4, 64 rows 18.7 / 18.5, 128 rows 20.5 / 26.6.
constexpr int kManyRows = 64, kManyTiles = 20;

}  // namespace

pkv_status launch_weigh(const char *who, const Params &p, const WeighParams &wp, int head_dim, int64_t rows, int64_t keys, cudaStream_t s) {
    const unsigned L = static_cast<unsigned>(p.tab.max_len), B = static_cast<unsigned>(p.batch), H = static_cast<unsigned>(p.hkv);
    pkv_status st;
    // (max_seq_len 0: the blocks of weigh_kernel that check the requests)
    const bool many = L > 0 && (rows >= kManyRows || keys * p.hkv / kTcKeys >= static_cast<int64_t>(kManyTiles) * std::max(1, sm_count()));
    if (many && p.batch <= kTcBatch) {
        Params q = p;
        if (boxes(p.t_shift, head_dim)) {   // the pool as lines of 128 bytes; a box is K's of a tile and head
            const uint32_t lines = static_cast<uint32_t>((head_dim << p.t_shift) / 128);
            const uint64_t dims[3] = {64, static_cast<uint64_t>(p.hkv) * 2 * lines,
                                      static_cast<uint64_t>(std::max<int64_t>(1, p.tab.num_pages << p.tab.ps_shift >> p.t_shift))};
            const uint64_t strides[2] = {128, static_cast<uint64_t>(p.tile_stride)};
            const uint32_t box[3] = {64, lines, 1};
            if (!encode_tmap_bf16(&q.map, p.pool, 3, dims, strides, box))   // (pairs of bytes)
                return fail(PKV_ERR_CUDA, "%s: cuTensorMapEncodeTiled rejected the pool", who);
        }
        auto *kern = head_dim == 128 ? weigh_many_kernel<128> : weigh_many_kernel<64>;
        const size_t smem = (head_dim == 128 ? TcSmem<128>::kBytes : TcSmem<64>::kBytes) + 1024;
        if (raise_smem_limit(reinterpret_cast<const void *>(kern)) < smem)
            return fail(PKV_ERR_CUDA, "%s: cannot raise the shared-memory limit", who);
        st = launch_status(launch_chained(kern, dim3(static_cast<unsigned>(std::max(1, sm_count()))), dim3(kTcThreads), smem, s, q, wp), who);
    } else {
        auto *kern = head_dim == 128 ? weigh_kernel<128> : weigh_kernel<64>;
        st = launch_status(launch_chained(kern, dim3(std::max(1u, (L + kWeighKeys - 1) / kWeighKeys), H, B), dim3(kWeighWarps * 32), 0, s, p, wp), who);
    }
    if (st != PKV_OK || L == 0) return st;
    return launch_status(launch_chained(add_kernel, dim3((L + 255) / 256, B), dim3(256), 0, s, p, wp), who);
}

pkv_status launch_finish(const char *who, const Params &p, const WeighParams &wp, cudaStream_t s) {
    return launch_status(launch_chained(finish_kernel, dim3((static_cast<unsigned>(p.tab.max_len) + kFinishKeys - 1) / kFinishKeys,
                                                            static_cast<unsigned>(p.batch)), dim3(256), 0, s, p, wp), who);
}

}  // namespace qattn
}  // namespace pkv
