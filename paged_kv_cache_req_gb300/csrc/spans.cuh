// What attention over a quantised pool shares, whatever the pool's format: the work of a call
// cut into spans or units, the walk over a span's tiles, the kernels around the math of a
// tile, the copy of held keys, and the host's plan.
//
// A format F gives the rest: kDim and kT (see its copy), the warps of an SM and the stages of a
// warp's ring, the size and address of a piece (one kv head's part of a pool tile), the copies of a tile
// into a stage, the math of 32 keys, and the start and the end of a segment.
#pragma once

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "extend_held.cuh"
#include "quant.cuh"

namespace pkv {
namespace qattn {

using quant::Table;

constexpr int kTile = 64;           // keys that a block of the copy of held keys takes at a time
constexpr int kStep = 32;           // keys per step of the math: what 128 to 168 registers hold
constexpr int kGroups = kStep / 16; // of 16 keys: the MMAs' key rows
// A tile is F::kKeys keys: what a stage of the copies holds.
// Tiles' worth of work that starting and finishing a unit takes (16 rows: q is loaded in place).
template <class F>
__host__ __device__ constexpr int unit_cost(int nt) { return (nt == 1 ? 1 : 2) * 64 / F::kKeys; }
constexpr int kMostTiles = 1 << 30; // of all units together
constexpr int kTableInSmem = 1024;  // requests whose tile offsets every block computes for itself
constexpr int kReqInSmem = 128;     // requests whose lengths are kept beside them
constexpr float kLn2 = 0.69314718055994531f, kLog2e = 1.44269504088896341f;

// Weights are held times 2^kLift and the running maximum is raised only when a logit passes it by
// kLazy, so the largest weight lies between 2^11 and 2^15, below fp16's 65504.  (A maximum that is raised
// past 2^8 only, with a lift of 7: 76.5 us for 77.1 at 64 requests x 4 rows x up to 16384 keys, 79.3 for 81.4
// with scores four times as far apart; one row per request the same.)
constexpr float kLazy = 4.f, kLift = 11.f;
// Dynamic shared memory from the next multiple of kAlign on (formats that need more than 128 get the room).
template <int kAlign>
__device__ __forceinline__ uint8_t *aligned_smem(uint8_t *raw) {
    return kAlign <= 128 ? raw : raw + (kAlign - (smem_u32(raw) & (kAlign - 1)) & (kAlign - 1));
}

constexpr float kNoUnit = -1000.f;   // log2 of the unit of a sum that holds nothing yet
// 2^e of an integer e >= -126 as a float (0 below, infinity above 127).
__device__ __forceinline__ float power_of_two(float e) {
    return __int_as_float(max(0, min(255, static_cast<int>(e) + 127)) << 23);
}

struct Params {
    CUtensorMap map;         // formats that copy pieces as tensor boxes: the pool as [tiles][lines of 128 bytes]
    Table tab;
    int32_t batch, hq, hkv, g, t_shift;
    uint32_t g_magic;        // ceil(2^32 / g), for g > 1
    float scale_log2;
    int64_t total_q, tile_stride, q_stride;
    const uint16_t *q;
    const uint8_t *pool;
    const float *k_scale, *v_scale;
    const int32_t *qo_indptr, *kv_end;
    uint16_t *out;
    float *lse;
    int32_t *err;
    uint64_t wait_ns;
    int32_t span_tiles;      // tiles per span; 0: all spans of the grid's warps equal
    int32_t spans_max;
    float *part_unit;        // formats with a unit: log2 of that of each of the partial rows
    float *part_o, *part_ml; // per span two slots: [rows][D], and [rows] of (m, l)
    int32_t *off;            // [B + 1] first tile of each request, then the tiles of a span
    int32_t off_ready;       // written by plan_kernel (large batches)
    // per span: the unit that its first tile continues, {request (-1: none), row block * Hkv + kv
    // head, 2 x spans back to its first + (1 if it began inside that span), spans on to its last}
    int4 *cuts;
    float *logits;           // formats that keep them: base-2 logits [B][Hq][logit_stride], or null
    int64_t logit_stride;
    int32_t max_rows;        // > 0: requests with more rows per kv head are left to the held path
};

__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Three-input maximum, and two fp32 in one 64-bit register with the paired FMA and add.
__device__ __forceinline__ float fmax3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
// D += A B for m16n8k16 with fp16 operands and fp32 accumulators.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ constexpr int ilog2_of(int x) { return x <= 1 ? 0 : 1 + ilog2_of(x / 2); }
template <int kBytes>
__device__ __forceinline__ void cp_async_small(void *dst, const void *src) {   // 4 or 8 bytes
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(dst)), "l"(src), "n"(kBytes) : "memory");
}
__device__ __forceinline__ void arrive_with_copies(uint64_t *bar) {   // once this lane's copies so far have landed
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ const uint8_t *from_lane(const uint8_t *p, int lane) {
    return reinterpret_cast<const uint8_t *>(__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(p), lane));
}
// Bounded wait: false once `limit_ns` have passed.  The first poll returns at once, so that a
// limit of some nanoseconds means what it says; the later ones suspend the warp for a
// while (the time is looked at after the first of them and then after every 64).
__device__ __forceinline__ bool wait_for(uint64_t *bar, uint32_t parity, uint64_t limit_ns) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (ok) return true;
    if (limit_ns < 1000) return false;
    const uint64_t t0 = global_ns();
    for (uint32_t i = 1;; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 63) == 1 && global_ns() - t0 > limit_ns) return false;
    }
}

// ---------------------------------------------------------------- work
struct Req {
    int64_t base;
    int L, n, qo0;   // keys, query rows, first query row
};

// Request b from the inputs; malformed ones have no rows (flags raised with `report`).
__device__ __forceinline__ Req load_req(const Params &p, int b, bool report) {
    Req r;
    r.L = quant::key_count(p.tab, b, r.base, p.err, report);
    r.n = 1;
    r.qo0 = b;
    if (p.qo_indptr) {
        const int64_t lo = p.qo_indptr[b], hi = p.qo_indptr[b + 1];
        r.n = static_cast<int>(hi - lo);
        r.qo0 = static_cast<int>(lo);
        if (lo < 0 || hi < lo || hi > p.total_q || (!p.kv_end && r.n > r.L)) {
            if (report) raise_flag(p.err, PKV_DEVERR_RANGE);
            r.n = 0;
        }
        if (p.max_rows && r.n * p.g > p.max_rows) r.n = 0;
    }
    return r;
}
// A unit enters the sequence as unit_cost stand-in tiles and its real ones, so that a span
// of many short units holds no more work than one inside a long unit.
template <class F>
__device__ __forceinline__ int real_tiles(int L) { return max(1, (L + F::kKeys - 1) / F::kKeys); }
template <int NT>
__device__ __forceinline__ int row_blocks(const Params &p, int n) { return (n * p.g + 8 * NT - 1) / (8 * NT); }

// Token of row r of a request and kv head: r / g, by a multiplication (for r < 2^28, which
// the host checks, the estimate is at most one off).
__device__ __forceinline__ int token_of(const Params &p, int r) {
    if (p.g == 1) return r;
    const int q = static_cast<int>(__umulhi(static_cast<uint32_t>(r), p.g_magic));
    return q - (q * p.g > r ? 1 : 0);
}

struct Table1 {
    int *off;    // [B + 2]
    Req *req;    // [B], or nullptr: read again where needed
};

// off[b] = first tile of request b's units, off[B] = all tiles, off[B + 1] = tiles per
// span, by the block's threads.  The host has checked that the tiles of well-formed inputs
// fit the spans; row ranges that overlap could exceed that, and then no request has any.
template <class F, int NT, int kBlock>
__device__ __forceinline__ void build_table(const Params &p, const Table1 &tb, long long *scratch, bool report) {
    int *off = tb.off;
    const int B = p.batch, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int seg = (B + kBlock - 1) / kBlock, lo = min(B, tid * seg), hi = min(B, lo + seg);
    long long local = 0;
    for (int b = lo; b < hi; ++b) {
        const Req r = load_req(p, b, report);
        if (tb.req) tb.req[b] = r;
        local += static_cast<long long>(row_blocks<NT>(p, r.n)) * p.hkv * (unit_cost<F>(NT) + real_tiles<F>(r.L));
        off[b + 1] = static_cast<int>(local);
    }
    long long incl = local;
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    long long before = incl - local, total = 0;
    for (int w = 0; w < kBlock / 32; ++w) {
        if (w < warp) before += scratch[w];
        total += scratch[w];
    }
    const bool fits = total <= (p.span_tiles ? min(static_cast<long long>(kMostTiles), static_cast<long long>(p.span_tiles) * p.spans_max)
                                             : static_cast<long long>(kMostTiles));
    for (int b = lo; b < hi; ++b) off[b + 1] = fits ? off[b + 1] + static_cast<int>(before) : 0;
    if (tid == 0) {
        if (!fits && report) raise_flag(p.err, PKV_DEVERR_RANGE);
        off[0] = 0;
        off[B + 1] = p.span_tiles ? p.span_tiles : max(1, (static_cast<int>(fits ? total : 0) + p.spans_max - 1) / p.spans_max);
    }
    __syncthreads();
}

template <class F, int NT>
__global__ void __launch_bounds__(1024) plan_kernel(const Params p) {
    pdl_wait();          // inputs may come from the previous kernel of the stream
    pdl_launch_next();
    __shared__ long long scratch[32];
    build_table<F, NT, 1024>(p, Table1{p.off, nullptr}, scratch, true);
}

// A unit and its place in the sequence of all units' tiles.
struct Unit {
    int64_t base;            // of the request's page list
    int b, rb, kh;
    int L, n, qo0;           // the request's keys, query rows and first query row
    int first, tiles;        // first real tile in the sequence; real tiles
};

__device__ __forceinline__ Req get_req(const Params &p, const Table1 &tb, int b) {
    return tb.req ? tb.req[b] : load_req(p, b, false);
}
template <class F>
__device__ __forceinline__ void set_req(Unit &u, const Req &r, int b) {
    u.b = b;
    u.L = r.L;
    u.n = r.n;
    u.qo0 = r.qo0;
    u.base = r.base;
    u.tiles = real_tiles<F>(r.L);
}
// The unit that holds tile `pos` of the sequence.
template <class F, int NT>
__device__ __forceinline__ Unit find_unit(const Params &p, const Table1 &tb, int pos) {
    const int *off = tb.off;
    int lo = 0, hi = p.batch;   // the last request with off[b] <= pos (those without rows have no tiles)
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (off[mid] <= pos) lo = mid; else hi = mid;
    }
    Unit u;
    set_req<F>(u, get_req(p, tb, lo), lo);
    const int all = u.tiles + unit_cost<F>(NT), rem = pos - off[lo], i = rem / all;
    u.rb = i / p.hkv;
    u.kh = i - u.rb * p.hkv;
    u.first = pos - (rem - i * all) + unit_cost<F>(NT);
    return u;
}
// The unit after u (there is one): the next kv head, row block or request.
template <class F, int NT>
__device__ __forceinline__ void next_unit(const Params &p, const Table1 &tb, Unit &u) {
    const int end = u.first + u.tiles;
    if (end == tb.off[u.b + 1]) {
        int b = u.b + 1;
        while (tb.off[b + 1] == end) ++b;   // requests without rows
        set_req<F>(u, get_req(p, tb, b), b);
        u.rb = u.kh = 0;
    } else if (++u.kh == p.hkv) {
        u.kh = 0;
        ++u.rb;
    }
    u.first = end + unit_cost<F>(NT);
}

// Keys that some row of the unit may see: the causal bound of its last token, or all.
template <int NT>
__device__ __forceinline__ int unit_keys(const Params &p, const Unit &u) {
    if (!p.qo_indptr || p.kv_end) return u.L;
    const int last = min(u.n, token_of(p, (u.rb + 1) * 8 * NT - 1) + 1);   // tokens up to the block's last row
    return u.L - u.n + last;
}

// What the math needs of a segment: a warp's queue of them lies in shared memory.
struct Work {
    int kh, rb, L, n, qo0;
    int t, t_end, keys;      // tiles with keys that some row sees; unit_keys
    int slot;                // of its partial; -1: the segment is the whole unit
    int pad[3];
};
constexpr int kQueue = 8;    // segments that the copies may be ahead by (at most a ring's stages + 1)

// A segment without keys: zeros and -inf where it is the whole unit, else an empty partial.
// (Given bounds leave a unit without keys only where the request has none.)
template <int D, int NT>
__device__ __forceinline__ void write_empty(const Params &p, const Unit &s, int slot, int lane) {
    for (int lr = 0; lr < 8 * NT; ++lr) {
        const int row = s.rb * 8 * NT + lr, tok = token_of(p, row);
        if (tok >= s.n) return;
        if (p.kv_end && s.kh == 0 && lane == 0 && p.kv_end[s.qo0 + tok] != 0) raise_flag(p.err, PKV_DEVERR_RANGE);
        const int64_t at = static_cast<int64_t>(s.qo0 + tok) * p.hq + s.kh * p.g + (row - tok * p.g);
        if (slot < 0) {
            if (lane < D / 8) *reinterpret_cast<uint4 *>(p.out + at * D + lane * 8) = make_uint4(0, 0, 0, 0);
            if (lane == 0 && p.lse) p.lse[at] = -INFINITY;
        } else if (lane == 0) {
            reinterpret_cast<float2 *>(p.part_ml)[static_cast<int64_t>(slot) * 8 * NT + lr] = make_float2(-INFINITY, 0.f);
        }
    }
}

// A stage of a warp's ring: what the copies fill, and the format's few bytes beside it.
struct Stage {
    uint8_t *codes, *aux;
};

// Walks the warp's spans and issues the copies of their tiles, one call of fetch() per tile,
// and queues the segments for the math.  A piece is a pool tile (a page, or a page's next 64
// keys); the pool addresses of 64 consecutive pieces (a window) are held by the lanes, two
// each, and each lane issues the copies of its own.  Slots are looked up before they are
// needed: the next window's with a window, a new segment's one tile ahead.
template <class F, int NT>
struct Fetcher {
    Unit u;
    int sp, span_end, next;  // the span; tiles of all units: its end, the next segment's start
    int t, t_end, keys;      // next tile of the unit; end of those with keys; unit_keys
    bool done, fresh, bad;   // no tile left; the window is not entered yet; a piece of it lies on a bad page
    const uint8_t *src[2];   // pieces 64 w + lane, + 32 of the window; nullptr: past the keys, or a bad page
    int nxt[2];              // slots of the next window's
    uint32_t queued;         // segments so far

    // log2 of the keys of a piece
    __device__ __forceinline__ static int shift(const Params &p) { return F::kT == 64 ? 6 : F::kT == 16 ? 4 : p.t_shift; }
    // and of the tiles that 64 pieces are
    __device__ __forceinline__ static int window_shift(const Params &p) { return shift(p) + 6 - ilog2_of(F::kKeys); }
    __device__ __forceinline__ void look_up(const Params &p, int window, int lane) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t key = static_cast<int64_t>(window * 64 + 32 * i + lane) << shift(p);
            nxt[i] = key < keys && key < static_cast<int64_t>(t_end) * F::kKeys
                         ? static_cast<int>(quant::slot_of(p.tab, u.base, static_cast<int>(key)))
                         : -3;
        }
    }
    // the looked-up window becomes the current one
    __device__ __forceinline__ void enter_window(const Params &p, int lane) {
        int flags = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            src[i] = nxt[i] >= 0 ? F::piece(p, nxt[i], u.kh) : nullptr;
            if (nxt[i] == -1) flags |= PKV_DEVERR_RANGE;
            if (nxt[i] == -2) flags |= PKV_DEVERR_CONTIG;
        }
        if (flags) raise_flag(p.err, flags);
        bad = __any_sync(0xffffffffu, flags);
        look_up(p, (t >> window_shift(p)) + 1, lane);
        fresh = false;
    }
    // To the next segment that has keys.
    __device__ __forceinline__ void advance(const Params &p, const Table1 &tb, Work *queue, int lane) {
        for (;;) {
            if (next < span_end) {
                next_unit<F, NT>(p, tb, u);
            } else {   // the warp's next span
                const int total = tb.off[p.batch], per = tb.off[p.batch + 1];
                for (;;) {
                    sp += gridDim.x * F::warps(NT);
                    if (sp >= p.spans_max) {
                        done = true;
                        return;
                    }
                    // (sp * per stays below total + spans_max * per: checked to fit on the host)
                    next = sp * per;
                    if (next < total) break;
                    if (lane == 0) p.cuts[sp] = make_int4(-1, 0, 0, 0);
                }
                span_end = min(total, next + per);
                u = find_unit<F, NT>(p, tb, next);
                if (lane == 0) {   // cut: the unit has real tiles on both sides of the boundary
                    int4 cut = make_int4(-1, 0, 0, 0);
                    if (u.first < next) {
                        const int s0 = u.first / per, s1 = (u.first + u.tiles - 1) / per;
                        cut = make_int4(u.b, u.rb * p.hkv + u.kh, (sp - s0) * 2 + (u.first > s0 * per ? 1 : 0), s1 - sp);
                    }
                    p.cuts[sp] = cut;
                }
            }
            const int begin = span_end - u.first;   // (tiles of the unit before the span's end)
            const int t0 = max(next - u.first, 0), t1 = min(u.tiles, begin);
            const bool starts_inside = t0 == 0 && next < u.first;
            next = min(u.first + u.tiles, span_end);
            if (t0 >= t1) continue;
            const int slot = t0 == 0 && t1 == u.tiles ? -1 : sp * 2 + (starts_inside ? 1 : 0);
            keys = unit_keys<NT>(p, u);
            t = t0;
            t_end = min(t1, (keys + F::kKeys - 1) / F::kKeys);
            if (t >= t_end) {
                write_empty<F::kDim, NT>(p, u, slot, lane);
                continue;
            }
            look_up(p, t >> window_shift(p), lane);
            if (lane == 0) queue[queued % kQueue] = Work{u.kh, u.rb, u.L, u.n, u.qo0, t, t_end, keys, slot, {0, 0, 0}};
            ++queued;
            fresh = true;
            return;
        }
    }
    __device__ __forceinline__ void start(const Params &p, const Table1 &tb, Work *queue, int lane) {
        // the warps of a block take spans far apart: what short units really cost differs along
        // the sequence, and so evens out over an SM
        sp = static_cast<int>((threadIdx.x >> 5) * gridDim.x + blockIdx.x) - static_cast<int>(gridDim.x) * F::warps(NT);
        next = span_end = 0;
        queued = 0;
        done = false;
        advance(p, tb, queue, lane);
    }
    // Copies the next tile into `stage`, completing on `bar`, and moves on.
    __device__ __forceinline__ void fetch(const Params &p, const Table1 &tb, Work *queue, const Stage &stage, uint64_t *bar, int lane) {
        if (fresh) enter_window(p, lane);
        constexpr int kShift = ilog2_of(F::kKeys);
        const int ps = shift(p), in_window = (1 << window_shift(p)) - 1;
        const int first = ((t & in_window) << kShift) >> ps;   // the tile's first piece within the window
        const int n = ps >= kShift ? 1 : min(1 << (kShift - ps), (keys - t * F::kKeys + (1 << ps) - 1) >> ps);
        if (bad) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int j = 32 * i + lane - first;
                if (j >= 0 && j < n && !src[i]) {   // a bad page reads as zeros
                    F::zero_piece(stage, j, ps);
                    fence_proxy_async_smem();       // before later copies into this stage
                }
            }
            __syncwarp();
        }
        uint32_t live = n;
        if (bad && !F::gathers(ps)) {
            live = 0;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int j = 32 * i + lane - first;
                live += __popc(__ballot_sync(0xffffffffu, j >= 0 && j < n && src[i]));
            }
        }
        F::copy(p, u.kh, src, first, n, live, ps, (t << kShift) & ((1 << ps) - 1), stage, bar, lane);
        if (++t >= t_end)
            advance(p, tb, queue, lane);
        else if ((t & in_window) == 0)
            fresh = true;
    }
};

template <int D, int NT>
struct State {
    uint32_t q[D / 16][NT][2];     // fp16 fragments of q
    float f[NT][2];                // score -> base-2 logit, per row of this lane's columns
    int end[NT][2];                // key bound of those rows
    float nm[NT][2];               // kLift minus the running maximum (0 before the first key)
    float limit[NT][2];            // the maximum is raised when logit + nm is past this: kLift + kLazy (-inf before the first key)
    float l[NT][2];                // this lane's share of the sum
    float o[D / 16][NT][4];        // O^T
};


// This lane's row of q as an MMA column (row 8 n + r of the unit, dims D/4 c ...), as it lies
// in memory.
template <int D, int NT>
__device__ __forceinline__ void load_q(const Params &p, const Work &s, int n, uint32_t (&w)[D / 8], int lane) {
    const int r = lane >> 2, c = lane & 3;
    const int row = s.rb * 8 * NT + n * 8 + r, tok = token_of(p, row), hh = row - tok * p.g;
    if (tok < s.n) {
        const uint4 *src = reinterpret_cast<const uint4 *>(p.q + static_cast<int64_t>(s.qo0 + tok) * p.q_stride +
                                                           (s.kh * p.g + hh) * D + c * (D / 4));
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            const uint4 x = __ldg(src + i);
            w[4 * i] = x.x; w[4 * i + 1] = x.y; w[4 * i + 2] = x.z; w[4 * i + 3] = x.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < D / 8; ++i) w[i] = 0;
    }
}

// q fragments, score factors and bounds of a segment's rows; a fresh softmax state.  At NT =
// 1 the rows of q are in `ahead`, loaded a tile ago.  Factors are at least `least`: a normal number
// where masked scores (-inf) are multiplied by them, 0 for formats whose keys have scales to join first.
template <int D, int NT, class State>
__device__ __forceinline__ void start_segment(const Params &p, const Work &s, State &st, const uint32_t (&ahead)[D / 8],
                                              int lane, float least = 1.2e-38f) {
    const int r = lane >> 2, c = lane & 3;
    const float gk = p.k_scale ? p.k_scale[s.kh] : 1.f;
    const float small = fminf(p.scale_log2, gk), large = fmaxf(p.scale_log2, gk);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        uint32_t w[D / 8];
        if (NT == 1) {
#pragma unroll
            for (int i = 0; i < D / 8; ++i) w[i] = ahead[i];
        } else {
            load_q<D, NT>(p, s, n, w, lane);
        }
        uint32_t mx = 0;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) mx = __vmaxu2(mx, w[i] & 0x7fff7fffu);
        uint32_t top = max(mx & 0xffffu, mx >> 16);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^e brings the largest magnitude's exponent (top >> 7, biased) to 6
        int e = min(126, 6 + 127 - static_cast<int>(top >> 7));
        if (top == 0 || top >= 0x7f80u) e = 0;
        const float up = __int_as_float((e + 127) << 23);
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t x = w[2 * j + i];
                st.q[j][n][i] = pack_f16x2(bf16_lo(x) * up, bf16_hi(x) * up);
            }
#pragma unroll
        for (int v = 0; v < 2; ++v) {   // this lane's rows as columns of S^T: 8 n + 2 c + v
            const int ev = __shfl_sync(0xffffffffu, e, (2 * c + v) * 4);
            // kept normal and finite, so that -inf (a masked key) stays -inf and 0 stays 0
            // (the power of two joins the factor that it brings nearer to 1: scale x g alone may be 0)
            const float down = __int_as_float((127 - ev) << 23);
            st.f[n][v] = fminf(fmaxf(ev < 0 ? small * down * large : large * down * small, least), 3.4e38f);
            const int rv = s.rb * 8 * NT + n * 8 + 2 * c + v, tv = token_of(p, rv);
            int end = s.L;   // rows past the last (zeros, never written) ask for no masking
            if (tv < s.n) {
                end = !p.qo_indptr ? s.L : p.kv_end ? __ldg(p.kv_end + s.qo0 + tv) : s.L - s.n + tv + 1;
                if (end < 0 || end > s.L) {
                    if (r == 0 && s.kh == 0 && s.t == 0) raise_flag(p.err, PKV_DEVERR_RANGE);
                    end = 0;
                }
            }
            st.end[n][v] = end;
            st.nm[n][v] = 0.f;
            st.limit[n][v] = -INFINITY;
            st.l[n][v] = 0.f;
        }
#pragma unroll
        for (int t = 0; t < D / 16; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) st.o[t][n][i] = 0.f;
    }
}

template <class F, int NT>
__global__ void __launch_bounds__(F::warps(NT) * 32, 1) attend_kernel(const __grid_constant__ Params p) {
    constexpr int D = F::kDim, kWarps = F::warps(NT), kThreads = kWarps * 32;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[kWarps * F::stages(NT)];
    __shared__ long long scratch[kWarps];
    __shared__ __align__(16) Work queues[kWarps][kQueue];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr uint32_t stage_bytes = F::kStageBytes;
    constexpr int S = F::stages(NT);
    uint8_t *smem = aligned_smem<F::kAlign>(smem_raw);
    uint8_t *ring = smem + static_cast<uint32_t>(warp * S) * stage_bytes;
    uint8_t *aux = smem + static_cast<uint32_t>(kWarps * S) * stage_bytes + warp * S * F::kAux;
    uint64_t *bar = bars + warp * S;
    if (lane == 0) {
        for (int i = 0; i < S; ++i) mbar_init(&bar[i], F::arrivals(p.t_shift));
        mbar_init_fence();
    }
    __syncwarp();
    pdl_wait();          // inputs may come from the previous kernel of the stream
    pdl_launch_next();
    Table1 tb{p.off, nullptr};
    if (!p.off_ready) {
        uint8_t *mine = smem + static_cast<uint32_t>(kWarps * S) * (stage_bytes + F::kAux);
        if (p.batch <= kReqInSmem) {
            tb.req = reinterpret_cast<Req *>(mine);
            mine += p.batch * sizeof(Req);
        }
        tb.off = reinterpret_cast<int *>(mine);
        build_table<F, NT, kThreads>(p, tb, scratch, blockIdx.x == 0);
    }
    if (blockIdx.x == 0 && warp < 2) {   // unusable head scales
        const float *g = warp ? p.v_scale : p.k_scale;
        for (int h = lane; g && h < p.hkv; h += 32)
            if (!quant::good_scale(g[h])) raise_flag(p.err, PKV_DEVERR_RANGE);
    }
    uint32_t issued = 0, used = 0;   // tiles whose copies were issued, and awaited
    uint32_t put = 0, take = 0, phase = 0;   // stages of the next copy and of the next tile; its barrier's phase
    uint32_t seg = 0;                // segments whose math began
    bool ok = true;
    typename F::template State<NT> st;
    Work w{};
    int low = 0;                     // every row of the segment sees the keys below it
    Fetcher<F, NT> f;
    Work *queue = queues[warp];
    f.start(p, tb, queue, lane);
    uint32_t q_raw[D / 8];           // the next segment's rows of q
    bool q_ahead = false;
    if (NT == 1 && f.queued > 0) {
        __syncwarp();
        load_q<D, NT>(p, queue[0], 0, q_raw, lane);
        q_ahead = true;
    }
    for (;;) {
        // (one place for the copies and one for the math: the instructions of a cold start come
        // from memory too)
        while (!f.done && issued - used < S) {
            f.fetch(p, tb, queue, Stage{ring + put * stage_bytes, aux + put * F::kAux}, &bar[put], lane);
            put = put == S - 1 ? 0 : put + 1;
            ++issued;
        }
        if (issued == used) break;
        if (w.t >= w.t_end) {
            __syncwarp();
            w = queue[seg++ % kQueue];
            if (NT == 1 && !q_ahead) load_q<D, NT>(p, w, 0, q_raw, lane);
            q_ahead = false;
            F::template start<NT>(p, w, st, q_raw, lane);
            low = w.L;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int v = 0; v < 2; ++v) low = min(low, st.end[n][v]);
            low = __reduce_min_sync(0xffffffffu, low);
        }
        ok = wait_for(&bar[take], phase, p.wait_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const Stage stage{ring + take * stage_bytes, aux + take * F::kAux};
        if (NT == 1 && w.t + 1 >= w.t_end && f.queued > seg) {   // the next segment's q on its way
            __syncwarp();   // lane 0 wrote the entry, maybe in the fetch() just above; a vote orders no memory
            load_q<D, NT>(p, queue[seg % kQueue], 0, q_raw, lane);
            q_ahead = true;
        }
        const int key0 = w.t * F::kKeys;
#pragma unroll 1
        for (int h = 0; h < F::kKeys / kStep; ++h) {
            const int k = key0 + h * kStep;
            if (k + kStep <= low)
                F::template step<NT, false>(p, st, stage, h, k, w.keys, w.kh, lane);
            else if (k < w.keys)
                F::template step<NT, true>(p, st, stage, h, k, w.keys, w.kh, lane);
        }
        ++used;
        if (++take == S) {
            take = 0;
            phase ^= 1;
        }
        if (++w.t >= w.t_end) F::template finish<NT>(p, w, st, lane);
        __syncwarp();
    }
    if (!ok) {   // a wait ran out: the copies in flight land before the block's memory is given back
        if (lane == 0) {
            raise_flag(p.err, PKV_DEVERR_TIMEOUT);
            // merge_kernel reads the record of every span, this warp's later ones too
            for (int sp = f.sp + gridDim.x * kWarps; sp < p.spans_max; sp += gridDim.x * kWarps) p.cuts[sp] = make_int4(-1, 0, 0, 0);
        }
        for (; used < issued; ++used) mbar_wait(&bar[used % S], (used / S) & 1);
    }
}

// ---------------------------------------------------------------- small calls
// One block per unit: its warps take the tiles in turn and combine their states in shared
// memory, in one launch with no table of tiles before and no merge after it (a request of more
// row blocks than the host expects: each block takes several in turn).  For calls whose time
// is latency: 4 requests of up to 255 keys x 8 kv heads take 7 us so and 12 us with spans;
// with more work the spans' even shares win.
// kRows: query rows by qo_indptr; else one per request (known to the compiler, 0.4 us of 7).
template <class F, int NT, bool kRows>
__global__ void __launch_bounds__(F::warps(NT) * 32, 1) unit_kernel(const __grid_constant__ Params p) {
    constexpr int D = F::kDim, kWarps = F::warps(NT), S = F::stages(NT);
    extern __shared__ __align__(128) uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[kWarps * S];
    __shared__ float2 ml[kWarps][8 * NT];
    __shared__ float unit_of[kWarps];   // log2 of the unit of a warp's sums (formats with one)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    const int shift = F::kT == 64 ? 6 : F::kT == 16 ? 4 : p.t_shift, pieces = max(1, F::kKeys >> shift);
    constexpr uint32_t stage_bytes = F::kStageBytes;
    uint8_t *smem = aligned_smem<F::kAlign>(smem_raw);
    uint8_t *ring = smem + static_cast<uint32_t>(warp * S) * stage_bytes;
    uint8_t *aux = smem + static_cast<uint32_t>(kWarps * S) * stage_bytes + warp * S * F::kAux;
    uint64_t *bar = bars + warp * S;
    if (lane == 0) {
        for (int i = 0; i < S; ++i) mbar_init(&bar[i], F::arrivals(p.t_shift));
        mbar_init_fence();
    }
    __syncwarp();
    pdl_wait();          // inputs may come from the previous kernel of the stream
    pdl_launch_next();
    const int b = blockIdx.x, kh = blockIdx.y;
    const int rb0 = kRows ? blockIdx.z : 0;
    const bool first = kh == 0 && rb0 == 0;
    if (first && b == 0 && warp < 2) {   // unusable head scales
        const float *g = warp ? p.v_scale : p.k_scale;
        for (int h = lane; g && h < p.hkv; h += 32)
            if (!quant::good_scale(g[h])) raise_flag(p.err, PKV_DEVERR_RANGE);
    }
    Req req;
    if (kRows) {
        req = load_req(p, b, first && threadIdx.x == 0);
    } else {
        req.L = quant::key_count(p.tab, b, req.base, p.err, first && threadIdx.x == 0);
        req.n = 1;
        req.qo0 = b;
    }
    const int64_t base = req.base;
    const int rows = kRows ? req.n * p.g : p.g;
    bool ok = true;
    int stage = 0, phase = 0;
    for (int rb = rb0; !kRows || rb * 8 * NT < rows; rb += gridDim.z) {
        Unit u{};
        u.rb = rb;
        u.L = req.L;
        u.n = req.n;
        const int keys = kRows ? unit_keys<NT>(p, u) : req.L, tiles = (keys + F::kKeys - 1) / F::kKeys;
        const Work w{kh, rb, req.L, req.n, req.qo0, 0, tiles, keys, -1, {0, 0, 0}};
        uint32_t q_raw[D / 8];
        if (NT == 1) load_q<D, NT>(p, w, 0, q_raw, lane);
        // slots of the pieces of tile t: piece lane, + 32
        auto look_up = [&](int t, int (&slot)[2]) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int64_t key = static_cast<int64_t>(t) * F::kKeys + (static_cast<int64_t>(32 * i + lane) << shift);
                slot[i] = 32 * i + lane < pieces && key < keys ? static_cast<int>(quant::slot_of(p.tab, base, static_cast<int>(key))) : -3;
            }
        };
        auto fetch = [&](const int (&slot)[2], int t, int stage) {
            const Stage dst{ring + stage * stage_bytes, aux + stage * F::kAux};
            const uint8_t *src[2];
            uint32_t live = 0;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                src[i] = slot[i] >= 0 ? F::piece(p, slot[i], kh) : nullptr;
                live += __popc(__ballot_sync(0xffffffffu, slot[i] >= 0));
                if (slot[i] == -1 || slot[i] == -2) {   // a bad page reads as zeros
                    raise_flag(p.err, slot[i] == -1 ? PKV_DEVERR_RANGE : PKV_DEVERR_CONTIG);
                    F::zero_piece(dst, 32 * i + lane, shift);
                    fence_proxy_async_smem();   // before later copies into this stage
                }
            }
            F::copy(p, kh, src, 0, pieces, live, shift, (t * F::kKeys) & ((1 << shift) - 1), dst, &bar[stage], lane);
            __syncwarp();
        };
        int slots[S][2];
#pragma unroll
        for (int i = 0; i < S; ++i) look_up(warp + i * kWarps, slots[i]);
#pragma unroll
        for (int i = 0; i < S; ++i)
            if (ok && warp + i * kWarps < tiles) fetch(slots[i], warp + i * kWarps, (stage + i) % S);
        typename F::template State<NT> st;
        F::template start<NT>(p, w, st, q_raw, lane);
        int low = req.L;   // every row sees the keys below it
        if (kRows) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int v = 0; v < 2; ++v) low = min(low, st.end[n][v]);
            low = __reduce_min_sync(0xffffffffu, low);
        }
        const bool was_ok = ok;
        int t = warp;
        for (; ok && t < tiles; t += kWarps) {
            int next[2];
            look_up(t + S * kWarps, next);
            ok = __all_sync(0xffffffffu, wait_for(&bar[stage], phase, p.wait_ns));
            if (!ok) break;
#pragma unroll 1
            for (int h = 0; h < F::kKeys / kStep; ++h) {
                const int k = t * F::kKeys + h * kStep;
                if (k + kStep <= low)
                    F::template step<NT, false>(p, st, Stage{ring + stage * stage_bytes, aux + stage * F::kAux}, h, k, keys, kh, lane);
                else if (k < keys)
                    F::template step<NT, true>(p, st, Stage{ring + stage * stage_bytes, aux + stage * F::kAux}, h, k, keys, kh, lane);
            }
            __syncwarp();
            if (t + S * kWarps < tiles) fetch(next, t + S * kWarps, stage);
            if (++stage == S) {
                stage = 0;
                phase ^= 1;
            }
        }
        if (was_ok && !ok) {   // a wait ran out: the copies in flight land before the block's memory is given back
            if (lane == 0) raise_flag(p.err, PKV_DEVERR_TIMEOUT);
            for (int i = 0; i < S && t < tiles; ++i, t += kWarps) {
                mbar_wait(&bar[stage], phase);
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        // the warps' states, each over its own (drained) ring
        float *red = reinterpret_cast<float *>(ring);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                float l = st.l[n][v];
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
                const int row = n * 8 + 2 * c + v;
                if (r == 0) ml[warp][row] = make_float2(l == 0.f ? -INFINITY : -st.nm[n][v], l);
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
                    *reinterpret_cast<float2 *>(red + row * D + r * (D / 8) + 2 * i) = make_float2(st.o[i][n][v], st.o[i][n][2 + v]);
            }
        if constexpr (F::kUnits)
            if (lane == 0) unit_of[warp] = st.unit;
        __syncthreads();
        const float head = p.v_scale ? p.v_scale[kh] : 1.f;
        const int live = min(8 * NT, rows - rb * 8 * NT);
        for (int e = threadIdx.x; e < live * (D / 4); e += kWarps * 32) {
            const int row = e / (D / 4), d0 = e % (D / 4) * 4;
            float m = -INFINITY, l = 0.f;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) m = fmaxf(m, ml[i][row].x);
            const float base_m = m == -INFINITY ? 0.f : m;
            float unit = kNoUnit;
            if constexpr (F::kUnits)
#pragma unroll
                for (int i = 0; i < kWarps; ++i) unit = ml[i][row].y == 0.f ? unit : fmaxf(unit, unit_of[i]);
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < kWarps; ++i) {
                const float2 x = ml[i][row];
                if (x.y == 0.f) continue;   // no key of the row
                const float wgt = ex2(x.x - base_m);
                float in = wgt;   // the weight in the common unit
                if constexpr (F::kUnits) in = wgt * ex2(unit_of[i] - unit);
                const float4 y = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(smem + static_cast<uint32_t>(i * S) * stage_bytes) + row * D + d0);
                l = fmaf(x.y, wgt, l);
                o.x = fmaf(y.x, in, o.x);
                o.y = fmaf(y.y, in, o.y);
                o.z = fmaf(y.z, in, o.z);
                o.w = fmaf(y.w, in, o.w);
            }
            const int r0 = rb * 8 * NT + row, tok = kRows ? token_of(p, r0) : 0;
            const int64_t at = static_cast<int64_t>(req.qo0 + tok) * p.hq + kh * p.g + (r0 - tok * p.g);
            const float inv = l == 0.f ? 0.f : rcp(l);
            float gv = head;
            if constexpr (F::kUnits) gv = power_of_two(unit);
            *reinterpret_cast<uint2 *>(p.out + at * D + d0) =
                make_uint2(pack_bf16x2(o.x * inv * gv, o.y * inv * gv), pack_bf16x2(o.z * inv * gv, o.w * inv * gv));
            if (d0 == 0 && p.lse) p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
        }
        if (!kRows) break;
        if ((rb + static_cast<int>(gridDim.z)) * 8 * NT < rows) {
            fence_proxy_async_smem();   // the states, before the next rows' copies over them
            __syncthreads();
        }
    }
}

// Combines the partials of the units that span boundaries cut: o = sum 2^(m_i - M) o_i /
// sum 2^(m_i - M) l_i.  A block per boundary; the P - 1 boundaries that cut a unit into P
// partials share its outputs (four dims of a row each) evenly, and where that leaves
// threads over, 2, 4 ... 32 of them share an output's partials.  Its time (5 us alone, 11 us with
// a cold cache) is the latency of the records and then of the partials.
constexpr int kMergeThreads = 128;

template <class F, int NT>
__global__ void __launch_bounds__(kMergeThreads) merge_kernel(const Params p) {
    constexpr int D = F::kDim;
    pdl_wait();          // inputs may come from the previous kernel of the stream
    pdl_launch_next();
    const int4 c = p.cuts[blockIdx.x];
    if (c.x < 0) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int back = c.z >> 1, parts = back + c.w + 1, rb = c.y / p.hkv, kh = c.y - rb * p.hkv;
    const int64_t s0 = static_cast<int>(blockIdx.x) - back;
    const int qo0 = p.qo_indptr ? p.qo_indptr[c.x] : c.x, n = p.qo_indptr ? p.qo_indptr[c.x + 1] - qo0 : 1;
    float gv = p.v_scale ? p.v_scale[kh] : 1.f;
    const int rows = min(8 * NT, n * p.g - rb * 8 * NT);
    const int outs = rows * (D / 4), share = (outs + parts - 2) / (parts - 1);
    int group = 1;   // outputs a warp works on at a time (the other lanes share their partials)
    while (group < 32 && group * (kMergeThreads / 32) < share) group *= 2;
    const int sub = lane / group, subs = 32 / group;
    const int end = min(outs, back * share);
    for (int o0 = (back - 1) * share; o0 < end; o0 += group * (kMergeThreads / 32)) {
        const int out = o0 + warp * group + lane % group;
        const bool live = out < end;
        const int lr = live ? out / (D / 4) : 0, d0 = live ? out % (D / 4) * 4 : 0;
        float m = -INFINITY, l = 0.f, unit = kNoUnit;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        // (no branch in the loop: the loads of several partials are in flight at a time)
#pragma unroll 8
        for (int i = sub; i < parts; i += subs) {
            const int64_t at = ((s0 + i) * 2 + (i == 0 ? c.z & 1 : 0)) * 8 * NT + lr;
            const float2 ml = reinterpret_cast<const float2 *>(p.part_ml)[at];
            float4 x = *reinterpret_cast<const float4 *>(p.part_o + at * D + d0);
            const bool some = ml.y != 0.f;   // else no key of the row in that span, and x was not written
            x.x = some ? x.x : 0.f;
            x.y = some ? x.y : 0.f;
            x.z = some ? x.z : 0.f;
            x.w = some ? x.w : 0.f;
            const float mn = some ? fmaxf(m, ml.x) : m, base = mn == -INFINITY ? 0.f : mn;
            const float c0 = ex2(m - base), c1 = some ? ex2(ml.x - base) : 0.f;
            float u0 = c0, u1 = c1;   // the weights in the common unit
            if constexpr (F::kUnits) {
                const float theirs = some ? p.part_unit[at] : kNoUnit, un = fmaxf(unit, theirs);
                u0 *= ex2(unit - un);
                u1 *= ex2(theirs - un);
                unit = un;
            }
            m = mn;
            l = l * c0 + ml.y * c1;
            o.x = o.x * u0 + x.x * u1;
            o.y = o.y * u0 + x.y * u1;
            o.z = o.z * u0 + x.z * u1;
            o.w = o.w * u0 + x.w * u1;
        }
        for (int off = group; off < 32; off <<= 1) {
            const float m2 = __shfl_xor_sync(0xffffffffu, m, off), l2 = __shfl_xor_sync(0xffffffffu, l, off);
            const float4 x = make_float4(__shfl_xor_sync(0xffffffffu, o.x, off), __shfl_xor_sync(0xffffffffu, o.y, off),
                                         __shfl_xor_sync(0xffffffffu, o.z, off), __shfl_xor_sync(0xffffffffu, o.w, off));
            const float mn = fmaxf(m, m2), base = mn == -INFINITY ? 0.f : mn;
            const float c0 = ex2(m - base), c1 = ex2(m2 - base);
            float u0 = c0, u1 = c1;
            if constexpr (F::kUnits) {
                const float theirs = __shfl_xor_sync(0xffffffffu, unit, off), un = fmaxf(unit, theirs);
                u0 *= ex2(unit - un);
                u1 *= ex2(theirs - un);
                unit = un;
            }
            m = mn;
            l = l * c0 + l2 * c1;
            o.x = o.x * u0 + x.x * u1;
            o.y = o.y * u0 + x.y * u1;
            o.z = o.z * u0 + x.z * u1;
            o.w = o.w * u0 + x.w * u1;
        }
        if (sub || !live) continue;
        const int row = rb * 8 * NT + lr, tok = token_of(p, row);
        const int64_t at = static_cast<int64_t>(qo0 + tok) * p.hq + kh * p.g + (row - tok * p.g);
        // (a division, not rcp(): with that the compiler orders the loop's loads otherwise, 77 us for 69 at
        // 1 request x 131072 keys x 1 kv head)
        const float inv = l == 0.f ? 0.f : 1.f / l;
        if constexpr (F::kUnits) gv = power_of_two(unit);
        *reinterpret_cast<uint2 *>(p.out + at * D + d0) =
            make_uint2(pack_bf16x2(o.x * inv * gv, o.y * inv * gv), pack_bf16x2(o.z * inv * gv, o.w * inv * gv));
        if (d0 == 0 && p.lse) p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    }
}

// ---------------------------------------------------------------- held keys
// Requests with many query rows: their keys and values are taken out of the pool once, K as
// bf16 and V as fp16 (both exact, without the head scales), for the tcgen05 kernel of
// extend.cu: per key and head that moves 4.6 D bytes once, against 4 D flops for each of the
// many rows.  Layout [D/64][kv heads][rows][64], request after request.  A key whose V
// holds a NaN block gets a NaN K and a zero V: a zero weight times NaN would reach rows that
// do not see the key.  A thread takes 16 dims of a key and writes 32 bytes, a whole sector; six
// blocks of 256 threads fill an SM.  Bound by the writes: 20325 keys of 8 requests x 8 kv heads of
// 128 (83 MB written, 23 MB read) 27 us with a cold cache.
constexpr int kHoldThreads = 256, kHoldCtas = 6;   // threads of a block, blocks per SM

struct HoldParams {
    uint16_t *k, *v;
    int64_t rows;
    int32_t *first_row, *counter, *order;
    int32_t min_rows;
};
constexpr int kSorted = 1024;   // requests up to which their items go longest first

template <class F>
__global__ void __launch_bounds__(kHoldThreads, kHoldCtas) hold_kernel(const Params p, const HoldParams h) {
    constexpr int D = F::kDim;
    extern __shared__ __align__(16) int32_t table[];   // [B + 1] first rows, [B + 1] first tiles
    __shared__ long long scratch[kHoldThreads / 32];
    __shared__ long long carry_s[2];
    pdl_wait();          // inputs may come from the previous kernel of the stream
    pdl_launch_next();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = p.batch;
    int32_t *first = table, *tile0 = table + B + 1;
    if (tid < 2) carry_s[tid] = 0;
    if (tid == 0) first[0] = tile0[0] = 0;
    __syncthreads();
    for (int b0 = 0; b0 < B; b0 += kHoldThreads) {
        const int b = b0 + tid;
        int L = 0;
        if (b < B) {
            const Req r = load_req(p, b, blockIdx.x == 0);
            if (static_cast<int64_t>(r.n) * p.g > h.min_rows) L = r.L;
        }
        // one scan of both sums: rows below, tiles above bit 36
        long long v = L + (static_cast<long long>((L + kTile - 1) / kTile) << 36), incl = v;
        for (int o = 1; o < 32; o <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        if (lane == 31) scratch[warp] = incl;
        __syncthreads();
        long long before = carry_s[0];
        for (int w = 0; w < warp; ++w) before += scratch[w];
        incl += before;
        __syncthreads();
        if (tid == kHoldThreads - 1) carry_s[0] = incl;
        if (b < B) {
            first[b + 1] = static_cast<int32_t>(incl & ((1ll << 36) - 1));
            tile0[b + 1] = static_cast<int32_t>(incl >> 36);
        }
        __syncthreads();
    }
    if (blockIdx.x == 0) {
        for (int i = tid; i <= B; i += kHoldThreads) h.first_row[i] = first[i];
        for (int b = tid; b < B; b += kHoldThreads) {
            int place = b;
            if (B <= kSorted) {
                const int L = first[b + 1] - first[b];
                place = 0;
                for (int j = 0; j < B; ++j) {
                    const int x = first[j + 1] - first[j];
                    place += x > L || (x == L && j < b) ? 1 : 0;
                }
            }
            h.order[place] = b;
        }
        if (tid == 0) {
            *h.counter = 0;
            if (first[B] > h.rows) raise_flag(p.err, PKV_DEVERR_CAPACITY);
        }
        if (warp < 2) {   // unusable head scales
            const float *g = warp ? p.v_scale : p.k_scale;
            for (int i = lane; g && i < p.hkv; i += 32)
                if (!quant::good_scale(g[i])) raise_flag(p.err, PKV_DEVERR_RANGE);
        }
    }
    constexpr int kPerRow = D / 16, kRowThreads = 2 * kPerRow;   // threads of a row: K blocks, then V blocks
    constexpr int kRowsAtOnce = kHoldThreads / kRowThreads;
    const int j = tid % kPerRow, row_in = tid / kRowThreads;
    const bool is_v = (tid / kPerRow) & 1;
    const uint32_t group = (kRowThreads == 16 ? 0xffffu : 0xffu) << (lane / kRowThreads * kRowThreads);
    const int64_t items = static_cast<int64_t>(tile0[B]) * p.hkv;
    for (int64_t w = blockIdx.x; w < items; w += gridDim.x) {
        const int tl = static_cast<int>(w / p.hkv), kh = static_cast<int>(w - static_cast<int64_t>(tl) * p.hkv);
        int lo = 0, hi = B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (tile0[mid] <= tl) lo = mid; else hi = mid;
        }
        const int L = first[lo + 1] - first[lo];
        int64_t base;
        quant::key_count(p.tab, lo, base, p.err, false);
        const int key0 = (tl - tile0[lo]) * kTile;
        uint16_t *dst = (is_v ? h.v : h.k) + ((static_cast<int64_t>(j / 4) * p.hkv + kh) * h.rows + first[lo]) * 64 + (j % 4) * 16;
#pragma unroll
        for (int i = 0; i < kTile / kRowsAtOnce; ++i) {
            const int key = key0 + i * kRowsAtOnce + row_in;
            const bool in = key < L && first[lo] + key < h.rows;
            const int64_t slot = in ? quant::slot_of(p.tab, base, key) : -3;
            typename F::Block block{};
            if (slot >= 0) {
                block = F::load_block(p, slot, kh, is_v, j);
            } else if (slot != -3 && kh == 0 && j == 0 && !is_v) {
                raise_flag(p.err, slot == -1 ? PKV_DEVERR_RANGE : PKV_DEVERR_CONTIG);
            }
            const uint32_t any = __ballot_sync(0xffffffffu, is_v && F::has_nan(block)) & group;
            uint32_t x[8];
            F::hold(block, is_v, any != 0, x);
            if (in) {
                quant::store_32(dst + static_cast<int64_t>(key) * 64, x);
            }
        }
    }
}

// ------------------------------------------------------------------ host side
// What the plan has to know of a format at a head_dim and page size.
struct Shape {
    // at NT = 1 and 2: warps, stages of each, unit_cost, keys of a tile, bytes of a stage
    int warps[2], stages[2], cost[2], keys[2];
    size_t stage[2];
    size_t slack;              // bytes for the alignment of the first stage
    bool units;                // sums have a unit
    int64_t tile;              // bytes of a pool tile
};
template <class F1, class F2>
static Shape shape(int64_t tile) {
    return Shape{{F1::warps(1), F2::warps(2)}, {F1::stages(1), F2::stages(2)}, {unit_cost<F1>(1), unit_cost<F2>(2)}, {F1::kKeys, F2::kKeys},
                 {F1::kStageBytes + F1::kAux, F2::kStageBytes + F2::kAux}, F1::kAlign > 128 ? F1::kAlign : 0, F1::kUnits, tile};
}

// (`needs_out`: the call writes the attention's output)
template <class A>
static pkv_status validate(const char *who, const A *a, bool extend, bool check_ptrs, int64_t (*tile_of)(const A *), bool needs_out = true) {
    if (a->batch < 0 || a->num_q_heads < 1 || a->num_kv_heads < 1 || a->total_q < 0 || a->total_kv < 0 ||
        a->max_seq_len < 0 || a->max_q_len < 0 || a->num_tiles < 0)
        return fail(PKV_ERR_INVALID_ARG, "%s: negative or zero size", who);
    if (a->num_q_heads % a->num_kv_heads) return fail(PKV_ERR_INVALID_ARG, "%s: Hq not a multiple of Hkv", who);
    if (a->num_q_heads / a->num_kv_heads > 16) return fail(PKV_ERR_UNSUPPORTED, "%s: Hq/Hkv must be 16 or less", who);
    if (a->head_dim != 64 && a->head_dim != 128) return fail(PKV_ERR_UNSUPPORTED, "%s: head_dim 64 or 128", who);
    if (!is_pow2(a->page_size) || a->page_size > 1024)
        return fail(PKV_ERR_UNSUPPORTED, "%s: page_size must be a power of two in [1, 1024]", who);
    if (a->layout != PKV_LAYOUT_CSR && a->layout != PKV_LAYOUT_BLOCK_TABLE && a->layout != PKV_LAYOUT_REQ_TO_TOKEN)
        return fail(PKV_ERR_INVALID_ARG, "%s: layout must be CSR, BLOCK_TABLE or REQ_TO_TOKEN", who);
    if (a->layout == PKV_LAYOUT_REQ_TO_TOKEN &&
        (a->r2t_rows < 0 || a->r2t_width < 0 || a->r2t_row_stride < a->r2t_width || a->r2t_width > INT32_MAX))
        return fail(PKV_ERR_INVALID_ARG, "%s: bad req_to_token shape", who);
    if (!(a->sm_scale > 0.f) || std::isinf(a->sm_scale))
        return fail(PKV_ERR_INVALID_ARG, "%s: sm_scale must be positive and finite", who);
    if (a->kv_chunk < 0 || a->kv_chunk % 64) return fail(PKV_ERR_INVALID_ARG, "%s: kv_chunk multiple of 64", who);
    const int t = std::min(a->page_size, quant::kMaxTile);
    if (a->tile_stride % 16 || a->tile_stride < tile_of(a))
        return fail(PKV_ERR_INVALID_ARG, "%s: the tile stride must hold all kv heads and be a multiple of 16 bytes", who);
    if (a->q_row_stride < static_cast<int64_t>(a->num_q_heads) * a->head_dim || a->q_row_stride % 8)
        return fail(PKV_ERR_INVALID_ARG, "%s: q_row_stride must hold Hq x head_dim and be 16-byte aligned", who);
    if (a->num_tiles > INT32_MAX / t) return fail(PKV_ERR_UNSUPPORTED, "%s: more than 2^31 pool slots", who);
    if (a->total_q > INT32_MAX || a->total_q * a->num_q_heads >= 1 << 28 ||
        static_cast<int64_t>(a->batch) * a->num_kv_heads > INT32_MAX)
        return fail(PKV_ERR_UNSUPPORTED, "%s: 2^28 (query row, head) pairs or more", who);
    if (a->batch == 0 || !check_ptrs) return PKV_OK;
    if (!a->q || !a->pool || (needs_out && !a->out)) return fail(PKV_ERR_INVALID_ARG, "%s: null q/pool/out", who);
    if (extend ? !a->qo_indptr : (a->qo_indptr || a->kv_end || a->total_q != a->batch))
        return fail(PKV_ERR_INVALID_ARG, extend ? "%s: null qo_indptr"
                                                : "%s: one query row per request, without qo_indptr and kv_end", who);
    if (!aligned(a->q, 16) || !aligned(a->pool, 16) || !aligned(a->out, 16))
        return fail(PKV_ERR_INVALID_ARG, "%s: q, pool and out must be 16-byte aligned", who);
    if (a->layout == PKV_LAYOUT_CSR && (!a->kv_indptr || !a->kv_indices || !a->kv_last_page_len))
        return fail(PKV_ERR_INVALID_ARG, "%s: CSR layout needs kv_indptr/kv_indices/kv_last_page_len", who);
    if (a->layout == PKV_LAYOUT_BLOCK_TABLE && (!a->block_table || !a->seq_lens || a->block_table_width < 0))
        return fail(PKV_ERR_INVALID_ARG, "%s: block-table layout needs block_table and seq_lens", who);
    if (a->layout == PKV_LAYOUT_REQ_TO_TOKEN && (!a->req_to_token || !a->req_pool_idx || !a->seq_lens))
        return fail(PKV_ERR_INVALID_ARG, "%s: token-table layout needs req_to_token, req_pool_idx, seq_lens", who);
    return PKV_OK;
}

// How a call runs: a block per unit, or the span kernel (its rows per unit, grid, spans), and
// for requests with many query rows the held path; with the workspace of each.
constexpr int kHeldRows = 128;     // rows per request and kv head up to which the span kernel is used
constexpr int kHeldBatch = 4096;   // requests whose tables fit the held path's shared memory

struct Plan {
    bool unit, spans, held, plan_launch;
    int nt, spans_max, span_tiles;
    dim3 grid;
    size_t smem, part_o, part_ml, part_unit, cuts, table;          // span kernel
    size_t hold_k, hold_first, ext;                     // held path: one of the two tensors, row table, extend.cu's own
    int64_t hold_rows;
    size_t span_bytes() const { return part_o + part_ml + part_unit + cuts + table; }
    size_t bytes() const { return (spans ? span_bytes() : 0) + (held ? 2 * hold_k + hold_first + ext : 0); }
};

static size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// The part of the arguments that extend.cu's kernel takes.
template <class A>
static pkv_extend_args extend_args(const A *a) {
    pkv_extend_args e{};
    e.batch = a->batch;
    e.num_q_heads = a->num_q_heads;
    e.num_kv_heads = a->num_kv_heads;
    e.head_dim = a->head_dim;
    e.page_size = 1;
    e.sm_scale = a->sm_scale;
    e.max_seq_len = a->max_seq_len;
    e.kv_chunk = a->kv_chunk;
    if (e.kv_chunk == 0) {
        // keys are split only when the blocks of 128 rows leave SMs idle: a split block writes
        // and reads back its fp32 rows (8192 rows over 16384 keys: 2140 us in pieces of 4096 keys,
        // 1170 us whole)
        const int g = 1 << ilog2(a->num_q_heads / a->num_kv_heads);
        const int64_t blocks = a->num_kv_heads * std::max<int64_t>(1, std::max<int64_t>(a->batch, a->total_q * g / 128));
        const int64_t pieces = std::max<int64_t>(1, 2ll * std::max(1, sm_count()) / blocks), L = std::max(1, a->max_seq_len);
        e.kv_chunk = static_cast<int32_t>(std::min<int64_t>((std::max<int64_t>(512, (L + pieces - 1) / pieces) + 127) / 128 * 128,
                                                            INT32_MAX / 128 * 128));
    }
    e.total_q = a->total_q;
    e.q = a->q;
    e.qo_indptr = a->qo_indptr;
    e.kv_end = a->kv_end;
    e.out = a->out;
    e.lse = a->lse;
    return e;
}

template <class A>
static bool make_plan(const A *a, bool extend, const Shape &f, Plan &pl) {
    pl = Plan{};
    const int g = a->num_q_heads / a->num_kv_heads;
    const int64_t batch = std::max(a->batch, 1), total_q = std::max<int64_t>(a->total_q, 1);
    // rows of a request and kv head: at most max_q_len's, or what the average says
    const int64_t rows = (extend && a->max_q_len > 0 ? std::min<int64_t>(a->max_q_len, total_q) : (total_q + batch - 1) / batch) * g;
    // (a batch too large for the held path's tables, or keys past its counters and coordinates, take
    // the spans whatever their rows)
    pl.hold_rows = std::max<int64_t>(1, a->total_kv > 0 ? a->total_kv : batch * a->max_seq_len);
    pl.held = extend && rows > kHeldRows && a->batch <= kHeldBatch && batch * a->max_seq_len <= INT32_MAX &&
              pl.hold_rows <= INT32_MAX / (static_cast<int64_t>(a->num_kv_heads) * (a->head_dim / 64));
    const int64_t sms = std::max(1, sm_count());
    if (!pl.held && a->kv_chunk == 0) {
        // What the two kernels take, in parts of about 0.75 us: a block per unit starts, then makes
        // `rounds` of its warps over the unit's tiles, unit after unit where there are more than SMs;
        // spans start more slowly, share the tiles evenly and are merged.  The longest request
        // counts for the first, the sum for the second (total_kv, or half of what max_seq_len
        // allows: lengths are rarely equal).  Measured (8 kv heads of 128, us; unit / spans): decodes of
        // 16 x 768 keys 7.0 / 12.9, 16 x 3000 17.7 / 24.8, 32 x 700 12.7 / 15.8, 4 x 2048 11.5 / 12.5, but
        // 64 x 256 18.3 / 15.0 and 64 x 64 17.5 / 10.3; 16 rows per head, 4 x 512 keys 9.0 / 15.1, 16 x 2000
        // 17.4 / 25.8, 32 x 256 15.0 / 19.4; 48 rows, 4 x 1000 11.9 / 18.6.  (The same rule at 64 dims,
        // whose tiles are half the bytes and take some two thirds of the time.)
        // (Calls of more units than a grid's side take the spans in any case.)
        const int nt = rows <= 8 ? 1 : 2, warps = f.warps[nt - 1], keys = f.keys[nt - 1];
        const int64_t blocks = (rows + 8 * nt - 1) / (8 * nt), units = batch * a->num_kv_heads * blocks;
        if (units <= 65535) {
            const int64_t tiles = (std::max(1, a->max_seq_len) + keys - 1) / keys;
            const int64_t rounds = (tiles + warps - 1) / warps, waves = (units + sms - 1) / sms;
            const int64_t of_all = a->total_kv > 0 ? std::min(a->total_kv / keys, batch * tiles) : batch * tiles / 2;
            const int64_t all = of_all * a->num_kv_heads * blocks + units;
            pl.unit = 5 + waves * (2 + 3 * rounds * keys / 64) <= 13 + 3 * ((all + sms * warps - 1) / (sms * warps)) * keys / 64;
        }
    }
    pl.spans = !pl.unit && (!pl.held || batch > 1);
    if (pl.unit) {
        pl.nt = rows <= 8 ? 1 : 2;
        pl.grid = dim3(static_cast<unsigned>(batch), static_cast<unsigned>(a->num_kv_heads),
                       static_cast<unsigned>((rows + 8 * pl.nt - 1) / (8 * pl.nt)));
        pl.smem = static_cast<size_t>(f.warps[pl.nt - 1] * f.stages[pl.nt - 1]) * f.stage[pl.nt - 1] + f.slack;
    }
    if (pl.spans) {
        const int64_t few = pl.held ? kHeldRows : rows;
        pl.nt = few <= 8 ? 1 : 2;
        const int warps = f.warps[pl.nt - 1];
        pl.grid = dim3(static_cast<unsigned>(sms));
        pl.plan_launch = a->batch > kTableInSmem;
        pl.smem = static_cast<size_t>(warps * f.stages[pl.nt - 1]) * f.stage[pl.nt - 1] + f.slack;
        if (!pl.plan_launch) pl.smem += (static_cast<size_t>(a->batch) + 2) * 4 + (a->batch <= kReqInSmem ? a->batch * sizeof(Req) : 0);
        int64_t spans = sms * warps;
        // all units' tiles, at most (beside held keys the requests with few rows only)
        const int64_t all_rows = pl.held ? std::min<int64_t>(a->total_q * g, batch * kHeldRows) : a->total_q * g;
        const int64_t blocks = (all_rows + 8 * pl.nt - 1) / (8 * pl.nt) + a->batch;
        const int64_t tiles = blocks * a->num_kv_heads * ((std::max(1, a->max_seq_len) + f.keys[pl.nt - 1] - 1) / f.keys[pl.nt - 1] + f.cost[pl.nt - 1]);
        if (a->kv_chunk > 0) {
            pl.span_tiles = a->kv_chunk / f.keys[pl.nt - 1];
            spans = (tiles + pl.span_tiles - 1) / pl.span_tiles;
        }
        if (spans > INT32_MAX / 64 || tiles > kMostTiles) return false;
        pl.spans_max = static_cast<int>(spans);
        const size_t slots = static_cast<size_t>(spans) * 2 * 8 * pl.nt;
        pl.part_o = up256(slots * a->head_dim * 4);
        pl.part_ml = up256(slots * 8);
        pl.part_unit = f.units ? up256(slots * 4) : 0;
        pl.cuts = up256(static_cast<size_t>(spans) * 16);
        pl.table = up256((static_cast<size_t>(a->batch) + 2) * 4);
    }
    if (pl.held) {
        pl.hold_k = up256(static_cast<size_t>(pl.hold_rows) * a->num_kv_heads * a->head_dim * 2);
        pl.hold_first = up256((static_cast<size_t>(a->batch) * 2 + 1) * 4);   // first rows, and the order
        const pkv_extend_args e = extend_args(a);
        pl.ext = up256(ext::held_workspace(&e));
        if (pl.ext == 0) return false;
    }
    return true;
}

template <class A>
static size_t workspace_size(const A *a, bool extend, const Shape &f) {
    Plan pl;
    return make_plan(a, extend, f, pl) ? std::max<size_t>(pl.bytes(), 256) : 0;
}

template <class A>
static Params params(const A *a, int32_t *err) {
    Params p{};
    Table &t = p.tab;
    t.layout = a->layout;
    t.ps_shift = ilog2(a->page_size);
    t.ps_mask = a->page_size - 1;
    t.bt_width = a->block_table_width;
    t.max_len = a->max_seq_len;
    p.t_shift = std::min(t.ps_shift, ilog2(quant::kMaxTile));
    t.num_pages = (a->num_tiles << p.t_shift) >> t.ps_shift;
    t.kv_indices_len = a->kv_indices_len;
    t.kv_indptr = a->kv_indptr;
    t.kv_indices = a->kv_indices;
    t.kv_last = a->kv_last_page_len;
    t.block_table = a->block_table;
    t.seq_lens = a->seq_lens;
    t.r2t = a->req_to_token;
    t.req_pool_idx = a->req_pool_idx;
    t.kv_start = a->kv_start;
    t.r2t_rows = a->r2t_rows;
    t.r2t_stride = a->r2t_row_stride;
    t.r2t_width = a->r2t_width;
    p.batch = a->batch;
    p.hq = a->num_q_heads;
    p.hkv = a->num_kv_heads;
    p.g = a->num_q_heads / a->num_kv_heads;
    p.g_magic = static_cast<uint32_t>(((1ull << 32) + p.g - 1) / p.g);
    p.scale_log2 = a->sm_scale * kLog2e;
    p.total_q = a->total_q;
    p.tile_stride = a->tile_stride;
    p.q_stride = a->q_row_stride;
    p.q = static_cast<const uint16_t *>(a->q);
    p.pool = static_cast<const uint8_t *>(a->pool);
    p.qo_indptr = a->qo_indptr;
    p.kv_end = a->kv_end;
    p.out = static_cast<uint16_t *>(a->out);
    p.lse = a->lse;
    p.err = err;
    return p;
}

// Fm<D, kT, NT>: the format at a head_dim, for pools of tiles of kT slots (0: others; 1: fewer than kSmall) and 8 NT rows.
template <template <int, int, int> class Fm, int D, int NT>
static pkv_status launch(const char *who, const Params &p, const Plan &pl, cudaStream_t s) {
    auto pick = [&](auto f) {
        using F = decltype(f);
        return !pl.unit ? attend_kernel<F, NT> : p.qo_indptr ? unit_kernel<F, NT, true> : unit_kernel<F, NT, false>;
    };
    auto *kern = p.t_shift == 6 ? pick(Fm<D, 64, NT>{}) : p.t_shift == 4 ? pick(Fm<D, 16, NT>{}) : pick(Fm<D, 0, NT>{});
    if constexpr (Fm<D, 0, NT>::kSmall > 0)   // formats that take small pieces another way
        if (1 << p.t_shift < Fm<D, 0, NT>::kSmall) kern = pick(Fm<D, 1, NT>{});
    if (raise_smem_limit(reinterpret_cast<const void *>(kern)) < pl.smem)
        return fail(PKV_ERR_CUDA, "%s: cannot raise the shared-memory limit", who);
    pkv_status st = PKV_OK;
    if (pl.plan_launch) {
        st = launch_status(launch_chained(plan_kernel<Fm<D, 0, NT>, NT>, dim3(1), dim3(1024), 0, s, p), who);
        if (st != PKV_OK) return st;
    }
    st = launch_status(launch_chained(kern, pl.grid, dim3(Fm<D, 0, NT>::warps(NT) * 32), pl.smem, s, p), who);
    if (st != PKV_OK || pl.unit) return st;
    return launch_status(launch_chained(merge_kernel<Fm<D, 0, NT>, NT>, dim3(pl.spans_max), dim3(kMergeThreads), 0, s, p), who);
}

template <template <int, int, int> class Fm, int D, class A>
static pkv_status launch_held(const A *a, const Params &p, const Plan &pl, char *ws, cudaStream_t s) {
    const pkv_extend_args e = extend_args(a);
    char *own = ws + 2 * pl.hold_k + pl.hold_first;
    HoldParams h{};
    h.k = reinterpret_cast<uint16_t *>(ws);
    h.v = reinterpret_cast<uint16_t *>(ws + pl.hold_k);
    h.rows = pl.hold_rows;
    h.first_row = reinterpret_cast<int32_t *>(ws + 2 * pl.hold_k);
    h.order = h.first_row + a->batch + 1;
    h.counter = reinterpret_cast<int32_t *>(own + ext::held_counter_offset(&e));
    h.min_rows = pl.spans ? kHeldRows : 0;
    auto *kern = hold_kernel<Fm<D, 0, 1>>;
    const size_t smem = (static_cast<size_t>(a->batch) + 1) * 8;
    if (raise_smem_limit(reinterpret_cast<const void *>(kern)) < smem)
        return fail(PKV_ERR_CUDA, "%s: cannot raise the shared-memory limit", Fm<D, 0, 1>::kExtend);
    const int64_t items = (pl.hold_rows / kTile + a->batch) * a->num_kv_heads;
    const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(items, static_cast<int64_t>(kHoldCtas) * std::max(1, sm_count())));
    const pkv_status st = launch_status(launch_chained(kern, dim3(static_cast<unsigned>(grid)), dim3(kHoldThreads), smem, s, p, h),
                                        Fm<D, 0, 1>::kExtend);
    if (st != PKV_OK) return st;
    const ext::Held held{h.k, h.v, h.rows, h.first_row, h.order, p.k_scale, p.v_scale, a->q_row_stride, h.min_rows, Fm<D, 0, 1>::kHeldBf16V,
                         Fm<D, 0, 1>::kExtend};
    return ext::held_launch(&e, held, own, p.err, s);
}

// Checked arguments: the plan `pl`, parameters `p` but for the workspace's parts.
template <template <int, int, int> class Fm, class A>
static pkv_status attend(const char *who, const A *a, const Plan &pl, Params &p, char *at, cudaStream_t s) {
    p.wait_ns = wait_limit_ns();
    if (pl.held) {
        const pkv_status r = a->head_dim == 128 ? launch_held<Fm, 128>(a, p, pl, at, s) : launch_held<Fm, 64>(a, p, pl, at, s);
        if (r != PKV_OK || !pl.spans) return r;
        p.max_rows = kHeldRows;
        at += 2 * pl.hold_k + pl.hold_first + pl.ext;
    }
    p.span_tiles = pl.span_tiles;
    p.spans_max = pl.spans_max;
    p.part_o = reinterpret_cast<float *>(at);
    p.part_ml = reinterpret_cast<float *>(at + pl.part_o);
    p.part_unit = reinterpret_cast<float *>(at + pl.part_o + pl.part_ml);
    at += pl.part_o + pl.part_ml + pl.part_unit;
    p.cuts = reinterpret_cast<int4 *>(at);
    p.off = reinterpret_cast<int32_t *>(at + pl.cuts);
    p.off_ready = pl.plan_launch;
    if (a->head_dim == 128)
        return pl.nt == 1 ? launch<Fm, 128, 1>(who, p, pl, s) : launch<Fm, 128, 2>(who, p, pl, s);
    return pl.nt == 1 ? launch<Fm, 64, 1>(who, p, pl, s) : launch<Fm, 64, 2>(who, p, pl, s);
}
// The workspace of a call that needs `need` bytes.
static pkv_status check_workspace(const char *who, const void *ws, size_t ws_bytes, size_t need) {
    if (ws_bytes < need) return fail(PKV_ERR_CAPACITY, "%s: workspace of %zu bytes, %zu needed", who, ws_bytes, need);
    if (!ws || !aligned(ws, 256))
        return fail(PKV_ERR_INVALID_ARG, "%s: workspace must be non-null and 256-byte aligned", who);
    return PKV_OK;
}

}  // namespace qattn
}  // namespace pkv
