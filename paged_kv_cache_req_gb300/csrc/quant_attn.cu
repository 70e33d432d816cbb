// pkv_quant_decode / pkv_quant_extend: attention over a 4-bit K/V pool.
//
// Work: a unit is (request, block of 8 NT query rows, kv head); its rows are the (token,
// query head) pairs of the heads that share the kv head, its keys tiles of 64.  All units'
// tiles in order (request, row block, kv head) form one sequence that is cut into equal
// spans, one per warp of a persistent grid, whatever the requests' lengths.  A warp works
// alone: it fetches the tiles of its span into its own ring of stages with bulk copies
// (one per page of at most 64 keys: the pool keeps all that attention reads of it in one
// piece), and no warp waits for another.  A unit inside one span is written by its warp; one
// that a span boundary cuts leaves an fp32 partial per span for merge_kernel.
//
// Math per tile, in the warp's registers, keys as MMA rows so that 8 query rows fill an
// n = 8 tile: S^T = K q^T, then P^T through movmatrix, O^T += V^T P^T, all m16n8k16 with
// fp16 operands and fp32 sums.  A code times its block scale is exact in fp16; q (bf16) is
// taken into fp16 exactly too, after a power of two per row that brings its largest
// magnitude to [64, 128) (elements 2^-30 below the largest lose bits).  The dims are
// assigned to the MMA's contraction (and output row) indices so that a lane reads
// contiguous codes: lane (r, c) = (lane / 4, lane % 4) holds dims D/4 c ... of key row r for
// K, and dims D/8 r ... of keys of column c for V.  Softmax in base 2 with a running
// maximum per row.
#include <algorithm>
#include <cmath>

#include "quant.cuh"

namespace pkv {
namespace qattn {

using quant::Table;

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kTile = 64;           // keys per stage
constexpr int kMaxStages = 4;
constexpr int kTableInSmem = 256;   // requests whose tile offsets every CTA computes for itself
constexpr float kLn2 = 0.69314718055994531f, kLog2e = 1.44269504088896341f;

struct Params {
    Table tab;
    int32_t batch, hq, hkv, g, t_shift, stages;
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
    float *part_o, *part_ml; // per span two slots: [rows][D], and [rows] of (m, l)
    int64_t *off;            // [B + 1] first tile of each request, then the tiles of a span
    int32_t off_ready;       // written by plan_kernel (large batches)
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Two floats -> fp16 pair (to nearest even), lo in the low half.
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
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
__device__ __forceinline__ bool wait_for(uint64_t *bar, uint32_t parity, uint64_t limit_ns) {
    if (mbar_try_wait(bar, parity)) return true;
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
    }
    return r;
}
__device__ __forceinline__ int unit_tiles(int L) { return max(1, (L + kTile - 1) / kTile); }
template <int NT>
__device__ __forceinline__ int row_blocks(const Params &p, int n) { return (n * p.g + 8 * NT - 1) / (8 * NT); }

// off[b] = first tile of request b's units, off[B] = all tiles, off[B + 1] = tiles per
// span, by the block's threads.
template <int NT, int kBlock>
__device__ __forceinline__ void build_table(const Params &p, int64_t *off, long long *scratch, bool report) {
    const int B = p.batch, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int seg = (B + kBlock - 1) / kBlock, lo = min(B, tid * seg), hi = min(B, lo + seg);
    long long local = 0;
    for (int b = lo; b < hi; ++b) {
        const Req r = load_req(p, b, report);
        local += static_cast<long long>(row_blocks<NT>(p, r.n)) * p.hkv * unit_tiles(r.L);
        off[b + 1] = local;
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
    for (int b = lo; b < hi; ++b) off[b + 1] += before;
    if (tid == 0) {
        off[0] = 0;
        off[B + 1] = p.span_tiles ? p.span_tiles : max(1ll, (total + p.spans_max - 1) / p.spans_max);
    }
    __syncthreads();
}

template <int NT>
__global__ void __launch_bounds__(1024) plan_kernel(const Params p) {
    pdl_wait();          // inputs may come from the previous kernel of the stream
    pdl_launch_next();
    __shared__ long long scratch[32];
    build_table<NT, 1024>(p, p.off, scratch, true);
}

// The part of one unit that lies in one span.
struct Segment {
    int64_t base;            // of the request's page list
    int64_t pos, end;        // its tiles in the sequence of all tiles
    int b, kh, rb, L, n, qo0;
    int t0, t1;              // its tiles within the unit
    int tiles;               // of the unit
};

template <int NT>
__device__ __forceinline__ Segment segment_at(const Params &p, const int64_t *off, int64_t pos, int64_t span_end) {
    int lo = 0, hi = p.batch;   // the last request with off[b] <= pos (those without rows have no tiles)
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (off[mid] <= pos) lo = mid; else hi = mid;
    }
    Segment s;
    const Req r = load_req(p, lo, false);
    s.b = lo;
    s.L = r.L;
    s.n = r.n;
    s.qo0 = r.qo0;
    s.base = r.base;
    s.tiles = unit_tiles(r.L);
    const int64_t rem = pos - off[lo];
    const int64_t u = rem / s.tiles;
    s.t0 = static_cast<int>(rem - u * s.tiles);
    s.rb = static_cast<int>(u / p.hkv);
    s.kh = static_cast<int>(u - static_cast<int64_t>(s.rb) * p.hkv);
    s.t1 = static_cast<int>(min(static_cast<int64_t>(s.tiles), s.t0 + span_end - pos));
    s.pos = pos;
    s.end = pos + (s.t1 - s.t0);
    return s;
}

// Keys that some row of the unit may see: the causal bound of its last token, or all.
template <int NT>
__device__ __forceinline__ int unit_keys(const Params &p, const Segment &s) {
    if (!p.qo_indptr || p.kv_end) return s.L;
    const int last = min(s.n, ((s.rb + 1) * 8 * NT - 1) / p.g + 1);   // tokens up to the block's last row
    return s.L - s.n + last;
}

// Walks the tiles of a span that have keys to fetch, one call per tile.
template <int NT>
struct Fetcher {
    Segment s;
    int64_t span_end;
    int t, t_end, keys;      // next tile of the segment; end of those with keys; unit_keys
    bool done;

    __device__ __forceinline__ void enter(const Params &p, const int64_t *off, int64_t pos) {
        for (;;) {
            if (pos >= span_end) {
                done = true;
                return;
            }
            s = segment_at<NT>(p, off, pos, span_end);
            keys = unit_keys<NT>(p, s);
            t = s.t0;
            t_end = min(s.t1, (keys + kTile - 1) / kTile);
            if (t < t_end) return;
            pos = s.end;
        }
    }
    __device__ __forceinline__ void start(const Params &p, const int64_t *off, int64_t begin, int64_t end) {
        span_end = end;
        done = false;
        enter(p, off, begin);
    }
    __device__ __forceinline__ void next(const Params &p, const int64_t *off) {
        if (++t >= t_end) enter(p, off, s.end);
    }
};

// Pieces (pages, or their first 64 keys) of a tile that lane `lane` fetches: piece lane and,
// on pages of one key, lane + 32.  -3: past the unit's keys.
struct Pieces {
    int64_t slot[2];
};
template <int NT>
__device__ __forceinline__ Pieces look_up(const Params &p, const Fetcher<NT> &f, int lane) {
    Pieces x;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int key = f.t * kTile + ((lane + 32 * i) << p.t_shift);
        x.slot[i] = -3;
        if (!f.done && ((lane + 32 * i) << p.t_shift) < kTile && key < f.keys) x.slot[i] = quant::slot_of(p.tab, f.s.base, key);
    }
    return x;
}
template <int D>
__device__ __forceinline__ void fetch(const Params &p, const Pieces &x, int kh, uint8_t *stage, uint64_t *bar, int lane) {
    const uint32_t bytes = quant::tile_bytes(1 << p.t_shift, D);
    const uint32_t live = __popc(__ballot_sync(0xffffffffu, x.slot[0] >= 0)) +
                          __popc(__ballot_sync(0xffffffffu, x.slot[1] >= 0));
    if (lane == 0) mbar_arrive_expect_tx(bar, live * bytes);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint8_t *dst = stage + (lane + 32 * i) * bytes;
        if (x.slot[i] >= 0) {
            bulk_load(dst, p.pool + (x.slot[i] >> p.t_shift) * p.tile_stride + static_cast<int64_t>(kh) * bytes, bytes, bar);
        } else if (x.slot[i] != -3) {   // a bad page reads as zeros
            raise_flag(p.err, x.slot[i] == -1 ? PKV_DEVERR_RANGE : PKV_DEVERR_CONTIG);
            for (uint32_t o = 0; o < bytes; o += 16) *reinterpret_cast<uint4 *>(dst + o) = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();   // before later copies into this stage
        }
    }
    __syncwarp();
}

// Where the rows of a 16-key group lie in a stage.
template <int D, bool kSmall>
struct Rows {
    const uint8_t *base;   // pages of >= 16 keys: the piece, moved to the group's first key
    int t_shift, in;       // group's first key within its piece
    const uint8_t *stage;
    int key0;
    __device__ __forceinline__ Rows(const uint8_t *st, int k0, int shift) : t_shift(shift), stage(st), key0(k0) {
        const int t = 1 << shift;
        in = k0 & (t - 1);
        base = st + (k0 >> shift) * quant::tile_bytes(t, D);
    }
    // codes of row k of the group (part 0 = K, 1 = V), and its scales
    __device__ __forceinline__ const uint8_t *codes(int part, int k) const {
        const int t = 1 << t_shift;
        if (kSmall) {
            const int key = key0 + k;
            return stage + (key >> t_shift) * quant::tile_bytes(t, D) + part * t * (D / 2) + (key & (t - 1)) * (D / 2);
        }
        return base + part * t * (D / 2) + (in + k) * (D / 2);
    }
    __device__ __forceinline__ const uint8_t *scales(int part, int k) const {
        const int t = 1 << t_shift;
        if (kSmall) {
            const int key = key0 + k;
            return stage + (key >> t_shift) * quant::tile_bytes(t, D) + t * D + part * t * (D / 16) + (key & (t - 1)) * (D / 16);
        }
        return base + t * D + part * t * (D / 16) + (in + k) * (D / 16);
    }
};

// Key of row / column i of a 16-key group: i with its low bit flipped in the upper half of
// each eight, so that the four keys a quarter-warp reads of V lie in two bank groups.
__device__ __forceinline__ int key_of(int i) { return i ^ ((i >> 2) & 1); }

template <int D, int NT>
struct State {
    uint32_t q[D / 16][NT][2];     // fp16 fragments of q
    float f[NT][2];                // score -> base-2 logit, per row of this lane's columns
    int end[NT][2];                // key bound of those rows
    float m[NT][2], l[NT][2];      // running maximum; this lane's share of the sum
    float o[D / 16][NT][4];        // O^T
};

// One tile: keys 64 t ... of the unit.  With kMask some row's bound or the unit's last key
// lies inside the tile.
template <int D, int NT, bool kSmall, bool kMask>
__device__ __forceinline__ void tile_step(const Params &p, State<D, NT> &st, const uint8_t *stage, int key0, int keys,
                                          int lane) {
    const int r = lane >> 2, c = lane & 3;
    constexpr int KS = D / 16;     // contraction steps of q.k, and 16-row blocks of O^T
    float s[4][NT][4];
#pragma unroll
    for (int kt = 0; kt < 4; ++kt) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[kt][n][i] = 0.f;
        const Rows<D, kSmall> rows(stage, kt * 16, p.t_shift);
        uint32_t h[2][D / 8];      // fp16 pairs of this lane's D/4 dims of rows r and r + 8
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int k = key_of(r) + 8 * u;
            const uint8_t *cp = rows.codes(0, k) + c * (D / 8), *sp = rows.scales(0, k) + c * (D / 64);
            if (D == 128) {
                const uint4 w = *reinterpret_cast<const uint4 *>(cp);
                const uint32_t sc = quant::scales_to_f16(*reinterpret_cast<const uint16_t *>(sp));
                const uint32_t s0 = __byte_perm(sc, 0, 0x1010), s1 = __byte_perm(sc, 0, 0x3232);
                const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t x[4];
                    quant::codes_to_f16(ww[i], x);
#pragma unroll
                    for (int e = 0; e < 4; ++e) h[u][i * 4 + e] = quant::mul_f16x2(x[e], i < 2 ? s0 : s1);
                }
            } else {
                const uint2 w = *reinterpret_cast<const uint2 *>(cp);
                const uint32_t sc = quant::scales_to_f16(*sp);
                const uint32_t s0 = __byte_perm(sc, 0, 0x1010);
                const uint32_t ww[2] = {w.x, w.y};
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t x[4];
                    quant::codes_to_f16(ww[i], x);
#pragma unroll
                    for (int e = 0; e < 4; ++e) h[u][i * 4 + e] = quant::mul_f16x2(x[e], s0);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < KS; ++j)
#pragma unroll
            for (int n = 0; n < NT; ++n)
                mma_f16(s[kt][n], h[0][2 * j], h[1][2 * j], h[0][2 * j + 1], h[1][2 * j + 1], st.q[j][n][0], st.q[j][n][1]);
    }
    // softmax: s[kt][n][2 u + w] is key kt * 16 + key_of(r) + 8 u of row 8 n + 2 c + w
    uint32_t pt[4][NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            float top = -INFINITY;
#pragma unroll
            for (int kt = 0; kt < 4; ++kt)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    float &x = s[kt][n][2 * u + w];
                    if (kMask && key0 + kt * 16 + key_of(r) + 8 * u >= st.end[n][w]) x = -INFINITY;
                    top = fmaxf(top, x);
                }
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float mn = fmaxf(st.m[n][w], top * st.f[n][w]);
            const float base = mn == -INFINITY ? 0.f : mn;   // no key yet: every weight is 2^-inf
            const float corr = ex2(st.m[n][w] - base);
            st.m[n][w] = mn;
            float sum = 0.f;
#pragma unroll
            for (int kt = 0; kt < 4; ++kt)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    float &x = s[kt][n][2 * u + w];
                    x = ex2(fmaf(x, st.f[n][w], -base));
                    sum += x;
                }
            st.l[n][w] = fmaf(st.l[n][w], corr, sum);
#pragma unroll
            for (int t = 0; t < KS; ++t) {
                st.o[t][n][w] *= corr;
                st.o[t][n][2 + w] *= corr;
            }
        }
#pragma unroll
        for (int kt = 0; kt < 4; ++kt)
#pragma unroll
            for (int u = 0; u < 2; ++u)
                pt[kt][n][u] = transpose_8x8(pack_f16x2(s[kt][n][2 * u], s[kt][n][2 * u + 1]));
    }
#pragma unroll
    for (int kt = 0; kt < 4; ++kt) {
        const Rows<D, kSmall> rows(stage, kt * 16, p.t_shift);
        uint32_t a[2][2][KS];      // [keys 2c.. / 2c + 8..][even / odd dim][16-row block]
        bool bad = false;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            uint32_t x[2][KS];
            uint32_t sc[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int k = key_of(2 * c + e) + 8 * u;
                const uint8_t *cp = rows.codes(1, k) + r * (D / 16);
                sc[e] = rows.scales(1, k)[D == 128 ? r : r >> 1];
                if (kMask) {
                    // nothing of a key past the unit's last, and no NaN that only some rows may see
                    const bool in = key0 + kt * 16 + k < keys;
                    const bool nan = (sc[e] & 0x7f) == 0x7f;
                    bad |= in && nan;
                    if (!in || nan) sc[e] = 0;
                }
                if (D == 128) {
                    const uint2 w = *reinterpret_cast<const uint2 *>(cp);
                    quant::codes_to_f16(w.x, *reinterpret_cast<uint32_t(*)[4]>(x[e]));
                    quant::codes_to_f16(w.y, *reinterpret_cast<uint32_t(*)[4]>(x[e] + KS / 2));
                } else {
                    quant::codes_to_f16(*reinterpret_cast<const uint32_t *>(cp), *reinterpret_cast<uint32_t(*)[4]>(x[e]));
                }
            }
            const uint32_t sp = quant::scales_to_f16(sc[0] | (sc[1] << 8));
#pragma unroll
            for (int t = 0; t < KS; ++t) {
                a[u][0][t] = quant::mul_f16x2(__byte_perm(x[0][t], x[1][t], 0x5410), sp);
                a[u][1][t] = quant::mul_f16x2(__byte_perm(x[0][t], x[1][t], 0x7632), sp);
            }
        }
#pragma unroll
        for (int t = 0; t < KS; ++t)
#pragma unroll
            for (int n = 0; n < NT; ++n)
                mma_f16(st.o[t][n], a[0][0][t], a[0][1][t], a[1][0][t], a[1][1][t], pt[kt][n][0], pt[kt][n][1]);
        if (kMask && __any_sync(0xffffffffu, bad)) {
            // the rows that see a key whose V block is NaN get it in that block's dims
            for (int k = 0; k < 16; ++k) {
                const int key = key0 + kt * 16 + k;
                if (key >= keys || (rows.scales(1, k)[D == 128 ? r : r >> 1] & 0x7f) != 0x7f) continue;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int w = 0; w < 2; ++w)
                        if (key < st.end[n][w])
#pragma unroll
                            for (int t = 0; t < KS; ++t) st.o[t][n][w] = st.o[t][n][2 + w] = __int_as_float(0x7fffffff);
            }
        }
    }
}

// q fragments, score factors and bounds of a segment's rows; a fresh softmax state.
template <int D, int NT>
__device__ __forceinline__ void start_segment(const Params &p, const Segment &s, State<D, NT> &st, int lane) {
    const int r = lane >> 2, c = lane & 3;
    const float gk = p.k_scale ? p.k_scale[s.kh] : 1.f;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        // this lane's row as an MMA column of q: row 8 n + r, dims D/4 c ...
        const int row = s.rb * 8 * NT + n * 8 + r, tok = row / p.g, hh = row - tok * p.g;
        uint32_t w[D / 8];
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
            st.f[n][v] = fminf(fmaxf(p.scale_log2 * gk * __int_as_float((127 - ev) << 23), 1.2e-38f), 3.4e38f);
            const int rv = s.rb * 8 * NT + n * 8 + 2 * c + v, tv = rv / p.g;
            int end = s.L;   // rows past the last (zeros, never written) ask for no masking
            if (tv < s.n) {
                end = !p.qo_indptr ? s.L : p.kv_end ? __ldg(p.kv_end + s.qo0 + tv) : s.L - s.n + tv + 1;
                if (end < 0 || end > s.L) {
                    if (r == 0 && s.kh == 0 && s.t0 == 0) raise_flag(p.err, PKV_DEVERR_RANGE);
                    end = 0;
                }
            }
            st.end[n][v] = end;
            st.m[n][v] = -INFINITY;
            st.l[n][v] = 0.f;
        }
#pragma unroll
        for (int t = 0; t < D / 16; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) st.o[t][n][i] = 0.f;
    }
}

// The segment's rows: normalised to the output when it is the whole unit, else the partial
// of slot 0 of its span (a unit that began at or before it), or of slot 1.
template <int D, int NT>
__device__ __forceinline__ void finish_segment(const Params &p, const Segment &s, State<D, NT> &st, int64_t slot, int lane) {
    const int r = lane >> 2, c = lane & 3;
    constexpr int W = D / 8;   // dims of a lane: D/8 r ...
    const bool whole = s.t0 == 0 && s.t1 == s.tiles;
    const float gv = p.v_scale ? p.v_scale[s.kh] : 1.f;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            float l = st.l[n][v];
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            const int lr = n * 8 + 2 * c + v, row = s.rb * 8 * NT + lr, tok = row / p.g, hh = row - tok * p.g;
            if (tok >= s.n) continue;
            if (whole) {
                const int64_t at = static_cast<int64_t>(s.qo0 + tok) * p.hq + s.kh * p.g + hh;
                const float inv = l == 0.f ? 0.f : gv / l;
                uint32_t h[W / 2];
#pragma unroll
                for (int t = 0; t < D / 16; ++t) h[t] = pack_bf16x2(st.o[t][n][v] * inv, st.o[t][n][2 + v] * inv);
                uint4 *dst = reinterpret_cast<uint4 *>(p.out + at * D + r * W);
#pragma unroll
                for (int i = 0; i < W / 8; ++i) dst[i] = make_uint4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
                if (r == 0 && p.lse) p.lse[at] = l == 0.f ? -INFINITY : (st.m[n][v] + log2f(l)) * kLn2;
            } else {
                float4 *dst = reinterpret_cast<float4 *>(p.part_o + (slot * 8 * NT + lr) * D + r * W);
#pragma unroll
                for (int i = 0; i < W / 4; ++i)
                    dst[i] = make_float4(st.o[2 * i][n][v], st.o[2 * i][n][2 + v], st.o[2 * i + 1][n][v], st.o[2 * i + 1][n][2 + v]);
                if (r == 0) reinterpret_cast<float2 *>(p.part_ml)[slot * 8 * NT + lr] = make_float2(st.m[n][v], l);
            }
        }
}

template <int D, int NT, bool kSmall>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 3 : 2) attend_kernel(const Params p) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t bars[kWarps * kMaxStages];
    __shared__ long long scratch[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t stage_bytes = (kTile >> p.t_shift) * quant::tile_bytes(1 << p.t_shift, D);
    uint8_t *ring = smem + static_cast<uint32_t>(warp * p.stages) * stage_bytes;
    uint64_t *bar = bars + warp * kMaxStages;
    if (lane == 0) {
        for (int i = 0; i < p.stages; ++i) mbar_init(&bar[i], 1);
        mbar_init_fence();
    }
    __syncwarp();
    pdl_wait();          // inputs may come from the previous kernel of the stream
    pdl_launch_next();
    const int64_t *off = p.off;
    if (!p.off_ready) {
        int64_t *mine = reinterpret_cast<int64_t *>(smem + static_cast<uint32_t>(kWarps * p.stages) * stage_bytes);
        build_table<NT, kThreads>(p, mine, scratch, blockIdx.x == 0);
        if (blockIdx.x == 0)   // for merge_kernel
            for (int i = threadIdx.x; i < p.batch + 2; i += kThreads) p.off[i] = mine[i];
        off = mine;
    }
    if (blockIdx.x == 0 && warp < 2) {   // unusable head scales
        const float *g = warp ? p.v_scale : p.k_scale;
        for (int h = lane; g && h < p.hkv; h += 32)
            if (!quant::good_scale(g[h])) raise_flag(p.err, PKV_DEVERR_RANGE);
    }
    const int64_t total = off[p.batch], per = off[p.batch + 1];
    uint32_t issued = 0, used = 0;   // tiles whose copies were issued, and awaited
    bool ok = true;
    const uint32_t S = p.stages;
    State<D, NT> st;
    for (int64_t sp = static_cast<int64_t>(blockIdx.x) * kWarps + warp; ok && sp * per < total;
         sp += static_cast<int64_t>(gridDim.x) * kWarps) {
        const int64_t begin = sp * per, end = min(total, begin + per);
        Fetcher<NT> f;
        f.start(p, off, begin, end);
        Pieces ahead = look_up(p, f, lane);   // of the next tile to fetch
        auto fetch_next = [&]() {
            if (f.done) return;
            const uint32_t s = issued % S;
            const int kh = f.s.kh;
            const Pieces now = ahead;
            f.next(p, off);
            ahead = look_up(p, f, lane);
            fetch<D>(p, now, kh, ring + s * stage_bytes, &bar[s], lane);
            ++issued;
        };
        for (uint32_t i = 0; i < S; ++i) fetch_next();
        for (int64_t pos = begin; ok && pos < end;) {
            const Segment s = segment_at<NT>(p, off, pos, end);
            const int keys = unit_keys<NT>(p, s);
            start_segment<D, NT>(p, s, st, lane);
            int low = s.L;   // every row sees the keys below it
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int v = 0; v < 2; ++v) low = min(low, st.end[n][v]);
            low = __reduce_min_sync(0xffffffffu, low);
            const int t_end = min(s.t1, (keys + kTile - 1) / kTile);
            for (int t = s.t0; t < t_end; ++t) {
                const uint32_t b = used % S;
                ok = wait_for(&bar[b], (used / S) & 1, p.wait_ns);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if ((t + 1) * kTile <= low)
                    tile_step<D, NT, kSmall, false>(p, st, ring + b * stage_bytes, t * kTile, keys, lane);
                else
                    tile_step<D, NT, kSmall, true>(p, st, ring + b * stage_bytes, t * kTile, keys, lane);
                ++used;
                __syncwarp();
                fetch_next();
            }
            if (!ok) break;
            finish_segment<D, NT>(p, s, st, sp * 2 + (s.t0 == 0 && pos > begin ? 1 : 0), lane);
            pos = s.end;
        }
    }
    if (!ok) {   // a wait ran out: the copies in flight land before the block's memory is given back
        if (lane == 0) raise_flag(p.err, PKV_DEVERR_TIMEOUT);
        for (; used < issued; ++used) mbar_wait(&bar[used % S], (used / S) & 1);
    }
}

// Combines the partials of one row of a unit that spans cut: o = sum 2^(m_i - M) o_i / sum
// 2^(m_i - M) l_i, a warp per share of the partials.
constexpr int kMergeThreads = 256;

template <int D, int NT>
__global__ void __launch_bounds__(kMergeThreads) merge_kernel(const Params p) {
    pdl_wait();          // inputs may come from the previous kernel of the stream
    pdl_launch_next();
    constexpr int W = kMergeThreads / 32, V = D / 32;
    __shared__ float red[W][D];
    __shared__ float red_m[W], red_l[W];
    const int64_t *off = p.off;
    const int64_t per = off[p.batch + 1];
    // grid: (query row, query head)
    const int64_t row = blockIdx.x / p.hq;
    const int head = static_cast<int>(blockIdx.x - row * p.hq), kh = head / p.g;
    int b = static_cast<int>(row);
    if (p.qo_indptr) {
        int lo = 0, hi = p.batch;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (p.qo_indptr[mid] <= row) lo = mid; else hi = mid;
        }
        b = lo;
    }
    const Req rq = load_req(p, b, false);
    const int64_t tok = row - rq.qo0;
    if (tok < 0 || tok >= rq.n) return;
    const int64_t ur = tok * p.g + (head - kh * p.g);
    const int rb = static_cast<int>(ur / (8 * NT)), lr = static_cast<int>(ur - static_cast<int64_t>(rb) * 8 * NT);
    const int tiles = unit_tiles(rq.L);
    const int64_t u0 = off[b] + (static_cast<int64_t>(rb) * p.hkv + kh) * tiles, u1 = u0 + tiles;
    const int64_t s0 = u0 / per, s1 = (u1 - 1) / per;
    if (s0 == s1) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float m = -INFINITY, l = 0.f, o[V];
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = 0.f;
#pragma unroll 2
    for (int64_t s = s0 + warp; s <= s1; s += W) {
        const int64_t at = (s * 2 + (s == s0 && u0 > s * per ? 1 : 0)) * 8 * NT + lr;
        const float2 ml = reinterpret_cast<const float2 *>(p.part_ml)[at];
        if (ml.y == 0.f) continue;   // no key of this row in the span
        float x[V];
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = p.part_o[at * D + lane * V + i];
        const float mn = fmaxf(m, ml.x), base = mn == -INFINITY ? 0.f : mn;
        const float c0 = ex2(m - base), c1 = ex2(ml.x - base);
        m = mn;
        l = l * c0 + ml.y * c1;
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = o[i] * c0 + x[i] * c1;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) red[warp][lane * V + i] = o[i];
    if (lane == 0) {
        red_m[warp] = m;
        red_l[warp] = l;
    }
    __syncthreads();
    float M = -INFINITY, den = 0.f;
    for (int w = 0; w < W; ++w) M = fmaxf(M, red_m[w]);
    const float base = M == -INFINITY ? 0.f : M;
    for (int w = 0; w < W; ++w) den += red_l[w] * ex2(red_m[w] - base);
    const int64_t at = row * p.hq + head;
    const float gv = p.v_scale ? p.v_scale[kh] : 1.f;
    for (int d = threadIdx.x; d < D; d += kMergeThreads) {
        float num = 0.f;
        for (int w = 0; w < W; ++w) num = fmaf(red[w][d], ex2(red_m[w] - base), num);
        p.out[at * D + d] = static_cast<uint16_t>(pack_bf16x2(den == 0.f ? 0.f : num * (gv / den), 0.f));
    }
    if (threadIdx.x == 0 && p.lse) p.lse[at] = den == 0.f ? -INFINITY : (M + log2f(den)) * kLn2;
}

// ------------------------------------------------------------------ host side
static pkv_status validate(const char *who, const pkv_quant_args *a, bool extend, bool check_ptrs) {
    if (a->batch < 0 || a->num_q_heads < 1 || a->num_kv_heads < 1 || a->total_q < 0 || a->total_kv < 0 ||
        a->max_seq_len < 0 || a->num_tiles < 0)
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
    if (a->tile_stride % 16 || a->tile_stride < static_cast<int64_t>(a->num_kv_heads) * quant::tile_bytes(t, a->head_dim))
        return fail(PKV_ERR_INVALID_ARG, "%s: the tile stride must hold all kv heads and be a multiple of 16 bytes", who);
    if (a->q_row_stride < static_cast<int64_t>(a->num_q_heads) * a->head_dim || a->q_row_stride % 8)
        return fail(PKV_ERR_INVALID_ARG, "%s: q_row_stride must hold Hq x head_dim and be 16-byte aligned", who);
    if (a->total_q > INT32_MAX || a->num_tiles * t > INT32_MAX)
        return fail(PKV_ERR_UNSUPPORTED, "%s: more than 2^31 pool slots or query rows", who);
    if (a->batch == 0 || !check_ptrs) return PKV_OK;
    if (!a->q || !a->pool || !a->out) return fail(PKV_ERR_INVALID_ARG, "%s: null q/pool/out", who);
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

// The launch of attend_kernel: rows per unit, grid, spans and the workspace.
struct Plan {
    int nt, grid, stages, spans_max, span_tiles;
    bool plan_launch;
    size_t smem, part_o, part_ml, table;
    size_t bytes() const { return part_o + part_ml + table; }
};

static size_t up256(size_t x) { return (x + 255) / 256 * 256; }

static bool make_plan(const pkv_quant_args *a, Plan &pl) {
    const int g = a->num_q_heads / a->num_kv_heads;
    // rows of a request and kv head, on average: up to 8 fill one n = 8 tile
    const int64_t rows = (std::max<int64_t>(a->total_q, 1) + std::max(a->batch, 1) - 1) / std::max(a->batch, 1) * g;
    pl.nt = rows <= 8 ? 1 : 2;
    const int t = std::min(a->page_size, quant::kMaxTile);
    const size_t stage = static_cast<size_t>(kTile / t) * quant::tile_bytes(t, a->head_dim);
    pl.stages = a->head_dim == 128 ? 2 : 4;
    if (pl.nt == 2) pl.stages = a->head_dim == 128 ? 3 : 4;
    const int sms = std::max(1, sm_count());
    pl.grid = sms * (pl.nt == 1 ? 3 : 2);
    pl.plan_launch = a->batch > kTableInSmem;
    pl.smem = kWarps * pl.stages * stage + (pl.plan_launch ? 0 : (static_cast<size_t>(a->batch) + 2) * 8);
    int64_t spans = static_cast<int64_t>(pl.grid) * kWarps;
    pl.span_tiles = 0;
    if (a->kv_chunk > 0) {
        pl.span_tiles = a->kv_chunk / kTile;
        const int64_t blocks = (a->total_q * g + 8 * pl.nt - 1) / (8 * pl.nt) + a->batch;
        const int64_t tiles = blocks * a->num_kv_heads * ((std::max(1, a->max_seq_len) + kTile - 1) / kTile);
        spans = (tiles + pl.span_tiles - 1) / pl.span_tiles;
    }
    if (spans > INT32_MAX / 64) return false;
    pl.spans_max = static_cast<int>(spans);
    const size_t slots = static_cast<size_t>(spans) * 2 * 8 * pl.nt;
    pl.part_o = up256(slots * a->head_dim * 4);
    pl.part_ml = up256(slots * 8);
    pl.table = up256((static_cast<size_t>(a->batch) + 2) * 8);
    return true;
}

static size_t workspace_size(const pkv_quant_args *a) {
    Plan pl;
    return make_plan(a, pl) ? pl.bytes() : 0;
}

static Params params(const pkv_quant_args *a, int32_t *err) {
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
    p.scale_log2 = a->sm_scale * kLog2e;
    p.total_q = a->total_q;
    p.tile_stride = a->tile_stride;
    p.q_stride = a->q_row_stride;
    p.q = static_cast<const uint16_t *>(a->q);
    p.pool = static_cast<const uint8_t *>(a->pool);
    p.k_scale = a->k_scale;
    p.v_scale = a->v_scale;
    p.qo_indptr = a->qo_indptr;
    p.kv_end = a->kv_end;
    p.out = static_cast<uint16_t *>(a->out);
    p.lse = a->lse;
    p.err = err;
    return p;
}

template <int D, int NT>
static pkv_status launch(const char *who, const Params &p, const Plan &pl, cudaStream_t s) {
    auto *kern = p.t_shift < 4 ? attend_kernel<D, NT, true> : attend_kernel<D, NT, false>;
    std::atomic<int64_t> *set = device_memo(reinterpret_cast<const void *>(kern));
    if (!set) return fail(PKV_ERR_CUDA, "%s: cannot query the current device", who);
    if (set->load() < static_cast<int64_t>(pl.smem)) {   // kernel attributes are per device
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(pl.smem)) != cudaSuccess) {
            (void)cudaGetLastError();
            return fail(PKV_ERR_CUDA, "%s: cannot raise the shared-memory limit", who);
        }
        set->store(static_cast<int64_t>(pl.smem));
    }
    pkv_status st = PKV_OK;
    if (pl.plan_launch) {
        st = launch_status(launch_chained(plan_kernel<NT>, dim3(1), dim3(1024), 0, s, p), who);
        if (st != PKV_OK) return st;
    }
    st = launch_status(launch_chained(kern, dim3(pl.grid), dim3(kThreads), pl.smem, s, p), who);
    if (st != PKV_OK) return st;
    return launch_status(launch_chained(merge_kernel<D, NT>, dim3(static_cast<unsigned>(p.total_q * p.hq)),
                                        dim3(kMergeThreads), 0, s, p), who);
}

static pkv_status attend(const char *who, const pkv_quant_args *a, bool extend, void *ws, size_t ws_bytes, int32_t *err,
                         cudaStream_t s) {
    if (!a) return fail(PKV_ERR_INVALID_ARG, "%s: null args", who);
    if (!err) return fail(PKV_ERR_INVALID_ARG, "%s: err_flags is required", who);
    const pkv_status st = validate(who, a, extend, true);
    if (st != PKV_OK) return st;
    if (a->batch == 0 || a->total_q == 0) return ok();
    Plan pl;
    if (!make_plan(a, pl)) return fail(PKV_ERR_UNSUPPORTED, "%s: too many splits", who);
    const size_t need = pl.bytes();
    if (ws_bytes < need) return fail(PKV_ERR_CAPACITY, "%s: workspace of %zu bytes, %zu needed", who, ws_bytes, need);
    if (!ws || !aligned(ws, 256))
        return fail(PKV_ERR_INVALID_ARG, "%s: workspace must be non-null and 256-byte aligned", who);
    if (a->total_q * a->num_q_heads > INT32_MAX) return fail(PKV_ERR_UNSUPPORTED, "%s: too many query rows", who);
    Params p = params(a, err);
    p.stages = pl.stages;
    p.wait_ns = wait_limit_ns();
    p.span_tiles = pl.span_tiles;
    p.spans_max = pl.spans_max;
    p.part_o = static_cast<float *>(ws);
    p.part_ml = reinterpret_cast<float *>(static_cast<char *>(ws) + pl.part_o);
    p.off = reinterpret_cast<int64_t *>(static_cast<char *>(ws) + pl.part_o + pl.part_ml);
    p.off_ready = pl.plan_launch;
    if (a->head_dim == 128)
        return pl.nt == 1 ? launch<128, 1>(who, p, pl, s) : launch<128, 2>(who, p, pl, s);
    return pl.nt == 1 ? launch<64, 1>(who, p, pl, s) : launch<64, 2>(who, p, pl, s);
}

}  // namespace qattn
}  // namespace pkv

extern "C" size_t pkv_quant_decode_workspace_size(const pkv_quant_args *args) {
    using namespace pkv::qattn;
    if (!args || validate("pkv_quant_decode", args, false, false) != PKV_OK) return 0;
    return workspace_size(args);
}
extern "C" size_t pkv_quant_extend_workspace_size(const pkv_quant_args *args) {
    using namespace pkv::qattn;
    if (!args || validate("pkv_quant_extend", args, true, false) != PKV_OK) return 0;
    return workspace_size(args);
}
extern "C" pkv_status pkv_quant_decode(const pkv_quant_args *args, void *workspace, size_t workspace_bytes,
                                       int32_t *err_flags, pkv_stream_t stream) {
    return pkv::qattn::attend("pkv_quant_decode", args, false, workspace, workspace_bytes, err_flags,
                              reinterpret_cast<cudaStream_t>(stream));
}
extern "C" pkv_status pkv_quant_extend(const pkv_quant_args *args, void *workspace, size_t workspace_bytes,
                                       int32_t *err_flags, pkv_stream_t stream) {
    return pkv::qattn::attend("pkv_quant_extend", args, true, workspace, workspace_bytes, err_flags,
                              reinterpret_cast<cudaStream_t>(stream));
}
