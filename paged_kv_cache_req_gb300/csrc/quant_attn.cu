// pkv_quant_decode / pkv_quant_extend: attention over a 4-bit K/V pool, in three ways.
//
// Spans (attend_kernel, merge_kernel).  A unit is (request, block of 8 NT query rows, kv
// head); its rows are the (token, query head) pairs of the heads that share the kv head, its
// keys tiles of 64.  All units' tiles in order (request, row block, kv head) form one sequence
// that is cut into equal spans, one per warp of a grid of one block per SM, whatever the
// requests' lengths.  A warp works alone: it copies the tiles of its span into its own ring
// of stages, and no warp waits for another.  A unit inside one span is written by its warp;
// one that a span boundary cuts leaves an fp32 partial per span for merge_kernel.
// One block per unit (unit_kernel): small calls, whose time is latency.
// Held keys (hold_kernel, then the tcgen05 kernel of extend.cu): requests with many query rows.
//
// Math per 32 keys, in the warp's registers, keys as MMA rows so that 8 query rows fill an
// n = 8 tile: S^T = K q^T, then P^T through movmatrix, O^T += V^T P^T, all m16n8k16 with
// fp16 operands and fp32 sums.  (A decode has 1 to 16 rows per kv head: the 128 rows of a
// tcgen05 tile would be mostly padding, and K and V would first have to be written out to
// shared memory as 16-bit values, 3.6 times what is read.)  A code times its block scale is exact in fp16; q
// (bf16) is taken into fp16 exactly too, after a power of two per row that brings its
// largest magnitude to [64, 128) (elements more than 2^23 below the largest lose bits: 2^-31
// of it at most).  The
// dims are assigned to the MMA's contraction (and output row) indices so that a lane reads
// contiguous codes: lane (r, c) = (lane / 4, lane % 4) holds dims D/4 c ... of key row r for
// K, and dims D/8 r ... of keys of column c for V.  Softmax in base 2 with a running
// maximum per row.  P is rounded to fp16: by at most 2^-11 of a weight (2^-8 in the bf16 kernels)
// down to 2^-25 of the row's largest, where fp16's subnormals begin, and by at most 2^-36 of the
// largest below that, which is also where weights become 0 (the sum that divides them is fp32
// and keeps them).
//
// What bounds it: instructions as much as bytes.  At D = 128 a tile of 64 keys has 256
// conversions of two codes, which issue every second cycle, and 256 fp16 products at the
// same rate; an SM makes a tile in 174 ns, and its share of the copy rate is one in 206.
// Hence V's codes of two keys are interleaved before they are converted (a conversion then
// gives the pair of keys that the MMA wants, for half the permutes), the maximum is looked
// for across lanes only when some score passes it, and a step is 32 keys: 16 need fewer
// registers and less code but took 71 us where 32 take 66 (16 requests x 16384 keys x 8 kv
// heads), 64 gained 4 % on long requests of 64 dims and lost as much on short ones.
// Measured at 8 kv heads of 128, 32 query heads, page size 64: 128 requests of 128 to 16384
// keys 99 us, 5.0 TB/s, fixed costs included; 90 % of the copy rate per further request.
// Some 19 us of a call do not depend on the keys: start and tile table 6, first copies and
// last tiles, merge 5.
#include "spans.cuh"

namespace pkv {
namespace qattn {
namespace {

// The span kernel runs one block per SM, which holds all the shared memory: a second block of
// a persistent grid could be left without room where the launch before still has a block,
// and then starts when the others end.  Its warps (as many as their registers allow) and
// the stages of a warp's ring.
constexpr int warps_per_sm(int d, int nt) { return nt == 2 && d == 128 ? 8 : 12; }
constexpr int ring_stages(int d, int nt) { return d == 128 && nt == 1 ? 2 : 3; }
// The stage of a tile has the layout of a 64-slot pool tile, or of four 16-slot ones, whatever
// the pool's: with constant addresses the math of a tile takes less time than with the pool's
// tile size looked up.  kT is 64 or 16 for pools of such tiles, copied as they lie (a bulk
// copy each); 0 for the others, copied part by part: K codes, V codes, K scales, V scales.
// Of those, tiles of 32 slots are four bulk copies each, and those of up to 8 slots are copied
// 16 bytes per lane: a bulk copy keeps the SM's copy unit busy for some 18 cycles whatever its
// size.  Measured, in us, over bulk copies of whole pieces with their tile size looked up by
// the math: 16 requests x 16384 keys x 8 kv heads of 128, page size 1: 129 / 114, 2: 101 / 91,
// 4: 87 / 83, 8: 81 / 80, 32: 78 / 76; of 64: 105 / 79, 77 / 63, 62 / 55, 57 / 53, 54 / 51.
constexpr int kGatherShift = 3;   // log2 of the slots
template <int kT>
__device__ __forceinline__ bool gathers(int t_shift) { return kT == 0 && t_shift <= kGatherShift; }
// Copies the pieces of a tile (2^ps slots each) of 32 slots or fewer into the stage; piece i's
// address is lane (first + i) % 32's src[(first + i) / 32], null for one that is not copied.
// `bar` counts each lane's arrival where the warp copies itself, else the bytes.
template <int D>
__device__ __forceinline__ void copy_parts(const uint8_t *const (&src)[2], int first, int ps, uint8_t *stage, uint64_t *bar, int lane) {
    const uint8_t *low = first < 32 ? src[0] : src[1];   // (only 64 pieces lie in both)
    first &= 31;
    const int t = 1 << ps;
    if (!gathers<0>(ps)) {
        const int pieces = 64 >> ps, j = lane & (pieces - 1), part = lane >> (6 - ps);
        const uint8_t *a = from_lane(low, first + j);
        if (part < 4 && a) {
            const int size = part < 2 ? t * (D / 2) : t * (D / 16);
            const int before = part < 2 ? part * (D / 2) : D + (part - 2) * (D / 16);   // bytes per slot of the parts before
            bulk_load(stage + before * 64 + j * size, a + before * t, size, bar);
        }
        return;
    }
    // codes: 16 bytes per lane, whole pieces at a time, each K then V
    constexpr int kHalf = 64 * D / 16 / 32 / 2;          // rounds for 32 slots
    if (D == 128 && ps == 3) {                           // two rounds for a piece
#pragma unroll
        for (int i = 0; i < kHalf; ++i) {
            const uint8_t *a = from_lane(low, first + i);
            if (!a) continue;
            cp_async_16(stage + i * 512 + lane * 16, a + lane * 16, 16);
            cp_async_16(stage + 32 * D + i * 512 + lane * 16, a + 512 + lane * 16, 16);
        }
    } else {
        const int per = ilog2_of(D / 16) + ps;           // log2 of a piece's 16 bytes, at most 5
        const int in = lane & ((1 << per) - 1), part = in >> (per - 1), c = in & ((1 << (per - 1)) - 1);
        uint8_t *dst = stage + part * (32 * D) + (lane >> per) * (t * (D / 2)) + c * 16;
        const int step = 32 >> per;
        int j = first + (lane >> per);
#pragma unroll
        for (int i = 0; i < 2 * kHalf; ++i, j += step, dst += 512 / 2) {
            const uint8_t *a = from_lane(ps == 0 && i >= kHalf ? src[1] : low, j & 31);
            if (a) cp_async_16(dst, a + in * 16, 16);
        }
    }
    // scales: 4, 8 or 16 bytes per lane
    const int unit = min(4, ps + ilog2_of(D / 16));      // log2 of the bytes
    const int per = ps + ilog2_of(D / 8) - unit;         // log2 of a piece's
    const int in = lane & ((1 << per) - 1), part = in >> (per - 1), c = in & ((1 << (per - 1)) - 1);
    uint8_t *dst = stage + 64 * D + part * (4 * D) + (lane >> per) * (t * (D / 16)) + (c << unit);
    const int step = 32 >> per, rounds = (64 * D / 8 >> unit) / 32;
    int j = first + (lane >> per);
    for (int i = 0; i < rounds; ++i, j += step, dst += 16 << unit) {
        const uint8_t *a = from_lane(ps == 0 && i >= rounds / 2 ? src[1] : low, j & 31);
        if (!a) continue;
        a += t * D + (in << unit);
        if (unit == 4) cp_async_16(dst, a, 16);
        else if (unit == 3) cp_async_small<8>(dst, a);
        else cp_async_small<4>(dst, a);
    }
    arrive_with_copies(bar);
}
// Zeros in place of piece j.
template <int D, int kT>
__device__ __forceinline__ void zero_piece(uint8_t *stage, int j, int ps) {
    const int t = 1 << ps;
    if (kT != 0) {
        uint32_t *w = reinterpret_cast<uint32_t *>(stage + j * quant::tile_bytes(kT, D));
        for (int o = 0; o < quant::tile_bytes(kT, D) / 4; ++o) w[o] = 0;
        return;
    }
    for (int part = 0; part < 2; ++part) {
        uint32_t *codes = reinterpret_cast<uint32_t *>(stage + part * (32 * D) + j * t * (D / 2));
        uint32_t *scales = reinterpret_cast<uint32_t *>(stage + 64 * D + part * (4 * D) + j * t * (D / 16));
        for (int o = 0; o < t * (D / 8); ++o) codes[o] = 0;
        for (int o = 0; o < t * (D / 64); ++o) scales[o] = 0;
    }
}
// Where key `k` (a lane's part) of the 16-key group `kt` of a step lies: every address is a
// lane's base and a constant.
template <int D, int kT>
struct Rows {
    const uint8_t *codes_at, *scales_at;   // the step's first 16-slot tile, or its half of the 64-slot one
    __device__ __forceinline__ Rows(const uint8_t *stage, int step) {
        codes_at = scales_at = stage;
        if (kT != 16) {
            codes_at += step * (kStep * D / 2);
            scales_at += step * (kStep * D / 16);
        } else {
            codes_at += step * (kStep / 16) * quant::tile_bytes(16, D);
            scales_at = codes_at;
        }
    }
    static constexpr int kSlots = kT == 16 ? 16 : 64;
    __device__ __forceinline__ static int piece(int kt) { return kT == 16 ? kt * quant::tile_bytes(16, D) : 0; }
    __device__ __forceinline__ static int slot(int kt, int k) { return kT == 16 ? k : kt * 16 + k; }
    // its codes (part 0 = K, 1 = V), and its scales
    __device__ __forceinline__ const uint8_t *codes(int part, int kt, int k) const {
        return codes_at + piece(kt) + part * kSlots * (D / 2) + slot(kt, k) * (D / 2);
    }
    __device__ __forceinline__ const uint8_t *scales(int part, int kt, int k) const {
        return scales_at + piece(kt) + kSlots * D + part * kSlots * (D / 16) + slot(kt, k) * (D / 16);
    }
};

// Key of row / column i of a 16-key group: i with its low bit flipped in the upper half of
// each eight, so that the four keys a quarter-warp reads of V lie in two bank groups.
__device__ __forceinline__ int key_of(int i) { return i ^ ((i >> 2) & 1); }

// One step: 32 keys, the unit's key0 ..., in half `step` of a stage.  With kMask some row's
// bound or the unit's last key lies among them.
template <int D, int NT, int kT, bool kMask>
__device__ __forceinline__ void tile_step(const Params &p, State<D, NT> &st, const uint8_t *stage, int step, int key0,
                                          int keys, int lane) {
    const int r = lane >> 2, c = lane & 3;
    constexpr int KS = D / 16;     // contraction steps of q.k, and 16-row blocks of O^T
    const Rows<D, kT> rows(stage, step);
    float s[kGroups][NT][4];
    // q.k a word (eight dims per lane) at a time over the groups of 16 keys: their MMAs
    // are independent of one another
    uint32_t w[kGroups][2][D / 32], sc[kGroups][2];
#pragma unroll
    for (int kt = 0; kt < kGroups; ++kt)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int k = key_of(r) + 8 * u;
            const uint8_t *cp = rows.codes(0, kt, k) + c * (D / 8), *sp = rows.scales(0, kt, k) + c * (D / 64);
            if (D == 128) {
                const uint4 x = *reinterpret_cast<const uint4 *>(cp);
                w[kt][u][0] = x.x;
                w[kt][u][1] = x.y;
                w[kt][u][D / 64] = x.z;
                w[kt][u][D / 32 - 1] = x.w;
                sc[kt][u] = quant::scales_to_f16(*reinterpret_cast<const uint16_t *>(sp));
            } else {
                const uint2 x = *reinterpret_cast<const uint2 *>(cp);
                w[kt][u][0] = x.x;
                w[kt][u][1] = x.y;
                sc[kt][u] = quant::scales_to_f16(*sp);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) s[kt][n][2 * u] = s[kt][n][2 * u + 1] = 0.f;
        }
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int kt = 0; kt < kGroups; ++kt) {
            uint32_t h[2][4];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                // D = 128: the lane's 32 dims are two blocks, two words each
                const uint32_t sb = __byte_perm(sc[kt][u], 0, D == 64 || i < 2 ? 0x1010 : 0x3232);
                quant::codes_to_f16(w[kt][u][i], h[u]);
#pragma unroll
                for (int e = 0; e < 4; ++e) h[u][e] = quant::mul_f16x2(h[u][e], sb);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    mma_f16(s[kt][n], h[0][2 * j], h[1][2 * j], h[0][2 * j + 1], h[1][2 * j + 1], st.q[2 * i + j][n][0],
                            st.q[2 * i + j][n][1]);
        }
    // softmax: s[kt][n][2 u + w] is key kt * 16 + key_of(r) + 8 u of row 8 n + 2 c + w
    uint32_t pt[kGroups][NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        float top[2];   // of this lane's keys
#pragma unroll
        for (int w = 0; w < 2; ++w) {
#pragma unroll
            for (int kt = 0; kt < kGroups; ++kt)
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    if (kMask && key0 + kt * 16 + key_of(r) + 8 * u >= st.end[n][w]) s[kt][n][2 * u + w] = -INFINITY;
            top[w] = fmaxf(fmax3(s[0][n][w], s[0][n][2 + w], s[1][n][w]), s[1][n][2 + w]);
        }
        // the maximum is looked for across lanes only when some score passes it by 2^kLazy (by the
        // exponent that its weight would have, so that no weight is past fp16)
        if (__any_sync(0xffffffffu, fmaf(top[0], st.f[n][0], st.nm[n][0]) > st.limit[n][0] ||
                                        fmaf(top[1], st.f[n][1], st.nm[n][1]) > st.limit[n][1])) {
#pragma unroll
            for (int w = 0; w < 2; ++w) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) top[w] = fmaxf(top[w], __shfl_xor_sync(0xffffffffu, top[w], o));
                if (fmaf(top[w], st.f[n][w], st.nm[n][w]) > st.limit[n][w]) {
                    const bool fresh = st.limit[n][w] == -INFINITY;
                    const float nm = kLift - top[w] * st.f[n][w];
                    const float corr = fresh ? 0.f : ex2(nm - st.nm[n][w]);
                    st.nm[n][w] = nm;
                    st.limit[n][w] = kLift + kLazy;
                    st.l[n][w] *= corr;
#pragma unroll
                    for (int t = 0; t < KS; ++t) {
                        st.o[t][n][w] *= corr;
                        st.o[t][n][2 + w] *= corr;
                    }
                }
            }
        }
        const uint64_t f2 = pair(st.f[n][0], st.f[n][1]), nm2 = pair(st.nm[n][0], st.nm[n][1]);
        uint64_t sum = pair(st.l[n][0], st.l[n][1]);
#pragma unroll
        for (int kt = 0; kt < kGroups; ++kt)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const float2 y = unpair(fma2(pair(s[kt][n][2 * u], s[kt][n][2 * u + 1]), f2, nm2));
                const float x0 = ex2(y.x), x1 = ex2(y.y);
                sum = add2(sum, pair(x0, x1));
                pt[kt][n][u] = transpose_8x8(pack_f16x2(x0, x1));
            }
        const float2 l = unpair(sum);
        st.l[n][0] = l.x;
        st.l[n][1] = l.y;
    }
#pragma unroll
    for (int kt = 0; kt < kGroups; ++kt) {
        uint32_t a[2][2][KS];      // [keys 2c.. / 2c + 8..][even / odd dim][16-row block]
        bool bad = false;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            uint32_t w[2][D / 64];   // codes of the two keys, D/8 dims each
            uint32_t sc[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int k = key_of(2 * c + e) + 8 * u;
                const uint8_t *cp = rows.codes(1, kt, k) + r * (D / 16);
                sc[e] = rows.scales(1, kt, k)[D == 128 ? r : r >> 1];
                if (kMask) {
                    // nothing of a key past the unit's last, and no NaN that only some rows may see
                    const bool in = key0 + kt * 16 + k < keys;
                    const bool nan = (sc[e] & 0x7f) == 0x7f;
                    bad |= in && nan;
                    if (!in || nan) sc[e] = 0;
                }
                if (D == 128) {
                    const uint2 x = *reinterpret_cast<const uint2 *>(cp);
                    w[e][0] = x.x;
                    w[e][D / 64 - 1] = x.y;
                } else {
                    w[e][0] = *reinterpret_cast<const uint32_t *>(cp);
                }
            }
            const uint32_t sp = quant::scales_to_f16(sc[0] | (sc[1] << 8));
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                // bytes (first key, second key) of the even dims, and of the odd ones
                const uint32_t even = (w[0][i] & 0x0f0f0f0fu) | ((w[1][i] << 4) & 0xf0f0f0f0u);
                const uint32_t odd = ((w[0][i] >> 4) & 0x0f0f0f0fu) | (w[1][i] & 0xf0f0f0f0u);
                uint32_t x[4], y[4];
                quant::codes_to_f16(even, x);
                quant::codes_to_f16(odd, y);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    a[u][0][4 * i + t] = quant::mul_f16x2(x[t], sp);
                    a[u][1][4 * i + t] = quant::mul_f16x2(y[t], sp);
                }
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
                if (key >= keys || (rows.scales(1, kt, k)[D == 128 ? r : r >> 1] & 0x7f) != 0x7f) continue;
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

// The segment's rows: normalised to the output when it is the whole unit, else the partial
// of slot 0 of its span (a unit that began at or before it), or of slot 1.
template <int D, int NT>
__device__ __forceinline__ void finish_segment(const Params &p, const Work &s, State<D, NT> &st, int lane) {
    const int r = lane >> 2, c = lane & 3;
    constexpr int W = D / 8;   // dims of a lane: D/8 r ...
    const int64_t slot = s.slot;
    const bool whole = slot < 0;
    const float gv = p.v_scale ? p.v_scale[s.kh] : 1.f;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            float l = st.l[n][v];
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            const int lr = n * 8 + 2 * c + v, row = s.rb * 8 * NT + lr, tok = token_of(p, row), hh = row - tok * p.g;
            if (tok >= s.n) continue;
            if (whole) {
                const int64_t at = static_cast<int64_t>(s.qo0 + tok) * p.hq + s.kh * p.g + hh;
                const float inv = l == 0.f ? 0.f : rcp(l);   // (gv / l may be below fp32's normal numbers)
                uint32_t h[W / 2];
#pragma unroll
                for (int t = 0; t < D / 16; ++t) h[t] = pack_bf16x2(st.o[t][n][v] * inv * gv, st.o[t][n][2 + v] * inv * gv);
                uint4 *dst = reinterpret_cast<uint4 *>(p.out + at * D + r * W);
#pragma unroll
                for (int i = 0; i < W / 8; ++i) dst[i] = make_uint4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
                if (r == 0 && p.lse) p.lse[at] = l == 0.f ? -INFINITY : (log2f(l) - st.nm[n][v]) * kLn2;
            } else {
                float4 *dst = reinterpret_cast<float4 *>(p.part_o + (slot * 8 * NT + lr) * D + r * W);
#pragma unroll
                for (int i = 0; i < W / 4; ++i)
                    dst[i] = make_float4(st.o[2 * i][n][v], st.o[2 * i][n][2 + v], st.o[2 * i + 1][n][v], st.o[2 * i + 1][n][2 + v]);
                if (r == 0) reinterpret_cast<float2 *>(p.part_ml)[slot * 8 * NT + lr] = make_float2(l == 0.f ? -INFINITY : -st.nm[n][v], l);
            }
        }
}

template <int D, int kT_, int>
struct Quant4 {
    static constexpr int kDim = D, kT = kT_;
    static constexpr bool kUnits = false, kHeldBf16V = false;
    static constexpr int kAlign = 128, kKeys = 64, kAux = 0, kSmall = 0;
    static constexpr const char *kExtend = "pkv_quant_extend";
    static constexpr uint32_t kStageBytes = quant::tile_bytes(kKeys, D);
    static constexpr int warps(int nt) { return warps_per_sm(D, nt); }
    static constexpr int stages(int nt) { return ring_stages(D, nt); }
    template <int NT>
    using State = qattn::State<D, NT>;

    __device__ __forceinline__ static bool gathers(int t_shift) { return qattn::gathers<kT>(t_shift); }
    __device__ __forceinline__ static int arrivals(int t_shift) { return gathers(t_shift) ? 32 : 1; }   // at a stage's barrier
    __device__ __forceinline__ static const uint8_t *piece(const Params &p, int slot, int kh) {
        return p.pool + static_cast<int64_t>(slot >> p.t_shift) * p.tile_stride + static_cast<int64_t>(kh) * quant::tile_bytes(1 << p.t_shift, D);
    }
    __device__ __forceinline__ static void zero_piece(const Stage &stage, int j, int ps) { qattn::zero_piece<D, kT>(stage.codes, j, ps); }
    // Copies a tile's n pieces, `live` of them on good pages; piece i of the window is lane i % 32's src[i / 32].
    __device__ __forceinline__ static void copy(const Params &, int, const uint8_t *const (&src)[2], int first, int n, uint32_t live,
                                                int ps, int, const Stage &to, uint64_t *bar, int lane) {
        uint8_t *stage = to.codes;
        const uint32_t bytes = quant::tile_bytes(1 << ps, D);
        if (!gathers(ps)) {
            if (lane == (first & 31)) mbar_arrive_expect_tx(bar, live * bytes);
            if (kT != 64) __syncwarp();   // (with one piece the same lane copies)
        }
        if (kT == 64) {
            const uint8_t *a = first < 32 ? src[0] : src[1];
            if (lane == (first & 31) && a) bulk_load(stage, a, bytes, bar);
        } else if (kT == 16) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int j = 32 * i + lane - first;
                if (j >= 0 && j < n && src[i]) bulk_load(stage + j * bytes, src[i], bytes, bar);
            }
        } else {
            copy_parts<D>(src, first, ps, stage, bar, lane);
        }
    }
    template <int NT, bool kMask>
    __device__ __forceinline__ static void step(const Params &p, State<NT> &st, const Stage &stage, int step, int key0, int keys, int,
                                                int lane) {
        tile_step<D, NT, kT, kMask>(p, st, stage.codes, step, key0, keys, lane);
    }
    template <int NT>
    __device__ __forceinline__ static void start(const Params &p, const Work &w, State<NT> &st, const uint32_t (&ahead)[D / 8], int lane) {
        start_segment<D, NT>(p, w, st, ahead, lane);
    }
    template <int NT>
    __device__ __forceinline__ static void finish(const Params &p, const Work &w, State<NT> &st, int lane) {
        finish_segment<D, NT>(p, w, st, lane);
    }

    // Sixteen dims of a held row.
    struct Block {
        uint2 codes;
        uint32_t scale;
    };
    __device__ __forceinline__ static Block load_block(const Params &p, int64_t slot, int kh, bool is_v, int j) {
        constexpr int kPerRow = D / 16;
        const int t = 1 << p.t_shift, at = static_cast<int>(slot & (t - 1));
        const uint8_t *tile = p.pool + (slot >> p.t_shift) * p.tile_stride + static_cast<int64_t>(kh) * quant::tile_bytes(t, D);
        Block b;
        b.codes = __ldg(reinterpret_cast<const uint2 *>(tile + (is_v ? t * (D / 2) : 0) + at * (D / 2) + j * 8));
        b.scale = __ldg(tile + t * D + (is_v ? t * kPerRow : 0) + at * kPerRow + j);
        return b;
    }
    __device__ __forceinline__ static bool has_nan(const Block &b) { return (b.scale & 0x7f) == 0x7f; }
    // `any`: V holds a NaN for the key
    __device__ __forceinline__ static void hold(Block &b, bool is_v, bool any, uint32_t (&x)[8]) {
        if (any) b.scale = is_v ? 0 : quant::kNanScale;
        const uint32_t s2 = quant::scales_to_f16(b.scale | (b.scale << 8));
        quant::codes_to_f16(b.codes.x, *reinterpret_cast<uint32_t(*)[4]>(x));
        quant::codes_to_f16(b.codes.y, *reinterpret_cast<uint32_t(*)[4]>(x + 4));
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x[e] = quant::mul_f16x2(x[e], s2);
            if (!is_v) {
                const float2 f = quant::f16x2_to_f32(x[e]);
                x[e] = pack_bf16x2(f.x, f.y);
            }
        }
    }
};

int64_t tile_of(const pkv_quant_args *a) {
    return static_cast<int64_t>(a->num_kv_heads) * quant::tile_bytes(std::min(a->page_size, quant::kMaxTile), a->head_dim);
}
Shape shape_of(const pkv_quant_args *a) { return a->head_dim == 128 ? shape<Quant4<128, 0, 1>, Quant4<128, 0, 2>>(tile_of(a)) : shape<Quant4<64, 0, 1>, Quant4<64, 0, 2>>(tile_of(a)); }

size_t size_of(const char *who, const pkv_quant_args *a, bool extend) {
    if (!a || validate(who, a, extend, false, tile_of) != PKV_OK) return 0;
    return workspace_size(a, extend, shape_of(a));
}

pkv_status attend4(const char *who, const pkv_quant_args *a, bool extend, void *ws, size_t ws_bytes, int32_t *err, cudaStream_t s) {
    if (!a) return fail(PKV_ERR_INVALID_ARG, "%s: null args", who);
    if (!err) return fail(PKV_ERR_INVALID_ARG, "%s: err_flags is required", who);
    pkv_status st = validate(who, a, extend, true, tile_of);
    if (st != PKV_OK) return st;
    if (a->batch == 0 || a->total_q == 0) return ok();
    Plan pl;
    if (!make_plan(a, extend, shape_of(a), pl)) return fail(PKV_ERR_UNSUPPORTED, "%s: too many splits, keys or requests", who);
    st = check_workspace(who, ws, ws_bytes, std::max<size_t>(pl.bytes(), 256));
    if (st != PKV_OK) return st;
    Params p = params(a, err);
    p.k_scale = a->k_scale;
    p.v_scale = a->v_scale;
    return attend<Quant4>(who, a, pl, p, static_cast<char *>(ws), s);
}

}  // namespace
}  // namespace qattn
}  // namespace pkv

extern "C" size_t pkv_quant_decode_workspace_size(const pkv_quant_args *args) {
    return pkv::qattn::size_of("pkv_quant_decode", args, false);
}
extern "C" size_t pkv_quant_extend_workspace_size(const pkv_quant_args *args) {
    return pkv::qattn::size_of("pkv_quant_extend", args, true);
}
extern "C" pkv_status pkv_quant_decode(const pkv_quant_args *args, void *workspace, size_t workspace_bytes,
                                       int32_t *err_flags, pkv_stream_t stream) {
    return pkv::qattn::attend4("pkv_quant_decode", args, false, workspace, workspace_bytes, err_flags,
                               reinterpret_cast<cudaStream_t>(stream));
}
extern "C" pkv_status pkv_quant_extend(const pkv_quant_args *args, void *workspace, size_t workspace_bytes,
                                       int32_t *err_flags, pkv_stream_t stream) {
    return pkv::qattn::attend4("pkv_quant_extend", args, true, workspace, workspace_bytes, err_flags,
                               reinterpret_cast<cudaStream_t>(stream));
}
