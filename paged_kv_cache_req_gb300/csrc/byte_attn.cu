// pkv_byte_decode / pkv_byte_extend / pkv_byte_weights: attention over an 8-bit K/V pool.
//
// Work is cut and handed out as for the 4-bit pool (spans.cuh: spans of tiles, one per warp; a block
// per unit for small calls; held keys for requests with many rows).
//
// Math per 32 keys, in a warp's registers: S^T = K q^T and O^T += V^T P^T, all m16n8k16 with
// fp16 operands and fp32 sums, keys as MMA rows.  An e4m3 code is exact in fp16; q (bf16) is
// taken into fp16 after a power of two per row.  K's scale multiplies the scores.  V's cannot
// wait for the end, as it differs from tile to tile: a weight takes 2^(E - M) before it is rounded
// to fp16, M being the largest E of the warp's tiles so far (`unit`), and the sums are in units of
// 2^M; where M grows they are multiplied by 2^(M_old - M).  So nothing is past fp16 (weights
// are at most 2^15), and a weight is 2^-11 relative down to 2^(M - E - 25) of the row's largest.
//
// Lane (r, c) = (lane / 4, lane % 4) holds dims D/4 c ... of key row r for K, and dims D/8 r
// ... of keys of column c for V, as the 4-bit kernel's do; codes of two keys are interleaved before
// V's conversion, so that one gives the pair of keys that the MMA wants.
//
// What bounds it: with one row per head a large call reads the pool at 6.3 TB/s (64 requests x 16384 keys, 8 heads of
// 128: 344 us; 4096 keys: 97 us, of which 16 are the table, first copies, uneven ends and the merge).  On pages of 8, 4, 2
// and 1 the copies of small pieces bound it, made by the warps that do the math: 397, 425, 484 and 633 us.  With 9 to 16
// rows, 16 x 16384 keys take 105 us for 302 MB: 32 % of the tensor pipe, warps waiting for their own last instruction
// (8 warps of 250 registers).  With heads of 64 dims instructions bound it: 64 x 1500 keys x 20 heads in 52 us, 48 % of the ALU.
#include "byte_weigh.cuh"

namespace pkv {
namespace qattn {
namespace {

template <int D, int NT>
struct State8 : qattn::State<D, NT> {
    float unit;       // M - 127: the sums are in units of 2^unit (kNoUnit: no key yet)
    float *logits;    // row 2 c of the unit's logits, where they are asked for
    int rows;         // rows of the unit from there on
};

// 2^d of an integer d <= 0 (0 below the normal numbers).
__device__ __forceinline__ float down_by(float d) { return __int_as_float(max(0, static_cast<int>(d) + 127) << 23); }

template <int D, int kT_, int kNT>
struct Quant8 {
    static constexpr int kDim = D, kT = kT_;
    static constexpr bool kUnits = true, kHeldBf16V = true;
    static constexpr const char *kExtend = "pkv_byte_extend";
    // A stage is a tile of 64 keys, or of 32 (D = 128 and 16 rows, for 8 warps in place of 6: 64 requests x 4
    // rows over up to 16384 keys 98 us for 101): K codes [keys][D], V codes [keys][D], or where pieces are smaller but 2 KB or more (kT = 16, or 0: of
    // the pool's t slots) those as they lie.  In each line of 128 bytes the eight 16-byte chunks are swapped about, chunk x ^ (line %
    // 8), by the tensor copies or by the lanes that copy: the keys that eight lanes read at a time lie a
    // line apart or more, and so in different banks.  Beside it the scales: 16 bytes of a piece with its
    // own two among them, 4 where kT is 0 or 1.
    static constexpr int kKeys = D == 128 && kNT == 2 ? 32 : 64, kAlign = 1024, kAux = 256;
    static constexpr uint32_t kStageBytes = 2 * kKeys * D;
    static constexpr int kLines = kKeys == 64 ? D : D / 4;   // of the box that one tensor copy of a 64-slot tile brings
    static constexpr int warps(int nt) { return D == 64 ? 12 : nt == 2 ? 8 : 6; }
    static constexpr int stages(int nt) { return D == 128 && nt == 2 ? 3 : 2; }
    template <int NT>
    using State = State8<D, NT>;

    // Pieces of 2 KB or more are copied as boxes, smaller ones (kT = 1) 16 bytes per lane; where kT is 0 or 1 the
    // lanes copy the scales.  (One row of 64 requests x 4096 keys x 8 kv heads, per lane / as boxes: 128 dims, pages of 32
    // 111.2 / 103.4 us, 16 110.9 / 100.8, 8 113.3 / 111.8, 4 118.2 / 125.7; 64 dims, pages of 32 61.7 / 59.7, 8 63.1 / 64.3.)
    static constexpr int kSmall = 1024 / D;
    __host__ __device__ static constexpr bool gathers(int) { return kT == 1; }
    __device__ __forceinline__ static int arrivals(int) { return kT >= 16 ? 1 : kT == 1 ? 32 : 33; }   // at a stage's barrier
    // A piece: its address, or where it is copied as a box its tile, counted from 1.
    __device__ __forceinline__ static const uint8_t *piece(const Params &p, int slot, int kh) {
        if (!gathers(p.t_shift)) return reinterpret_cast<const uint8_t *>(static_cast<uintptr_t>((slot >> p.t_shift) + 1));
        return piece_at<D>(p, slot, kh);
    }
    __device__ __forceinline__ static void zero_piece(const Stage &stage, int j, int ps) {
        const int bytes = kT > kKeys ? 2 * kKeys * D : 2 * D << ps;
        if (gathers(ps)) {
            for (int part = 0; part < 2; ++part)
                for (int o = 0; o < bytes / 2; o += 16)
                    *reinterpret_cast<uint4 *>(stage.codes + part * kKeys * D + swapped(j * (bytes / 2) + o)) = make_uint4(0, 0, 0, 0);
        } else {   // (whole lines)
            for (int o = 0; o < bytes; o += 16) *reinterpret_cast<uint4 *>(stage.codes + j * bytes + o) = make_uint4(0, 0, 0, 0);
        }
        if (kT < 16)
            reinterpret_cast<uint32_t *>(stage.aux)[j] = 0x01010101u;
        else
            reinterpret_cast<uint4 *>(stage.aux)[j] = make_uint4(0x01010101u, 0x01010101u, 0x01010101u, 0x01010101u);
    }
    // Copies a tile's n pieces (from key `half` of a larger one on), `live` of them on good pages; piece i of
    // the window is lane i % 32's src[i / 32].
    __device__ __forceinline__ static void copy(const Params &p, int kh, const uint8_t *const (&src)[2], int first, int n,
                                                uint32_t live, int ps, int half, const Stage &stage, uint64_t *bar, int lane) {
        // the scale bytes of a tile, in whole units of `unit`
        auto scales = [&](int64_t tile, int unit) {
            return p.pool + tile * p.tile_stride + (static_cast<int64_t>(p.hkv) * 2 * D << p.t_shift) + (2 * kh & ~(unit - 1));
        };
        if constexpr (kT != 1) {
            const uint32_t bytes = kT > kKeys ? 2 * kKeys * D : 2 * D << ps;
            if (lane == (first & 31)) mbar_arrive_expect_tx(bar, live * (bytes + (kT == 0 ? 0 : 16)));
            if (kT != 64) __syncwarp();   // (with one piece the same lane copies)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int j = 32 * i + lane - first;
                if (j >= 0 && j < n && src[i]) {
                    const int tile = static_cast<int>(reinterpret_cast<uintptr_t>(src[i])) - 1;
                    const int line = kh * ((2 * D << p.t_shift) / 128);
                    if (kT > kKeys) {   // K's half of the tile, and V's
                        tma_load_3d(stage.codes, &p.map, 0, line + half * D / 128, tile, bar);
                        tma_load_3d(stage.codes + kKeys * D, &p.map, 0, line + (kT + half) * D / 128, tile, bar);
                    } else {
                        tma_load_3d(stage.codes + j * bytes, &p.map, 0, line, tile, bar);
                    }
                    if (kT == 0)
                        cp_async_small<4>(stage.aux + j * 4, scales(tile, 4));
                    else
                        bulk_load(stage.aux + j * 16, scales(tile, 16), 16, bar);
                }
            }
            if (kT == 0) arrive_with_copies(bar);
            return;
        }
        constexpr int kRow = D / 16, kRounds = kKeys * kRow / 32;   // 16 bytes per lane; rounds for K (and V)
        const uint8_t *low = first < 32 ? src[0] : src[1];          // (only 64 pieces lie in both)
        const int at = first & 31, c = lane % kRow;
#pragma unroll 8
        for (int i = 0; i < kRounds; ++i) {
            const int row = i * (32 / kRow) + lane / kRow, j = row >> ps;
            const uint8_t *a = from_lane(kKeys == 64 && ps == 0 && i >= kRounds / 2 ? src[1] : low, (at + j) & 31);
            if (!a) continue;
            a += (row & ((1 << ps) - 1)) * D + c * 16;
            uint8_t *dst = stage.codes + swapped(row * D + c * 16);
            cp_async_16(dst, a, 16);
            cp_async_16(dst + kKeys * D, a + (D << ps), 16);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int j = 32 * i + lane - first;
            if (j >= 0 && j < (kKeys >> ps) && src[i])
                cp_async_small<4>(stage.aux + j * 4, src[i] + (static_cast<int64_t>(p.hkv - kh) * 2 * D << ps) + (2 * kh & ~3));
        }
        arrive_with_copies(bar);
    }

    // Where byte `at` of a run of lines that begins on a multiple of 1024 is.
    __device__ __forceinline__ static int swapped(int at) { return at ^ ((at >> 3) & 0x70); }
    // Byte `at` of the codes (part 0 = K, 1 = V) of key k of the 16-key group kt of the stage's `step`-th 32 keys.
    // (Where the group's place does not depend on t it begins on a multiple of 1024, so the swap is a lane's own.)
    __device__ __forceinline__ static const uint8_t *codes(const Params &p, const Stage &stage, int step, int part, int kt, int k, int at) {
        const int group = step * kGroups + kt;
        if (kT == 0) {
            const int key = group * 16 + k, in = key & ((1 << p.t_shift) - 1);
            return stage.codes + swapped(((key - in) * 2 + in + (part << p.t_shift)) * D + at);
        }
        return stage.codes + (kT == 16 ? group * (32 * D) + part * (16 * D) : part * (kKeys * D) + group * (16 * D)) + swapped(k * D + at);
    }
    // Its two scale bytes.
    __device__ __forceinline__ static uint32_t scale_bytes(const Params &p, const Stage &stage, int step, int kt, int k, int kh) {
        const int group = step * kGroups + kt;
        int at = kT == 64 ? (2 * kh & 15) : group * 16 + (2 * kh & 15);
        if (kT < 16) at = ((group * 16 + k) >> p.t_shift) * 4 + (2 * kh & 3);
        return *reinterpret_cast<const uint16_t *>(stage.aux + at);
    }

    // One step: a stage's `step`-th 32 keys, the unit's key0 ....  With kMask some row's bound or the unit's
    // last key lies among them.
    template <int NT, bool kMask>
    __device__ __forceinline__ static void step(const Params &p, State<NT> &st, const Stage &stage, int step, int key0, int keys, int kh,
                                                int lane) {
        const int r = lane >> 2, c = lane & 3;
        constexpr int KS = D / 16;     // contraction steps of q.k, and 16-row blocks of O^T
        float s[kGroups][NT][4];
        uint32_t w[kGroups][2][D / 16];
        float ks[kGroups][2], ve[kGroups][2];   // K's scale and log2 of V's, of keys kt * 16 + r + 8 u
#pragma unroll
        for (int kt = 0; kt < kGroups; ++kt)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
#pragma unroll
                for (int i = 0; i < D / 64; ++i) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(codes(p, stage, step, 0, kt, r + 8 * u, c * (D / 4) + 16 * i));
                    w[kt][u][4 * i] = x.x; w[kt][u][4 * i + 1] = x.y; w[kt][u][4 * i + 2] = x.z; w[kt][u][4 * i + 3] = x.w;
                }
                const uint32_t e = scale_bytes(p, stage, step, kt, r + 8 * u, kh);
                ks[kt][u] = byte::scale_value(e & 0xff);
                ve[kt][u] = static_cast<float>(e >> 8) - 127.f;
                // (pieces past the last key were not copied)
                if (kMask && kT != 64 && key0 + kt * 16 + (kT == 16 ? 0 : r + 8 * u) >= keys) ve[kt][u] = kNoUnit;
#pragma unroll
                for (int n = 0; n < NT; ++n) s[kt][n][2 * u] = s[kt][n][2 * u + 1] = 0.f;
            }
#pragma unroll
        for (int i = 0; i < KS; ++i)
#pragma unroll
            for (int kt = 0; kt < kGroups; ++kt) {
                const uint32_t a0 = byte::lo_to_f16(w[kt][0][i]), a1 = byte::lo_to_f16(w[kt][1][i]);
                const uint32_t a2 = byte::hi_to_f16(w[kt][0][i]), a3 = byte::hi_to_f16(w[kt][1][i]);
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_f16(s[kt][n], a0, a1, a2, a3, st.q[i][n][0], st.q[i][n][1]);
            }
        {   // the unit of the sums
            float most = ve[0][0];
            if (kT != 64) {
                most = fmaxf(fmaxf(ve[0][0], ve[0][1]), fmaxf(ve[1][0], ve[1][1]));
                if (kT < 16) most = static_cast<float>(__reduce_max_sync(0xffffffffu, static_cast<int>(most)));
            }
            if (most > st.unit) {
                const float corr = down_by(st.unit - most);
                st.unit = most;
#pragma unroll
                for (int t = 0; t < KS; ++t)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) st.o[t][n][i] *= corr;
            }
#pragma unroll
            for (int kt = 0; kt < kGroups; ++kt)
#pragma unroll
                for (int u = 0; u < 2; ++u) ve[kt][u] = down_by(ve[kt][u] - st.unit);
        }
        // softmax: s[kt][n][2 u + w] is key kt * 16 + r + 8 u of row 8 n + 2 c + w, from here on a base-2 logit
        uint32_t pt[kGroups][NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float top[2];   // of this lane's keys
#pragma unroll
            for (int v = 0; v < 2; ++v) {
#pragma unroll
                for (int kt = 0; kt < kGroups; ++kt)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        float &x = s[kt][n][2 * u + v];
                        // (the factor stays normal and finite, so that 0 stays 0)
                        x *= fminf(fmaxf(st.f[n][v] * ks[kt][u], 1.2e-38f), 3.4e38f);
                        if (kMask && key0 + kt * 16 + r + 8 * u >= st.end[n][v]) x = -INFINITY;
                    }
                top[v] = fmaxf(fmax3(s[0][n][v], s[0][n][2 + v], s[1][n][v]), s[1][n][2 + v]);
            }
            if (p.logits) {   // (base 2; a key that no row sees is not among them)
#pragma unroll
                for (int v = 0; v < 2; ++v)
                    if (8 * n + v < st.rows)
#pragma unroll
                        for (int kt = 0; kt < kGroups; ++kt)
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                const int key = key0 + kt * 16 + r + 8 * u;
                                if (!kMask || key < keys) st.logits[(8 * n + v) * p.logit_stride + key] = s[kt][n][2 * u + v];
                            }
            }
            // the maximum is looked for across lanes only when some logit passes it by kLazy
            if (__any_sync(0xffffffffu, top[0] + st.nm[n][0] > st.limit[n][0] || top[1] + st.nm[n][1] > st.limit[n][1])) {
#pragma unroll
                for (int v = 0; v < 2; ++v) {
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) top[v] = fmaxf(top[v], __shfl_xor_sync(0xffffffffu, top[v], o));
                    if (top[v] + st.nm[n][v] > st.limit[n][v]) {
                        const bool fresh = st.limit[n][v] == -INFINITY;
                        const float nm = kLift - top[v];
                        const float corr = fresh ? 0.f : ex2(nm - st.nm[n][v]);
                        st.nm[n][v] = nm;
                        st.limit[n][v] = kLift + kLazy;
                        st.l[n][v] *= corr;
#pragma unroll
                        for (int t = 0; t < KS; ++t) {
                            st.o[t][n][v] *= corr;
                            st.o[t][n][2 + v] *= corr;
                        }
                    }
                }
            }
            const uint64_t nm2 = pair(st.nm[n][0], st.nm[n][1]);
            uint64_t sum = pair(st.l[n][0], st.l[n][1]);
#pragma unroll
            for (int kt = 0; kt < kGroups; ++kt)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float2 y = unpair(add2(pair(s[kt][n][2 * u], s[kt][n][2 * u + 1]), nm2));
                    const float x0 = ex2(y.x), x1 = ex2(y.y);
                    sum = add2(sum, pair(x0, x1));
                    pt[kt][n][u] = transpose_8x8(pack_f16x2(x0 * ve[kt][u], x1 * ve[kt][u]));
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
                uint32_t x[2][D / 32];   // codes of the two keys, D/8 dims each
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int k = 2 * c + e + 8 * u;
                    const uint8_t *cp = codes(p, stage, step, 1, kt, k, r * (D / 8));
                    if (D == 128) {
                        const uint4 y = *reinterpret_cast<const uint4 *>(cp);
                        x[e][0] = y.x; x[e][1] = y.y; x[e][D / 32 - 2] = y.z; x[e][D / 32 - 1] = y.w;
                    } else {
                        const uint2 y = *reinterpret_cast<const uint2 *>(cp);
                        x[e][0] = y.x; x[e][1] = y.y;
                    }
                    if (kMask) {
                        // nothing of a key past the unit's last, and no NaN that only some rows may see
                        const bool in = key0 + kt * 16 + k < keys;
#pragma unroll
                        for (int i = 0; i < D / 32; ++i) {
                            const uint32_t nan = byte::nan_bytes(x[e][i]);
                            bad |= in && nan;
                            x[e][i] = in ? x[e][i] & ~nan : 0;
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    const uint32_t lo = __byte_perm(x[0][i], x[1][i], 0x5140), hi = __byte_perm(x[0][i], x[1][i], 0x7362);
                    a[u][0][2 * i] = byte::lo_to_f16(lo);
                    a[u][1][2 * i] = byte::hi_to_f16(lo);
                    a[u][0][2 * i + 1] = byte::lo_to_f16(hi);
                    a[u][1][2 * i + 1] = byte::hi_to_f16(hi);
                }
            }
#pragma unroll
            for (int t = 0; t < KS; ++t)
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    mma_f16(st.o[t][n], a[0][0][t], a[0][1][t], a[1][0][t], a[1][1][t], pt[kt][n][0], pt[kt][n][1]);
            if (kMask && __any_sync(0xffffffffu, bad)) {
                // the rows that see a key with a NaN in V get it in that dim
                for (int k = 0; k < 16; ++k) {
                    const int key = key0 + kt * 16 + k;
                    if (key >= keys) continue;
                    const uint8_t *cp = codes(p, stage, step, 1, kt, k, r * (D / 8));
#pragma unroll
                    for (int t = 0; t < KS; ++t)
#pragma unroll
                        for (int odd = 0; odd < 2; ++odd) {
                            if ((cp[2 * t + odd] & 0x7f) != 0x7f) continue;
#pragma unroll
                            for (int n = 0; n < NT; ++n)
#pragma unroll
                                for (int v = 0; v < 2; ++v)
                                    if (key < st.end[n][v]) st.o[t][n][2 * odd + v] = __int_as_float(0x7fffffff);
                        }
                }
            }
        }
    }

    template <int NT>
    __device__ __forceinline__ static void start(const Params &p, const Work &w, State<NT> &st, const uint32_t (&ahead)[D / 8], int lane) {
        // (queries below 2^-119 have factors below fp32's normal numbers; large keys' scales bring them back)
        start_segment<D, NT>(p, w, st, ahead, lane, 0.f);
        st.unit = kNoUnit;
        if (p.logits) {   // (one query row per request)
            const int row = w.rb * 8 * NT + 2 * (lane & 3);
            st.logits = p.logits + (static_cast<int64_t>(w.qo0) * p.hq + w.kh * p.g + row) * p.logit_stride;
            st.rows = p.g - row;
        }
    }

    // The segment's rows: normalised to the output when it is the whole unit, else a partial
    // (see Work::slot).
    template <int NT>
    __device__ __forceinline__ static void finish(const Params &p, const Work &s, State<NT> &st, int lane) {
        const int r = lane >> 2, c = lane & 3;
        constexpr int W = D / 8;   // dims of a lane: D/8 r ...
        const int64_t slot = s.slot;
        const float one = power_of_two(st.unit);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                float l = st.l[n][v];
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
                const int lr = n * 8 + 2 * c + v, row = s.rb * 8 * NT + lr, tok = token_of(p, row), hh = row - tok * p.g;
                if (tok >= s.n) continue;
                if (slot < 0) {
                    const int64_t at = static_cast<int64_t>(s.qo0 + tok) * p.hq + s.kh * p.g + hh;
                    const float inv = l == 0.f ? 0.f : rcp(l);   // (one / l may be outside fp32's normal numbers)
                    uint32_t h[W / 2];
#pragma unroll
                    for (int t = 0; t < D / 16; ++t) h[t] = pack_bf16x2(st.o[t][n][v] * inv * one, st.o[t][n][2 + v] * inv * one);
                    uint4 *dst = reinterpret_cast<uint4 *>(p.out + at * D + r * W);
#pragma unroll
                    for (int i = 0; i < W / 8; ++i) dst[i] = make_uint4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
                    if (r == 0 && p.lse) p.lse[at] = l == 0.f ? -INFINITY : (log2f(l) - st.nm[n][v]) * kLn2;
                } else {
                    float4 *dst = reinterpret_cast<float4 *>(p.part_o + (slot * 8 * NT + lr) * D + r * W);
#pragma unroll
                    for (int i = 0; i < W / 4; ++i)
                        dst[i] = make_float4(st.o[2 * i][n][v], st.o[2 * i][n][2 + v], st.o[2 * i + 1][n][v], st.o[2 * i + 1][n][2 + v]);
                    if (r == 0) {
                        reinterpret_cast<float2 *>(p.part_ml)[slot * 8 * NT + lr] = make_float2(l == 0.f ? -INFINITY : -st.nm[n][v], l);
                        p.part_unit[slot * 8 * NT + lr] = st.unit;
                    }
                }
            }
    }

    // Two fp32 as bf16, at most its largest number: a value of 2^128 (code 256 at the largest scale) would be infinite, and
    // times the weight of a row that does not see its key, 0, NaN.  NaN stays.
    __device__ __forceinline__ static uint32_t to_bf16x2(float lo, float hi) {
        uint32_t r;
        asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
    // Sixteen dims of a held row: both as bf16, which has the range for any scale.
    struct Block {
        uint4 codes;
        uint32_t scale;
    };
    __device__ __forceinline__ static Block load_block(const Params &p, int64_t slot, int kh, bool is_v, int j) {
        const int t = 1 << p.t_shift, at = static_cast<int>(slot & (t - 1));
        const uint8_t *a = piece_at<D>(p, slot, kh);
        Block b;
        b.codes = __ldg(reinterpret_cast<const uint4 *>(a + (is_v ? t * D : 0) + at * D + j * 16));
        b.scale = __ldg(scales_at<D>(p, a, kh) + is_v);
        return b;
    }
    __device__ __forceinline__ static bool has_nan(const Block &b) {
        return (byte::nan_bytes(b.codes.x) | byte::nan_bytes(b.codes.y) | byte::nan_bytes(b.codes.z) | byte::nan_bytes(b.codes.w)) != 0;
    }
    // `any`: V holds a NaN for the key
    __device__ __forceinline__ static void hold(const Block &b, bool is_v, bool any, uint32_t (&x)[8]) {
        const uint32_t w[4] = {b.codes.x, b.codes.y, b.codes.z, b.codes.w};
        const float s = byte::scale_value(b.scale);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 f = quant::f16x2_to_f32(i % 2 ? byte::hi_to_f16(w[i / 2]) : byte::lo_to_f16(w[i / 2]));
            x[i] = any ? (is_v ? 0u : 0x7fff7fffu) : to_bf16x2(f.x * s, f.y * s);
        }
    }
};

// ---------------------------------------------------------------- host side
int64_t tile_of(const pkv_byte_args *a) {
    return byte::tile_bytes(std::min(a->page_size, quant::kMaxTile), a->head_dim, a->num_kv_heads);
}
Shape shape_of(const pkv_byte_args *a) { return a->head_dim == 128 ? shape<Quant8<128, 0, 1>, Quant8<128, 0, 2>>(tile_of(a)) : shape<Quant8<64, 0, 1>, Quant8<64, 0, 2>>(tile_of(a)); }

enum Call { kDecode, kExtend, kWeights };
const char *const kNames[] = {"pkv_byte_decode", "pkv_byte_extend", "pkv_byte_weights"};

pkv_status check(const pkv_byte_args *a, Call call, bool check_ptrs) {
    const char *who = kNames[call];
    const pkv_status st = validate(who, a, call != kDecode, check_ptrs, tile_of, call != kWeights);
    if (st != PKV_OK) return st;
    if (call == kExtend && (a->acc_out || a->acc_in))
        return fail(PKV_ERR_INVALID_ARG, "%s: acc_in and acc_out must be NULL (pkv_byte_weights takes the rows)", who);
    if (!a->acc_out && a->acc_in) return fail(PKV_ERR_INVALID_ARG, "%s: acc_in without acc_out", who);
    if (call == kWeights || a->acc_out) {
        if (a->layout != PKV_LAYOUT_REQ_TO_TOKEN) return fail(PKV_ERR_UNSUPPORTED, "%s: weights need the token-table layout", who);
        if (a->acc_row_stride < a->r2t_width) return fail(PKV_ERR_INVALID_ARG, "%s: acc_row_stride smaller than the table's width", who);
        if (a->batch > 65535 || a->num_kv_heads > 65535) return fail(PKV_ERR_UNSUPPORTED, "%s: weights of more than 65535 requests or kv heads", who);
    }
    if (call == kWeights && check_ptrs && a->batch > 0 && (!a->lse || !a->acc_out))
        return fail(PKV_ERR_INVALID_ARG, "%s: null lse/acc_out", who);
    return PKV_OK;
}

// Workspace of the weights: partial sums of given rows, or a decode's logits (and its lse where the
// caller wants none).  Logits move 8 bytes per key and query head, where reading K again moves
// head_dim per kv head and takes the scores a second time: for 32 requests of 128 to 8192 keys, 32
// heads over 8 of 128, decode and weights took 52 us together so (42 now), and 87 with a second pass over K.
struct WeighPlan {
    size_t part, lse;
    int64_t stride;          // floats of a row of logits
};
WeighPlan weigh_plan(const pkv_byte_args *a, Call call) {
    WeighPlan w{};
    w.stride = (static_cast<int64_t>(a->max_seq_len) + 7) / 8 * 8;
    const size_t rows = static_cast<size_t>(call == kDecode ? a->num_q_heads : a->num_kv_heads) * a->batch;
    w.part = up256(rows * static_cast<size_t>(call == kDecode ? w.stride : a->max_seq_len) * 4);
    w.lse = call == kWeights || a->lse ? 0 : up256(static_cast<size_t>(a->total_q) * a->num_q_heads * 4);
    return w;
}

size_t size_of(const pkv_byte_args *a, Call call) {
    if (!a || check(a, call, false) != PKV_OK) return 0;
    if (call == kWeights) return std::max<size_t>(weigh_plan(a, call).part, 256);
    const size_t n = workspace_size(a, call == kExtend, shape_of(a));
    if (n == 0 || call == kExtend || !a->acc_out) return n;
    const WeighPlan w = weigh_plan(a, call);
    return n + w.part + w.lse;
}

// The map of a pool whose pieces are copied as boxes.
bool encode_pool(const pkv_byte_args *a, int nt, Params &p) {
    if (1 << p.t_shift < (a->head_dim == 128 ? Quant8<128, 0, 1>::kSmall : Quant8<64, 0, 1>::kSmall)) return true;
    const uint32_t lines = static_cast<uint32_t>((2 * a->head_dim << p.t_shift) / 128);
    const uint64_t dims[3] = {64, static_cast<uint64_t>(a->num_kv_heads) * lines, static_cast<uint64_t>(std::max<int64_t>(1, a->num_tiles))};
    const uint64_t strides[2] = {128, static_cast<uint64_t>(a->tile_stride)};
    auto box_lines = [&](auto kt) {
        constexpr int kT = decltype(kt)::value;
        if (a->head_dim == 128) return nt == 1 ? Quant8<128, kT, 1>::kLines : Quant8<128, kT, 2>::kLines;
        return nt == 1 ? Quant8<64, kT, 1>::kLines : Quant8<64, kT, 2>::kLines;
    };
    const int height = p.t_shift == 6 ? box_lines(std::integral_constant<int, 64>{}) : static_cast<int>(lines);
    const uint32_t box[3] = {64, static_cast<uint32_t>(height), 1};
    return encode_tmap_bf16(&p.map, a->pool, 3, dims, strides, box);   // (pairs of bytes)
}

pkv_status run(const pkv_byte_args *a, Call call, void *ws, size_t ws_bytes, int32_t *err, cudaStream_t s) {
    const char *who = kNames[call];
    if (!a) return fail(PKV_ERR_INVALID_ARG, "%s: null args", who);
    if (!err) return fail(PKV_ERR_INVALID_ARG, "%s: err_flags is required", who);
    pkv_status st = check(a, call, true);
    if (st != PKV_OK) return st;
    if (a->batch == 0 || (a->total_q == 0 && call != kWeights)) return ok();
    Params p = params(a, err);
    const size_t need = size_of(a, call);
    if (need == 0) return fail(PKV_ERR_UNSUPPORTED, "%s: too many splits, keys or requests", who);
    st = check_workspace(who, ws, ws_bytes, need);
    if (st != PKV_OK) return st;
    char *at = static_cast<char *>(ws);
    if (call == kWeights) {
        p.wait_ns = wait_limit_ns();
        // rows of a request and kv head: at most max_q_len's, or what the average says
        const int64_t most = a->max_q_len > 0 ? a->max_q_len : (a->total_q + a->batch - 1) / a->batch;
        const WeighParams wp{a->lse, reinterpret_cast<float *>(at), a->acc_in, a->acc_out, a->acc_row_stride};
        // keys: total_kv, or half of what max_seq_len allows
        const int64_t keys = a->total_kv > 0 ? a->total_kv : static_cast<int64_t>(a->batch) * a->max_seq_len / 2;
        return launch_weigh(who, p, wp, a->head_dim, most * p.g, keys, s);
    }
    Plan pl;
    if (!make_plan(a, call == kExtend, shape_of(a), pl)) return fail(PKV_ERR_UNSUPPORTED, "%s: too many splits, keys or requests", who);
    if ((pl.unit || pl.spans) && !encode_pool(a, pl.nt, p)) return fail(PKV_ERR_CUDA, "%s: cuTensorMapEncodeTiled rejected the pool", who);
    if (!a->acc_out) return attend<Quant8>(who, a, pl, p, at, s);
    if (a->max_seq_len == 0) return attend<Quant8>(who, a, pl, p, at, s);
    const WeighPlan w = weigh_plan(a, call);
    p.logits = reinterpret_cast<float *>(at);
    p.logit_stride = w.stride;
    if (!p.lse) p.lse = reinterpret_cast<float *>(at + w.part);
    const Params q = p;
    st = attend<Quant8>(who, a, pl, p, at + w.part + w.lse, s);
    if (st != PKV_OK) return st;
    return launch_finish(who, q, WeighParams{q.lse, nullptr, a->acc_in, a->acc_out, a->acc_row_stride}, s);
}

}  // namespace
}  // namespace qattn
}  // namespace pkv

extern "C" size_t pkv_byte_decode_workspace_size(const pkv_byte_args *args) { return pkv::qattn::size_of(args, pkv::qattn::kDecode); }
extern "C" size_t pkv_byte_extend_workspace_size(const pkv_byte_args *args) { return pkv::qattn::size_of(args, pkv::qattn::kExtend); }
extern "C" size_t pkv_byte_weights_workspace_size(const pkv_byte_args *args) { return pkv::qattn::size_of(args, pkv::qattn::kWeights); }
extern "C" pkv_status pkv_byte_decode(const pkv_byte_args *args, void *workspace, size_t workspace_bytes, int32_t *err_flags,
                                    pkv_stream_t stream) {
    return pkv::qattn::run(args, pkv::qattn::kDecode, workspace, workspace_bytes, err_flags, reinterpret_cast<cudaStream_t>(stream));
}
extern "C" pkv_status pkv_byte_extend(const pkv_byte_args *args, void *workspace, size_t workspace_bytes, int32_t *err_flags,
                                    pkv_stream_t stream) {
    return pkv::qattn::run(args, pkv::qattn::kExtend, workspace, workspace_bytes, err_flags, reinterpret_cast<cudaStream_t>(stream));
}
extern "C" pkv_status pkv_byte_weights(const pkv_byte_args *args, void *workspace, size_t workspace_bytes, int32_t *err_flags,
                                     pkv_stream_t stream) {
    return pkv::qattn::run(args, pkv::qattn::kWeights, workspace, workspace_bytes, err_flags, reinterpret_cast<cudaStream_t>(stream));
}
