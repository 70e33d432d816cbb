// pkv_quant_decode / pkv_quant_extend: attention over a 4-bit K/V pool.
//
// One CTA per (query row, query head): each warp takes every kWarps-th key of the row's
// bound, its lanes the head dims, with its own online softmax; the warps' states are
// combined at the end.
#include <algorithm>
#include <cmath>

#include "quant.cuh"

namespace pkv {
namespace qattn {

using quant::Table;

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr float kLn2 = 0.69314718055994531f, kLog2e = 1.44269504088896341f;

struct Params {
    Table tab;
    int32_t batch, hq, hkv, g, t_shift;
    float scale_log2;
    int64_t total_q, tile_stride, q_stride;
    const uint16_t *q;
    const uint8_t *pool;
    const float *k_scale, *v_scale;
    const int32_t *qo_indptr, *kv_end;
    uint16_t *out;
    float *lse;
    int32_t *err;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Query rows of request b (0 for a malformed qo_indptr, or for causal rows without their keys).
__device__ __forceinline__ int q_count(const Params &p, int b, int L, bool report) {
    if (!p.qo_indptr) return 1;
    const int64_t lo = p.qo_indptr[b], hi = p.qo_indptr[b + 1];
    if (lo < 0 || hi < lo || hi > p.total_q || (!p.kv_end && hi - lo > L)) {
        if (report) raise_flag(p.err, PKV_DEVERR_RANGE);
        return 0;
    }
    return static_cast<int>(hi - lo);
}

template <int D>
__global__ void __launch_bounds__(kThreads) rows_kernel(const Params p) {
    pdl_wait();          // inputs may come from the previous kernel of the stream
    pdl_launch_next();
    __shared__ float red_o[kWarps][D];
    __shared__ float red_m[kWarps], red_l[kWarps];
    const int row = blockIdx.x / p.hq, head = blockIdx.x % p.hq, kh = head / p.g;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int b = row;
    if (p.qo_indptr) {
        int lo = 0, hi = p.batch;   // the last request that starts at or before the row
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (p.qo_indptr[mid] <= row) lo = mid; else hi = mid;
        }
        b = lo;
    }
    const bool report = head == 0 && threadIdx.x == 0;
    int64_t base;
    const int L = quant::key_count(p.tab, b, base, p.err, report);
    const int n = q_count(p, b, L, report);
    const int i = p.qo_indptr ? row - p.qo_indptr[b] : 0;
    if (i < 0 || i >= n) return;
    int end = !p.qo_indptr ? L : p.kv_end ? p.kv_end[row] : L - n + i + 1;
    if (end < 0 || end > L) {
        if (report) raise_flag(p.err, PKV_DEVERR_RANGE);
        end = 0;
    }
    const float gk = p.k_scale ? p.k_scale[kh] : 1.f, gv = p.v_scale ? p.v_scale[kh] : 1.f;
    if (report && kh == 0)
        for (int h = 0; h < p.hkv; ++h)
            if ((p.k_scale && !quant::good_scale(p.k_scale[h])) || (p.v_scale && !quant::good_scale(p.v_scale[h])))
                raise_flag(p.err, PKV_DEVERR_RANGE);
    constexpr int P = D / 64;   // pairs of dims per lane
    const int t = 1 << p.t_shift;
    float2 q[P], o[P];
    const uint32_t *qr = reinterpret_cast<const uint32_t *>(p.q + row * p.q_stride + static_cast<int64_t>(head) * D);
#pragma unroll
    for (int k = 0; k < P; ++k) {
        const uint32_t w = qr[lane + 32 * k];
        q[k] = make_float2(bf16_lo(w) * gk * p.scale_log2, bf16_hi(w) * gk * p.scale_log2);
        o[k] = make_float2(0.f, 0.f);
    }
    float m = -INFINITY, l = 0.f;
    for (int key = warp; key < end; key += kWarps) {
        const int64_t slot = quant::slot_of(p.tab, base, key);
        if (slot < 0 && lane == 0) raise_flag(p.err, slot == -1 ? PKV_DEVERR_RANGE : PKV_DEVERR_CONTIG);
        const uint8_t *tile = p.pool + (slot < 0 ? 0 : slot >> p.t_shift) * p.tile_stride +
                              static_cast<int64_t>(kh) * quant::tile_bytes(t, D);
        const int at = static_cast<int>(slot & (t - 1));
        auto value = [&](bool v, int k) -> float2 {
            if (slot < 0) return make_float2(0.f, 0.f);
            const int pr = lane + 32 * k;
            uint32_t h[4];
            quant::codes_to_f16(tile[(v ? t * (D / 2) : 0) + at * (D / 2) + pr], h);
            const float2 c = quant::f16x2_to_f32(h[0]);
            const float s = quant::f16x2_to_f32(quant::scales_to_f16(tile[t * D + (v ? t * (D / 16) : 0) + at * (D / 16) + pr / 8])).x;
            return make_float2(c.x * s, c.y * s);
        };
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < P; ++k) {
            const float2 x = value(false, k);
            s = fmaf(q[k].x, x.x, fmaf(q[k].y, x.y, s));
        }
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        const float mn = fmaxf(m, s);
        const float base_m = mn == -INFINITY ? 0.f : mn;
        const float corr = ex2(m - base_m), w = ex2(s - base_m);
        l = fmaf(l, corr, w);
#pragma unroll
        for (int k = 0; k < P; ++k) {
            const float2 x = value(true, k);
            o[k].x = fmaf(o[k].x, corr, w * x.x);
            o[k].y = fmaf(o[k].y, corr, w * x.y);
        }
        m = mn;
    }
#pragma unroll
    for (int k = 0; k < P; ++k) {
        red_o[warp][2 * (lane + 32 * k)] = o[k].x;
        red_o[warp][2 * (lane + 32 * k) + 1] = o[k].y;
    }
    if (lane == 0) {
        red_m[warp] = m;
        red_l[warp] = l;
    }
    __syncthreads();
    float M = -INFINITY, den = 0.f;
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, red_m[w]);
    const float base_m = M == -INFINITY ? 0.f : M;
    for (int w = 0; w < kWarps; ++w) den += red_l[w] * ex2(red_m[w] - base_m);
    const int64_t orow = static_cast<int64_t>(row) * p.hq + head;
    for (int d = threadIdx.x; d < D; d += kThreads) {
        float num = 0.f;
        for (int w = 0; w < kWarps; ++w) num = fmaf(red_o[w][d], ex2(red_m[w] - base_m), num);
        const float v = den == 0.f ? 0.f : num / den * gv;
        p.out[orow * D + d] = static_cast<uint16_t>(pack_bf16x2(v, 0.f));
    }
    if (threadIdx.x == 0 && p.lse) p.lse[orow] = den == 0.f ? -INFINITY : (M + log2f(den)) * kLn2;
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

static size_t workspace_size(const pkv_quant_args *) { return 256; }

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

static pkv_status attend(const char *who, const pkv_quant_args *a, bool extend, void *ws, size_t ws_bytes, int32_t *err,
                         cudaStream_t s) {
    if (!a) return fail(PKV_ERR_INVALID_ARG, "%s: null args", who);
    if (!err) return fail(PKV_ERR_INVALID_ARG, "%s: err_flags is required", who);
    const pkv_status st = validate(who, a, extend, true);
    if (st != PKV_OK) return st;
    if (a->batch == 0 || a->total_q == 0) return ok();
    const size_t need = workspace_size(a);
    if (ws_bytes < need) return fail(PKV_ERR_CAPACITY, "%s: workspace of %zu bytes, %zu needed", who, ws_bytes, need);
    if (!ws || !aligned(ws, 256))
        return fail(PKV_ERR_INVALID_ARG, "%s: workspace must be non-null and 256-byte aligned", who);
    const int64_t grid = a->total_q * a->num_q_heads;
    if (grid > INT32_MAX) return fail(PKV_ERR_UNSUPPORTED, "%s: too many query rows", who);
    auto *kern = a->head_dim == 128 ? rows_kernel<128> : rows_kernel<64>;
    return launch_status(launch_chained(kern, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, s, params(a, err)), who);
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
