// pkv_evict: the pages whose tokens received least attention go back to the free list.
//
// Two kernels, a cluster of blocks per request in each.  The first checks the requests, counts
// what each loses, and writes each page's score as a 32-bit key whose unsigned order is
// theirs.  The second finds the border key by digits (11, 11 and 10 bits: a histogram of the
// pages that share the digits so far, summed over the cluster), numbers the pages that stay and
// those that go, and moves the columns: chunk after chunk, each read by the whole
// cluster before any of it is written, so that a row may be compacted in place.
#include <algorithm>

#include "pkv_internal.cuh"

namespace pkv {
namespace evict {
namespace {

constexpr int kThreads = 1024;
constexpr int kMaxBatch = 8192, kMaxCluster = 8;
constexpr int kBins = 2048;
constexpr int kEach = 4;          // columns of a thread per chunk

struct Info {                     // a request, as the first kernel found it
    int64_t r2t, acc;             // its first column in the table and in acc
    int32_t L, gone, head, tail;  // tokens; pages to evict, of those in [head, tail)
    int32_t state, pad;           // kBad, kKeep (nothing to evict), kEvict
};
enum { kBad, kKeep, kEvict };

struct Params {
    pkv_evict_args a;
    int32_t *err;
    uint32_t *keys;               // [B][pages_max]; then each page's new place, or -1
    Info *info;                   // [B]
    int32_t *free_state;          // head and count as they were
    int64_t pages_max;
    int32_t ps_shift;
};

__device__ __forceinline__ int cluster_size() {
    uint32_t n;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;\n" : "=r"(n));
    return static_cast<int>(n);
}
__device__ __forceinline__ int block_sum_int(int v, int *scratch) {   // kThreads threads; every thread gets the sum
    v = __reduce_add_sync(0xffffffffu, v);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();
    if (lane == 0) scratch[warp] = v;
    __syncthreads();
    return __reduce_add_sync(0xffffffffu, scratch[lane]);
}
// Exclusive prefix over the block's threads; *total gets the sum.
__device__ __forceinline__ int block_scan(int v, int *scratch, int *total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int incl = v;
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    __syncthreads();
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    int x = scratch[lane], s = x;
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
    }
    *total = __shfl_sync(0xffffffffu, s, 31);
    return __shfl_sync(0xffffffffu, s - x, warp) + incl - v;
}
// Sum of the values that the cluster's blocks hold in `mine`, and of those before this block.
__device__ __forceinline__ int cluster_sum(int *mine, int rank, int size, int *before) {
    int all = 0, low = 0;
    for (int i = 0; i < size; ++i) {
        const int x = ld_cluster_s32(mapa(smem_u32(mine), i));
        if (i < rank) low += x;
        all += x;
    }
    *before = low;
    return all;
}

// Unsigned keys in the order of the scores; NaN above all.
__device__ __forceinline__ uint32_t key_of(float score) {
    if (score != score) return 0xffffffffu;
    const uint32_t u = __float_as_uint(score + 0.f);   // (-0 is 0)
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kThreads) score_kernel(const Params p) {
    __shared__ int scratch[32];
    __shared__ int flags_s;
    pdl_wait();          // inputs may come from the previous kernel of the stream
    pdl_launch_next();
    const pkv_evict_args &a = p.a;
    const int size = cluster_size(), rank = cluster_rank(), b = blockIdx.x / size, tid = threadIdx.x;
    if (blockIdx.x == 0 && tid < 2) p.free_state[tid] = a.free_state[tid];
    const int64_t row = a.req_pool_idx[b], s = a.kv_start ? a.kv_start[b] : 0, L = a.seq_lens[b];
    const int64_t budget = a.budget[b], first = a.keep_first ? a.keep_first[b] : 0, last = a.keep_last ? a.keep_last[b] : 0;
    const int mask = a.page_size - 1;
    bool bad = row < 0 || row >= a.r2t_rows || s < 0 || (s & mask) || L < 0 || s + L > a.r2t_width || budget < 0 || first < 0 || last < 0;
    int same = 0;
    for (int i = tid; i < a.batch; i += kThreads) same += i != b && a.req_pool_idx[i] == row;
    bad |= block_sum_int(same, scratch) != 0;
    const bool long_ = !bad && L > a.max_seq_len;
    Info f{};
    f.L = static_cast<int>(L);
    f.state = bad || long_ ? kBad : kKeep;
    int n = 0;
    if (f.state == kKeep) {
        f.r2t = row * a.r2t_row_stride + s;
        f.acc = row * a.acc_row_stride + s;
        n = static_cast<int>((L + mask) >> p.ps_shift);
        const int64_t head = (first + mask) >> p.ps_shift, tail = max(L - last, static_cast<int64_t>(0)) >> p.ps_shift;
        f.head = static_cast<int>(min(head, static_cast<int64_t>(n)));
        f.tail = static_cast<int>(max(static_cast<int64_t>(f.head), min(tail, static_cast<int64_t>(n - 1))));
        f.gone = static_cast<int>(min(static_cast<int64_t>(f.tail - f.head),
                                      max(static_cast<int64_t>(0), n - max(static_cast<int64_t>(1), budget >> p.ps_shift))));
        if (f.gone > 0) f.state = kEvict;
    }
    int flags = bad ? PKV_DEVERR_RANGE : long_ ? PKV_DEVERR_CAPACITY : 0;
    if (f.state == kEvict) {
        // the pages in [head, tail) are whole
        const int lanes = min(a.page_size, 32), shift = min(p.ps_shift, 5), sub = tid & (lanes - 1), each = a.page_size >> shift;
        const int groups = kThreads >> shift;   // pages at a time
        for (int64_t p0 = f.head + static_cast<int64_t>(rank) * groups; p0 < f.tail; p0 += static_cast<int64_t>(size) * groups) {
            const int64_t page = p0 + (tid >> shift);
            const bool in = page < f.tail;
            double sum = 0;
            if (in) {
                const float *x = a.acc + f.acc + (page << p.ps_shift) + sub;
                for (int i = 0; i < each; ++i) sum += x[i * lanes];
            }
            for (int o = 1; o < lanes; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (in && sub == 0) {
                p.keys[b * p.pages_max + page] = key_of(static_cast<float>(sum));
                const int64_t slot = a.req_to_token[f.r2t + (page << p.ps_shift)];
                if (slot < 0 || (slot >> p.ps_shift) >= a.num_pool_pages) flags |= PKV_DEVERR_RANGE;
                else if (slot & mask) flags |= PKV_DEVERR_CONTIG;
            }
        }
    }
    flags = __reduce_or_sync(0xffffffffu, flags);
    if (tid == 0) flags_s = 0;
    __syncthreads();
    if ((tid & 31) == 0 && flags) atomicOr(&flags_s, flags);
    __syncthreads();
    cluster_sync_all();
    if (rank == 0) {
        flags = 0;
        for (int i = 0; i < size; ++i) flags |= ld_cluster_s32(mapa(smem_u32(&flags_s), i));
        if (tid == 0) {
            if (flags) raise_flag(p.err, flags);
            if (flags && f.state == kEvict) {   // a bad page
                f.state = kKeep;
                f.gone = 0;
            }
            p.info[b] = f;
        }
    }
    __syncthreads();
    cluster_sync_all();   // (no block leaves while its shared memory is read)
}

__global__ void __launch_bounds__(kThreads) move_kernel(const Params p) {
    __shared__ int hist[3][kBins];
    __shared__ int scratch[32];
    __shared__ int found[2];
    __shared__ int ties_s, gone_s;
    pdl_wait();          // the first kernel's keys
    pdl_launch_next();
    const pkv_evict_args &a = p.a;
    const int size = cluster_size(), rank = cluster_rank(), b = blockIdx.x / size, tid = threadIdx.x;
    Info f = p.info[b];
    // pages that the requests before this one lose, and all of them
    int low = 0, all = 0;
    for (int i = tid; i < a.batch; i += kThreads) {
        const int g = p.info[i].gone;
        all += g;
        if (i < b) low += g;
    }
    all = block_sum_int(all, scratch);
    low = block_sum_int(low, scratch);
    const int64_t head = p.free_state[0], count = p.free_state[1];
    const bool room = all == 0 || (head >= all && head <= a.free_pages_len);
    if (blockIdx.x == 0 && tid == 0) {
        if (!room) raise_flag(p.err, PKV_DEVERR_CAPACITY);
        a.free_state_out[0] = static_cast<int32_t>(room ? head - all : head);
        a.free_state_out[1] = static_cast<int32_t>(room ? count + all : count);
    }
    if (!room) {
        f.gone = 0;
        if (f.state == kEvict) f.state = kKeep;
    }
    const int left = f.L - (f.gone << p.ps_shift);
    if (rank == 0 && tid == 0) a.seq_lens_out[b] = left;
    const bool move_table = a.req_to_token_out != a.req_to_token, move_acc = a.acc_out != a.acc;
    if (f.state == kBad || (f.gone == 0 && !move_table && !move_acc)) return;   // (the whole cluster)
    uint32_t *keys = p.keys + b * p.pages_max;
    if (f.gone > 0) {
        // ---- the border: the key of the best page that goes, and how many of that key go
        const int n = f.tail - f.head, seg = (n + size - 1) / size;
        const int lo = f.head + min(n, rank * seg), hi = f.head + min(n, (rank + 1) * seg);
        for (int i = tid; i < 3 * kBins; i += kThreads) (&hist[0][0])[i] = 0;
        __syncthreads();
        uint32_t border = 0, known = 0;   // its digits so far, and their mask
        int want = f.gone, ties = 0;      // pages to find among those that share them; pages that do
#pragma unroll 1
        for (int d = 0; d < 3; ++d) {
            const int shift = d == 0 ? 21 : d == 1 ? 10 : 0, bins = d == 2 ? 1024 : kBins;
            for (int i = lo + tid; i < hi; i += kThreads) {
                const uint32_t k = keys[i];
                if ((k & known) == border) atomicAdd(&hist[d][(k >> shift) & (bins - 1)], 1);
            }
            __syncthreads();
            cluster_sync_all();
            int x[2] = {0, 0};
            for (int r = 0; r < size; ++r)
#pragma unroll
                for (int i = 0; i < 2; ++i) x[i] += ld_cluster_s32(mapa(smem_u32(&hist[d][2 * tid + i]), r));
            int total;
            const int before = block_scan(x[0] + x[1], scratch, &total);
            if (before < want && want <= before + x[0]) {
                found[0] = 2 * tid;
                found[1] = before;
                ties_s = x[0];
            } else if (before + x[0] < want && want <= before + x[0] + x[1]) {
                found[0] = 2 * tid + 1;
                found[1] = before + x[0];
                ties_s = x[1];
            }
            __syncthreads();
            border |= static_cast<uint32_t>(found[0]) << shift;
            known |= static_cast<uint32_t>(bins - 1) << shift;
            want -= found[1];
            ties = ties_s;
            __syncthreads();
        }
        // ---- of the pages at the border the last `want` go: places of this thread's pages in order
        const int per = (hi - lo + kThreads - 1) / kThreads, i0 = min(hi, lo + tid * per), i1 = min(hi, i0 + per);
        int t = 0;
        for (int i = i0; i < i1; ++i) t += keys[i] == border;
        int sum, before;
        int tie = block_scan(t, scratch, &sum);
        if (tid == 0) ties_s = sum;
        __syncthreads();
        cluster_sync_all();
        cluster_sum(&ties_s, rank, size, &before);
        tie += before;
        const int stay = ties - want;
        int go = 0;
        {
            int x = tie;
            for (int i = i0; i < i1; ++i) {
                const uint32_t k = keys[i];
                go += k < border || (k == border && x++ >= stay);
            }
        }
        int gone = block_scan(go, scratch, &sum);
        if (tid == 0) gone_s = sum;
        __syncthreads();
        cluster_sync_all();
        cluster_sum(&gone_s, rank, size, &before);
        gone += before;
        int32_t *out = a.free_pages + head - all + low;
        for (int i = i0; i < i1; ++i) {
            const uint32_t k = keys[i];
            const bool goes = k < border || (k == border && tie++ >= stay);
            if (goes) out[gone] = a.req_to_token[f.r2t + (static_cast<int64_t>(i) << p.ps_shift)] >> p.ps_shift;
            keys[i] = goes ? 0xffffffffu : static_cast<uint32_t>(i - gone);
            gone += goes;
        }
        __syncthreads();
        cluster_sync_all();   // all places are known to the cluster
    }
    // ---- the columns
    const int mask = a.page_size - 1;
    const int from = move_table || move_acc ? 0 : f.head << p.ps_shift;   // (columns before head stay where they are)
    const int step = size * kThreads * kEach;
    for (int c0 = from; c0 < f.L; c0 += step) {
        int32_t slot[kEach];
        float w[kEach];
        int to[kEach];
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int c = c0 + (rank * kEach + e) * kThreads + tid;
            to[e] = -1;
            if (c >= f.L) continue;
            const int page = c >> p.ps_shift;
            int q = page;
            if (f.gone > 0 && page >= f.head) q = page < f.tail ? static_cast<int>(__ldcg(keys + page)) : page - f.gone;
            if (q < 0) continue;
            to[e] = (q << p.ps_shift) + (c & mask);
            slot[e] = a.req_to_token[f.r2t + c];
            w[e] = a.acc[f.acc + c];
        }
        __syncthreads();
        cluster_sync_all();   // the chunk has been read
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            if (to[e] < 0) continue;
            a.req_to_token_out[f.r2t + to[e]] = slot[e];
            a.acc_out[f.acc + to[e]] = w[e];
        }
    }
    // (a column behind the last kept one is nobody's target, and all of them have been read)
    for (int c = left + rank * kThreads + tid; c < f.L; c += size * kThreads) a.acc_out[f.acc + c] = 0.f;
    __syncthreads();
    cluster_sync_all();   // (no block leaves while its shared memory is read)
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

pkv_status launch(void (*kern)(Params), const Params &p, int batch, int cluster, cudaStream_t s) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(batch * cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return launch_status(cudaLaunchKernelEx(&cfg, kern, p), "pkv_evict");
}

}  // namespace
}  // namespace evict
}  // namespace pkv

extern "C" size_t pkv_evict_workspace_size(int32_t batch, int32_t max_seq_len, int32_t page_size) {
    using namespace pkv;
    using namespace pkv::evict;
    if (batch < 0 || batch > kMaxBatch || max_seq_len < 0 || !is_pow2(page_size) || page_size > 1024) return 0;
    const size_t pages = (static_cast<size_t>(max_seq_len) + page_size - 1) / page_size;
    return 256 + up256(batch * sizeof(Info)) + up256(batch * pages * 4);
}

extern "C" pkv_status pkv_evict(const pkv_evict_args *args, void *workspace, size_t workspace_bytes, int32_t *err_flags,
                                pkv_stream_t stream) {
    using namespace pkv;
    using namespace pkv::evict;
    if (!args) return fail(PKV_ERR_INVALID_ARG, "pkv_evict: null args");
    if (!err_flags) return fail(PKV_ERR_INVALID_ARG, "pkv_evict: err_flags is required");
    const pkv_evict_args &a = *args;
    if (a.batch < 0 || a.max_seq_len < 0 || a.num_pool_pages < 0 || a.r2t_rows < 0 || a.r2t_width < 0 ||
        a.r2t_row_stride < a.r2t_width || a.acc_row_stride < a.r2t_width || a.free_pages_len < 0)
        return fail(PKV_ERR_INVALID_ARG, "pkv_evict: bad sizes");
    if (a.batch > kMaxBatch) return fail(PKV_ERR_UNSUPPORTED, "pkv_evict: more than %d requests", kMaxBatch);
    if (!is_pow2(a.page_size) || a.page_size > 1024)
        return fail(PKV_ERR_UNSUPPORTED, "pkv_evict: page_size must be a power of two in [1, 1024]");
    if (a.r2t_width > INT32_MAX / 2 || a.num_pool_pages > INT32_MAX / a.page_size)
        return fail(PKV_ERR_UNSUPPORTED, "pkv_evict: more than 2^31 pool slots or 2^30 columns");
    const int32_t longest = static_cast<int32_t>(std::min<int64_t>(a.max_seq_len, a.r2t_width));
    if (!a.free_state || !a.free_state_out || (!a.free_pages && a.free_pages_len > 0))
        return fail(PKV_ERR_INVALID_ARG, "pkv_evict: null free list");
    if (a.batch > 0 && (!a.req_to_token || !a.req_to_token_out || !a.acc || !a.acc_out || !a.req_pool_idx || !a.seq_lens ||
                        !a.seq_lens_out || !a.budget))
        return fail(PKV_ERR_INVALID_ARG, "pkv_evict: null pointer");
    const size_t need = pkv_evict_workspace_size(a.batch, longest, a.page_size);
    if (workspace_bytes < need) return fail(PKV_ERR_CAPACITY, "pkv_evict: workspace of %zu bytes, %zu needed", workspace_bytes, need);
    if (!workspace || !aligned(workspace, 256))
        return fail(PKV_ERR_INVALID_ARG, "pkv_evict: workspace must be non-null and 256-byte aligned");
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (a.batch == 0) {
        if (a.free_state_out != a.free_state &&
            cudaMemcpyAsync(a.free_state_out, a.free_state, 8, cudaMemcpyDeviceToDevice, s) != cudaSuccess)
            return fail(PKV_ERR_CUDA, "pkv_evict: cannot copy the free list's state");
        return ok();
    }
    Params p{};
    p.a = a;
    p.a.max_seq_len = longest;
    p.err = err_flags;
    p.ps_shift = ilog2(a.page_size);
    p.pages_max = (static_cast<int64_t>(longest) + a.page_size - 1) / a.page_size;
    char *at = static_cast<char *>(workspace);
    p.free_state = reinterpret_cast<int32_t *>(at);
    p.info = reinterpret_cast<Info *>(at + 256);
    p.keys = reinterpret_cast<uint32_t *>(at + 256 + up256(a.batch * sizeof(Info)));
    // more blocks to a request while there are SMs for them and columns to share
    int cluster = 1;
    while (cluster < kMaxCluster && static_cast<int64_t>(longest) > 2048ll * cluster && 2ll * a.batch * cluster <= sm_count()) cluster *= 2;
    const pkv_status st = launch(score_kernel, p, a.batch, cluster, s);
    return st != PKV_OK ? st : launch(move_kernel, p, a.batch, cluster, s);
}
