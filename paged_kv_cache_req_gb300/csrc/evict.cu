// pkv_evict: the pages whose tokens received least attention go back to the free list.
//
// Two kernels, a cluster of blocks per request in each.  The first checks the requests and
// their pages and counts what each loses.  The second takes each page's score as a 32-bit key
// whose unsigned order is theirs (kept in shared memory where they fit), finds the border key by
// digits (11, 11 and 10 bits: a histogram of the pages that share the digits so far, summed over the
// cluster), numbers the pages that stay and those that go, and moves the columns: chunk after
// chunk, each read by the whole cluster before any of it is written, so that a row may be
// compacted in place.
//
// 128 requests of 8192 to 16384 pages of one token take 31 us (22 MB): a chain of dependent passes, half of the ALU
// busy; 32 requests of up to 4096 tokens in pages of 16 take 17, which is latency.  Two kernels, because
// what one request loses depends on whether the others' pages are good and the free list has room for all.
#include <algorithm>

#include "pkv_internal.cuh"

namespace pkv {
namespace evict {
namespace {

constexpr int kMaxBatch = 8192, kMaxCluster = 8;
constexpr int kBins = 2048;
constexpr int kEach = 8;          // columns of a thread per chunk
constexpr int kKeysInSmem = 16384;   // pages of a block up to which its keys are kept in shared memory

struct Info {                     // a request, as the first kernel found it
    int64_t r2t, acc;             // its first column in the table and in acc
    int32_t L, gone, head, tail;  // tokens; pages to evict, of those in [head, tail)
    int32_t state, pad;           // kBad, kKeep (nothing to evict), kEvict
};
enum { kBad, kKeep, kEvict };

struct Params {
    pkv_evict_args a;
    int32_t *err;
    uint32_t *places;             // [B][pages_max]: each page's new place, or -1 (before that its key, where keys are many)
    Info *info;                   // [B]
    int32_t *free_state;          // head and count as they were
    int64_t pages_max;
    int32_t ps_shift, cluster, smem_keys;
};

template <int T>
__device__ __forceinline__ int block_sum_int(int v, int *scratch) {   // every thread gets the sum
    v = __reduce_add_sync(0xffffffffu, v);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();
    if (lane == 0) scratch[warp] = v;
    __syncthreads();
    return __reduce_add_sync(0xffffffffu, lane < T / 32 ? scratch[lane] : 0);
}
// Exclusive prefix over the block's warps of a value per warp; *total gets the sum.
template <int T>
__device__ __forceinline__ int warps_scan(int v, int *scratch, int *total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();
    if (lane == 0) scratch[warp] = v;
    __syncthreads();
    const int x = lane < T / 32 ? scratch[lane] : 0;
    int s = x;
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
    }
    *total = __shfl_sync(0xffffffffu, s, 31);
    return __shfl_sync(0xffffffffu, s - x, warp);
}
// The same over its threads.
template <int T>
__device__ __forceinline__ int block_scan(int v, int *scratch, int *total) {
    const int lane = threadIdx.x & 31;
    int incl = v;
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    return warps_scan<T>(__shfl_sync(0xffffffffu, incl, 31), scratch, total) + incl - v;
}
// Makes shared and global writes of the cluster's blocks visible to all of them.
__device__ __forceinline__ void sync_all(int size) {
    __syncthreads();
    if (size > 1) cluster_sync_all();
}
// Sum of the values that the blocks before this one hold in `mine`.
__device__ __forceinline__ int sum_before(int *mine, int rank) {
    int low = 0;
    for (int i = 0; i < rank; ++i) low += ld_cluster_s32(mapa(smem_u32(mine), i));
    return low;
}

// Unsigned keys in the order of the scores; NaN above all.
__device__ __forceinline__ uint32_t key_of(float score) {
    if (score != score) return 0xffffffffu;
    const uint32_t u = __float_as_uint(score + 0.f);   // (-0 is 0)
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

template <int T>
__global__ void __launch_bounds__(T) check_kernel(const Params p) {
    __shared__ int scratch[32];
    __shared__ int flags_s;
    pdl_wait();          // inputs may come from the previous kernel of the stream
    pdl_launch_next();
    const pkv_evict_args &a = p.a;
    const int size = p.cluster, rank = size > 1 ? cluster_rank() : 0, b = blockIdx.x / size, tid = threadIdx.x;
    if (blockIdx.x == 0 && tid < 2) p.free_state[tid] = a.free_state[tid];
    const int64_t row = a.req_pool_idx[b], s = a.kv_start ? a.kv_start[b] : 0, L = a.seq_lens[b];
    const int64_t budget = a.budget[b], first = a.keep_first ? a.keep_first[b] : 0, last = a.keep_last ? a.keep_last[b] : 0;
    const int mask = a.page_size - 1;
    bool bad = row < 0 || row >= a.r2t_rows || s < 0 || (s & mask) || L < 0 || s + L > a.r2t_width || budget < 0 || first < 0 || last < 0;
    int same = 0;
    for (int i = tid; i < a.batch; i += T) same |= i != b && a.req_pool_idx[i] == row;
    bad |= __syncthreads_or(same) != 0;
    const bool too_long = !bad && L > a.max_seq_len;
    Info f{};
    f.L = static_cast<int>(L);
    f.state = bad || too_long ? kBad : kKeep;
    if (f.state == kKeep) {
        f.r2t = row * a.r2t_row_stride + s;
        f.acc = row * a.acc_row_stride + s;
        const int n = static_cast<int>((L + mask) >> p.ps_shift);
        const int64_t head = (first + mask) >> p.ps_shift, tail = max(L - last, static_cast<int64_t>(0)) >> p.ps_shift;
        f.head = static_cast<int>(min(head, static_cast<int64_t>(n)));
        f.tail = static_cast<int>(max(static_cast<int64_t>(f.head), min(tail, static_cast<int64_t>(n - 1))));
        f.gone = static_cast<int>(min(static_cast<int64_t>(f.tail - f.head),
                                      max(static_cast<int64_t>(0), n - max(static_cast<int64_t>(1), budget >> p.ps_shift))));
        if (f.gone > 0) f.state = kEvict;
    }
    int flags = bad ? PKV_DEVERR_RANGE : too_long ? PKV_DEVERR_CAPACITY : 0;
    if (f.state == kEvict) {
        const int32_t *table = a.req_to_token + f.r2t;
        const int step = size * T;
        for (int p0 = f.head + rank * T + tid; p0 < f.tail; p0 += step * 8) {
            int64_t slot[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) slot[i] = p0 + i * step < f.tail ? table[static_cast<int64_t>(p0 + i * step) << p.ps_shift] : 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (slot[i] < 0 || (slot[i] >> p.ps_shift) >= a.num_pool_pages) flags |= PKV_DEVERR_RANGE;
                else if (slot[i] & mask) flags |= PKV_DEVERR_CONTIG;
            }
        }
    }
    flags = __reduce_or_sync(0xffffffffu, flags);
    if ((tid & 31) == 0) scratch[tid >> 5] = flags;
    __syncthreads();
    flags = 0;
    for (int i = 0; i < T / 32; ++i) flags |= scratch[i];
    if (tid == 0) flags_s = flags;
    sync_all(size);
    if (rank == 0 && tid == 0) {
        for (int i = 1; i < size; ++i) flags |= ld_cluster_s32(mapa(smem_u32(&flags_s), i));
        if (flags) raise_flag(p.err, flags);
        if (flags && f.state == kEvict) {   // a bad page
            f.state = kKeep;
            f.gone = 0;
        }
        p.info[b] = f;
    }
    sync_all(size);   // (no block leaves while its shared memory is read)
}

// Keys of the pages [lo, hi) of a request: `keys[i - lo]` is page i's.
template <int T>
__device__ __forceinline__ void load_keys(const Params &p, const float *__restrict__ acc, int lo, int hi, uint32_t *keys) {
    const int tid = threadIdx.x;
    if (p.ps_shift == 0) {
        for (int i0 = lo + tid; i0 < hi; i0 += 8 * T) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = i0 + i * T < hi ? acc[i0 + i * T] : 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i0 + i * T < hi) keys[i0 + i * T - lo] = key_of(x[i]);
        }
        return;
    }
    // 4 columns to a lane (2 where a page has no more), a page to up to 32 lanes; these pages are whole
    const int cols = p.ps_shift == 1 ? 2 : 4, lane_shift = min(p.ps_shift - (cols == 4 ? 2 : 1), 5), lanes = 1 << lane_shift;
    const int sub = tid & (lanes - 1), each = (1 << p.ps_shift) / (cols * lanes);
    for (int i0 = lo; i0 < hi; i0 += T >> lane_shift) {
        const int page = i0 + (tid >> lane_shift);
        double sum = 0;
        if (page < hi) {
            const float *x = acc + (static_cast<int64_t>(page) << p.ps_shift) + sub * cols;
            for (int e = 0; e < each; ++e, x += lanes * cols)
                for (int c = 0; c < cols; ++c) sum += x[c];
        }
        for (int o = 1; o < lanes; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (page < hi && sub == 0) keys[page - lo] = key_of(static_cast<float>(sum));
    }
}

template <int T>
__global__ void __launch_bounds__(T) move_kernel(const Params p) {
    extern __shared__ uint32_t keys_s[];
    __shared__ int hist[3][kBins];
    __shared__ int scratch[32];
    __shared__ int found[3];
    __shared__ int ties_s, gone_s;
    pdl_wait();          // the first kernel's findings
    pdl_launch_next();
    const pkv_evict_args &a = p.a;
    const int size = p.cluster, rank = size > 1 ? cluster_rank() : 0, b = blockIdx.x / size, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Info f = p.info[b];
    // pages that the requests before this one lose, and all of them
    int low = 0, all = 0;
    for (int i = tid; i < a.batch; i += T) {
        const int g = p.info[i].gone;
        all += g;
        if (i < b) low += g;
    }
    for (int i = tid; i < 3 * kBins; i += T) (&hist[0][0])[i] = 0;
    const int n = f.tail - f.head, seg = (n + size - 1) / size;
    const int lo = f.head + min(n, rank * seg), hi = f.head + min(n, (rank + 1) * seg);
    uint32_t *places = p.places + b * p.pages_max, *keys = p.smem_keys ? keys_s : places + lo;
    if (f.gone > 0) load_keys<T>(p, a.acc + f.acc, lo, hi, keys);
    all = block_sum_int<T>(all, scratch);
    low = block_sum_int<T>(low, scratch);
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
    const bool elsewhere = a.req_to_token_out != a.req_to_token || a.acc_out != a.acc;
    if (f.state == kBad || (f.gone == 0 && !elsewhere)) return;   // (the whole cluster)
    if (f.gone > 0) {
        // ---- the border: the key of the best page that goes, and how many of that key go
        uint32_t border = 0, known = 0;   // its digits so far, and their mask
        int want = f.gone, ties = 0;      // pages to find among those that share them; pages that do
        __syncthreads();
#pragma unroll 1
        for (int d = 0; d < 3; ++d) {
            const int shift = d == 0 ? 21 : d == 1 ? 10 : 0, bins = d == 2 ? 1024 : kBins;
#pragma unroll 4
            for (int i = tid; i < hi - lo; i += T) {
                const uint32_t k = keys[i];
                if ((k & known) == border) atomicAdd(&hist[d][(k >> shift) & (bins - 1)], 1);
            }
            sync_all(size);
            constexpr int kOwn = kBins / T;   // bins of a thread
            int x[kOwn], sum = 0;
#pragma unroll
            for (int i = 0; i < kOwn; ++i) {
                x[i] = hist[d][kOwn * tid + i];
                for (int r = 1; r < size; ++r) x[i] += ld_cluster_s32(mapa(smem_u32(&hist[d][kOwn * tid + i]), (rank + r) % size));
                sum += x[i];
            }
            int total, before = block_scan<T>(sum, scratch, &total);
            if (before < want && want <= before + sum) {
#pragma unroll
                for (int i = 0; i < kOwn; ++i) {
                    if (before < want && want <= before + x[i]) {
                        found[0] = kOwn * tid + i;
                        found[1] = before;
                        found[2] = x[i];
                    }
                    before += x[i];
                }
            }
            __syncthreads();
            border |= static_cast<uint32_t>(found[0]) << shift;
            known |= static_cast<uint32_t>(bins - 1) << shift;
            want -= found[1];
            ties = found[2];
            if (ties == want) {   // all of them go, whatever their further digits
                border |= ~known;
                break;
            }
        }
        // ---- of the pages at the border the last `want` go.  Each warp has a run of pages, 32 at a time.
        const int per = ((hi - lo + T / 32 - 1) / (T / 32) + 31) / 32 * 32, i0 = min(hi - lo, warp * per), i1 = min(hi - lo, i0 + per);
        const int stay = ties - want;
        const uint32_t lower = (1u << lane) - 1;
        int tie = 0, sum;
        const bool all_go = ties == want;
        if (!all_go) {
            for (int i = i0 + lane; i < i1 + lane; i += 32) tie += __popc(__ballot_sync(0xffffffffu, i < i1 && keys[i] == border));
            tie = warps_scan<T>(tie, scratch, &sum);
            if (size > 1) {
                if (tid == 0) ties_s = sum;
                sync_all(size);
                tie += sum_before(&ties_s, rank);
            }
        }
        int gone = 0;
        if (all_go) {
#pragma unroll 4
            for (int i = i0 + lane; i < i1; i += 32) gone += keys[i] <= border;
            gone = __reduce_add_sync(0xffffffffu, gone);
        } else {
            for (int i = i0 + lane, x = tie; i < i1 + lane; i += 32) {
                const uint32_t k = i < i1 ? keys[i] : 0xffffffffu;
                const uint32_t eq = __ballot_sync(0xffffffffu, i < i1 && k == border);
                gone += __popc(__ballot_sync(0xffffffffu, i < i1 && (k < border || (k == border && x + __popc(eq & lower) >= stay))));
                x += __popc(eq);
            }
        }
        gone = warps_scan<T>(gone, scratch, &sum);
        if (size > 1) {
            if (tid == 0) gone_s = sum;
            sync_all(size);
            gone += sum_before(&gone_s, rank);
        }
        int32_t *out = a.free_pages + head - all + low;
        const int32_t *table = a.req_to_token + f.r2t + (static_cast<int64_t>(lo) << p.ps_shift);
        constexpr int kAhead = 8;   // table entries on their way before any place is written
        for (int j0 = i0; j0 < i1; j0 += 32 * kAhead) {
            int32_t slot[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int i = j0 + 32 * j + lane;
                slot[j] = i < i1 ? table[static_cast<int64_t>(i) << p.ps_shift] : 0;
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int i = j0 + 32 * j + lane;
                const uint32_t k = i < i1 ? keys[i] : 0xffffffffu;
                bool goes = i < i1 && k <= border;
                if (!all_go) {
                    const uint32_t eq = __ballot_sync(0xffffffffu, i < i1 && k == border);
                    goes = i < i1 && (k < border || (k == border && tie + __popc(eq & lower) >= stay));
                    tie += __popc(eq);
                }
                const uint32_t g = __ballot_sync(0xffffffffu, goes);
                const int at = gone + __popc(g & lower);
                if (goes) out[at] = slot[j] >> p.ps_shift;
                if (i < i1) places[lo + i] = goes ? 0xffffffffu : static_cast<uint32_t>(lo + i - at);
                gone += __popc(g);
            }
        }
        sync_all(size);   // all places are known to the cluster
    }
    // ---- the columns
    const int mask = a.page_size - 1;
    const int from = elsewhere ? 0 : f.head << p.ps_shift;   // (columns before head stay where they are)
    const int step = size * T * kEach;
    for (int c0 = from; c0 < f.L; c0 += step) {
        int32_t slot[kEach];
        float w[kEach];
        int to[kEach];
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int c = c0 + (rank * kEach + e) * T + tid, page = c >> p.ps_shift;
            int q = page;
            if (c >= f.L) q = -1;
            else if (f.gone > 0 && page >= f.head) q = page < f.tail ? static_cast<int>(__ldcg(places + page)) : page - f.gone;
            to[e] = q < 0 ? -1 : (q << p.ps_shift) + (c & mask);
            if (c < f.L) {   // (read whether it stays or not: the place is on its way)
                slot[e] = a.req_to_token[f.r2t + c];
                w[e] = a.acc[f.acc + c];
            }
        }
        sync_all(size);   // the chunk has been read
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            if (to[e] < 0) continue;
            a.req_to_token_out[f.r2t + to[e]] = slot[e];
            a.acc_out[f.acc + to[e]] = w[e];
        }
    }
    // (a column behind the last kept one is nobody's target, and all of them have been read)
    for (int c = left + rank * T + tid; c < f.L; c += size * T) a.acc_out[f.acc + c] = 0.f;
    sync_all(size);   // (no block leaves while its shared memory is read)
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

pkv_status launch(void (*kern)(Params), const Params &p, int threads, size_t smem, cudaStream_t s) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(p.a.batch * p.cluster));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(p.cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.cluster > 1 ? 2 : 1;
    return launch_status(cudaLaunchKernelEx(&cfg, kern, p), "pkv_evict");
}
template <int T>
pkv_status run(const Params &p, cudaStream_t s) {
    const size_t smem = p.smem_keys ? (static_cast<size_t>(p.pages_max) + p.cluster - 1) / p.cluster * 4 : 0;
    if (raise_smem_limit(reinterpret_cast<const void *>(move_kernel<T>)) < smem)
        return fail(PKV_ERR_CUDA, "pkv_evict: cannot raise the shared-memory limit");
    const pkv_status st = launch(check_kernel<T>, p, T, 0, s);
    return st != PKV_OK ? st : launch(move_kernel<T>, p, T, smem, s);
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
    p.places = reinterpret_cast<uint32_t *>(at + 256 + up256(a.batch * sizeof(Info)));
    // more blocks to a request while there are SMs for them and columns to share
    int cluster = 1;
    while (cluster < kMaxCluster && static_cast<int64_t>(longest) > 4096ll * cluster && 2ll * a.batch * cluster <= sm_count()) cluster *= 2;
    p.cluster = cluster;
    p.smem_keys = (p.pages_max + cluster - 1) / cluster <= kKeysInSmem;
    return longest > 2048 ? run<1024>(p, s) : run<256>(p, s);
}
