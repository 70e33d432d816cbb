// What keys of an 8-bit pool receive: the launches that byte_attn.cu makes of byte_weigh.cu.
#pragma once

#include "byte.cuh"
#include "spans.cuh"

namespace pkv {
namespace qattn {

struct WeighParams {
    const float *lse;
    float *part;             // given rows: [Hkv][B][max_len]
    const float *acc_in;
    float *acc_out;
    int64_t acc_stride;
};

// Kv head kh's piece of the tile that holds `slot`, and its scale bytes.
template <int D>
__device__ __forceinline__ const uint8_t *piece_at(const Params &p, int64_t slot, int kh) {
    return p.pool + (slot >> p.t_shift) * p.tile_stride + (static_cast<int64_t>(kh) * 2 * D << p.t_shift);
}
template <int D>
__device__ __forceinline__ const uint8_t *scales_at(const Params &p, const uint8_t *piece, int kh) {
    return piece + (static_cast<int64_t>(p.hkv - kh) * 2 * D << p.t_shift) + 2 * kh;
}

// acc_out = acc_in + the weights of the given rows (`rows`: what the host expects of a request and kv head, `keys`: of all requests).
pkv_status launch_weigh(const char *who, const Params &p, const WeighParams &wp, int head_dim, int64_t rows, int64_t keys,
                        cudaStream_t s);
// acc_out = acc_in + the weights of a decode whose logits are in p.logits.
pkv_status launch_finish(const char *who, const Params &p, const WeighParams &wp, cudaStream_t s);

}  // namespace qattn
}  // namespace pkv
