// What quant_attn.cu hands to the multi-query kernel of extend.cu: keys and values taken out
// of the 4-bit pool into workspace tensors.
#pragma once

#include "pkv_internal.cuh"

namespace pkv {
namespace ext {

struct Held {
    const void *k, *v;           // bf16 / fp16 [D/64][kv heads][rows][64]
    int64_t rows;
    const int32_t *first_row;    // device [B + 1]: request b's keys are rows first_row[b] .. first_row[b + 1] - 1
    const int32_t *order;        // device [B]: the requests, the longest first (their items are handed out so)
    const float *k_scale, *v_scale;
    int64_t q_row_stride;
    int32_t min_rows;            // requests with at most this many (token, head) rows per kv head are left out
};

// Bytes of the kernel's own workspace, the place of its item counter there (int32, to be
// zeroed on the stream before the launch), and the launch.  `a` gives the batch, heads,
// query rows, bounds, outputs and max_seq_len; its page-table fields are not used.
size_t held_workspace(const pkv_extend_args *a);
size_t held_counter_offset(const pkv_extend_args *a);
pkv_status held_launch(const pkv_extend_args *a, const Held &held, void *workspace, int32_t *err, cudaStream_t s);

}  // namespace ext
}  // namespace pkv
