// What the rotating append's kernel and its C entry share.
#pragma once

#include "ice_paged.cuh"

namespace ice {

// One call, passed by value.
struct RopeAppend {
    const void *q, *k, *v;
    void *q_out, *k_pages, *v_pages;
    const int* positions;
    const long long* slot_map;
    int* status;
    long long q_stride, q_out_stride, k_stride, v_stride;  // elements
    long long pos_stride, pos_offset, n_slots;
    int n_tokens, Hq, H, P;  // Hq = 0: no queries
    // made by the launch: warps that share a token's rows, the pairs' frequencies (2^-64 turns a position) and axes
    int parts, n_pairs;
    unsigned long long turn[64];
    unsigned char axis[64];
};

cudaError_t launch_rope_append(RopeAppend a, const ice_rope& r, int dtype, cudaStream_t s);

}  // namespace ice
