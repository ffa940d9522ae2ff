// What the kernels and the C entry of the verification of drafted tokens share.
#pragma once

#include "ice_paged.cuh"

namespace ice {

constexpr int kVerMaxDrafts = 63;
constexpr int kVerMaxVocab = 1 << 22;

// One call, passed by value. Strides in elements.
struct Verify {
    const void *target, *draft;  // draft NULL: drafts are certain, or greedy
    long long t_req, t_row, d_req, d_row;
    const int *tokens, *n_draft;
    const float* uniform;  // NULL: greedy
    int *out, *accepted, *n_new, *status;
    int n_req, K, V;
    int group;  // greedy: rows of a request that are read together
};

cudaError_t launch_verify(Verify a, int dtype, cudaStream_t s);

}  // namespace ice
