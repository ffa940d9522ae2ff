// What the kernels and the C entry of the verification of drafted tokens share.
#pragma once

#include "ice_paged.cuh"

namespace ice {

constexpr int kVerMaxDrafts = 63;
constexpr int kVerMaxVocab = 1 << 22;

constexpr int kVerGroups = 256;  // sampling: most parts of a row that are summed separately

// Scratch of a request; all but the sums is zero between calls.
struct VerifyScratch {
    unsigned long long best[kVerMaxDrafts + 1];  // greedy: a row's best entry
    float2 sum[kVerGroups];                      // sampling: a part's sum, as two numbers
    int count[kVerMaxDrafts + 1];                // groups of a row that are done (greedy), blocks of the request (the first; sampling)
    int wrong;                                   // greedy: kVerMaxDrafts + 1 - the first row known to end the request
    int rows;                                    // greedy: rows that are done
};

// One call, passed by value. Strides in elements.
struct Verify {
    const void *target, *draft;  // draft NULL: drafts are certain, or greedy
    long long t_req, t_row, d_req, d_row;
    const int *tokens, *n_draft;
    const float* uniform;  // NULL: greedy
    int *out, *accepted, *n_new, *status;
    VerifyScratch* scratch;  // [n_req]
    int n_req, K, V;
    int groups, blocks;  // of a row; sampling: blocks of a request
};

cudaError_t launch_verify(const Verify& a, int dtype, cudaStream_t s);

}  // namespace ice
