// The handle of the plain paged cache and the checks that its C entries share.
#pragma once

#include <nvtx3/nvToolsExt.h>

#include "ice_paged.cuh"

struct ice_paged {
    ice_paged_params p;
    int G = 0, device = 0, n_sm = 0, debug = 0;
    long long rows_cap = 0;    // rows of partial results
    float* part_o = nullptr;   // rows_cap x D
    float2* part_ml = nullptr; // rows_cap
    int* words = nullptr;      // status word, ticket, item counters, plan, then [max_requests] of the plan
    void* verify = nullptr;    // scratch of ice_paged_verify, VerifyScratch [max_requests]
    char* share = nullptr;     // scratch of the calls on shared pages, made by the first of them
};

namespace ice {

struct ApiRange {
    explicit ApiRange(const char* name) { nvtxRangePushA(name); }
    ~ApiRange() { nvtxRangePop(); }
};

enum { kWordStatus = 0, kWordTicket = 1, kWordNext = 2, kWordPlan = 4, kWords = 16 };

inline bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

// Memory that the kernels can use for a caller's buffer: device memory of the handle's
// GPU, or managed memory. While `stream` is being captured no driver query is made
// (the eager calls before a capture check the same buffers).
struct Buffers {
    const ice_paged* pg;
    bool capturing = false, ok = true;
    Buffers(const ice_paged* h, void* stream) : pg(h) {
        int dev = -1;
        cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
        if (cudaGetDevice(&dev) != cudaSuccess || dev != h->device ||
            cudaStreamIsCapturing((cudaStream_t)stream, &cs) != cudaSuccess) {
            cudaGetLastError();
            ok = false;
        }
        capturing = cs != cudaStreamCaptureStatusNone;
    }
    Buffers& need(const void* p, size_t align) {
        if (!p || !aligned(p, align)) ok = false;
        return opt(p);
    }
    Buffers& opt(const void* p) {
        if (!ok || capturing || !p) return *this;
        cudaPointerAttributes a;
        if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
            cudaGetLastError();
            ok = false;
        } else if (!((a.type == cudaMemoryTypeDevice && a.device == pg->device) ||
                     a.type == cudaMemoryTypeManaged)) {
            ok = false;
        }
        return *this;
    }
};

// A launch's result as a status. A failed one leaves no error behind that the caller's next, unrelated check of
// the runtime would find.
inline int launched(cudaError_t e) {
    if (e == cudaSuccess) return ICE_OK;
    cudaGetLastError();
    return ICE_ERR_CUDA;
}

inline int es_of(const ice_paged* pg) { return pg->p.dtype == ICE_BF16 ? 2 : 4; }

// A token stride in elements: at least the row, a multiple of 16 bytes.
inline bool stride_ok(const ice_paged* pg, int64_t stride, int heads) {
    return stride >= (int64_t)heads * kD && stride * es_of(pg) % 16 == 0 && stride <= (1LL << 30);
}

}  // namespace ice
