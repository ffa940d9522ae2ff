// C ABI of the plain paged cache: argument checks and launches. See include/ice.h for
// the contract of each call.
#include <algorithm>
#include <new>

#include <nvtx3/nvToolsExt.h>

#include "ice_paged.cuh"

using namespace ice;

struct ice_paged {
    ice_paged_params p;
    int G = 0, device = 0, n_sm = 0, debug = 0;
    long long rows_cap = 0;    // rows of partial results
    float* part_o = nullptr;   // rows_cap x D
    float2* part_ml = nullptr; // rows_cap
    int* words = nullptr;      // status word, ticket, item counters, plan, then [max_requests] of the plan
};

namespace {

struct ApiRange {
    explicit ApiRange(const char* name) { nvtxRangePushA(name); }
    ~ApiRange() { nvtxRangePop(); }
};

enum { kWordStatus = 0, kWordTicket = 1, kWordNext = 2, kWordPlan = 4, kWords = 16 };

bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

int check(const ice_paged_params* p) {
    if (!p) return ICE_ERR_INVALID_ARG;
    if (p->d != kD) return ICE_ERR_UNSUPPORTED;
    if (p->n_kv_heads < 1 || p->n_q_heads < p->n_kv_heads || p->n_q_heads % p->n_kv_heads)
        return ICE_ERR_INVALID_ARG;
    const int G = p->n_q_heads / p->n_kv_heads;
    if (!(G == 1 || G == 2 || G == 4 || G == 8) || p->n_q_heads > 4096) return ICE_ERR_UNSUPPORTED;
    if (p->page_size < 1 || p->page_size > kMaxP) return ICE_ERR_INVALID_ARG;
    if (p->dtype != ICE_F32 && p->dtype != ICE_BF16) return ICE_ERR_INVALID_ARG;
    if (p->max_requests < 1 || p->max_requests > kPagedMaxRequests) return ICE_ERR_INVALID_ARG;
    if (p->max_blocks < 1 || (long long)p->max_blocks * p->page_size > (1LL << 30)) return ICE_ERR_INVALID_ARG;
    if (p->max_tokens < 1 || p->max_tokens > (1 << 20)) return ICE_ERR_INVALID_ARG;
    if (p->n_pages < 1) return ICE_ERR_INVALID_ARG;
    if (p->n_pages > 0x7FFFFFFFLL / ((long long)p->n_kv_heads * p->page_size)) return ICE_ERR_UNSUPPORTED;
    return ICE_OK;
}

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

void free_all(ice_paged* pg) {
    cudaFree(pg->part_o);
    cudaFree(pg->part_ml);
    cudaFree(pg->words);
}

// A launch's result as a status. A failed one leaves no error behind that the caller's next, unrelated check of
// the runtime would find.
int launched(cudaError_t e) {
    if (e == cudaSuccess) return ICE_OK;
    cudaGetLastError();
    return ICE_ERR_CUDA;
}

int es_of(const ice_paged* pg) { return pg->p.dtype == ICE_BF16 ? 2 : 4; }

// A token stride in elements: at least the row, a multiple of 16 bytes.
bool stride_ok(const ice_paged* pg, int64_t stride, int heads) {
    return stride >= (int64_t)heads * kD && stride * es_of(pg) % 16 == 0 && stride <= (1LL << 30);
}

}  // namespace

extern "C" {

int ice_paged_create(const ice_paged_params* params, ice_paged** out) {
    ApiRange range_("ice_paged_create");
    if (!out) return ICE_ERR_INVALID_ARG;
    *out = nullptr;
    const int rc = check(params);
    if (rc != ICE_OK) return rc;
    ice_paged* pg = new (std::nothrow) ice_paged();
    if (!pg) return ICE_ERR_CAPACITY;
    pg->p = *params;
    pg->G = params->n_q_heads / params->n_kv_heads;
    const long long R = (long long)params->max_tokens * params->n_q_heads;
    pg->rows_cap = std::max(3 * R, std::min(128 * R, 262144LL));
    if (cudaGetDevice(&pg->device) != cudaSuccess ||
        cudaDeviceGetAttribute(&pg->n_sm, cudaDevAttrMultiProcessorCount, pg->device) != cudaSuccess ||
        paged_prepare() != cudaSuccess) {
        cudaGetLastError();
        delete pg;
        return ICE_ERR_CUDA;
    }
    if (cudaMalloc(&pg->part_o, (size_t)pg->rows_cap * kD * 4) != cudaSuccess ||
        cudaMalloc(&pg->part_ml, (size_t)pg->rows_cap * 8) != cudaSuccess ||
        cudaMalloc(&pg->words, (kWords + params->max_requests) * 4) != cudaSuccess) {
        cudaGetLastError();
        free_all(pg);
        delete pg;
        return ICE_ERR_CAPACITY;
    }
    // complete before the call returns, whatever stream is used first
    if (cudaMemset(pg->words, 0, kWords * 4) != cudaSuccess || cudaStreamSynchronize(nullptr) != cudaSuccess) {
        cudaGetLastError();
        free_all(pg);
        delete pg;
        return ICE_ERR_CUDA;
    }
    *out = pg;
    return ICE_OK;
}

void ice_paged_destroy(ice_paged* pg) {
    if (!pg) return;
    int dev = 0;
    const bool had = cudaGetDevice(&dev) == cudaSuccess;
    cudaSetDevice(pg->device);
    cudaDeviceSynchronize();
    free_all(pg);
    if (had) cudaSetDevice(dev);
    cudaGetLastError();
    delete pg;
}

int ice_paged_get_error(ice_paged* pg, void* stream) {
    if (!pg) return ICE_ERR_INVALID_ARG;
    int code = 0;
    cudaStream_t st = (cudaStream_t)stream;
    if (cudaMemcpyAsync(&code, pg->words + kWordStatus, sizeof(int), cudaMemcpyDeviceToHost, st) != cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess) {
        cudaGetLastError();
        return ICE_ERR_CUDA;
    }
    if (code != 0 && cudaMemsetAsync(pg->words + kWordStatus, 0, sizeof(int), st) != cudaSuccess) {
        cudaGetLastError();
        return ICE_ERR_CUDA;
    }
    return code;
}

int ice_paged_debug_set_flags(ice_paged* pg, int32_t flags) {
    if (!pg || (flags & ~ICE_DEBUG_STALL_ATTN)) return ICE_ERR_INVALID_ARG;
    pg->debug = flags;
    return ICE_OK;
}

int ice_paged_tables(ice_paged* pg, int32_t n_req, const int32_t* seq_len, const int32_t* n_new,
                     int32_t* block_table, int32_t* free_pages, const int64_t* free_state,
                     int32_t* seq_len_out, int64_t* free_state_out, int32_t* q_start,
                     int64_t* slot_map, int32_t* positions, int32_t n_slots, void* stream) {
    ApiRange range_("ice_paged_tables");
    if (!pg || n_req < 1 || n_req > pg->p.max_requests || n_slots < 0 || n_slots > (1 << 30))
        return ICE_ERR_INVALID_ARG;
    Buffers b(pg, stream);
    b.need(seq_len, 4).need(n_new, 4).need(block_table, 4).need(free_pages, 4).need(free_state, 8);
    b.need(seq_len_out, 4).need(free_state_out, 8).need(q_start, 4);
    if (n_slots > 0) b.need(slot_map, 8).opt(positions);
    if (!b.ok || !aligned(positions, 4)) return ICE_ERR_INVALID_ARG;
    const cudaError_t e = launch_paged_tables(
        n_req, pg->p.max_blocks, pg->p.page_size, pg->p.n_pages, seq_len, n_new, block_table, free_pages,
        (const long long*)free_state, seq_len_out, (long long*)free_state_out, q_start, (long long*)slot_map,
        positions, n_slots, (unsigned*)pg->words + kWordTicket, pg->words + kWordStatus, (cudaStream_t)stream);
    return launched(e);
}

int ice_paged_append(ice_paged* pg, int32_t n_tokens, const void* k, int64_t k_stride, const void* v,
                     int64_t v_stride, const int64_t* slot_map, void* k_pages, void* v_pages,
                     void* stream) {
    ApiRange range_("ice_paged_append");
    if (!pg || n_tokens < 0) return ICE_ERR_INVALID_ARG;
    if (!stride_ok(pg, k_stride, pg->p.n_kv_heads) || !stride_ok(pg, v_stride, pg->p.n_kv_heads))
        return ICE_ERR_INVALID_ARG;
    if (n_tokens == 0) return ICE_OK;
    Buffers b(pg, stream);
    b.need(k, 16).need(v, 16).need(slot_map, 8).need(k_pages, 16).need(v_pages, 16);
    if (!b.ok) return ICE_ERR_INVALID_ARG;
    const cudaError_t e =
        launch_paged_append(n_tokens, pg->p.n_kv_heads, pg->p.page_size, es_of(pg), pg->p.n_pages, k, k_stride, v,
                            v_stride, (const long long*)slot_map, k_pages, v_pages, pg->words + kWordStatus,
                            (cudaStream_t)stream);
    return launched(e);
}

int ice_paged_attn(ice_paged* pg, int32_t n_req, int32_t n_tokens, const void* q, int64_t q_stride,
                   const int32_t* q_start, const int32_t* seq_len, const int32_t* block_table,
                   const int32_t* prefix_table, int32_t prefix_len, const void* k_pages,
                   const void* v_pages, void* out, void* stream) {
    ApiRange range_("ice_paged_attn");
    if (!pg || n_req < 1 || n_req > pg->p.max_requests || n_tokens < 0 || n_tokens > pg->p.max_tokens)
        return ICE_ERR_INVALID_ARG;
    if (prefix_len < 0 || prefix_len > (1 << 30) || !stride_ok(pg, q_stride, pg->p.n_q_heads))
        return ICE_ERR_INVALID_ARG;
    if (n_tokens == 0) return ICE_OK;
    const uintptr_t es = es_of(pg), q0 = (uintptr_t)q, o0 = (uintptr_t)out;
    const uintptr_t row = (uintptr_t)pg->p.n_q_heads * kD * es;
    if (q0 < o0 + n_tokens * row && o0 < q0 + (n_tokens - 1) * (uintptr_t)q_stride * es + row) return ICE_ERR_INVALID_ARG;
    Buffers b(pg, stream);
    b.need(q, 16).need(q_start, 4).need(seq_len, 4).need(block_table, 4);
    if (prefix_len > 0) b.need(prefix_table, 4);
    b.need(k_pages, 16).need(v_pages, 16).need(out, 16);
    if (!b.ok) return ICE_ERR_INVALID_ARG;
    PagedAttn a = {};
    a.q = q;
    a.q_stride = q_stride;
    a.q_start = q_start;
    a.seq_len = seq_len;
    a.block_table = block_table;
    a.prefix_table = prefix_table;
    a.k_pages = k_pages;
    a.v_pages = v_pages;
    a.out = out;
    a.part_o = pg->part_o;
    a.part_ml = pg->part_ml;
    a.plan = pg->words + kWordPlan;
    a.first_long = pg->words + kWords;
    a.next = (unsigned*)pg->words + kWordNext;
    a.status = pg->words + kWordStatus;
    a.scale_log2 = 1.44269504088896341f * 0.08838834764831845f;  // log2(e) / sqrt(128)
    a.n_req = n_req;
    a.n_tokens = n_tokens;
    a.H = pg->p.n_kv_heads;
    a.G = pg->G;
    a.P = pg->p.page_size;
    a.max_blocks = pg->p.max_blocks;
    a.prefix_len = prefix_len;
    a.n_pages = pg->p.n_pages;
    a.debug = pg->debug;
    const cudaError_t e = launch_paged_attn(a, pg->p.dtype, pg->rows_cap, pg->n_sm, (cudaStream_t)stream);
    return launched(e);
}

}  // extern "C"
