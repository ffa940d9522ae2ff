// The plain paged cache of a batch whose requests share a prefix: what its
// kernels and its C entries share.
//
// Pages of one layer: k_pages, v_pages [n_pages][H][P][D] T, so that a page's
// rows of one KV head are P * D contiguous elements.
#pragma once

#include "ice_internal.cuh"

namespace ice {

constexpr int kPagedMaxRequests = 8192;
constexpr int kPagedMaxPrefixSplits = 64;  // parts of the prefix that are attended separately

// Attention of one call, passed by value. The work is a list of items, each a
// block of rows (new tokens x the G query heads of a KV head) against a range of
// key tiles: first the prefix items, whose rows are the whole batch's, then the
// items of the requests' own tokens. Items of one row are joined afterwards.
struct PagedAttn {
    const void* q;
    long long q_stride;  // elements
    const int* q_start;
    const int* seq_len;
    const int* block_table;
    const int* prefix_table;
    const void* k_pages;
    const void* v_pages;
    void* out;
    float* part_o;   // [slot][n_tokens * Hq][D]: a part's output, normalised
    float2* part_ml; // [slot][n_tokens * Hq]: its maximum (log2 units) and sum
    int* plan;       // kPlanWords, written by the attention kernel for the joining kernel
    int* status;
    float scale_log2;  // log2(e) / sqrt(d)
    int n_req, n_tokens, H, G, P, max_blocks, prefix_len;
    long long n_pages;
    int prefix_splits;  // parts of the prefix: slots 0 .. prefix_splits - 1
    int max_splits;     // most parts of a request's own tokens (slots after the prefix's)
    int target_items;   // items of own tokens aimed at
};

enum { kPlanOk = 0, kPlanChunk = 1, kPlanOwn = 2, kPlanWords = 4 };

cudaError_t launch_paged_tables(int n_req, int max_blocks, int P, long long n_pages, const int* seq_len,
                                const int* n_new, int* block_table, int* free_pages,
                                const long long* free_state, int* seq_len_out, long long* free_state_out,
                                int* q_start, long long* slot_map, int* positions, int n_slots,
                                unsigned* ticket, int* status, cudaStream_t s);
cudaError_t launch_paged_append(int n_tokens, int H, int P, int es, long long n_pages, const void* k,
                                long long k_stride, const void* v, long long v_stride,
                                const long long* slot_map, void* k_pages, void* v_pages, int* status,
                                cudaStream_t s);
// rows_cap: rows of partial results that part_o and part_ml hold
cudaError_t launch_paged_attn(PagedAttn a, int dtype, long long rows_cap, int n_sm, cudaStream_t s);
cudaError_t paged_prepare();

// ---- the plan of an attention call, made by every block from the lengths ---------
// Keys per tile KT, new tokens per row block TB. Request r with nq new tokens
// and s own tokens is ceil(nq / TB) row blocks, each against up to ceil(s / KT)
// tiles, cut into ceil(ceil(s / KT) / chunk) parts; chunk is the least that keeps
// the items near target_items and the parts within max_splits.
__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

__device__ __forceinline__ int plan_splits(int nq, int s, int KT, int chunk) {
    return nq > 0 && s > 0 ? ceil_div(ceil_div(s, KT), chunk) : 0;
}

struct PlanShared {
    long long w[32];  // per warp: tiles of all row blocks
    int mx[32];       // per warp: most tiles of a request
    int bad[32];
    int sum[32];
    int ok, chunk, items;  // items: of own tokens and one KV head
};

// Fills cum[0 .. n_req] (items before each request, one KV head) and sh; all threads of the
// block call it. Block-uniform results after the last barrier.
template <int NT>
__device__ __forceinline__ void make_plan(const PagedAttn& a, int KT, int TB, int* cum, PlanShared& sh) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int NW = NT / 32;
    const int n = a.n_req, per = (n + NT - 1) / NT;
    const int r0 = min(tid * per, n), r1 = min(r0 + per, n);
    const long long cap = (long long)a.max_blocks * a.P;
    long long w = 0;
    int mx = 0, bad = 0;
    for (int r = r0; r < r1; ++r) {
        const int b = a.q_start[r], e = a.q_start[r + 1], s = a.seq_len[r];
        if (b < 0 || e < b || e > a.n_tokens || s < 0 || s > cap || (r == 0 && b != 0)) {
            bad = 1;
        } else if (e > b && s > 0) {
            const int t = ceil_div(s, KT);
            w += (long long)t * ceil_div(e - b, TB);
            mx = max(mx, t);
        }
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        w += __shfl_xor_sync(0xffffffffu, w, o);
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        bad |= __shfl_xor_sync(0xffffffffu, bad, o);
    }
    if (lane == 0) {
        sh.w[warp] = w;
        sh.mx[warp] = mx;
        sh.bad[warp] = bad;
    }
    __syncthreads();
    w = 0, mx = 0, bad = 0;
#pragma unroll
    for (int k = 0; k < NW; ++k) {
        w += sh.w[k];
        mx = max(mx, sh.mx[k]);
        bad |= sh.bad[k];
    }
    long long chunk = max((w * a.H + a.target_items - 1) / a.target_items, 1LL);
    chunk = max(chunk, (long long)ceil_div(mx, a.max_splits));
    const int ch = (int)min(chunk, (long long)(1 << 30));
    int mine = 0;
    if (!bad)
        for (int r = r0; r < r1; ++r) {
            const int nq = a.q_start[r + 1] - a.q_start[r];
            mine += ceil_div(max(nq, 0), TB) * plan_splits(nq, a.seq_len[r], KT, ch);
        }
    int inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
    }
    if (lane == 31) sh.sum[warp] = inc;
    __syncthreads();
    int before = inc - mine, total = 0;
#pragma unroll
    for (int k = 0; k < NW; ++k) {
        if (k < warp) before += sh.sum[k];
        total += sh.sum[k];
    }
    if (!bad)
        for (int r = r0; r < r1; ++r) {
            cum[r] = before;
            const int nq = a.q_start[r + 1] - a.q_start[r];
            before += ceil_div(max(nq, 0), TB) * plan_splits(nq, a.seq_len[r], KT, ch);
        }
    if (tid == 0) {
        cum[n] = total;
        sh.ok = !bad;
        sh.chunk = ch;
        sh.items = total;
        if (blockIdx.x == 0) {
            a.plan[kPlanOk] = !bad;
            a.plan[kPlanChunk] = ch;
            a.plan[kPlanOwn] = total;
            if (bad) set_status(a.status, ICE_ERR_BOUNDS);
        }
    }
    __syncthreads();
}

// One item of work: rows of new tokens tok0 .. tok0 + ntok - 1 of KV head h against
// key tiles kt0 .. kt1 - 1 of a page list. Token t sees keys below
// min(kv_len, t + lim_off).
struct PagedItem {
    const int* table;
    int h, tok0, ntok, kt0, kt1, kv_len, lim_off, slot;
    bool direct;  // the rows have no other part: write the output itself
};

// Most items there can be is known on the host only as a bound; item index i runs
// over prefix items and then own items. False when i is past the last.
__device__ __forceinline__ bool get_item(const PagedAttn& a, int KT, int TB, const int* cum,
                                         const PlanShared& sh, long long i, PagedItem& it) {
    const int nb = ceil_div(a.n_tokens, TB);
    const long long n_pre = (long long)nb * a.H * a.prefix_splits;
    if (i < n_pre) {
        // row blocks fastest: the blocks that run together read the same keys (from L2)
        it.tok0 = (int)(i % nb) * TB;
        i /= nb;
        it.h = (int)(i % a.H);
        it.slot = (int)(i / a.H);
        it.ntok = min(TB, a.n_tokens - it.tok0);
        const int nt = ceil_div(a.prefix_len, KT);
        it.kt0 = (int)((long long)nt * it.slot / a.prefix_splits);
        it.kt1 = (int)((long long)nt * (it.slot + 1) / a.prefix_splits);
        it.kv_len = a.prefix_len;
        it.lim_off = 1 << 30;
        it.table = a.prefix_table;
        it.direct = a.prefix_splits == 1 && sh.items == 0;
        return true;
    }
    i -= n_pre;
    if (i >= (long long)sh.items * a.H) return false;
    it.h = (int)(i % a.H);  // heads fastest: neighbours in a page
    const int k = (int)(i / a.H);
    int lo = 0, hi = a.n_req;  // the last r with cum[r] <= k
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cum[mid] <= k) lo = mid;
        else hi = mid;
    }
    const int b = a.q_start[lo], e = a.q_start[lo + 1], s = a.seq_len[lo];
    const int splits = plan_splits(e - b, s, KT, sh.chunk);
    const int rb = (k - cum[lo]) / splits, part = (k - cum[lo]) - rb * splits;
    it.tok0 = b + rb * TB;
    it.ntok = min(TB, e - it.tok0);
    it.lim_off = s - e + 1;  // the last new token, e - 1, sees all s
    it.kv_len = s;
    const int seen = min(s, it.tok0 + it.ntok - 1 + it.lim_off);
    const int nt = seen > 0 ? ceil_div(seen, KT) : 0;
    it.kt0 = (int)((long long)nt * part / splits);
    it.kt1 = (int)((long long)nt * (part + 1) / splits);
    it.slot = a.prefix_splits + part;
    it.table = a.block_table + (long long)lo * a.max_blocks;
    it.direct = a.prefix_splits == 0 && splits == 1;
    return true;
}

}  // namespace ice
