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
    // Parts, by slot and KV head; row R = token * G + head in the group, RP = n_tokens * G
    // rounded up to 32. Rows are innermost: a warp of the attention holds 32 rows, one a
    // lane, and writes full lines (as [row][d] the stores of an item took 7 us).
    float* part_o;   // [slot][H][D][RP]: a part's output, normalised
    float2* part_ml; // [slot][H][RP]: its maximum (log2 units) and sum
    int* plan;       // kPlanWords, written by the attention kernel for the joining kernel
    unsigned* next;  // [2]: items handed out beyond the first of each block, blocks done; zero between calls
    int* status;
    float scale_log2;  // log2(e) / sqrt(d)
    int n_req, n_tokens, H, G, P, max_blocks, prefix_len;
    long long n_pages;
    int RP;
    int prefix_splits;  // parts of the prefix: slots 0 .. prefix_splits - 1 (even in number or one a
                        // tile where two are attended side by side)
    int max_splits;     // most parts of a request's own tokens (slots after the prefix's), >= 2
    int target_items;   // items of own tokens aimed at where they are few
};
constexpr int kPagedMaxSlots = 128;

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
// and s own tokens is ceil(nq / TB) row blocks, each against up to t = ceil(s / KT)
// tiles, cut into ceil(t / chunk) ranges. Where the rows of a request fill
// one row tile or less (nq <= TD), a range is cut once more, into two parts that one
// block attends side by side. chunk gives about target_items items in all, but no range is
// longer than kPagedMaxRange tiles (the last items to end are then short), and keeps the
// parts within max_splits.
constexpr int kPagedMaxRange = 48;

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

struct PagedTiles {
    int KT, TB, TD;  // TD = 0: no second cut
};

__device__ __forceinline__ int plan_parts(int nq, int s, const PagedTiles& z, int chunk) {
    if (nq <= 0 || s <= 0) return 0;
    const int t = ceil_div(s, z.KT), ranges = ceil_div(t, chunk);
    return nq <= z.TD ? min(t, 2 * ranges) : ranges;
}
// Items of a row block of the request.
__device__ __forceinline__ int plan_items(int nq, int parts, const PagedTiles& z) {
    return nq <= z.TD ? (parts + 1) >> 1 : parts;
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
__device__ __forceinline__ void make_plan(const PagedAttn& a, const PagedTiles& z, int* cum, PlanShared& sh) {
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
            const int t = ceil_div(s, z.KT);
            w += (long long)t * ceil_div(e - b, z.TB);
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
    long long chunk = min(max((w * a.H + a.target_items - 1) / a.target_items, 1LL), (long long)kPagedMaxRange);
    chunk = max(chunk, (long long)ceil_div(mx, z.TD > 0 ? a.max_splits / 2 : a.max_splits));
    const int ch = (int)chunk;
    int mine = 0;
    if (!bad)
        for (int r = r0; r < r1; ++r) {
            const int nq = a.q_start[r + 1] - a.q_start[r];
            mine += ceil_div(nq, z.TB) * plan_items(nq, plan_parts(nq, a.seq_len[r], z, ch), z);
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
            before += ceil_div(nq, z.TB) * plan_items(nq, plan_parts(nq, a.seq_len[r], z, ch), z);
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
// key tiles of a page list. Token t sees keys below min(kv_len, t + lim_off).
struct PagedItem {
    const int* table;
    int h, tok0, ntok, kv_len, lim_off;
    int kt0, n[2];  // tiles kt0 .. kt0 + n[0] - 1; a second part, if any: the n[1] tiles that follow
    int parts;      // 1, or 2 (slots slot and slot + 1)
    int slot;
    int direct;     // the rows have no other part: write the output itself
};

// Items of the prefix: row blocks x heads x ranges; ranges are cut into two parts where
// all the rows fill one row tile or less.
__device__ __forceinline__ int prefix_items(const PagedAttn& a, const PagedTiles& z) {
    return ceil_div(a.n_tokens, z.TB) * a.H * plan_items(a.n_tokens, a.prefix_splits, z);
}

// Fits an int: the scratch for the rows alone would pass the GPU's memory before.
__device__ __forceinline__ int item_count(const PagedAttn& a, const PagedTiles& z, const PlanShared& sh) {
    return prefix_items(a, z) + sh.items * a.H;
}

// Item i < item_count. Prefix items and own items alternate as long as there are both: the
// former are bound by arithmetic, the latter by memory, and they overlap on
// different SMs.
__device__ __forceinline__ void get_item(const PagedAttn& a, const PagedTiles& z, const int* cum,
                                         const PlanShared& sh, int i, PagedItem& out) {
    PagedItem it;
    const int n_pre = prefix_items(a, z), n_own = sh.items * a.H;
    const int both = 2 * min(n_pre, n_own);
    bool pre;
    if (i < both) {
        pre = !(i & 1);
        i >>= 1;
    } else {
        pre = n_pre > n_own;
        i -= both >> 1;
    }
    it.n[1] = 0;
    it.parts = 1;
    int nt, parts, p0, twin;
    if (pre) {
        // row blocks fastest: the blocks that run together read the same keys (from L2)
        const int nb = ceil_div(a.n_tokens, z.TB);
        const int rb = i % nb, k = i / nb;
        it.tok0 = rb * z.TB;
        it.h = k % a.H;
        it.ntok = min(z.TB, a.n_tokens - it.tok0);
        it.kv_len = a.prefix_len;
        it.lim_off = 1 << 30;
        it.table = a.prefix_table;
        it.direct = a.prefix_splits == 1 && sh.items == 0;
        nt = ceil_div(a.prefix_len, z.KT);
        parts = a.prefix_splits;
        twin = a.n_tokens <= z.TD;
        p0 = (k / a.H) << twin;
        it.slot = p0;
    } else {
        const int k = i / a.H;
        it.h = i - k * a.H;  // heads fastest: neighbours in a page
        int lo = 0, hi = a.n_req;  // the last r with cum[r] <= k
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (cum[mid] <= k) lo = mid;
            else hi = mid;
        }
        const int b = a.q_start[lo], e = a.q_start[lo + 1], s = a.seq_len[lo];
        parts = plan_parts(e - b, s, z, sh.chunk);
        const int x0 = k - cum[lo], items = plan_items(e - b, parts, z);
        const int rb = x0 / items;
        it.tok0 = b + rb * z.TB;
        it.ntok = min(z.TB, e - it.tok0);
        it.lim_off = s - e + 1;  // the last new token, e - 1, sees all s
        it.kv_len = s;
        it.table = a.block_table + (long long)lo * a.max_blocks;
        it.direct = a.prefix_splits == 0 && parts == 1;
        const int seen = min(s, it.tok0 + it.ntok - 1 + it.lim_off);
        nt = seen > 0 ? ceil_div(seen, z.KT) : 0;
        twin = e - b <= z.TD;
        p0 = (x0 - rb * items) << twin;
        it.slot = a.prefix_splits + p0;
    }
    auto edge = [&](int p) { return (int)((long long)nt * p / parts); };
    it.kt0 = edge(p0);
    const int kt1 = edge(p0 + 1);
    it.n[0] = kt1 - it.kt0;
    if (twin && p0 + 1 < parts) {
        it.parts = 2;
        it.n[1] = edge(p0 + 2) - kt1;
    }
    out = it;
}

}  // namespace ice
