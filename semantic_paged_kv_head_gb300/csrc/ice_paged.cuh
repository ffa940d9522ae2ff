// The plain paged cache of a batch whose requests share a prefix: what its
// kernels and its C entries share.
//
// Pages of one layer: k_pages, v_pages [n_pages][H][P][D] T, so that a page's
// rows of one KV head are P * D contiguous elements.
#pragma once

#include <limits.h>

#include "ice_internal.cuh"

namespace ice {

constexpr int kPagedMaxRequests = 8192;
constexpr int kPagedMaxPrefixSplits = 64;  // parts of the prefix that are attended separately

// Attention of one call, passed by value. The work is a list of items, each a
// block of rows (new tokens x the G query heads of a KV head) against a range of
// key tiles: prefix items, whose rows are the whole batch's, and items of single
// requests. The parts of one row are joined afterwards.
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
    // Parts, by slot and KV head; row R = token * G + head in the group, RP = n_tokens * G.
    float* part_o;   // [slot][H][RP][D]: a part's output, normalised
    float2* part_ml; // [slot][H][RP]: its maximum (log2 units) and sum
    int* plan;       // kPlanWords, written by the attention kernel for the joining kernel
    int* first_long; // [n_req]: number of each request's first row block x head, if it is long
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
    int debug;          // ICE_DEBUG_* flags (tests only), 0 in normal use
};
constexpr int kPagedMaxSlots = 128;

// plan words: lengths in range, tiles of a range of own tokens, the two of PagedLong, whether the
// prefix items write the output themselves
enum { kPlanOk = 0, kPlanChunk = 1, kPlanWhole = 2, kPlanSplit = 3, kPlanDirect = 4, kPlanWords = 5 };

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

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
        " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}\n"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
// ---- the plan of an attention call, made by every block from the lengths ---------
// Keys per tile KT, new tokens per row block TB. Tiles are numbered through the
// prefix's NP and on through a request's own.
//
// A request of more than TS new tokens has row blocks of its own. Full ones gain nothing by
// sharing, so their items run through the prefix and the request's own tokens in one pass
// and have nothing to join (one of little more than TS tokens would gain: with G = 8, 8 requests of 17
// on 32k take 200 us, of 16, which share, 116), except those of the last, incomplete wave over the GPU, which are cut
// into `split` parts each. The other requests' rows share the prefix items, and their own tokens
// are cut into ranges of `chunk` tiles; with TD > 0 one block attends two streams side
// by side: two KV heads, or the two halves of a range where there is one head.
// chunk gives about target_items items in all, but no stream is longer than
// kPagedMaxRange tiles (the last items to end are then short), and keeps the parts
// within max_splits.
constexpr int kPagedMaxRange = 24;

__host__ __device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

struct PagedTiles {
    int KT, TB, TS, TD;  // TD = TS, or 0: one stream at a time
    int NP, pages;       // tiles of the prefix, pages of a tile (TD > 0)
};

// Parts of the own tokens of a request that shares the prefix items: one a range, or two.
__device__ __forceinline__ int plan_parts(int s, int H, const PagedTiles& z, int chunk) {
    if (s <= 0) return 0;
    const int t = ceil_div(s, z.KT), ranges = ceil_div(t, chunk);
    return z.TD > 0 && H == 1 ? min(t, 2 * ranges) : ranges;
}

// Row blocks x heads of long requests are numbered: request by request, head by head. Those
// below `whole` are one item each, the others `split`.
struct PagedLong {
    int whole, split;
};
// Of a long request whose first number is g0, those that are one item each.
__device__ __forceinline__ int long_whole(int g0, int n, const PagedLong& f) { return min(max(f.whole - g0, 0), n); }

__device__ __forceinline__ int long_blocks(int nq, int s, const PagedTiles& z) {
    return nq > z.TS && (z.NP > 0 || s > 0) ? ceil_div(nq, z.TB) : 0;
}
// Items of a request.
__device__ __forceinline__ int plan_items(int nq, int s, int H, int g0, const PagedTiles& z, int chunk, const PagedLong& f) {
    if (nq <= 0) return 0;
    if (nq > z.TS) {
        const int n = long_blocks(nq, s, z) * H, w = long_whole(g0, n, f);
        return w + (n - w) * f.split;
    }
    const int parts = plan_parts(s, H, z, chunk);
    return z.TD == 0 ? parts * H : H == 1 ? (parts + 1) >> 1 : parts * ((H + 1) >> 1);
}

struct PlanShared {
    // sums over the requests: tiles of the own tokens of requests that share the prefix, tiles and
    // number of the row blocks of long ones; the most own tiles of one of the former
    unsigned long long w, wl;
    unsigned nl, mx;
    unsigned fl;  // 1 bad length, 2 a request that shares the prefix, 4 one with own tokens
    int sum[32], sum2[32];                   // per warp: items, row blocks of long requests
    int ok, chunk, own, pre, direct;         // items of requests, of the prefix
    int some_long;
    PagedLong f;
    const int *q_start, *seq_len;            // in shared memory where they fit
    const int* first_long;
};

// Bytes of shared memory for the plan's lists: items before each request, and (where the
// room for kPagedMaxRequests allows) the lengths.
__host__ __device__ constexpr int plan_ints(int n_req) {
    return 4 * (n_req + 1) <= kPagedMaxRequests + 1 ? 4 * (n_req + 1) : n_req + 1;
}

// Sum of the values of the warps before, from their inclusive scan; every thread's exclusive sum.
__device__ __forceinline__ int block_scan(int mine, int* sums, int& total, int nw) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = mine;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
    }
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    const int v = lane < nw ? sums[lane] : 0;
    total = __reduce_add_sync(0xffffffffu, v);
    return __reduce_add_sync(0xffffffffu, lane < warp ? v : 0) + inc - mine;
}

// Fills cum[0 .. n_req] (items before each request) and sh; all threads of the block call
// it. Block-uniform results after the last barrier. Every block comes to the same plan (integer
// sums). Nothing is unrolled: the code runs once, and at the start of a call it comes from memory.
template <int NT>
__device__ __forceinline__ void make_plan(const PagedAttn& a, const PagedTiles& z, int* cum, PlanShared& sh) {
    const int tid = threadIdx.x, lane = tid & 31;
    constexpr int NW = NT / 32;
    const int n = a.n_req, per = (n + NT - 1) / NT;
    const int r0 = min(tid * per, n), r1 = min(r0 + per, n);
    const bool keep = plan_ints(n) > n + 1;
    int *qs = cum + n + 1, *sl = qs + n + 1, *gl = sl + n + 1;
    if (tid == 0) sh.w = sh.wl = 0, sh.nl = sh.mx = sh.fl = 0;
    __syncthreads();
    unsigned long long w = 0, wl = 0;
    unsigned mx = 0, nl = 0, fl = 0;
#pragma unroll 1
    for (int r = r0; r < r1; ++r) {
        const int b = a.q_start[r], e = a.q_start[r + 1], s = a.seq_len[r];
        if (keep) {
            qs[r] = b;
            sl[r] = s;
            if (r == n - 1) qs[n] = e;
        }
        if (b < 0 || e < b || e > a.n_tokens || s < 0 || s > a.max_blocks * a.P || (r == 0 && b != 0)) {
            fl |= 1;
        } else if (e - b > z.TS) {
            const int blocks = long_blocks(e - b, s, z);
            nl += blocks;
            wl += (unsigned long long)blocks * (z.NP + ceil_div(s, z.KT));
        } else if (e > b) {
            fl |= s > 0 ? 6 : 2;
            const unsigned t = ceil_div(s, z.KT);
            w += t;
            mx = max(mx, t);
        }
    }
    if (w) atomicAdd(&sh.w, w);
    if (wl) atomicAdd(&sh.wl, wl);
    nl = __reduce_add_sync(0xffffffffu, nl);
    mx = __reduce_max_sync(0xffffffffu, mx);
    fl = __reduce_or_sync(0xffffffffu, fl);
    if (lane == 0) {
        if (nl) atomicAdd(&sh.nl, nl);
        atomicMax(&sh.mx, mx);
        atomicOr(&sh.fl, fl);
    }
    __syncthreads();
    nl = sh.nl, mx = sh.mx, fl = sh.fl;
    const bool bad = fl & 1;
    // with two streams of one head a range is two parts: twice the tiles, an even number of parts
    const int halves = z.TD > 0 && a.H == 1 ? 2 : 1;
    const float want = (float)sh.w * (float)a.H / (float)(a.target_items * (z.TD > 0 ? 2 : 1));
    const int chunk = halves * max(max((int)fminf(ceilf(want), (float)kPagedMaxRange), 1),
                                   ceil_div((int)mx, a.max_splits / halves * halves));
    // parts of the last wave's: waves x (tiles of a part + the fixed cost of an item, and of
    // joining it, in tiles), the least of 1 to 16
    // (where the lengths do not fit in shared memory, with thousands of requests, all are whole)
    PagedLong f = {INT_MAX, 1};
    if (nl > 0 && keep) {
        const int all = nl * a.H, rest = all % a.target_items, mean = (int)((float)sh.wl / (float)nl);
        f.whole = all - rest;  // the last `rest` are an incomplete wave
        int best = INT_MAX;
        const int most = rest > 0 ? min(16, min(a.max_splits, max(mean, 1))) : 0;
#pragma unroll 1
        for (int k = 1; k <= most; ++k) {
            const int t = ceil_div(rest * k, a.target_items) * (ceil_div(mean, k) + (k > 1 ? 6 : 3));
            if (t < best) {
                best = t;
                f.split = k;
            }
        }
    }
    // long row blocks before each thread's requests, then items
    int g0 = 0, total;
    if (nl > 0) {
        int mine = 0;
#pragma unroll 1
        for (int r = r0; r < r1 && !bad; ++r) mine += long_blocks(a.q_start[r + 1] - a.q_start[r], a.seq_len[r], z);
        g0 = block_scan(mine, sh.sum2, total, NW) * a.H;
    }
    int before = 0;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
        int g = g0, mine = 0;
#pragma unroll 1
        for (int r = r0; r < r1 && !bad; ++r) {
            const int nq = a.q_start[r + 1] - a.q_start[r], s = a.seq_len[r];
            if (pass) {
                cum[r] = before + mine;
                if (nl > 0 && keep) {
                    gl[r] = g;
                    if (blockIdx.x == 0) a.first_long[r] = g;  // for the joining kernel
                }
            }
            mine += plan_items(nq, s, a.H, g, z, chunk, f);
            g += long_blocks(nq, s, z) * a.H;
        }
        if (pass == 0) before = block_scan(mine, sh.sum, total, NW);
    }
    if (tid == 0) {
        cum[n] = total;
        sh.ok = !bad;
        sh.chunk = chunk;
        sh.f = f;
        sh.own = total;
        sh.some_long = nl > 0;
        // the prefix's: row blocks x heads x ranges, cut in two where all rows fit one stream
        const int ranges = z.TD > 0 && a.n_tokens <= z.TD ? (a.prefix_splits + 1) >> 1 : a.prefix_splits;
        sh.pre = fl & 2 ? ceil_div(a.n_tokens, z.TB) * a.H * ranges : 0;
        sh.direct = a.prefix_splits == 1 && !(fl & 4) && nl == 0;
        sh.q_start = keep ? qs : a.q_start;
        sh.seq_len = keep ? sl : a.seq_len;
        sh.first_long = gl;
        if (blockIdx.x == 0) {
            a.plan[kPlanOk] = !bad;
            a.plan[kPlanChunk] = chunk;
            a.plan[kPlanWhole] = f.whole;
            a.plan[kPlanSplit] = f.split;
            a.plan[kPlanDirect] = sh.direct;
            if (bad) set_status(a.status, ICE_ERR_BOUNDS);
        }
    }
    __syncthreads();
}

// Rows of new tokens tok0 .. tok0 + ntok - 1 of KV head h against tiles kt0 .. kt0 + n - 1.
// Token t sees the prefix and the own tokens below min(own_len, t + lim_off).
struct PagedStream {
    const int* own_table;
    int h, tok0, ntok, own_len, lim_off, kt0, n, slot;
    int direct;  // the rows have no other part: write the output itself
};

struct PagedItem {
    PagedStream st[2];
    int ns;      // streams: 1 or 2 (0: nothing to do)
    int shared;  // both streams, row tiles of one block, read the same key tiles
    int same_q;  // both streams, parts of one range, have the same rows
};

// A tile of a stream: its page list, the first key in it, the list's keys.
struct PagedTile {
    const int* table;
    int key0, len;
    bool own;
};
__device__ __forceinline__ PagedTile tile_of(const PagedAttn& a, const PagedTiles& z, const PagedStream& s, int x) {
    PagedTile t;
    t.own = x >= z.NP;
    t.table = t.own ? s.own_table : a.prefix_table;
    t.key0 = (t.own ? x - z.NP : x) * z.KT;
    t.len = t.own ? s.own_len : a.prefix_len;
    return t;
}

// The last r in [0, n) with v[r] <= i (v[0] <= i).
__device__ __forceinline__ int find_last(const int* v, int n, int i) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (v[mid] <= i) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Item i < sh.pre + sh.own. The items of the prefix are the longer ones. Up to one a block they
// come first; with more of them they are every third item while they last: they are bound by
// arithmetic and own tokens of few rows by memory, and the two overlap on different SMs.
__device__ __forceinline__ void get_item(const PagedAttn& a, const PagedTiles& z, const int* cum,
                                         const PlanShared& sh, int i, PagedItem& out) {
    const int every = min(3, (sh.pre + sh.own) / max(sh.pre, 1));
    const int span = sh.pre * every;
    bool pre;
    if (sh.pre <= a.target_items) {
        pre = i < sh.pre;
        if (!pre) i -= sh.pre;
    } else if (i < span) {
        const int k = i / every;
        pre = i == k * every;
        i = pre ? k : i - k - 1;
    } else {
        pre = false;
        i -= sh.pre;
    }
    const int NP = z.NP;
    const int tpt = z.TD > 0 ? z.TD : z.TB;  // tokens of a row tile
    PagedStream st;
    int ns = 1, shared = 0, base, nt, parts, p0;
    bool twin = false, two_heads = false;
    if (pre) {
        // row blocks fastest: the blocks that run together read the same keys (from L2)
        const int nb = ceil_div(a.n_tokens, z.TB);
        const int k = i / nb, rb = i - k * nb;
        st.tok0 = rb * z.TB;
        st.h = k % a.H;
        st.ntok = min(z.TB, a.n_tokens - st.tok0);
        st.own_table = nullptr;
        st.own_len = 0;
        st.lim_off = 0;
        st.direct = sh.direct;
        base = 0;
        nt = NP;
        parts = a.prefix_splits;
        twin = z.TD > 0 && a.n_tokens <= z.TD;
        p0 = (k / a.H) << (int)twin;
        st.slot = p0;
        if (sh.some_long) {  // nothing to do where the block's tokens are all of long requests
            bool any = false;
            for (int r = find_last(sh.q_start, a.n_req, st.tok0); r < a.n_req && !any; ++r) {
                const int b = sh.q_start[r], e = sh.q_start[r + 1];
                if (b >= st.tok0 + st.ntok) break;
                any = e > max(b, st.tok0) && e - b <= z.TS;
            }
            if (!any) ns = 0;
        }
    } else {
        const int lo = find_last(cum, a.n_req, i);
        const int b = sh.q_start[lo], e = sh.q_start[lo + 1], s = sh.seq_len[lo], x = i - cum[lo];
        st.own_table = a.block_table + (long long)lo * a.max_blocks;
        st.own_len = s;
        st.lim_off = s - e + 1;  // the last new token, e - 1, sees all s
        int rb = 0;
        if (e - b > z.TS) {
            const int blocks = ceil_div(e - b, z.TB), n = blocks * a.H;
            const int whole = long_whole(sh.f.whole == INT_MAX ? 0 : sh.first_long[lo], n, sh.f);
            int y = x;  // head, row block: the blocks of a head run together
            p0 = 0;
            parts = 1;
            if (x >= whole) {
                p0 = (x - whole) / (n - whole);
                y = x - p0 * (n - whole);
                parts = sh.f.split;
            }
            st.h = y / blocks;
            rb = y - st.h * blocks;
            base = 0;
            st.direct = parts == 1;
        } else {
            parts = plan_parts(s, a.H, z, sh.chunk);
            base = NP;
            twin = z.TD > 0 && a.H == 1 && parts > 1;
            two_heads = z.TD > 0 && a.H > 1;
            const int hs = two_heads ? (a.H + 1) >> 1 : a.H, k = x / hs;
            st.h = (x - k * hs) << (int)two_heads;
            p0 = k << (int)twin;
            st.direct = a.prefix_splits == 0 && parts == 1;
        }
        st.tok0 = b + rb * z.TB;
        st.ntok = min(z.TB, e - st.tok0);
        st.slot = a.prefix_splits + p0;
        const int seen = min(s, st.tok0 + st.ntok - 1 + st.lim_off);
        nt = NP - base + (seen > 0 ? ceil_div(seen, z.KT) : 0);
    }
    // fits 32 bits: at most 2^25 tiles and 16 parts, or 2^24 and 128
    auto edge = [&](int p) { return base + (int)((unsigned)nt * (unsigned)p / (unsigned)parts); };
    st.kt0 = edge(p0);
    const int kt1 = edge(p0 + 1);
    st.n = kt1 - st.kt0;
    out.st[1] = st;
    out.same_q = twin && p0 + 1 < parts;
    if (out.same_q) {
        ns *= 2;
        out.st[1].kt0 = kt1;
        out.st[1].n = edge(p0 + 2) - kt1;
        out.st[1].slot = st.slot + 1;
    } else if (two_heads && st.h + 1 < a.H) {
        ns *= 2;
        out.st[1].h = st.h + 1;
    } else if (st.ntok > tpt) {
        ns *= 2;
        shared = 1;
        out.st[1].tok0 = st.tok0 + tpt;
        out.st[1].ntok = st.ntok - tpt;
        st.ntok = tpt;
    }
    out.st[0] = st;
    out.ns = ns;
    out.shared = shared;
}

}  // namespace ice
