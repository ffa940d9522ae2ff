// Pages that several requests hold: forking, block tables with copy on write, compaction of the pool, copies of pages.
#include <cooperative_groups.h>

#include <algorithm>

#include "ice_paged_scan.cuh"
#include "ice_paged_share.cuh"

namespace cg = cooperative_groups;

namespace ice {

// One cluster of blocks.
template <typename Arg>
static cudaError_t launch_cluster(void (*kern)(Arg), int blocks, int threads, size_t smem, cudaStream_t s, const Arg& a) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = blocks;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see pdl_wait_then_release
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

// ---------------------------------------------------------------------------
// Forking: a row of page ids copied and each page's count raised. Every block checks the whole call by itself (the
// destinations as a bitmap in shared memory) and does its share of pieces of 256 columns; the lengths, which may be replaced
// in place, are written by the last block to have read them. Bound by latency: 15 forks of 2304 pages 7.1 us, 3584 of 22 pages at
// most 10.6 us (21 with blocks of 256 threads, whose checks take four times the rounds).
// ---------------------------------------------------------------------------
constexpr int kForkThreads = 1024, kForkFewThreads = 256;  // the latter for few forks
constexpr int kForkPiece = 256;

template <int NT>
__global__ void __launch_bounds__(NT) fork_kernel(Fork a) {
    __shared__ unsigned s_dst[kPagedMaxRequests / 32];
    __shared__ int s_last;
    const int tid = threadIdx.x, lane = tid & 31;
    for (int i = tid; i < kPagedMaxRequests / 32; i += NT) s_dst[i] = 0;
    __syncthreads();
    pdl_wait_then_release();
    const long long cap = (long long)a.max_blocks * a.P;
    auto length = [&](int i) { return a.fork_len ? a.fork_len[i] : a.seq_len[a.src[i]]; };
    bool bad = false;
    for (int i = tid; i < a.n_fork; i += NT) {
        const int s = a.src[i], d = a.dst[i];
        if (s < 0 || s >= a.n || d < 0 || d >= a.n) {
            bad = true;
            continue;
        }
        const int have = a.seq_len[s], len = length(i);
        bad |= (atomicOr(&s_dst[d >> 5], 1u << (d & 31)) >> (d & 31)) & 1;  // a destination given twice
        bad |= have < 0 || have > cap || len < 0 || len > have || a.seq_len[d] != 0;
    }
    __syncthreads();
    for (int i = tid; i < a.n_fork; i += NT) {
        const int s = a.src[i];
        bad |= s >= 0 && s < a.n && ((s_dst[s >> 5] >> (s & 31)) & 1);
    }
    const bool ok = !__syncthreads_or(bad);
    if (ok) {
        const int pieces = (a.max_blocks + kForkPiece - 1) / kForkPiece;
        const long long items = (long long)a.n_fork * pieces;
        const int step = gridDim.x * (NT / 32);
        bool range = false;
        for (long long x = blockIdx.x * (NT / 32) + (tid >> 5); x < items; x += step) {
            const int i = (int)(x / pieces), c0 = (int)(x - (long long)i * pieces) * kForkPiece;
            const int n = min((length(i) + a.P - 1) / a.P, c0 + kForkPiece);
            const int* from = a.block_table + (long long)a.src[i] * a.max_blocks;
            int* to = a.block_table + (long long)a.dst[i] * a.max_blocks;
#pragma unroll 4
            for (int c = c0 + lane; c < n; c += 32) {
                const int p = from[c];
                to[c] = p;
                if (p >= 0 && p < a.n_pages) atomicAdd(a.page_refs + p, 1);
                else range = true;
            }
        }
        if (range) set_status(a.status, ICE_ERR_BOUNDS);
    }
    __syncthreads();
    if (tid == 0) {
        __threadfence();
        s_last = gridDim.x == 1 || atomicAdd(&a.head->ticket, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!s_last) return;
    if (a.seq_len_out != a.seq_len)
        for (int r = tid; r < a.n; r += NT)
            if (!ok || !((s_dst[r >> 5] >> (r & 31)) & 1)) a.seq_len_out[r] = a.seq_len[r];
    if (ok)
        for (int i = tid; i < a.n_fork; i += NT) a.seq_len_out[a.dst[i]] = length(i);  // no source is a destination
    if (tid == 0) {
        if (!ok) set_status(a.status, ICE_ERR_BOUNDS);
        a.head->ticket = 0;
    }
}

cudaError_t launch_fork(const Fork& a, cudaStream_t s) {
    const bool few = a.n_fork <= kForkFewThreads;
    const int threads = few ? kForkFewThreads : kForkThreads;
    const long long items = (long long)a.n_fork * ((a.max_blocks + kForkPiece - 1) / kForkPiece);
    const int blocks = (int)std::max<long long>(1, std::min<long long>(152, (items + threads / 32 - 1) / (threads / 32)));
    return launch_pdl(few ? fork_kernel<kForkFewThreads> : fork_kernel<kForkThreads>, dim3(blocks), dim3(threads), 0, s, a);
}

// ---------------------------------------------------------------------------
// One step's block tables where pages may have several holders. Three phases:
//
// claim  A request lets go of the pages that it no longer touches, and of the page that it is about to write
//        into (its last, incomplete one): each lowers the page's count by one, and leaves its name with the page.
//        The largest name stays: a request that writes goes before one that leaves, then the later request before
//        the earlier. A name carries the call's number, so that names of earlier calls lose and are never cleared.
// count  A page whose count came to 0 has lost all its holders. If its name is of one that writes, that request
//        keeps it; else the named request gives it back to the ring. A request that writes and does not keep its page
//        takes a new one and copies. So each request knows how many pages it takes and gives back.
// fill   As without sharing: sums over the requests, after which every entry is a function of what is there.
//
// Names make the result independent of the order in which the blocks run; the counts are whole numbers. If the step cannot be
// carried out the claims are taken back by adding them again.
//
// A warp takes eight requests and 32 columns at once: requests forked from one hold the same page in the same column, so where they
// are neighbours one claim and one look-up serve all of them (16 requests that share 2304 pages, their end: 28 us with a claim
// a request, 14 so). Which pages a request gives back is noted, a bit an entry, by the second phase for the third.
//
// Bound by latency: loads that depend on each other, three phases and the barriers between them. One thread-block cluster runs the
// phases of most steps: 256 requests of a token, 128 columns, 12.2 us, their end 12.4. See the launch for the other form.
// ---------------------------------------------------------------------------
constexpr int kShrThreads = 1024, kShrGridThreads = 256;
constexpr int kShrCluster = 8;
constexpr int kShrFew = kShrThreads;  // requests of a call that a cluster may serve
constexpr int kShrSlots = 4;    // consecutive slots of a thread
constexpr int kShrRows = 8;     // requests that a warp takes at once, with 32 columns
constexpr int kShrLong = 256;   // columns above which a block instead of a warp gives a request's pages back

__device__ __forceinline__ unsigned long long claim_name(unsigned long long epoch, bool writes, int r) {
    // above every word that a compaction leaves in the claims (below 2^31)
    return (epoch + (1ull << 20)) << 16 | (writes ? 1u << 15 : 0u) | (unsigned)(r + 1);
}

// A request's lengths in tokens and pages, and the columns whose pages it lets go of. grows: it writes into a page that is
// there, and lets go of that one alone.
struct ShareReq {
    int old_len, new_len, had, has, lo, hi;
    int bad;
    bool grows;
};
__device__ __forceinline__ ShareReq share_req(const SharedTables& a, int r) {
    ShareReq q;
    const long long cap = (long long)a.max_blocks * a.P, o = a.seq_len[r], w = o + a.n_new[r];
    q.bad = o < 0 || o > cap || w < 0 ? kBadBounds : w > cap ? kBadCapacity : 0;
    q.old_len = (int)o, q.new_len = (int)w;
    q.had = q.has = q.lo = q.hi = 0;
    q.grows = false;
    if (q.bad) return q;
    q.had = (q.old_len + a.P - 1) / a.P, q.has = (q.new_len + a.P - 1) / a.P;  // lengths up to 2^30
    q.grows = w > o && q.old_len != q.had * a.P;
    q.lo = q.grows ? q.had - 1 : q.has, q.hi = q.had;
    return q;
}

// The work of the first two phases: kShrRows requests and 32 columns an item, a column a lane.
struct ShareItems {
    int groups, words;  // of requests, of 32 columns
    long long n;
};
__device__ __forceinline__ ShareItems share_items(const SharedTables& a) {
    ShareItems x;
    x.groups = (a.n + kShrRows - 1) / kShrRows, x.words = (a.max_blocks + 31) / 32;
    x.n = (long long)x.groups * x.words;
    return x;
}

// An item's requests (request r0 + k with lane k < kShrRows; none has hi = 0) and, if any lets go of pages among its columns, the
// pages (-1: none). Returns whether an id was out of range.
struct ShareItem {
    int r0, word;
    ShareReq q;  // of this lane's request
    bool any;
    int p[kShrRows];
};
__device__ __forceinline__ bool share_item(const SharedTables& a, const ShareItems& items, long long x, ShareItem& it) {
    const int lane = threadIdx.x & 31;
    const int g = (int)(x / items.words), word = (int)(x - (long long)g * items.words);
    it.r0 = g * kShrRows, it.word = word;
    it.q = {};
    if (lane < kShrRows && it.r0 + lane < a.n) it.q = share_req(a, it.r0 + lane);
    it.any = __any_sync(0xffffffffu, max(it.q.lo, 32 * word) < min(it.q.hi, 32 * word + 32));
    bool bad = false;
    if (!it.any) return bad;
    const int c = 32 * word + lane;
    const int* row = a.block_table + (long long)it.r0 * a.max_blocks + c;
    bool in[kShrRows];
#pragma unroll
    for (int k = 0; k < kShrRows; ++k) {
        const int lo = __shfl_sync(0xffffffffu, it.q.lo, k), hi = __shfl_sync(0xffffffffu, it.q.hi, k);
        in[k] = c >= lo && c < hi;
        it.p[k] = in[k] ? row[(long long)k * a.max_blocks] : -1;
    }
#pragma unroll
    for (int k = 0; k < kShrRows; ++k)
        if (in[k] && (it.p[k] < 0 || it.p[k] >= a.n_pages)) it.p[k] = -1, bad = true;
    return bad;
}

// Ids that the ring holds for the step are looked at before anything is written for good, by the last warps: they have the fewest items.
// Beside the claims, so at no cost in a step of few tokens a request (up to 0.2 us); 1.2 us of 18 where 64000 pages of one token are taken.
__device__ __forceinline__ void share_ring(const SharedTables& a, int warp, int warps) {
    const int lane = threadIdx.x & 31;
    int i = 32 * (warps - 1 - warp) + lane;
    if (i >= a.most_taken) return;
    const long long head = a.free_state[0], tail = a.free_state[1];
    if (head < 0 || tail < head || tail - head > a.n_pages) return;  // another fault
    const long long at = head % a.n_pages, n = min(tail - head, (long long)a.most_taken);
    for (; i < n; i += 32 * warps) {
        const int p = a.free_pages[at + i < a.n_pages ? at + i : at + i - a.n_pages];
        if (p < 0 || p >= a.n_pages) atomicMax(&a.w.head->ring_bad, kRingNone - (unsigned)i);
    }
}

__device__ __forceinline__ void share_claim(const SharedTables& a, int warp, int warps) {
    share_ring(a, warp, warps);
    const unsigned long long epoch = a.w.head->epoch;
    const int lane = threadIdx.x & 31;
    const ShareItems items = share_items(a);
    ShareItem it;
    for (long long x = warp; x < items.n; x += warps) {
        int bad = share_item(a, items, x, it) ? kBadBounds : 0;
        bad |= it.q.bad;
        const unsigned writes = __ballot_sync(0xffffffffu, it.q.grows);
        if (it.any) {
            // neighbouring requests that hold the same page, as forks of one do: one claim for all of them
            int held = 0;
            bool write = false;
            unsigned long long name = 0;
#pragma unroll
            for (int k = 0; k < kShrRows; ++k) {
                if (it.p[k] < 0) continue;
                const bool w = writes >> k & 1;
                ++held;
                if (w || !write) name = claim_name(epoch, w, it.r0 + k);  // the later, those that write first
                write |= w;
                if (k + 1 < kShrRows && it.p[k + 1] == it.p[k]) continue;
                atomicSub(a.page_refs + it.p[k], held);
                atomicMax(a.w.claim + it.p[k], name);
                held = 0;
                write = false;
            }
        }
        if (bad) atomicOr(&a.w.head->flags, bad);
        if (it.word == 0 && lane < kShrRows && it.r0 + lane < a.n)
            a.w.req[it.r0 + lane] = make_int4(max(it.q.new_len - it.q.old_len, 0), max(it.q.has - it.q.had, 0), 0, it.q.grows ? kReqKeeps : 0);
    }
}

__device__ __forceinline__ void share_count(const SharedTables& a, int warp, int warps) {
    const unsigned long long epoch = a.w.head->epoch;
    const int lane = threadIdx.x & 31;
    const ShareItems items = share_items(a);
    ShareItem it;
    for (long long x = warp; x < items.n; x += warps) {
        share_item(a, items, x, it);
        if (!it.any) continue;
        const unsigned writes = __ballot_sync(0xffffffffu, it.q.grows);
        unsigned long long claim[kShrRows];
        int refs[kShrRows];
        bool bad = false;
#pragma unroll
        for (int k = 0; k < kShrRows; ++k) {
            claim[k] = 0, refs[k] = 1;
            if (it.p[k] < 0 || (k > 0 && it.p[k] == it.p[k - 1])) continue;
            claim[k] = __ldcg(a.w.claim + it.p[k]);
            refs[k] = __ldcg(a.page_refs + it.p[k]);
        }
#pragma unroll
        for (int k = 0; k < kShrRows; ++k) {
            if (k > 0 && it.p[k] >= 0 && it.p[k] == it.p[k - 1]) claim[k] = claim[k - 1], refs[k] = refs[k - 1];
            bad |= refs[k] < 0;  // more holders than the page's count
        }
        unsigned bits = 0;  // with lane k: the columns whose pages are request r0 + k's to decide on
#pragma unroll
        for (int k = 0; k < kShrRows; ++k) {
            const unsigned m = __ballot_sync(0xffffffffu, refs[k] == 0 && claim[k] == claim_name(epoch, writes >> k & 1, it.r0 + k));
            if (lane == k) bits = m;
        }
        if (bad) atomicOr(&a.w.head->flags, kBadBounds);
        if (max(it.q.lo, 32 * it.word) < min(it.q.hi, 32 * it.word + 32)) {
            const int r = it.r0 + lane;
            if (it.q.grows) {
                if (!bits) a.w.req[r].w = kReqCopies;
            } else {
                a.w.freed[(long long)r * items.words + it.word] = bits;
                if (bits) atomicAdd(&a.w.req[r].z, __popc(bits));
            }
        }
    }
}

__host__ __device__ constexpr size_t share_smem(int n) { return (size_t)(n + 1) * 17; }

// CLUSTER: the grid is one cluster
template <int NT, bool CLUSTER>
__device__ __forceinline__ void share_fill(const SharedTables& a) {
    extern __shared__ int shr_smem[];
    __shared__ TabSums sums;
    __shared__ int s_last;
    const int tid = threadIdx.x, lane = tid & 31, n = a.n, P = a.P;
    int* tok_cum = shr_smem;           // [n + 1] new tokens before each request
    int* pop_cum = tok_cum + n + 1;    // [n + 1] pages taken
    int* push_cum = pop_cum + n + 1;   // [n + 1] pages given back
    int* old_len = push_cum + n + 1;   // [n] tokens
    unsigned char* kinds = reinterpret_cast<unsigned char*>(old_len + n);  // [n] kReq*
    const long long head = a.free_state[0], tail = a.free_state[1], n_pages = a.n_pages;
    const unsigned long long epoch = a.w.head->epoch;
    const int flags = __ldcg(&a.w.head->flags);
    const int per = (n + NT - 1) / NT, r0 = min(tid * per, n), r1 = min(r0 + per, n);
    unsigned x[3] = {0, 0, 0}, tot[3];
    int turns = 0;
    auto copied = [&](int r) { return (int)(kinds[r] == kReqCopies); };
    constexpr int kPer = CLUSTER ? kShrFew / NT : kPagedMaxRequests / NT;
    int4 c[kPer];  // this thread's requests, all asked for at once
    int had[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int r = r0 + k;
        c[k] = make_int4(0, 0, 0, 0);
        if (r < r1) c[k] = __ldcg(a.w.req + r), had[k] = a.seq_len[r];
    }
    __shared__ int s_at[2];  // the ring's head and tail; the division is long, so one warp's
    if (tid < 2) {
        const long long at = tid == 0 ? head : tail;
        s_at[tid] = at >= 0 ? (int)(at % n_pages) : 0;
    }
    __shared__ unsigned s_ring_bad;
    if (tid == 32) s_ring_bad = __ldcg(&a.w.head->ring_bad);
    bool over = false;
    if (!flags) {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            x[0] += c[k].x;
            x[1] += c[k].y + (c[k].w == kReqCopies);
            x[2] += c[k].z;
            over |= (x[0] | x[1] | x[2]) >> 31;  // each term is below 2^31: seen before a sum can wrap
        }
    }
    bool wrapped;
    scan3<NT>(x, tot, wrapped, sums);
    over = __syncthreads_or(over);
    const int hm = s_at[0], tm = s_at[1];
    // every block comes to the same verdict
    int code = ICE_OK;
    if ((flags & kBadBounds) || head < 0 || tail < head || tail - head > n_pages) code = ICE_ERR_BOUNDS;
    else if ((flags & kBadCapacity) || over || wrapped || tot[1] > tail - head || tot[0] > (unsigned)a.n_slots) code = ICE_ERR_CAPACITY;
    else if (tail - head + tot[2] > n_pages || (s_ring_bad && kRingNone - s_ring_bad < tot[1])) code = ICE_ERR_BOUNDS;
    const bool ok = code == ICE_OK;
    const int n_tok = ok ? (int)tot[0] : 0, n_pop = ok ? (int)tot[1] : 0, n_push = ok ? (int)tot[2] : 0;
    if (ok) {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int r = r0 + k;
            if (r >= r1) break;
            tok_cum[r] = (int)x[0];
            pop_cum[r] = (int)x[1];
            push_cum[r] = (int)x[2];
            old_len[r] = had[k];
            kinds[r] = (unsigned char)c[k].w;
            x[0] += c[k].x;
            x[1] += c[k].y + (c[k].w == kReqCopies);
            x[2] += c[k].z;
        }
    }
    if (tid == 0) {
        tok_cum[n] = n_tok;
        pop_cum[n] = n_pop;
        push_cum[n] = n_push;
    }
    __syncthreads();
    auto ring = [&](int base, int j) {  // base, j < n_pages < 2^31: the sum may pass 2^31
        const long long p = (long long)base + j;
        return (int)(p < n_pages ? p : p - n_pages);
    };
    // The jobs below are independent. Each begins at another block, so that short ones run side by side.
    const int step = gridDim.x * NT;
    int first = blockIdx.x * NT + tid;
    auto turn = [&]() { first = (int)((blockIdx.x + (gridDim.x + 3) / 4 * ++turns) % gridDim.x) * NT + tid; };
    const bool wide = ((uintptr_t)a.slot_map & 15) == 0 && ((uintptr_t)a.positions & 15) == 0;
    for (long long i4 = (long long)first * kShrSlots; i4 < a.n_slots; i4 += (long long)step * kShrSlots) {
        const int i0 = (int)i4;
        long long slot[kShrSlots];
        int pos[kShrSlots];
        // the slot's request, its first slot and that of the one after; page, its id, offset in it; pages that the
        // request keeps
        int r = 0, b = 0, next = 0, pg = 0, id = 0, off = 0, held = 0;
        auto page_id = [&]() {
            id = pg < held ? a.block_table[(long long)r * a.max_blocks + pg] : a.free_pages[ring(hm, pop_cum[r] + pg - held)];
        };
        if (i0 < n_tok) r = find_row(tok_cum, n, i0);
#pragma unroll
        for (int k = 0; k < kShrSlots; ++k) {
            const int i = i0 + k;
            slot[k] = -1;
            pos[k] = 0;
            if (i < n_tok) {
                if (k == 0 || i >= next) {
                    while (tok_cum[r + 1] <= i) ++r;
                    b = tok_cum[r], next = tok_cum[r + 1];
                    const int o = old_len[r], p = o + i - b;
                    // a page that is copied is the first of those taken
                    held = (o + P - 1) / P - copied(r);
                    pg = p / P;
                    off = p - pg * P;
                    page_id();
                } else if (++off == P) {
                    off = 0;
                    ++pg;
                    page_id();
                }
                pos[k] = pg * P + off;
                slot[k] = (long long)id * P + off;
            }
        }
        if (wide && i0 + kShrSlots <= a.n_slots) {
            longlong2* d = reinterpret_cast<longlong2*>(a.slot_map + i0);
            d[0] = make_longlong2(slot[0], slot[1]);
            d[1] = make_longlong2(slot[2], slot[3]);
            if (a.positions) *reinterpret_cast<int4*>(a.positions + i0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        } else {
#pragma unroll
            for (int k = 0; k < kShrSlots; ++k)
                if (i0 + k < a.n_slots) {
                    a.slot_map[i0 + k] = slot[k];
                    if (a.positions) a.positions[i0 + k] = pos[k];
                }
        }
    }
    turn();
    for (long long jj = first; jj < n_pop; jj += step) {
        const int j = (int)jj, p = a.free_pages[ring(hm, j)];
        const int r = find_row(pop_cum, n, j), k = j - pop_cum[r], copies = copied(r);
        int* e = a.block_table + (long long)r * a.max_blocks + (old_len[r] + P - 1) / P - copies + k;
        if (copies && k == 0) {
            a.copy_src[r] = *e;
            a.copy_dst[r] = p;
        }
        *e = p;
        a.page_refs[p] = 1;
    }
    turn();
    for (int r = first; r <= n; r += step) a.q_start[r] = ok ? tok_cum[r] : 0;
    for (int r = first; r < n; r += step) {
        const int kind = ok ? kinds[r] : 0;
        if (kind != kReqCopies) a.copy_src[r] = a.copy_dst[r] = -1;
        if (kind == kReqKeeps) a.page_refs[a.block_table[(long long)r * a.max_blocks + (old_len[r] - 1) / P]] = 1;  // nobody else's
    }
    turn();
    const ShareItems items = share_items(a);
    if (!ok) {  // the claims taken back
        ShareItem it;
        for (long long y = first >> 5; y < items.n; y += step >> 5) {
            share_item(a, items, y, it);
            if (!it.any) continue;
#pragma unroll
            for (int k = 0; k < kShrRows; ++k)
                if (it.p[k] >= 0) atomicAdd(a.page_refs + it.p[k], 1);
        }
    } else if (a.max_blocks <= kShrLong) {  // pages given back, in order: a warp a request, or where rows are long a block
        constexpr int U = kShrLong / 32;
        for (int r = first >> 5; r < n; r += step >> 5) {
            if (push_cum[r + 1] == push_cum[r]) continue;
            const ShareReq q = share_req(a, r);
            int p[U];
            unsigned m[U];
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int c = 32 * k + lane;
                p[k] = c >= q.lo && c < q.hi ? a.block_table[(long long)r * a.max_blocks + c] : -1;
                m[k] = 32 * k < q.hi && 32 * k + 32 > q.lo ? __ldcg(a.w.freed + (long long)r * items.words + k) : 0;
            }
            int at = push_cum[r];
#pragma unroll
            for (int k = 0; k < U; ++k) {
                if (m[k] >> lane & 1) a.free_pages[ring(tm, at + __popc(m[k] & ((1u << lane) - 1)))] = p[k];
                at += __popc(m[k]);
            }
        }
    } else {
        constexpr int U = 4;  // columns of a thread, whose loads are under way together
        __shared__ int s_warp[U][NT / 32];
        const int warp = tid >> 5;
        for (int r = blockIdx.x; r < n; r += gridDim.x) {
            if (push_cum[r + 1] == push_cum[r]) continue;
            const ShareReq q = share_req(a, r);
            int at = push_cum[r];
            for (int c0 = q.lo / 32 * 32; c0 < q.hi; c0 += U * NT) {
                int p[U];
                unsigned m[U];
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    const int c = c0 + k * NT + tid;
                    p[k] = c >= q.lo && c < q.hi ? a.block_table[(long long)r * a.max_blocks + c] : -1;
                    m[k] = c - lane < q.hi ? __ldcg(a.w.freed + (long long)r * items.words + (c >> 5)) : 0;
                }
                __syncthreads();
#pragma unroll
                for (int k = 0; k < U; ++k)
                    if (lane == 0) s_warp[k][warp] = __popc(m[k]);
                __syncthreads();
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    const int c = lane < NT / 32 ? s_warp[k][lane] : 0;
                    const int before = __reduce_add_sync(0xffffffffu, lane < warp ? c : 0);
                    if (m[k] >> lane & 1) a.free_pages[ring(tm, at + before + __popc(m[k] & ((1u << lane) - 1)))] = p[k];
                    at += __reduce_add_sync(0xffffffffu, c);
                }
            }
        }
    }
    // last, when every block has read the lengths, the ring's state and the flags: what may replace them
    if (CLUSTER) {
        cg::this_cluster().sync();
        if (blockIdx.x != 0) return;
    } else {
        __syncthreads();
        if (tid == 0) {
            __threadfence();
            s_last = gridDim.x == 1 || atomicAdd(&a.w.head->ticket, 1u) == gridDim.x - 1;
        }
        __syncthreads();
        if (!s_last) return;
    }
    for (int r = tid; r < n; r += NT) a.seq_len_out[r] = ok ? a.seq_len[r] + a.n_new[r] : a.seq_len[r];
    if (tid == 0) {
        a.free_state_out[0] = head + n_pop;
        a.free_state_out[1] = tail + n_push;
        if (!ok) set_status(a.status, code);
        a.w.head->ticket = 0;
        a.w.head->flags = 0;
        a.w.head->ring_bad = 0;
        a.w.head->epoch = epoch + 1;
    }
}

__global__ void __launch_bounds__(kShrGridThreads) share_claim_kernel(SharedTables a) {
    pdl_wait_then_release();
    share_claim(a, (blockIdx.x * kShrGridThreads + threadIdx.x) >> 5, gridDim.x * kShrGridThreads >> 5);
}

__global__ void __launch_bounds__(kShrGridThreads) share_count_kernel(SharedTables a) {
    pdl_wait_then_release();
    share_count(a, (blockIdx.x * kShrGridThreads + threadIdx.x) >> 5, gridDim.x * kShrGridThreads >> 5);
}

__global__ void __launch_bounds__(kShrThreads) share_fill_kernel(SharedTables a) {
    pdl_wait_then_release();
    share_fill<kShrThreads, false>(a);
}

// The blocks of one cluster; its barrier orders their writes.
__global__ void __launch_bounds__(kShrThreads) share_step_kernel(SharedTables a) {
    pdl_wait_then_release();
    const cg::cluster_group cl = cg::this_cluster();
    const int warp = (threadIdx.x >> 5) * gridDim.x + blockIdx.x, warps = gridDim.x * kShrThreads >> 5;  // few items: on all SMs
    share_claim(a, warp, warps);
    cl.sync();
    share_count(a, warp, warps);
    cl.sync();
    share_fill<kShrThreads, true>(a);
}

cudaError_t launch_shared_tables(SharedTables a, cudaStream_t s) {
    const size_t smem = share_smem(a.n);
    // a request of g new tokens takes at most ceil(g / P) pages, and one that it copies to
    a.most_taken = a.n_slots / a.P + 2 * a.n;
    // One cluster of 8 SMs, or three launches on all. The first has 5 us less on the host, and up to 2 less on the GPU where the tables are
    // small. Towards the bound of 2^16 entries the GPU loses 1 to 5 us (17 where 1024 requests that share no page end in one call),
    // which only an eager caller has back from the host; beyond it more than that. A step / the end of all requests, one cluster
    // (three launches): 16 with 128 columns 11.1 / 10.5 us (12.4 / 12.4), 16 with 2310 11.5 / 14.0 (12.5 / 12.6), 1024 with 64 14.4 / 19.7
    // (12.8 / 15.1), with no page shared 15.8 / 32 (15.3 / 15.5), 64 with 2048 17.4 / 31.3 (13.1 / 13.7), 256 with 2048 42.2 / 102
    // (13.9 / 19.3).
    if (a.n <= kShrFew && a.n_slots <= 65536 && (long long)a.n * a.max_blocks <= 1 << 16)
        return launch_cluster(share_step_kernel, kShrCluster, kShrThreads, smem, s, a);
    const int per = kShrGridThreads / 32;
    const long long items = (long long)((a.n + kShrRows - 1) / kShrRows) * ((a.max_blocks + 31) / 32);
    const dim3 grid((unsigned)std::min<long long>(152 * 8, (items + per - 1) / per));
    // with blocks of their own for the ring's ids
    const dim3 claim(grid.x + std::min(152, (a.most_taken + kShrGridThreads - 1) / kShrGridThreads));
    cudaError_t e = launch_pdl(share_claim_kernel, claim, dim3(kShrGridThreads), 0, s, a);
    if (e == cudaSuccess) e = launch_pdl(share_count_kernel, grid, dim3(kShrGridThreads), 0, s, a);
    const int blocks = std::max(1, std::min(152, std::max(a.n_slots / 1024, a.max_blocks > kShrLong ? a.n : a.n / 32)));
    if (e == cudaSuccess) e = launch_pdl(share_fill_kernel, dim3(blocks), dim3(kShrThreads), smem, s, a);
    return e;
}

// ---------------------------------------------------------------------------
// Compaction: with L pages in use, the pages in use at L and behind go to the free ones before L, in order: the k-th of
// the former to the k-th of the latter. Ranks are sums of flags, so three passes do it: flags counted by
// chunk (and every list checked), ranks and lists of moves, then the tables. A page that moves leaves its
// number k in its claim, where the tables' pass finds it. Bound by latency: 1000 pages 8.5 us, 32768 pages 14 us.
// ---------------------------------------------------------------------------
constexpr int kCmpThreads = 256, kCmpStepThreads = 1024;
constexpr int kCmpPer = 4;  // pages of a thread; a block's chunk is one pass over them
static_assert(kCmpChunk == kCmpThreads * kCmpPer, "the smaller chunk decides how many counts there are");

template <int NT>
__device__ __forceinline__ int block_sum(int x, int* s_sum) {
    x = __reduce_add_sync(0xffffffffu, x);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = x;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    return __reduce_add_sync(0xffffffffu, lane < NT / 32 ? s_sum[lane] : 0);
}

template <int NT>
__device__ __forceinline__ void compact_count(const Compact& a) {
    constexpr int kChunk = NT * kCmpPer;
    __shared__ int s_sum[NT / 32];
    const int tid = threadIdx.x, lane = tid & 31;
    const int chunks = (int)((a.n_pages + kChunk - 1) / kChunk);
    bool bad = false;
    for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
        int live = 0;
#pragma unroll
        for (int k = 0; k < kCmpPer; ++k) {
            const long long p = (long long)c * kChunk + k * NT + tid;
            const int f = p < a.n_pages ? a.page_refs[p] : 0;
            live += f > 0;
            bad |= f < 0;
        }
        live = block_sum<NT>(live, s_sum);
        if (tid == 0) a.w.count[c] = live;
    }
    // every page that is named is one in use
    auto named = [&](int p) { return p >= 0 && p < a.n_pages && a.page_refs[p] > 0; };
    const long long cap = (long long)a.max_blocks * a.P;
    const int warps = gridDim.x * (NT / 32), warp = blockIdx.x * (NT / 32) + (tid >> 5);
    for (int r = warp; r < a.n; r += warps) {
        const int len = a.seq_len[r];
        if (len < 0 || len > cap) {
            bad = true;
            continue;
        }
        const int pages = (len + a.P - 1) / a.P;
#pragma unroll 4
        for (int c = lane; c < pages; c += 32) bad |= !named(a.block_table[(long long)r * a.max_blocks + c]);
    }
    for (long long i = blockIdx.x * NT + tid; i < a.n_extra; i += gridDim.x * NT) bad |= !named(a.extra[i]);
    if (bad) atomicOr(&a.w.head->flags, kBadBounds);
}

template <int NT>
__device__ __forceinline__ void compact_move(const Compact& a) {
    constexpr int kChunk = NT * kCmpPer;
    __shared__ int s_sum[NT / 32], s_warp[NT / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int chunks = (int)((a.n_pages + kChunk - 1) / kChunk);
    // this block's chunks, the pages in use before them and in all
    const int c0 = (int)((long long)chunks * blockIdx.x / gridDim.x), c1 = (int)((long long)chunks * (blockIdx.x + 1) / gridDim.x);
    int before = 0, all = 0;
    for (int c = tid; c < chunks; c += NT) {
        const int x = __ldcg(a.w.count + c);
        all += x;
        if (c < c0) before += x;
    }
    before = block_sum<NT>(before, s_sum);
    const int L = block_sum<NT>(all, s_sum);
    // those in use before page L
    int low = 0;
    for (int c = tid; c < L / kChunk; c += NT) low += __ldcg(a.w.count + c);
    for (long long p = L / kChunk * kChunk + tid; p < L; p += NT) low += a.page_refs[p] > 0;
    low = block_sum<NT>(low, s_sum);
    const int moves = L - low;
    const int code = __ldcg(&a.w.head->flags) ? ICE_ERR_BOUNDS : moves > a.n_moves ? ICE_ERR_CAPACITY : ICE_OK;
    const bool ok = code == ICE_OK;
    for (int c = c0; ok && c < c1; ++c) {
        // neighbouring pages a thread: ranks in order
        const long long p0 = (long long)c * kChunk + tid * kCmpPer;
        int f[kCmpPer], mine = 0;
#pragma unroll
        for (int k = 0; k < kCmpPer; ++k) {
            f[k] = p0 + k < a.n_pages && a.page_refs[p0 + k] > 0;
            mine += f[k];
        }
        int inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        __syncthreads();
        if (lane == 31) s_warp[warp] = inc;
        __syncthreads();
        const int of_warp = lane < NT / 32 ? s_warp[lane] : 0;
        int rank = before + inc - mine + __reduce_add_sync(0xffffffffu, lane < warp ? of_warp : 0);
        before += __reduce_add_sync(0xffffffffu, of_warp);
#pragma unroll
        for (int k = 0; k < kCmpPer; ++k) {
            const long long p = p0 + k;
            if (p >= a.n_pages) break;
            if (p >= L) {
                a.free_pages[p - L] = (int)p;
                if (f[k]) {
                    a.move_src[rank - low] = (int)p;
                    a.w.claim[p] = (unsigned long long)(rank - low);
                }
            } else if (!f[k]) {
                a.move_dst[p - rank] = (int)p;
            }
            rank += f[k];
        }
    }
    for (long long k = (ok ? moves : 0) + blockIdx.x * NT + tid; k < a.n_moves; k += gridDim.x * NT)
        a.move_src[k] = a.move_dst[k] = -1;
    if (blockIdx.x == 0 && tid == 0) {
        a.w.head->plan[0] = ok;
        a.w.head->plan[1] = L;
        a.w.head->plan[2] = moves;
        if (ok) {
            a.free_state_out[0] = 0;
            a.free_state_out[1] = a.n_pages - L;
        } else {
            set_status(a.status, code);
        }
    }
}

template <int NT>
__device__ __forceinline__ void compact_apply(const Compact& a) {
    const int tid = threadIdx.x, lane = tid & 31;
    const bool ok = __ldcg(&a.w.head->plan[0]);
    const int L = __ldcg(&a.w.head->plan[1]), moves = __ldcg(&a.w.head->plan[2]);
    const int first = blockIdx.x * NT + tid, step = gridDim.x * NT;
    if (first == 0) a.w.head->flags = 0;
    auto goes = [&](int p) { return ok && p >= L ? __ldcg(a.move_dst + (int)__ldcg(a.w.claim + p)) : p; };
    const long long cap = (long long)a.max_blocks * a.P;
    for (int r = first >> 5; r < a.n; r += step >> 5) {
        const int len = a.seq_len[r];
        // a length that is out of range, with which nothing moves: the whole row
        const int pages = len < 0 || len > cap ? a.max_blocks : (len + a.P - 1) / a.P;
        const long long row = (long long)r * a.max_blocks;
#pragma unroll 4
        for (int c = lane; c < pages; c += 32) a.block_table_out[row + c] = goes(a.block_table[row + c]);
    }
    for (long long i = first; i < a.n_extra; i += step) a.extra_out[i] = goes(a.extra[i]);
    // counts: a page that moves takes its own along
    if (ok) {
        for (long long k = first; k < moves; k += step) {
            const int s = __ldcg(a.move_src + k), f = a.page_refs[s];
            a.page_refs_out[__ldcg(a.move_dst + k)] = f;
            a.page_refs_out[s] = 0;
        }
    }
    if (a.page_refs_out != a.page_refs) {
        for (long long p = first; p < a.n_pages; p += step) {
            const int f = a.page_refs[p];
            if (!ok) a.page_refs_out[p] = f;
            else if (p >= L) a.page_refs_out[p] = 0;
            else if (f > 0) a.page_refs_out[p] = f;
        }
    }
}

__global__ void __launch_bounds__(kCmpThreads) compact_count_kernel(Compact a) {
    pdl_wait_then_release();
    compact_count<kCmpThreads>(a);
}

__global__ void __launch_bounds__(kCmpThreads) compact_move_kernel(Compact a) {
    pdl_wait_then_release();
    compact_move<kCmpThreads>(a);
}

__global__ void __launch_bounds__(kCmpThreads) compact_apply_kernel(Compact a) {
    pdl_wait_then_release();
    compact_apply<kCmpThreads>(a);
}

// The blocks of one cluster; its barrier orders their writes.
__global__ void __launch_bounds__(kCmpStepThreads) compact_step_kernel(Compact a) {
    pdl_wait_then_release();
    const cg::cluster_group cl = cg::this_cluster();
    compact_count<kCmpStepThreads>(a);
    cl.sync();
    compact_move<kCmpStepThreads>(a);
    cl.sync();
    compact_apply<kCmpStepThreads>(a);
}

cudaError_t launch_compact(const Compact& a, cudaStream_t s) {
    const int chunks = (int)((a.n_pages + kCmpChunk - 1) / kCmpChunk);
    // one cluster for small pools (1000 pages 8.3 us, as three launches 8.6 and 5 us more on the host); 32768 pages: 17.2 us, 14.3 as
    // three launches
    if (a.n_pages <= 16384 && (long long)a.n * a.max_blocks <= 1 << 19 && a.n_extra <= 65536)
        return launch_cluster(compact_step_kernel, kShrCluster, kCmpStepThreads, 0, s, a);
    const dim3 block(kCmpThreads);
    const dim3 wide(std::max(1, std::min(152 * 4, std::max(chunks * kCmpPer, std::max(a.n, a.n_extra / 32) / 8))));
    cudaError_t e = launch_pdl(compact_count_kernel, wide, block, 0, s, a);
    if (e == cudaSuccess) e = launch_pdl(compact_move_kernel, dim3(std::min(152 * 4, chunks)), block, 0, s, a);
    if (e == cudaSuccess) e = launch_pdl(compact_apply_kernel, wide, block, 0, s, a);
    return e;
}

// ---------------------------------------------------------------------------
// Pages copied by a list of pairs, in every layer, K and V. A warp takes pieces of 2 KB, four 16-byte loads a lane
// under way together. A block looks up the entries of its share of the list at once and goes on with those that are
// pairs: most entries of a step's list are -1. Where the list is short, blocks in y share an entry. Sources stay in the caches:
// forked requests copy one page several times. Bound by memory: 8229 pages of 32 KB, K and V, 158 us, 6.8 TB/s of read and
// write (the measured copy rate).
// ---------------------------------------------------------------------------
constexpr int kCpyThreads = 256, kCpyBatch = 4;

__global__ void __launch_bounds__(kCpyThreads) page_copy_kernel(int n, const int* src, const int* dst, int n_layers, long long layer_vecs,
                                                                int page_vecs, long long n_pages, uint4* k_pages, uint4* v_pages,
                                                                int* status) {
    __shared__ int2 s_pair[kCpyThreads];
    __shared__ int s_n;
    const int tid = threadIdx.x, lane = tid & 31;
    const int w = blockIdx.y * (kCpyThreads / 32) + (tid >> 5), warps = gridDim.y * (kCpyThreads / 32);
    const int pieces = (page_vecs + 32 * kCpyBatch - 1) / (32 * kCpyBatch), units = n_layers * 2 * pieces;
    pdl_wait_then_release();
    for (long long e0 = blockIdx.x; e0 < n; e0 += (long long)gridDim.x * kCpyThreads) {
        __syncthreads();
        if (tid == 0) s_n = 0;
        __syncthreads();
        const long long e = e0 + (long long)tid * gridDim.x;
        if (e < n) {
            const int s = src[e], d = dst[e];
            if (s >= 0 && s < n_pages && d >= 0 && d < n_pages) s_pair[atomicAdd(&s_n, 1)] = make_int2(s, d);
            else if (!(s == -1 || d == -1)) set_status(status, ICE_ERR_BOUNDS);
        }
        __syncthreads();
        const int m = s_n;
        // pieces of all pairs in turn
        for (long long x = w; x < (long long)m * units; x += warps) {
            const int i = (int)(x / units), u = (int)(x - (long long)i * units);
            const int y = u / pieces, at = (u - y * pieces) * 32 * kCpyBatch + lane;
            uint4* pool = (y & 1 ? v_pages : k_pages) + (long long)(y >> 1) * layer_vecs;
            const int2 p = s_pair[i];
            const uint4* from = pool + (long long)p.x * page_vecs;
            uint4* to = pool + (long long)p.y * page_vecs;
            uint4 v[kCpyBatch];
#pragma unroll
            for (int k = 0; k < kCpyBatch; ++k)
                if (at + 32 * k < page_vecs) v[k] = from[at + 32 * k];
#pragma unroll
            for (int k = 0; k < kCpyBatch; ++k)
                if (at + 32 * k < page_vecs) to[at + 32 * k] = v[k];
        }
    }
}

cudaError_t launch_page_copy(int n, const int* src, const int* dst, int n_layers, long long layer_bytes, long long page_bytes,
                             long long n_pages, void* k_pages, void* v_pages, int* status, cudaStream_t s) {
    const int page_vecs = (int)(page_bytes / 16);
    const long long pieces = (page_vecs + 32 * kCpyBatch - 1) / (32 * kCpyBatch), units = n_layers * 2 * pieces;
    const int most = 152 * 64;  // blocks of few pieces: the last ones end together (152 * 8: 32768 pages' moves 172 us, with these 158)
    const int x = std::min(n, most);
    const int y = (int)std::max<long long>(1, std::min<long long>(most / x, (units + 7) / 8));
    return launch_pdl(page_copy_kernel, dim3(x, y), dim3(kCpyThreads), 0, s, n, src, dst, n_layers, layer_bytes / 16, page_vecs,
                      n_pages, (uint4*)k_pages, (uint4*)v_pages, status);
}

cudaError_t share_prepare() {
    cudaError_t e = cudaFuncSetAttribute(share_fill_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)share_smem(kPagedMaxRequests));
    return e;
}

}  // namespace ice
