// Block tables and slot maps of one step from the requests' lengths, and the rows of
// new tokens written by the slot map.
#include <algorithm>

#include "ice_paged_scan.cuh"

namespace ice {

// ---------------------------------------------------------------------------
// Request r goes from old to new = old + n_new tokens, ceil(old / P) to
// ceil(new / P) pages. With exclusive sums over the requests of new tokens, pages
// taken and pages given back, every output entry is a function of the inputs
// alone: token i of the step lies in the request whose sum interval holds i, the
// j-th page taken is ring entry head + j. So each block makes the sums itself
// (all lengths, 8 B a request from L2) and then fills its share of the entries;
// no block waits for another. What a call may replace in place (lengths, ring
// state) is written by the last block to have read it, found by a ticket.
// Bound by latency: the launch, the scan and the look-ups in a row, 5.5 us for 16 requests,
// 7.8 us for 256. 4096 requests with 1.03 million new tokens: 13.8 us, 12.8 MB written; four
// slots a thread take one search, one divide and a wide store (one slot a thread: 21 us, a divide
// a slot 14.9, eight slots a thread 14.4 and 1.7 us more for the small calls).
// ---------------------------------------------------------------------------
constexpr int kTabThreads = 1024, kTabFewThreads = 256;  // the latter where the requests are few
constexpr int kTabSlots = 4;  // consecutive slots of a thread: one search for them, wide stores

template <int NT>
__global__ void __launch_bounds__(NT) tables_kernel(
    int n, int max_blocks, int P, long long n_pages, const int* seq_len, const int* n_new,
    int* block_table, int* free_pages, const long long* free_state, int* seq_len_out,
    long long* free_state_out, int* q_start, long long* slot_map, int* positions, int n_slots,
    unsigned* ticket, int* status) {
    extern __shared__ int tab_smem[];
    __shared__ TabSums sums;
    __shared__ int s_last, s_bad;
    int* tok_cum = tab_smem;             // [n + 1] new tokens before each request
    int* pop_cum = tok_cum + n + 1;      // [n + 1] pages taken
    int* push_cum = pop_cum + n + 1;     // [n + 1] pages given back
    const int tid = threadIdx.x;
    if (tid == 0) s_bad = 0;
    pdl_wait_then_release();
    __syncthreads();
    const long long head = free_state[0], tail = free_state[1];
    const int per = (n + NT - 1) / NT;
    const int r0 = min(tid * per, n), r1 = min(r0 + per, n);
    const long long cap = (long long)max_blocks * P;
    unsigned x[3] = {0, 0, 0}, tot[3];
    int bad = 0;  // 1: an impossible length, 2: the table's columns do not suffice
    for (int r = r0; r < r1; ++r) {
        const long long o = seq_len[r], w = o + n_new[r];
        if (o < 0 || o > cap || w < 0) {
            bad |= 1;
        } else if (w > cap) {
            bad |= 2;
        } else {
            const int had = ((int)o + P - 1) / P, has = ((int)w + P - 1) / P;
            x[0] += max((int)(w - o), 0);
            x[1] += max(has - had, 0);
            x[2] += max(had - has, 0);
            if ((x[0] | x[1] | x[2]) >> 31) bad |= 2;  // each term is below 2^31: seen before a sum can wrap
        }
    }
    if (bad) atomicOr(&s_bad, bad);
    bool wrapped;
    scan3<NT>(x, tot, wrapped, sums);  // its barrier also orders s_bad
    // every block comes to the same verdict
    int code = ICE_OK;
    if ((s_bad & 1) || head < 0 || tail < head || tail - head > n_pages) code = ICE_ERR_BOUNDS;
    else if ((s_bad & 2) || wrapped || tot[1] > tail - head || tot[0] > (unsigned)n_slots) code = ICE_ERR_CAPACITY;
    else if (tail - head + tot[2] > n_pages) code = ICE_ERR_BOUNDS;
    const bool ok = code == ICE_OK;
    const int n_tok = ok ? (int)tot[0] : 0, n_pop = ok ? (int)tot[1] : 0, n_push = ok ? (int)tot[2] : 0;
    if (ok) {
        for (int r = r0; r < r1; ++r) {
            tok_cum[r] = (int)x[0];
            pop_cum[r] = (int)x[1];
            push_cum[r] = (int)x[2];
            const int o = seq_len[r], w = o + n_new[r], had = (o + P - 1) / P, has = (w + P - 1) / P;
            x[0] += max(w - o, 0);
            x[1] += max(has - had, 0);
            x[2] += max(had - has, 0);
        }
    }
    if (tid == 0) {
        tok_cum[n] = n_tok;
        pop_cum[n] = n_pop;
        push_cum[n] = n_push;
    }
    __syncthreads();
    const int hm = n_pages > 0 && ok ? (int)(head % n_pages) : 0, tm = n_pages > 0 && ok ? (int)(tail % n_pages) : 0;
    auto ring = [&](int base, int j) {  // base, j < n_pages < 2^31: the sum may pass 2^31
        const long long p = (long long)base + j;
        return (int)(p < n_pages ? p : p - n_pages);
    };
    const int first = blockIdx.x * NT + tid, step = gridDim.x * NT;
    for (int r = first; r <= n; r += step) q_start[r] = ok ? tok_cum[r] : 0;
    const bool wide = ((uintptr_t)slot_map & 15) == 0 && ((uintptr_t)positions & 15) == 0;
    for (long long i4 = (long long)first * kTabSlots; i4 < n_slots; i4 += (long long)step * kTabSlots) {
        const int i0 = (int)i4;
        long long slot[kTabSlots];
        int pos[kTabSlots];
        // the slot's request, its first slot and that of the one after; page, its id, offset in it; pages
        // that the request had
        int r = 0, b = 0, next = 0, pg = 0, id = 0, off = 0, had = 0;
        auto page_id = [&]() {
            id = pg < had ? block_table[(long long)r * max_blocks + pg] : free_pages[ring(hm, pop_cum[r] + pg - had)];
        };
        if (i0 < n_tok) r = find_row(tok_cum, n, i0);
#pragma unroll
        for (int k = 0; k < kTabSlots; ++k) {
            const int i = i0 + k;
            slot[k] = -1;
            pos[k] = 0;
            if (i < n_tok) {
                if (k == 0 || i >= next) {
                    while (tok_cum[r + 1] <= i) ++r;
                    b = tok_cum[r], next = tok_cum[r + 1];
                    const int o = seq_len[r], p = o + i - b;
                    had = (o + P - 1) / P;
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
        if (wide && i0 + kTabSlots <= n_slots) {
            longlong2* d = reinterpret_cast<longlong2*>(slot_map + i0);
            d[0] = make_longlong2(slot[0], slot[1]);
            d[1] = make_longlong2(slot[2], slot[3]);
            if (positions) *reinterpret_cast<int4*>(positions + i0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        } else {
#pragma unroll
            for (int k = 0; k < kTabSlots; ++k)
                if (i0 + k < n_slots) {
                    slot_map[i0 + k] = slot[k];
                    if (positions) positions[i0 + k] = pos[k];
                }
        }
    }
    for (int j = first; j < n_pop; j += step) {
        const int r = find_row(pop_cum, n, j);
        const int had = (seq_len[r] + P - 1) / P;
        block_table[(long long)r * max_blocks + had + j - pop_cum[r]] = free_pages[ring(hm, j)];
    }
    for (int j = first; j < n_push; j += step) {
        const int r = find_row(push_cum, n, j);
        const int has = (seq_len[r] + n_new[r] + P - 1) / P;
        free_pages[ring(tm, j)] = block_table[(long long)r * max_blocks + has + j - push_cum[r]];
    }
    // the last block to come here: every block has read the lengths and the ring's state
    __syncthreads();
    if (tid == 0) {
        __threadfence();
        s_last = gridDim.x == 1 || atomicAdd(ticket, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!s_last) return;
    for (int r = tid; r < n; r += NT) seq_len_out[r] = ok ? seq_len[r] + n_new[r] : seq_len[r];
    if (tid == 0) {
        free_state_out[0] = head + n_pop;
        free_state_out[1] = tail + n_push;
        if (!ok) set_status(status, code);
        *ticket = 0;
    }
}

cudaError_t launch_paged_tables(int n_req, int max_blocks, int P, long long n_pages, const int* seq_len,
                                const int* n_new, int* block_table, int* free_pages,
                                const long long* free_state, int* seq_len_out, long long* free_state_out,
                                int* q_start, long long* slot_map, int* positions, int n_slots,
                                unsigned* ticket, int* status, cudaStream_t s) {
    const int blocks = std::max(1, std::min(152, std::max(n_slots / 1024, n_req / 32)));
    // a scan of 8 warps instead of 32 while a thread has one request and one group of slots at most:
    // 16 requests 6.4 -> 5.5 us, 256 requests 8.2 -> 7.6 us
    const bool few = n_req <= kTabFewThreads && n_slots <= 152 * kTabFewThreads * kTabSlots;
    return launch_pdl(few ? tables_kernel<kTabFewThreads> : tables_kernel<kTabThreads>, dim3(blocks),
                      dim3(few ? kTabFewThreads : kTabThreads), (size_t)(n_req + 1) * 12, s, n_req, max_blocks,
                      P, n_pages, seq_len, n_new, block_table, free_pages, free_state,
                      seq_len_out, free_state_out, q_start, slot_map, positions, n_slots, ticket, status);
}

// ---------------------------------------------------------------------------
// Rows of new tokens into their slots: a copy whose destination is looked up.
// A row (one token, KV head, K or V) is 16 or 32 pieces of 16 bytes; consecutive
// threads take consecutive pieces, four of each thread under way together. Bound by memory:
// 32768 tokens of 8 heads in bf16 46.0 us, 5.8 TB/s of read and write (86 % of the measured
// copy rate); one token for each of 64 requests 2.7 us, the launch.
// ---------------------------------------------------------------------------
constexpr int kAppThreads = 256;
constexpr int kAppBatch = 4;  // pieces of a thread that are under way together

__global__ void __launch_bounds__(kAppThreads) append_kernel(
    int n_tokens, int H, int P, int shift, long long n_slots, const uint4* k, long long k_stride,
    const uint4* v, long long v_stride, const long long* slot_map, uint4* k_pages, uint4* v_pages,
    int* status) {
    pdl_wait_then_release();
    const unsigned per_kv = H << shift, per_tok = 2 * per_kv;  // pieces of a token's K, of a token
    const long long total = (long long)n_tokens * per_tok;
    for (long long i0 = (long long)blockIdx.x * kAppThreads * kAppBatch + threadIdx.x; i0 < total;
         i0 += (long long)gridDim.x * kAppThreads * kAppBatch) {
        uint4 x[kAppBatch];
        uint4* dst[kAppBatch];
#pragma unroll
        for (int u = 0; u < kAppBatch; ++u) {
            const long long i = i0 + (long long)u * kAppThreads;
            dst[u] = nullptr;
            if (i >= total) continue;
            const long long t = total <= 0xFFFFFFFFll ? (long long)((unsigned)i / per_tok) : i / per_tok;
            unsigned c = (unsigned)(i - t * per_tok);
            const long long slot = slot_map[t];
            if (slot < 0 || slot >= n_slots) {
                if (slot != -1) set_status(status, ICE_ERR_BOUNDS);
                continue;
            }
            const bool is_v = c >= per_kv;
            if (is_v) c -= per_kv;
            const unsigned page = (unsigned)slot / (unsigned)P;  // n_slots < 2^31
            const int off = (int)((unsigned)slot - page * P), h = c >> shift, piece = c & ((1 << shift) - 1);
            x[u] = __ldcs(is_v ? v + t * v_stride + c : k + t * k_stride + c);
            dst[u] = (is_v ? v_pages : k_pages) + (((((long long)page * H + h) * P + off) << shift) + piece);
        }
#pragma unroll
        for (int u = 0; u < kAppBatch; ++u)
            if (dst[u] != nullptr) *dst[u] = x[u];
    }
}

cudaError_t launch_paged_append(int n_tokens, int H, int P, int es, long long n_pages, const void* k,
                                long long k_stride, const void* v, long long v_stride,
                                const long long* slot_map, void* k_pages, void* v_pages, int* status,
                                cudaStream_t s) {
    const int shift = es == 2 ? 4 : 5;  // 16-byte pieces of a row of 128 elements
    const long long total = (long long)n_tokens * 2 * ((long long)H << shift);
    const int per_block = kAppThreads * kAppBatch;
    const int blocks = (int)std::min<long long>((total + per_block - 1) / per_block, 152 * 8);
    return launch_pdl(append_kernel, dim3(blocks), dim3(kAppThreads), 0, s, n_tokens, H, P, shift,
                      n_pages * P, (const uint4*)k, k_stride * es / 16, (const uint4*)v, v_stride * es / 16,
                      slot_map, (uint4*)k_pages, (uint4*)v_pages, status);
}

cudaError_t paged_tables_prepare() {
    return cudaFuncSetAttribute(tables_kernel<kTabThreads>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (kPagedMaxRequests + 1) * 12);
}

}  // namespace ice
