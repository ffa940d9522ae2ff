// Block tables and slot maps of one step from the requests' lengths, and the rows of
// new tokens written by the slot map.
#include <algorithm>

#include "ice_paged.cuh"

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
// ---------------------------------------------------------------------------
constexpr int kTabThreads = 1024;

struct TabSums {
    long long v[3][32];
};

// Inclusive block scan of three values per thread; total in tot.
__device__ __forceinline__ void scan3(long long (&x)[3], long long (&tot)[3], TabSums& sh) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const long long y = __shfl_up_sync(0xffffffffu, x[k], o);
            if (lane >= o) x[k] += y;
        }
    if (lane == 31)
#pragma unroll
        for (int k = 0; k < 3; ++k) sh.v[k][warp] = x[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        long long y = sh.v[k][lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long z = __shfl_up_sync(0xffffffffu, y, o);
            if (lane >= o) y += z;
        }
        tot[k] = __shfl_sync(0xffffffffu, y, 31);
        const long long before = __shfl_sync(0xffffffffu, y, max(warp - 1, 0));
        if (warp > 0) x[k] += before;
    }
}

// The last r in [0, n) with cum[r] <= i (cum[0] = 0).
__device__ __forceinline__ int find_row(const int* cum, int n, int i) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cum[mid] <= i) lo = mid;
        else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kTabThreads) tables_kernel(
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
    const int per = (n + kTabThreads - 1) / kTabThreads;
    const int r0 = min(tid * per, n), r1 = min(r0 + per, n);
    const long long cap = (long long)max_blocks * P;
    long long x[3] = {0, 0, 0}, tot[3];
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
        }
    }
    if (bad) atomicOr(&s_bad, bad);
    long long e[3] = {x[0], x[1], x[2]};
    scan3(x, tot, sums);  // its barrier also orders s_bad
    // every block comes to the same verdict
    int code = ICE_OK;
    if ((s_bad & 1) || head < 0 || tail < head || tail - head > n_pages || tail - head + tot[2] > n_pages)
        code = ICE_ERR_BOUNDS;
    else if ((s_bad & 2) || tot[1] > tail - head || tot[0] > n_slots)
        code = ICE_ERR_CAPACITY;
    const bool ok = code == ICE_OK;
    const int n_tok = ok ? (int)tot[0] : 0, n_pop = ok ? (int)tot[1] : 0, n_push = ok ? (int)tot[2] : 0;
    if (ok) {
#pragma unroll
        for (int k = 0; k < 3; ++k) e[k] = x[k] - e[k];
        for (int r = r0; r < r1; ++r) {
            tok_cum[r] = (int)e[0];
            pop_cum[r] = (int)e[1];
            push_cum[r] = (int)e[2];
            const int o = seq_len[r], w = o + n_new[r], had = (o + P - 1) / P, has = (w + P - 1) / P;
            e[0] += max(w - o, 0);
            e[1] += max(has - had, 0);
            e[2] += max(had - has, 0);
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
    const int first = blockIdx.x * kTabThreads + tid, step = gridDim.x * kTabThreads;
    for (int r = first; r <= n; r += step) q_start[r] = ok ? tok_cum[r] : 0;
    for (int i = first; i < n_slots; i += step) {
        long long slot = -1;
        int pos = 0;
        if (i < n_tok) {
            const int r = find_row(tok_cum, n, i);
            const int o = seq_len[r];
            pos = o + i - tok_cum[r];
            const int had = (o + P - 1) / P, pg = pos / P;
            const int id = pg < had ? block_table[(long long)r * max_blocks + pg]
                                    : free_pages[ring(hm, pop_cum[r] + pg - had)];
            slot = (long long)id * P + (pos - pg * P);
        }
        slot_map[i] = slot;
        if (positions) positions[i] = pos;
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
        s_last = atomicAdd(ticket, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!s_last) return;
    for (int r = tid; r < n; r += kTabThreads) seq_len_out[r] = ok ? seq_len[r] + n_new[r] : seq_len[r];
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
    const int blocks = std::max(1, std::min(152, std::max(n_slots / 4096, n_req / 512)));
    return launch_pdl(tables_kernel, dim3(blocks), dim3(kTabThreads), (size_t)(n_req + 1) * 12, s, n_req,
                      max_blocks, P, n_pages, seq_len, n_new, block_table, free_pages, free_state,
                      seq_len_out, free_state_out, q_start, slot_map, positions, n_slots, ticket, status);
}

// ---------------------------------------------------------------------------
// Rows of new tokens into their slots: a copy whose destination is looked up.
// A row (one token, KV head, K or V) is 16 or 32 pieces of 16 bytes; consecutive
// threads take consecutive pieces.
// ---------------------------------------------------------------------------
constexpr int kAppThreads = 256;

__global__ void __launch_bounds__(kAppThreads) append_kernel(
    int n_tokens, int H, int P, int shift, long long n_slots, const uint4* k, long long k_stride,
    const uint4* v, long long v_stride, const long long* slot_map, uint4* k_pages, uint4* v_pages,
    int* status) {
    pdl_wait_then_release();
    const int per_kv = H << shift;  // pieces of a token's K
    const long long total = (long long)n_tokens * 2 * per_kv;
    const long long step = (long long)gridDim.x * kAppThreads;
    for (long long i = (long long)blockIdx.x * kAppThreads + threadIdx.x; i < total; i += step) {
        const long long t = i / (2 * per_kv);
        int c = (int)(i - t * (2 * per_kv));
        const long long slot = slot_map[t];
        if (slot < 0 || slot >= n_slots) {
            if (slot != -1) set_status(status, ICE_ERR_BOUNDS);
            continue;
        }
        const bool is_v = c >= per_kv;
        if (is_v) c -= per_kv;
        const long long page = slot / P;
        const int off = (int)(slot - page * P), h = c >> shift, piece = c & ((1 << shift) - 1);
        const uint4 x = is_v ? v[t * v_stride + c] : k[t * k_stride + c];
        uint4* dst = is_v ? v_pages : k_pages;
        dst[(((page * H + h) * P + off) << shift) + piece] = x;
    }
}

cudaError_t launch_paged_append(int n_tokens, int H, int P, int es, long long n_pages, const void* k,
                                long long k_stride, const void* v, long long v_stride,
                                const long long* slot_map, void* k_pages, void* v_pages, int* status,
                                cudaStream_t s) {
    const int shift = es == 2 ? 4 : 5;  // 16-byte pieces of a row of 128 elements
    const long long total = (long long)n_tokens * 2 * ((long long)H << shift);
    const int blocks = (int)std::min<long long>((total + kAppThreads - 1) / kAppThreads, 152 * 8);
    return launch_pdl(append_kernel, dim3(blocks), dim3(kAppThreads), 0, s, n_tokens, H, P, shift,
                      n_pages * P, (const uint4*)k, k_stride * es / 16, (const uint4*)v, v_stride * es / 16,
                      slot_map, (uint4*)k_pages, (uint4*)v_pages, status);
}

cudaError_t paged_tables_prepare() {
    return cudaFuncSetAttribute(tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (kPagedMaxRequests + 1) * 12);
}

}  // namespace ice
