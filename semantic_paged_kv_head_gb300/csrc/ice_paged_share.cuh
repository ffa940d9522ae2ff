// What the kernels and the C entries of shared pages have in common.
#pragma once

#include "ice_paged.cuh"

namespace ice {

// Scratch of a handle, made by the first call that needs it: this head, then the arrays of ShareScratch.
struct ShareHead {
    unsigned long long epoch;  // calls so far
    unsigned ticket;
    int flags;                 // kBad*, zero between calls
    int plan[4];               // of a compaction: 1 if it is carried out, pages in use, pages moved
    unsigned ring_bad;         // of a step: kRingNone - the first place behind the ring's head whose id is no page's; zero between calls
    int pad[7];
};
static_assert(sizeof(ShareHead) == 64, "claims begin at a multiple of 8 bytes");
enum { kBadBounds = 1, kBadCapacity = 2 };
constexpr unsigned kRingNone = 1u << 31;  // above every place in a ring
constexpr int kCmpChunk = 1024;  // pages that a block of a compaction counts at once

// what becomes of the page that a request writes into: kept, or copied
enum { kReqKeeps = 2, kReqCopies = 1 };

struct ShareScratch {
    ShareHead* head;
    unsigned long long* claim;  // [n_pages]
    int4* req;                  // [max_requests] of a step: new tokens, pages more, pages given back, kReq*
    unsigned* freed;            // [max_requests][ceil(max_blocks / 32)] of a step: which entries' pages are given back, a bit each
    int* count;                 // [ceil(n_pages / kCmpChunk)] of a compaction: pages in use
};

struct SharedTables {
    const int *seq_len, *n_new;
    int *block_table, *free_pages, *page_refs;
    const long long* free_state;
    int* seq_len_out;
    long long* free_state_out;
    int* q_start;
    long long* slot_map;
    int *positions, *copy_src, *copy_dst, *status;
    ShareScratch w;
    long long n_pages;
    int n, max_blocks, P, n_slots;
    int most_taken;  // made by the launch: no step that is carried out takes more pages
};

struct Fork {
    const int *src, *dst, *fork_len, *seq_len;
    int *block_table, *page_refs, *seq_len_out, *status;
    ShareHead* head;
    long long n_pages;
    int n_fork, n, max_blocks, P;
};

struct Compact {
    const int *seq_len, *block_table, *page_refs, *extra;
    int *block_table_out, *page_refs_out, *extra_out, *free_pages;
    long long* free_state_out;
    int *move_src, *move_dst, *status;
    ShareScratch w;
    long long n_pages;
    int n, max_blocks, P, n_extra, n_moves;
};

cudaError_t launch_shared_tables(SharedTables a, cudaStream_t s);
cudaError_t launch_fork(const Fork& a, cudaStream_t s);
cudaError_t launch_compact(const Compact& a, cudaStream_t s);
// page_bytes, layer_bytes: multiples of 16
cudaError_t launch_page_copy(int n, const int* src, const int* dst, int n_layers, long long layer_bytes, long long page_bytes,
                             long long n_pages, void* k_pages, void* v_pages, int* status, cudaStream_t s);
cudaError_t share_prepare();

}  // namespace ice
