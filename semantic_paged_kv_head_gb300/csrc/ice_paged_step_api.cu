// C ABI of the calls around the paged cache's attention: rotating append, shared pages, verification of drafts. See
// include/ice.h for the contract of each call.
#include <cmath>
#include <utility>

#include "ice_paged_handle.cuh"
#include "ice_paged_rope.cuh"
#include "ice_paged_share.cuh"
#include "ice_paged_verify.cuh"

using namespace ice;

namespace {

bool rope_ok(const ice_rope* r) {
    if (!r || r->n_axes < 1 || r->n_axes > 4 || r->n_pairs < 8 || r->n_pairs > kD / 2 || r->n_pairs % 8) return false;
    if ((r->interleaved != 0 && r->interleaved != 1) || r->reserved != 0) return false;
    for (int i = 0; i < r->n_pairs; ++i)
        if (!std::isfinite(r->freq[i]) || r->axis[i] < 0 || r->axis[i] >= r->n_axes) return false;
    return true;
}

// The handle's scratch for shared pages, allocated and cleared (on `stream`) the first time.
int share_scratch(ice_paged* pg, const Buffers& b, void* stream, ShareScratch* w) {
    const size_t chunks = (size_t)((pg->p.n_pages + kCmpChunk - 1) / kCmpChunk);
    const size_t req = sizeof(ShareHead), claims = req + sizeof(int4) * (size_t)pg->p.max_requests;
    const size_t count = claims + 8 * (size_t)pg->p.n_pages;
    const size_t freed = count + 4 * chunks;
    const size_t bytes = freed + 4 * (size_t)pg->p.max_requests * ((pg->p.max_blocks + 31) / 32);
    if (!pg->share) {
        if (b.capturing) return ICE_ERR_INVALID_ARG;
        char* p = nullptr;
        if (cudaMalloc(&p, bytes) != cudaSuccess) {
            cudaGetLastError();
            return ICE_ERR_CAPACITY;
        }
        if (cudaMemsetAsync(p, 0, freed, (cudaStream_t)stream) != cudaSuccess) {
            cudaGetLastError();
            cudaFree(p);
            return ICE_ERR_CUDA;
        }
        pg->share = p;
    }
    w->head = (ShareHead*)pg->share;
    w->claim = (unsigned long long*)(pg->share + claims);
    w->req = (int4*)(pg->share + req);
    w->count = (int*)(pg->share + count);
    w->freed = (unsigned*)(pg->share + freed);
    return ICE_OK;
}

// Whether n rows of `row` bytes each share memory: those at a + i sa and at b + j sb. With equal strides (>= row) exact: columns of one
// buffer share none. Else by the spans from the first row to the end of the last.
bool rows_overlap(uintptr_t a, int64_t sa, uintptr_t b, int64_t sb, int64_t row, int64_t n) {
    if (a > b) std::swap(a, b), std::swap(sa, sb);
    const uint64_t apart = b - a;  // b's first row begins so far behind a's
    if (apart >= (uint64_t)(n - 1) * (uint64_t)sa + (uint64_t)row) return false;
    if (sa != sb) return true;
    const uint64_t off = apart % (uint64_t)sa, k = apart / (uint64_t)sa;  // it begins in or behind row k of a, k < n
    return off < (uint64_t)row || (k + 1 < (uint64_t)n && off + (uint64_t)row > (uint64_t)sa);
}

bool req_ok(const ice_paged* pg, int32_t n_req) { return pg && n_req >= 1 && n_req <= pg->p.max_requests; }

}  // namespace

extern "C" {

int ice_paged_rope_append(ice_paged* pg, int32_t n_tokens, const ice_rope* rope, const int32_t* positions,
                          int64_t pos_stride, int64_t pos_offset, const void* q, int64_t q_stride, void* q_out,
                          int64_t q_out_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                          const int64_t* slot_map, void* k_pages, void* v_pages, void* stream) {
    ApiRange range_("ice_paged_rope_append");
    if (!pg || n_tokens < 0 || !rope_ok(rope)) return ICE_ERR_INVALID_ARG;
    if (!stride_ok(pg, k_stride, pg->p.n_kv_heads) || !stride_ok(pg, v_stride, pg->p.n_kv_heads)) return ICE_ERR_INVALID_ARG;
    if (rope->n_axes > 1 && (pos_stride < n_tokens || pos_stride > (1LL << 40))) return ICE_ERR_INVALID_ARG;
    if (pos_offset < -(1LL << 31) || pos_offset >= 1LL << 31) return ICE_ERR_INVALID_ARG;
    const int Hq = q || q_out ? pg->p.n_q_heads : 0;
    if (Hq && (!stride_ok(pg, q_stride, Hq) || !stride_ok(pg, q_out_stride, Hq))) return ICE_ERR_INVALID_ARG;
    if (n_tokens == 0) return ICE_OK;
    if (Hq && !(q == q_out && q_stride == q_out_stride)) {
        const int64_t es = es_of(pg), row = (int64_t)Hq * kD * es;
        if (rows_overlap((uintptr_t)q, q_stride * es, (uintptr_t)q_out, q_out_stride * es, row, n_tokens)) return ICE_ERR_INVALID_ARG;
    }
    Buffers b(pg, stream);
    if (Hq) b.need(q, 16).need(q_out, 16);
    b.need(positions, 4).need(k, 16).need(v, 16).need(slot_map, 8).need(k_pages, 16).need(v_pages, 16);
    if (!b.ok) return ICE_ERR_INVALID_ARG;
    RopeAppend a = {};
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_out = q_out;
    a.k_pages = k_pages;
    a.v_pages = v_pages;
    a.positions = positions;
    a.slot_map = (const long long*)slot_map;
    a.status = pg->words + kWordStatus;
    a.q_stride = q_stride;
    a.q_out_stride = q_out_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.pos_stride = rope->n_axes > 1 ? pos_stride : 0;
    a.pos_offset = pos_offset;
    a.n_slots = pg->p.n_pages * pg->p.page_size;
    a.n_tokens = n_tokens;
    a.Hq = Hq;
    a.H = pg->p.n_kv_heads;
    a.P = pg->p.page_size;
    return launched(launch_rope_append(a, *rope, pg->p.dtype, (cudaStream_t)stream));
}

int ice_paged_fork(ice_paged* pg, int32_t n_fork, const int32_t* src, const int32_t* dst,
                   const int32_t* fork_len, int32_t n_req, const int32_t* seq_len, int32_t* block_table,
                   int32_t* page_refs, int32_t* seq_len_out, void* stream) {
    ApiRange range_("ice_paged_fork");
    if (!req_ok(pg, n_req) || n_fork < 0 || n_fork > n_req) return ICE_ERR_INVALID_ARG;
    Buffers b(pg, stream);
    if (n_fork > 0) b.need(src, 4).need(dst, 4).opt(fork_len);
    b.need(seq_len, 4).need(block_table, 4).need(page_refs, 4).need(seq_len_out, 4);
    if (!b.ok || !aligned(fork_len, 4)) return ICE_ERR_INVALID_ARG;
    ShareScratch w;
    const int rc = share_scratch(pg, b, stream, &w);
    if (rc != ICE_OK) return rc;
    Fork a = {};
    a.src = src;
    a.dst = dst;
    a.fork_len = fork_len;
    a.seq_len = seq_len;
    a.block_table = block_table;
    a.page_refs = page_refs;
    a.seq_len_out = seq_len_out;
    a.status = pg->words + kWordStatus;
    a.head = w.head;
    a.n_pages = pg->p.n_pages;
    a.n_fork = n_fork;
    a.n = n_req;
    a.max_blocks = pg->p.max_blocks;
    a.P = pg->p.page_size;
    return launched(launch_fork(a, (cudaStream_t)stream));
}

int ice_paged_tables_shared(ice_paged* pg, int32_t n_req, const int32_t* seq_len, const int32_t* n_new,
                            int32_t* block_table, int32_t* free_pages, const int64_t* free_state,
                            int32_t* page_refs, int32_t* seq_len_out, int64_t* free_state_out, int32_t* q_start,
                            int64_t* slot_map, int32_t* positions, int32_t n_slots, int32_t* copy_src,
                            int32_t* copy_dst, void* stream) {
    ApiRange range_("ice_paged_tables_shared");
    if (!req_ok(pg, n_req) || n_slots < 0 || n_slots > (1 << 30)) return ICE_ERR_INVALID_ARG;
    Buffers b(pg, stream);
    b.need(seq_len, 4).need(n_new, 4).need(block_table, 4).need(free_pages, 4).need(free_state, 8).need(page_refs, 4);
    b.need(seq_len_out, 4).need(free_state_out, 8).need(q_start, 4).need(copy_src, 4).need(copy_dst, 4);
    if (n_slots > 0) b.need(slot_map, 8).opt(positions);
    if (!b.ok || !aligned(positions, 4)) return ICE_ERR_INVALID_ARG;
    SharedTables a = {};
    const int rc = share_scratch(pg, b, stream, &a.w);
    if (rc != ICE_OK) return rc;
    a.seq_len = seq_len;
    a.n_new = n_new;
    a.block_table = block_table;
    a.free_pages = free_pages;
    a.page_refs = page_refs;
    a.free_state = (const long long*)free_state;
    a.seq_len_out = seq_len_out;
    a.free_state_out = (long long*)free_state_out;
    a.q_start = q_start;
    a.slot_map = (long long*)slot_map;
    a.positions = positions;
    a.copy_src = copy_src;
    a.copy_dst = copy_dst;
    a.status = pg->words + kWordStatus;
    a.n_pages = pg->p.n_pages;
    a.n = n_req;
    a.max_blocks = pg->p.max_blocks;
    a.P = pg->p.page_size;
    a.n_slots = n_slots;
    return launched(launch_shared_tables(a, (cudaStream_t)stream));
}

int ice_paged_copy(ice_paged* pg, int32_t n, const int32_t* src, const int32_t* dst, int32_t n_layers,
                   int64_t layer_stride, void* k_pages, void* v_pages, void* stream) {
    ApiRange range_("ice_paged_copy");
    if (!pg || n < 0 || n_layers < 1 || n_layers > 4096) return ICE_ERR_INVALID_ARG;
    const int64_t es = es_of(pg), page = (int64_t)pg->p.n_kv_heads * pg->p.page_size * kD;
    if (n_layers == 1) layer_stride = 0;
    else if (layer_stride < page * pg->p.n_pages || layer_stride > (1LL << 45) || layer_stride * es % 16) return ICE_ERR_INVALID_ARG;
    if (n == 0) return ICE_OK;
    Buffers b(pg, stream);
    b.need(src, 4).need(dst, 4).need(k_pages, 16).need(v_pages, 16);
    if (!b.ok) return ICE_ERR_INVALID_ARG;
    return launched(launch_page_copy(n, src, dst, n_layers, layer_stride * es, page * es, pg->p.n_pages, k_pages, v_pages,
                                     pg->words + kWordStatus, (cudaStream_t)stream));
}

int ice_paged_compact(ice_paged* pg, int32_t n_req, const int32_t* seq_len, const int32_t* block_table,
                      int32_t n_extra, const int32_t* extra, const int32_t* page_refs, int32_t* free_pages,
                      int64_t* free_state_out, int32_t n_moves, int32_t* move_src, int32_t* move_dst,
                      int32_t* block_table_out, int32_t* extra_out, int32_t* page_refs_out, void* stream) {
    ApiRange range_("ice_paged_compact");
    if (!req_ok(pg, n_req) || n_extra < 0 || n_moves < 0) return ICE_ERR_INVALID_ARG;
    Buffers b(pg, stream);
    b.need(seq_len, 4).need(block_table, 4).need(page_refs, 4).need(free_pages, 4).need(free_state_out, 8);
    b.need(block_table_out, 4).need(page_refs_out, 4);
    if (n_extra > 0) b.need(extra, 4).need(extra_out, 4);
    if (n_moves > 0) b.need(move_src, 4).need(move_dst, 4);
    if (!b.ok) return ICE_ERR_INVALID_ARG;
    Compact a = {};
    const int rc = share_scratch(pg, b, stream, &a.w);
    if (rc != ICE_OK) return rc;
    a.seq_len = seq_len;
    a.block_table = block_table;
    a.page_refs = page_refs;
    a.extra = extra;
    a.block_table_out = block_table_out;
    a.page_refs_out = page_refs_out;
    a.extra_out = extra_out;
    a.free_pages = free_pages;
    a.free_state_out = (long long*)free_state_out;
    a.move_src = move_src;
    a.move_dst = move_dst;
    a.status = pg->words + kWordStatus;
    a.n_pages = pg->p.n_pages;
    a.n = n_req;
    a.max_blocks = pg->p.max_blocks;
    a.P = pg->p.page_size;
    a.n_extra = n_extra;
    a.n_moves = n_moves;
    return launched(launch_compact(a, (cudaStream_t)stream));
}

int ice_paged_verify(ice_paged* pg, int32_t n_req, int32_t n_draft_max, int32_t vocab, int32_t dtype,
                     const int32_t* draft_tokens, const int32_t* n_draft, const void* target,
                     int64_t target_req_stride, int64_t target_row_stride, const void* draft,
                     int64_t draft_req_stride, int64_t draft_row_stride, const float* uniform, int32_t* tokens,
                     int32_t* n_accepted, int32_t* n_new, void* stream) {
    ApiRange range_("ice_paged_verify");
    if (!req_ok(pg, n_req) || n_draft_max < 0 || vocab < 1) return ICE_ERR_INVALID_ARG;
    if (dtype != ICE_F32 && dtype != ICE_BF16) return ICE_ERR_INVALID_ARG;
    const int64_t most = 1LL << 45;
    if (target_req_stride < 0 || target_req_stride > most || target_row_stride < 0 || target_row_stride > most) return ICE_ERR_INVALID_ARG;
    const bool has_draft = draft && uniform && n_draft_max > 0;
    if (has_draft && (draft_req_stride < 0 || draft_req_stride > most || draft_row_stride < 0 || draft_row_stride > most))
        return ICE_ERR_INVALID_ARG;
    if (n_draft_max > kVerMaxDrafts || vocab > kVerMaxVocab) return ICE_ERR_UNSUPPORTED;
    const size_t es = dtype == ICE_BF16 ? 2 : 4;
    Buffers b(pg, stream);
    b.need(n_draft, 4).need(target, es).need(tokens, 4).need(n_accepted, 4).need(n_new, 4).opt(uniform);
    if (n_draft_max > 0) b.need(draft_tokens, 4);
    if (has_draft) b.need(draft, es);
    if (!b.ok || !aligned(uniform, 4)) return ICE_ERR_INVALID_ARG;
    Verify a = {};
    a.target = target;
    a.draft = has_draft ? draft : nullptr;
    a.t_req = target_req_stride;
    a.t_row = target_row_stride;
    a.d_req = draft_req_stride;
    a.d_row = draft_row_stride;
    a.tokens = draft_tokens;
    a.n_draft = n_draft;
    a.uniform = uniform;
    a.out = tokens;
    a.accepted = n_accepted;
    a.n_new = n_new;
    a.status = pg->words + kWordStatus;
    a.scratch = (VerifyScratch*)pg->verify;
    a.n_req = n_req;
    a.K = n_draft_max;
    a.V = vocab;
    return launched(launch_verify(a, dtype, (cudaStream_t)stream));
}

}  // extern "C"
