// Drafted tokens against the target model's probabilities, or its logits.
#include <cooperative_groups.h>

#include <algorithm>

#include "ice_paged_verify.cuh"

namespace cg = cooperative_groups;

namespace ice {

// ---------------------------------------------------------------------------
// Speculative sampling (Leviathan et al. 2023, Chen et al. 2023): draft i with token x stays if u_i q_i(x) < p_i(x). The
// first that does not is replaced by a token drawn from max(p - q, 0); behind the last one that stays a token is drawn
// from p. Drawing is by the inverse of the cumulative sum: the first j with w_0 + ... + w_j > u W, W the sum of all.
//
// A border between two tokens may lie anywhere, so sums have to be near those of exact arithmetic: with 2^17 tokens of
// like weight fp32 sums would move one draw in ten. A thread's sums carry what each addition and each p - q cut off (two-sum,
// Knuth 1969; 46 bits or more), and are added over the lanes and tiles in fp64, whose units do a 32nd of
// the additions that way.
//
// One thread-block cluster a request. Its blocks find the first rejected draft by themselves (K gathers), each sums its
// share of the vocabulary, tile by tile; after one exchange of the blocks' sums through distributed shared memory one
// of them holds the drawn token: it looks up the tile by the tiles' sums, and reads that tile again.
// Only the rows that decide are read: two of the 2 K + 1.
// ---------------------------------------------------------------------------
constexpr int kVerThreads = 512, kVerWarps = kVerThreads / 32;
constexpr int kVerTile = 1024;                          // elements of a row that a warp takes at once
constexpr int kVerTiles = kVerMaxVocab / kVerTile;

// What an entry counts for: NaN, negative and huge ones nothing (2^22 of 2^100 have a sum in fp32).
__device__ __forceinline__ float clean(float x) { return x <= 1.2676506e30f ? fmaxf(x, 0.0f) : 0.0f; }

__device__ __forceinline__ float clamp_uniform(float u) { return fminf(fmaxf(u, 0.0f), 0.99999994f); }

// 16 bytes at p, which is aligned to an element only: from one or two aligned words. The caller has checked that
// both lie in the row.
template <bool ALIGNED>
__device__ __forceinline__ uint4 load16(const char* p) {
    if (ALIGNED) return __ldcs(reinterpret_cast<const uint4*>(p));
    const unsigned sh = (unsigned)(uintptr_t)p & 15;
    const uint4* b = reinterpret_cast<const uint4*>(p - sh);
    const uint4 x = __ldg(b), y = sh ? __ldg(b + 1) : x;
    unsigned w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    if (sh & 8) {
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    }
    if (sh & 4) {
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
    const unsigned bits = (sh & 3) * 8;
    return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits), __funnelshift_r(w[2], w[3], bits),
                      __funnelshift_r(w[3], w[4], bits));
}

template <typename T> constexpr int kVec = 16 / sizeof(T);  // elements of 16 bytes

template <typename T> __device__ __forceinline__ void unpack(const uint4& w, float (&v)[kVec<T>]);
template <> __device__ __forceinline__ void unpack<float>(const uint4& w, float (&v)[4]) {
    v[0] = __uint_as_float(w.x), v[1] = __uint_as_float(w.y), v[2] = __uint_as_float(w.z), v[3] = __uint_as_float(w.w);
}
template <> __device__ __forceinline__ void unpack<__nv_bfloat16>(const uint4& w, float (&v)[8]) {
    const unsigned u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(u[i] << 16), v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
}

// Whether a tile's 16-byte loads stay in the row.
template <typename T>
__device__ __forceinline__ bool whole_tile(const T* row, int V, int e0) {
    const unsigned sh = (unsigned)(uintptr_t)row & 15;  // a tile is a multiple of 16 bytes
    return e0 + kVerTile + (sh ? kVec<T> : 0) <= V && (sh == 0 || e0 > 0);
}

// A sum of terms >= 0 with the parts that its additions cut off.
struct Sum2 {
    float hi = 0.0f, lo = 0.0f;
    __device__ __forceinline__ void add(float d, float e) {
        const float s = hi + d, b = s - hi;
        lo += ((hi - (s - b)) + (d - b)) + e;
        hi = s;
    }
    // max(p - q, 0), exactly: where p > q >= 0 the difference's own error is (p - d) - q
    __device__ __forceinline__ void add_above(float p, float q) {
        const float d = p - q;
        if (d > 0.0f) add(d, (p - d) - q);
    }
};

__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Sum of a tile's weights, the same in every lane. q: the draft's row or NULL; sure: the token that the draft was certain of,
// or -1.
template <typename T, bool ALIGNED, bool HAS_Q>
__device__ __forceinline__ double sum_whole_tile(const T* p, const T* q, int e0) {
    constexpr int N = kVerTile / 32 / kVec<T>;
    const int at = e0 + (threadIdx.x & 31) * kVec<T>;
    uint4 x[N], y[HAS_Q ? N : 1];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        x[i] = load16<ALIGNED>(reinterpret_cast<const char*>(p + at + i * 32 * kVec<T>));
        if (HAS_Q) y[i] = load16<ALIGNED>(reinterpret_cast<const char*>(q + at + i * 32 * kVec<T>));
    }
    Sum2 s;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float a[kVec<T>], b[kVec<T>];
        unpack<T>(x[i], a);
        if (HAS_Q) unpack<T>(y[i], b);
#pragma unroll
        for (int j = 0; j < kVec<T>; ++j) {
            if (HAS_Q) s.add_above(clean(a[j]), clean(b[j]));
            else s.add(clean(a[j]), 0.0f);
        }
    }
    return warp_sum((double)s.hi + (double)s.lo);
}

template <typename T>
__device__ __forceinline__ double weight(const T* p, const T* q, int sure, int j) {
    const double b = q != nullptr ? (double)clean(to_f<T>(q[j])) : j == sure ? 1.0 : 0.0;
    return fmax((double)clean(to_f<T>(p[j])) - b, 0.0);
}

template <typename T>
__device__ __forceinline__ double sum_tile(const T* p, const T* q, int sure, int V, int e0) {
    const bool whole = whole_tile(p, V, e0) && (q == nullptr || whole_tile(q, V, e0)) && !(sure >= e0 && sure < e0 + kVerTile);
    if (whole) {
        const bool aligned = (((uintptr_t)p | (uintptr_t)q) & 15) == 0;
        if (q != nullptr) return aligned ? sum_whole_tile<T, true, true>(p, q, e0) : sum_whole_tile<T, false, true>(p, q, e0);
        return aligned ? sum_whole_tile<T, true, false>(p, q, e0) : sum_whole_tile<T, false, false>(p, q, e0);
    }
    double s = 0.0;
    const int end = min(e0 + kVerTile, V);
#pragma unroll 8
    for (int j = e0 + (threadIdx.x & 31); j < end; j += 32) s += weight(p, q, sure, j);
    return warp_sum(s);
}

// Block's share of the tiles.
__device__ __forceinline__ void share_of(int tiles, int rank, int size, int& t0, int& t1) {
    t0 = (int)((long long)tiles * rank / size);
    t1 = (int)((long long)tiles * (rank + 1) / size);
}

struct VerifyShared {
    double total;                 // of this block's tiles; read by the cluster
    unsigned long long best[2][kVerMaxDrafts + 1];  // greedy: this block's best of each row of a group; read by the cluster
    double warp[kVerWarps];
    double x;                     // what is left of u W before the tile
    unsigned keep[2];
    int tile, token;
};

// Entry j of the greedy comparison: larger is better, of equal values the lower index. NaN is nothing.
__device__ __forceinline__ unsigned long long greedy_key(float x, int j) {
    const unsigned b = __float_as_uint(x + 0.0f);  // -0 as 0
    const unsigned o = b & 0x80000000u ? ~b : b | 0x80000000u;
    return (unsigned long long)o << 32 | (0xffffffffu - (unsigned)j);
}

struct Best {
    float x = -INFINITY;
    int j = -1;  // none yet
    __device__ __forceinline__ void look(float y, int at) {
        if (y > x || (j < 0 && y == x)) x = y, j = at;
    }
};

template <typename T, bool ALIGNED>
__device__ __forceinline__ void best_of_whole_tile(const T* p, int e0, Best& best) {
    constexpr int N = kVerTile / 32 / kVec<T>;
    const int at = e0 + (threadIdx.x & 31) * kVec<T>;
    uint4 w[N];
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = load16<ALIGNED>(reinterpret_cast<const char*>(p + at + i * 32 * kVec<T>));
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float v[kVec<T>];
        unpack<T>(w[i], v);
        float m = v[0];
#pragma unroll
        for (int j = 1; j < kVec<T>; ++j) m = fmaxf(m, v[j]);  // a NaN is passed over
        if (m > best.x || (best.j < 0 && m == best.x)) {  // rare: the index only where there is a new best
#pragma unroll
            for (int j = 0; j < kVec<T>; ++j) best.look(v[j], at + i * 32 * kVec<T> + j);
        }
    }
}

template <typename T>
__device__ __forceinline__ unsigned long long best_of_tile(const T* p, int V, int e0) {
    Best best;
    if (whole_tile(p, V, e0)) {
        if (((uintptr_t)p & 15) == 0) best_of_whole_tile<T, true>(p, e0, best);
        else best_of_whole_tile<T, false>(p, e0, best);
    } else {
        const int end = min(e0 + kVerTile, V);
#pragma unroll 8
        for (int j = e0 + (threadIdx.x & 31); j < end; j += 32) best.look(to_f<T>(p[j]), j);
    }
    unsigned long long k = best.j < 0 ? 0ull : greedy_key(best.x, best.j);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const unsigned long long y = __shfl_xor_sync(0xffffffffu, k, o);
        k = y > k ? y : k;
    }
    return k;
}

template <typename T, bool GREEDY>
__global__ void __launch_bounds__(kVerThreads) verify_kernel(Verify a) {
    __shared__ VerifyShared sh;
    __shared__ double s_tile[GREEDY ? 1 : kVerTiles];
    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank(), size = (int)cl.num_blocks();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int r = blockIdx.x / size;
    pdl_wait_then_release();
    const int K = a.K, V = a.V, nd = a.n_draft[r];
    int* const out = a.out + (long long)r * (K + 1);
    if (nd < 0 || nd > K) {  // a request that waits; the whole cluster comes here
        if (rank == 0) {
            for (int i = tid; i <= K; i += kVerThreads) out[i] = -1;
            if (tid == 0) {
                a.accepted[r] = a.n_new[r] = 0;
                if (nd != -1) set_status(a.status, ICE_ERR_BOUNDS);
            }
        }
        return;
    }
    const T* const target = (const T*)a.target + r * a.t_req;
    const int* const tokens = a.tokens + (long long)r * K;
    const int tiles = (V + kVerTile - 1) / kVerTile;
    int t0, t1;
    share_of(tiles, rank, size, t0, t1);
    int kept = 0, token = -1;  // sampling: token in the block that owns the drawn one
    bool none = false;         // the deciding row leaves nothing
    if (rank == 0 && tid < nd && (tokens[tid] < 0 || tokens[tid] >= V)) set_status(a.status, ICE_ERR_BOUNDS);
    if (GREEDY) {
        bool done = false;
        for (int g0 = 0, buf = 0; !done; g0 += a.group, buf ^= 1) {
            const int rows = min(a.group, nd + 1 - g0), n = t1 - t0;
            if (tid < rows) sh.best[buf][tid] = 0;
            __syncthreads();
            for (int i = warp; i < rows * n; i += kVerWarps) {
                const int y = i / n, t = t0 + i - y * n;
                const unsigned long long k = best_of_tile(target + (g0 + y) * a.t_row, V, t * kVerTile);
                if (lane == 0 && k) atomicMax(&sh.best[buf][y], k);
            }
            cl.sync();
            for (int y = 0; y < rows && !done; ++y) {
                unsigned long long k = lane < size ? cl.map_shared_rank(&sh.best[buf][y], lane)[0] : 0ull;
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) {
                    const unsigned long long z = __shfl_xor_sync(0xffffffffu, k, o);
                    k = z > k ? z : k;
                }
                k = __shfl_sync(0xffffffffu, k, 0);
                none = k == 0;
                token = none ? -1 : (int)(0xffffffffu - (unsigned)k);
                if (kept < nd && !none && tokens[kept] == token) ++kept;
                else done = true;
            }
        }
    } else {
        if (warp < 2) {  // the drafts that stay: one a lane
            bool keep = false;
            if (tid < nd) {
                const int x = tokens[tid];
                if (x >= 0 && x < V) {
                    const float p = clean(to_f<T>(target[tid * a.t_row + x]));
                    const float q = a.draft ? clean(to_f<T>(((const T*)a.draft + r * a.d_req)[tid * a.d_row + x])) : 1.0f;
                    // 48 bits: exact
                    keep = (double)clamp_uniform(a.uniform[(long long)r * (K + 1) + tid]) * (double)q < (double)p;
                }
            }
            const unsigned m = __ballot_sync(0xffffffffu, keep);
            if (lane == 0) sh.keep[warp] = m;
        }
        const double u = clamp_uniform(a.uniform[(long long)r * (K + 1) + K]);
        __syncthreads();
        const unsigned long long m = (unsigned long long)sh.keep[1] << 32 | sh.keep[0];
        kept = __ffsll((long long)~m) - 1;  // bit 63 is never set
        const T* const p = target + kept * a.t_row;
        const T* q = nullptr;
        int sure = -1;
        if (kept < nd) {
            if (a.draft) q = (const T*)a.draft + r * a.d_req + kept * a.d_row;
            else sure = tokens[kept];
        }
        // at most twice: where the target is nowhere above the draft, a token of the target's own
        for (int pass = 0; pass < 2; ++pass) {
            for (int t = t0 + warp; t < t1; t += kVerWarps) {
                const double s = sum_tile(p, q, sure, V, t * kVerTile);
                if (lane == 0) s_tile[t - t0] = s;
            }
            __syncthreads();
            // sums up to each lane's range of tiles
            const int n = t1 - t0, per = (n + 31) >> 5, b = min(lane * per, n), e = min(b + per, n);
            double mine = 0.0, upto = 0.0;
            if (warp == 0) {
                for (int t = b; t < e; ++t) mine += s_tile[t];
                upto = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const double y = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= o) upto += y;
                }
                if (lane == 31) sh.total = upto;
            }
            cl.sync();
            // every block comes to the same owner of the drawn token
            double before = 0.0, all = 0.0, start = 0.0;
            int owner = -1;
            for (int k = 0; k < size; ++k) all += *cl.map_shared_rank(&sh.total, k);
            const double want = u * all;
            for (int k = 0; k < size; ++k) {
                const double s = *cl.map_shared_rank(&sh.total, k);
                if (s > 0.0 && !(owner >= 0 && want < start + *cl.map_shared_rank(&sh.total, owner))) {
                    owner = k;  // the first whose end lies beyond `want`, else the last that has any weight
                    start = before;
                }
                before += s;
            }
            cl.sync();  // the sums have been read
            if (owner < 0) {
                none = true;
                if (q == nullptr && sure < 0) break;
                q = nullptr, sure = -1;
                continue;
            }
            none = false;
            if (owner == rank) {
                if (warp == 0) {
                    double x = want - start, low = __shfl_up_sync(0xffffffffu, upto, 1);
                    if (lane == 0) low = 0.0;
                    const unsigned some = __ballot_sync(0xffffffffu, mine > 0.0), over = some & __ballot_sync(0xffffffffu, upto > x);
                    if (lane == (over ? __ffs(over) - 1 : 31 - __clz(some))) {
                        int found = b;
                        double base = low;
                        for (int t = b; t < e; ++t) {
                            if (s_tile[t] > 0.0) {
                                found = t;
                                base = low;
                                if (low + s_tile[t] > x) break;
                            }
                            low += s_tile[t];
                        }
                        sh.tile = found;
                        sh.x = x - base;
                        sh.token = INT_MAX;
                    }
                }
                __syncthreads();
                // the tile again, two neighbouring elements a thread, and their sums up to each
                const int j = (t0 + sh.tile) * kVerTile + 2 * tid;
                const double w0 = j < V ? weight(p, q, sure, j) : 0.0, w1 = j + 1 < V ? weight(p, q, sure, j + 1) : 0.0;
                double c = w0 + w1;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const double y = __shfl_up_sync(0xffffffffu, c, o);
                    if (lane >= o) c += y;
                }
                if (lane == 31) sh.warp[warp] = c;
                __syncthreads();
                double base = 0.0;
                for (int k = 0; k < warp; ++k) base += sh.warp[k];
                double c1 = __shfl_up_sync(0xffffffffu, c, 1);
                if (lane == 0) c1 = 0.0;
                if (w0 > 0.0 && base + c1 + w0 > sh.x) atomicMin(&sh.token, j);
                else if (w1 > 0.0 && base + c > sh.x) atomicMin(&sh.token, j + 1);
                __syncthreads();
                if (sh.token == INT_MAX) {  // by the roundings none: the last that has any weight
                    __syncthreads();
                    if (tid == 0) sh.token = -1;
                    __syncthreads();
                    if (w1 > 0.0) atomicMax(&sh.token, j + 1);
                    else if (w0 > 0.0) atomicMax(&sh.token, j);
                    __syncthreads();
                }
                token = sh.token;
                if (tid == 0) out[kept] = token;
            }
            break;
        }
    }
    if (GREEDY) cl.sync();  // the blocks' bests have been read
    if (rank != 0) return;
    for (int i = tid; i <= K; i += kVerThreads) {
        if (i < kept) out[i] = tokens[i];
        else if (i > kept) out[i] = -1;
        else if (GREEDY || none) out[i] = token;
    }
    if (tid == 0) {
        a.accepted[r] = kept;
        a.n_new[r] = kept - nd;
        if (none) set_status(a.status, ICE_ERR_BOUNDS);
    }
}

cudaError_t launch_verify(Verify a, int dtype, cudaStream_t s) {
    const int tiles = (a.V + kVerTile - 1) / kVerTile;
    int size = 8;
    while (size > 1 && size > tiles) size >>= 1;
    a.group = a.n_req * size <= 2 * 152 ? kVerMaxDrafts + 1 : 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.n_req * size);
    cfg.blockDim = dim3(kVerThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = size;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see pdl_wait_then_release
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    const bool greedy = a.uniform == nullptr;
    if (dtype == ICE_BF16)
        return cudaLaunchKernelEx(&cfg, greedy ? verify_kernel<__nv_bfloat16, true> : verify_kernel<__nv_bfloat16, false>, a);
    return cudaLaunchKernelEx(&cfg, greedy ? verify_kernel<float, true> : verify_kernel<float, false>, a);
}

}  // namespace ice
