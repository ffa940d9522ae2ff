// Attention of a batch that shares a prefix: the fp32 kernel on the CUDA cores, the joining
// of the parts, and the choice of the parts.
#include <algorithm>

#include "ice_paged.cuh"

namespace ice {

// ---------------------------------------------------------------------------
// One block takes items in turn: up to 64 rows (new tokens x G heads) against a
// range of tiles of 64 keys, in one pass with a running maximum m and sum l a
// row: m' = max(m, max_t s_t), l' = l 2^(m - m') + sum_t 2^(s_t - m'), and the same
// factor on the output, with s_t = q . k_t log2(e) / sqrt(d). Threads form a 16 x 16
// grid: RT rows by 4 keys each of the scores, RT rows by 8 dimensions each of the
// output, so that a row's 16 threads are half a warp and the statistics need
// shuffles only.
// ---------------------------------------------------------------------------
constexpr int kSimtThreads = 256;
constexpr int kSimtRows = 64;
constexpr int kSimtKeys = 64;
constexpr int kSimtStrideK = kD + 4;          // floats a row: consecutive rows 4 banks apart
constexpr int kSimtStrideP = kSimtKeys + 4;
constexpr int kSimtSmem = 4 * (kSimtRows * kSimtStrideK + kSimtKeys * kSimtStrideK + kSimtKeys * kD +
                               kSimtRows * kSimtStrideP);

__global__ void __launch_bounds__(kSimtThreads) paged_simt_kernel(PagedAttn a, PagedTiles z) {
    extern __shared__ __align__(16) float simt_smem[];
    __shared__ PlanShared sh;
    float* sQ = simt_smem;
    float* sK = sQ + kSimtRows * kSimtStrideK;
    float* sV = sK + kSimtKeys * kSimtStrideK;
    float* sP = sV + kSimtKeys * kD;
    int* cum = reinterpret_cast<int*>(sP + kSimtRows * kSimtStrideP);
    const int tid = threadIdx.x, rg = tid >> 4, kg = tid & 15;
    pdl_wait_then_release();
    make_plan<kSimtThreads>(a, z, cum, sh);
    if (!sh.ok) return;
    const int valid_tok = a.q_start[a.n_req];
    const int n_items = sh.pre + sh.own;
    PagedItem item;
    for (int i = blockIdx.x; i < n_items; i += gridDim.x) {
        get_item(a, z, cum, sh, i, item);
        if (item.ns == 0) continue;
        const PagedStream& it = item.st[0];
        const int nrow = it.ntok * a.G;
        __syncthreads();
        // row r: token tok0 + r / G, head h G + r % G; rows past the item's are zero
        for (int x = tid; x < kSimtRows * (kD / 4); x += kSimtThreads) {
            const int r = x / (kD / 4), c = (x % (kD / 4)) * 4;
            float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (r < nrow)
                load4((const float*)a.q + (it.tok0 + r / a.G) * a.q_stride + (it.h * a.G + r % a.G) * kD + c, v);
            *reinterpret_cast<float4*>(sQ + r * kSimtStrideK + c) = make_float4(v[0], v[1], v[2], v[3]);
        }
        float m[4], l[4], o[4][8];
        int lim[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            m[j] = -INFINITY;
            l[j] = 0.0f;
            const int r = rg * 4 + j;
            lim[j] = r < nrow ? min(it.own_len, it.tok0 + r / a.G + it.lim_off) : 0;  // of own tokens
#pragma unroll
            for (int k = 0; k < 8; ++k) o[j][k] = 0.0f;
        }
        for (int kt = it.kt0; kt < it.kt0 + it.n; ++kt) {
            const PagedTile t = tile_of(a, z, it, kt);
            const int key0 = t.key0;
            __syncthreads();
            for (int x = tid; x < kSimtKeys * (kD / 4); x += kSimtThreads) {
                const int r = x / (kD / 4), c = (x % (kD / 4)) * 4, key = key0 + r;
                float vk[4] = {0.0f, 0.0f, 0.0f, 0.0f}, vv[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                if (key < t.len) {
                    const int page = t.table[key / a.P];
                    if (page >= 0 && page < a.n_pages) {
                        const long long row = ((long long)page * a.H + it.h) * a.P + key % a.P;
                        load4((const float*)a.k_pages + row * kD + c, vk);
                        load4((const float*)a.v_pages + row * kD + c, vv);
                    } else {
                        set_status(a.status, ICE_ERR_BOUNDS);
                    }
                }
                *reinterpret_cast<float4*>(sK + r * kSimtStrideK + c) = make_float4(vk[0], vk[1], vk[2], vk[3]);
                *reinterpret_cast<float4*>(sV + r * kD + c) = make_float4(vv[0], vv[1], vv[2], vv[3]);
            }
            __syncthreads();
            float s[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k) s[j][k] = 0.0f;
#pragma unroll 4
            for (int c = 0; c < kD; c += 4) {
                float4 qv[4], kv[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    qv[j] = *reinterpret_cast<const float4*>(sQ + (rg * 4 + j) * kSimtStrideK + c);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    kv[k] = *reinterpret_cast<const float4*>(sK + (kg + 16 * k) * kSimtStrideK + c);
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        s[j][k] += qv[j].x * kv[k].x + qv[j].y * kv[k].y + qv[j].z * kv[k].z + qv[j].w * kv[k].w;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float mx = m[j];
                const int end = t.own ? lim[j] : t.len;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    s[j][k] = key0 + kg + 16 * k < end ? s[j][k] * a.scale_log2 : -INFINITY;
                    mx = fmaxf(mx, s[j][k]);
                }
#pragma unroll
                for (int d = 8; d >= 1; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                const float mu = mx == -INFINITY ? 0.0f : mx;  // nothing seen yet: all weights 0
                const float f = exp2_approx(m[j] - mu);
                m[j] = mx;
                l[j] *= f;
#pragma unroll
                for (int k = 0; k < 8; ++k) o[j][k] *= f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float p = exp2_approx(s[j][k] - mu);
                    l[j] += p;
                    sP[(rg * 4 + j) * kSimtStrideP + kg + 16 * k] = p;
                }
            }
            __syncwarp();  // a row's weights are written and read by one warp
#pragma unroll 2
            for (int k0 = 0; k0 < kSimtKeys; k0 += 4) {
                float4 pv[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    pv[j] = *reinterpret_cast<const float4*>(sP + (rg * 4 + j) * kSimtStrideP + k0);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const float4 v0 = *reinterpret_cast<const float4*>(sV + (k0 + u) * kD + kg * 4);
                    const float4 v1 = *reinterpret_cast<const float4*>(sV + (k0 + u) * kD + 64 + kg * 4);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float p = u == 0 ? pv[j].x : u == 1 ? pv[j].y : u == 2 ? pv[j].z : pv[j].w;
                        o[j][0] += p * v0.x; o[j][1] += p * v0.y; o[j][2] += p * v0.z; o[j][3] += p * v0.w;
                        o[j][4] += p * v1.x; o[j][5] += p * v1.y; o[j][6] += p * v1.z; o[j][7] += p * v1.w;
                    }
                }
            }
            __syncwarp();
        }
        __syncthreads();  // the key tile's memory takes the output, [d][row]
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float sum = l[j];
#pragma unroll
            for (int d = 8; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            const int r = rg * 4 + j;
            const float inv = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                sK[((k >> 2) * 64 + kg * 4 + (k & 3)) * (kSimtRows + 1) + r] = o[j][k] * inv;
            if (kg == 0 && r < nrow && !it.direct)
                a.part_ml[((long long)it.slot * a.H + it.h) * a.RP + it.tok0 * a.G + r] = make_float2(m[j], sum);
        }
        __syncthreads();
        if (it.direct) {
            for (int x = tid; x < nrow * kD; x += kSimtThreads) {
                const int r = x / kD, c = x % kD, tok = it.tok0 + r / a.G;
                if (tok < valid_tok)
                    ((float*)a.out)[((long long)tok * a.H * a.G + it.h * a.G + r % a.G) * kD + c] =
                        sK[c * (kSimtRows + 1) + r];
            }
        } else {
            float* dst = a.part_o + ((long long)it.slot * a.H + it.h) * kD * a.RP + it.tok0 * a.G;
            const int r = tid % kSimtRows;
            if (r < nrow)
                for (int c = tid / kSimtRows; c < kD; c += kSimtThreads / kSimtRows)
                    dst[(long long)c * a.RP + r] = sK[c * (kSimtRows + 1) + r];
        }
    }
}

// ---------------------------------------------------------------------------
// Joining: a block for 32 rows of a KV head, a lane a row. With parts (m_i, l_i, o_i),
// M = max m_i and w_i = l_i 2^(m_i - M): out = sum w_i o_i / sum w_i, zeros where
// nothing was seen. Rows with one part were written by the attention kernel. Bound by the
// parts' bytes, read once, where there are many rows, and by the latency of a
// chain of loads where there are few. PW of the 8 warps therefore share the parts of 16
// dimensions (and the block has 8 / PW groups of 16): one where the rows fill the GPU,
// eight where a row has many parts and little else runs.
// ---------------------------------------------------------------------------
constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kJoinDims = 16;

template <typename T, int PW>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(PagedAttn a, PagedTiles z) {
    constexpr int kDims = kJoinDims * (kJoinWarps / PW);  // dimensions of the block
    __shared__ float wt[kPagedMaxSlots][32];  // weights of the parts, by row
    __shared__ float tile[PW][32][kDims + 1];
    __shared__ float red[kJoinWarps][32];
    __shared__ int req_of[32], blk_of[32];    // request of each token, its row block
    __shared__ int own_of[32], len_of[32];    // new and own tokens of each token's request, then its parts
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int h = blockIdx.y, R0 = blockIdx.x * 32, d0 = blockIdx.z * kDims, G = a.G;
    // Before the wait: q_start and seq_len were complete when the attention kernel's blocks let
    // this one be scheduled (they wait for the kernels before them first).
    const int valid_tok = a.q_start[a.n_req];
    for (int t = warp; t < 32 / G; t += kJoinWarps) {
        const int tok = R0 / G + t;
        int nq = -1, own_len = 0;
        if (tok < valid_tok) {
            int lo = 0, hi = a.n_req;  // q_start[lo] <= tok < q_start[hi]; 32 probes a step
            while (hi - lo > 1) {
                const int w = (hi - lo + 31) / 32, probe = lo + lane * w;
                const unsigned le =
                    __ballot_sync(0xffffffffu, probe < hi && a.q_start[min(probe, a.n_req)] <= tok);
                const int k = 31 - __clz(le);  // lane 0 always holds
                hi = min(hi, lo + (k + 1) * w);
                lo = lo + k * w;
            }
            nq = a.q_start[lo + 1] - a.q_start[lo];
            own_len = a.seq_len[lo];
            if (lane == 0) {
                req_of[t] = lo;
                blk_of[t] = (tok - a.q_start[lo]) / z.TB;
            }
        }
        if (lane == 0) {
            own_of[t] = nq;
            len_of[t] = own_len;
        }
    }
    pdl_wait_then_release();
    if (!a.plan[kPlanOk]) return;
    const int chunk = a.plan[kPlanChunk], pre_direct = a.plan[kPlanDirect];
    const PagedLong f = {a.plan[kPlanWhole], a.plan[kPlanSplit]};
    __syncthreads();
    if (tid < 32 / G) {
        // the parts' first slot and number; none where the attention kernel wrote the output itself
        const int nq = own_of[tid], s = len_of[tid];
        int first = 0, parts = -1;
        if (nq > z.TS) {
            const int blocks = long_blocks(nq, s, z);
            first = a.prefix_splits;
            const bool whole = f.whole == INT_MAX || a.first_long[req_of[tid]] + h * blocks + blk_of[tid] < f.whole;
            parts = blocks == 0 ? 0 : whole || f.split == 1 ? -1 : f.split;
        } else if (nq > 0) {
            const int own = plan_parts(s, z, chunk);
            parts = (a.prefix_splits == 0 && own == 1) || pre_direct ? -1 : a.prefix_splits + own;
        }
        own_of[tid] = parts;
        len_of[tid] = first;
    }
    __syncthreads();
    const int n = max(own_of[lane / G], 0);  // parts of row R0 + lane
    const int first = len_of[lane / G];
    const float2* ml = a.part_ml + ((long long)first * a.H + h) * a.RP + R0 + lane;
    const long long ml_step = (long long)a.H * a.RP;
    float M = -INFINITY;
#pragma unroll 4
    for (int p = warp; p < n; p += kJoinWarps) M = fmaxf(M, ml[p * ml_step].x);
    red[warp][lane] = M;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kJoinWarps; ++k) M = fmaxf(M, red[k][lane]);
    if (M == -INFINITY) M = 0.0f;
    for (int p = warp; p < n; p += kJoinWarps) {
        const float2 x = ml[p * ml_step];
        wt[p][lane] = x.y * exp2_approx(x.x - M);
    }
    __syncthreads();
    const int pw = warp % PW, dw = warp / PW;
    const float* src = a.part_o + (((long long)first * a.H + h) * kD + d0 + dw * kJoinDims) * a.RP + R0 + lane;
    const long long step = (long long)a.H * kD * a.RP;
    float W = 0.0f, acc[kJoinDims];
#pragma unroll
    for (int k = 0; k < kJoinDims; ++k) acc[k] = 0.0f;
#pragma unroll 2
    for (int p = pw; p < n; p += PW) {
        const float w = wt[p][lane];
        W += w;
#pragma unroll
        for (int k = 0; k < kJoinDims; ++k) acc[k] = fmaf(w, src[p * step + (long long)k * a.RP], acc[k]);
    }
    if (PW > 1) {  // the whole sum of weights
        red[warp][lane] = W;
        __syncthreads();
        W = 0.0f;
#pragma unroll
        for (int k = 0; k < PW; ++k) W += red[dw * PW + k][lane];
    }
    const float inv = W > 0.0f ? 1.0f / W : (W == 0.0f ? 0.0f : W);
#pragma unroll
    for (int k = 0; k < kJoinDims; ++k) tile[pw][lane][dw * kJoinDims + k] = acc[k] * inv;
    __syncthreads();
    for (int x = tid; x < 32 * kDims; x += kJoinThreads) {
        const int r = x / kDims, c = x % kDims;
        if (own_of[r / G] < 0) continue;
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < PW; ++k) v += tile[k][r][c];
        ((T*)a.out)[((long long)((R0 + r) / G) * a.H * G + h * G + (R0 + r) % G) * kD + d0 + c] = from_f<T>(v);
    }
}

template <typename T>
static cudaError_t launch_join(const PagedAttn& a, const PagedTiles& z, int n_sm, cudaStream_t s) {
    // warps that share a row's parts: as many as leave the blocks near two a SM
    const long long groups = (long long)(a.RP / 32) * a.H;
    const dim3 block(kJoinThreads);
    auto grid = [&](int pw) { return dim3((unsigned)(a.RP / 32), (unsigned)a.H, (unsigned)pw); };
    if (groups >= 2 * n_sm) return launch_pdl(paged_join_kernel<T, 1>, grid(1), block, 0, s, a, z);
    if (groups >= n_sm / 2) return launch_pdl(paged_join_kernel<T, 4>, grid(4), block, 0, s, a, z);
    return launch_pdl(paged_join_kernel<T, 8>, grid(8), block, 0, s, a, z);
}

static int simt_bytes(int n_req) { return kSimtSmem + plan_ints(n_req) * 4; }

cudaError_t paged_tables_prepare();
cudaError_t paged_tc_prepare();
PagedTiles paged_tc_tiles(int P, int G);
cudaError_t launch_paged_tc(const PagedAttn& a, const PagedTiles& z, int n_sm, cudaStream_t s);

cudaError_t paged_prepare() {
    cudaError_t e = paged_tables_prepare();
    if (e != cudaSuccess) return e;
    e = paged_tc_prepare();
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(paged_simt_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kSimtSmem + (kPagedMaxRequests + 1) * 4);
}

// Ranges of the prefix: n_base row blocks x heads, each range a wave's share of
// tiles. The time of s ranges is taken as waves x (tiles of a range + the fixed cost of
// an item, in tiles); the least wins, the fewest ranges among equals.
static int prefix_ranges(long long n_base, int tiles, int limit, int n_sm) {
    constexpr int kItemCost = 3;
    int best = 1;
    long long best_t = -1;
    for (int s = 1; s <= std::min(limit, tiles); ++s) {
        const long long waves = (n_base * s + n_sm - 1) / n_sm;
        const long long t = waves * ((tiles + s - 1) / s + kItemCost);
        if (best_t < 0 || t < best_t) {
            best_t = t;
            best = s;
        }
    }
    return best;
}

cudaError_t launch_paged_attn(PagedAttn a, int dtype, long long rows_cap, int n_sm, cudaStream_t s) {
    const bool tc = dtype == ICE_BF16;
    PagedTiles z = tc ? paged_tc_tiles(a.P, a.G) : PagedTiles{kSimtKeys, kSimtRows / a.G, kSimtRows / a.G, 0, 0, 0};
    z.NP = (a.prefix_len + z.KT - 1) / z.KT;
    a.RP = (a.n_tokens * a.G + 31) / 32 * 32;
    const int slots = (int)std::min<long long>(rows_cap / ((long long)a.H * a.RP), kPagedMaxSlots);  // >= 3
    const long long n_base = (long long)((a.n_tokens + z.TB - 1) / z.TB) * a.H;
    a.prefix_splits = 0;
    if (a.prefix_len > 0) {
        const int tiles = z.NP, limit = std::min(slots / 2, kPagedMaxPrefixSplits);
        const bool twin = a.n_tokens <= z.TD;  // two parts a range
        a.prefix_splits = prefix_ranges(n_base, tiles, twin ? std::max(1, limit / 2) : limit, n_sm);
        if (twin) a.prefix_splits = std::min(std::min(2 * a.prefix_splits, limit), tiles);
    }
    a.max_splits = slots - a.prefix_splits;
    a.target_items = n_sm;
    cudaError_t e;
    if (tc)
        e = launch_paged_tc(a, z, n_sm, s);
    else
        e = launch_pdl(paged_simt_kernel, dim3(n_sm), dim3(kSimtThreads), (size_t)simt_bytes(a.n_req), s, a, z);
    if (e != cudaSuccess) return e;
    return tc ? launch_join<__nv_bfloat16>(a, z, n_sm, s) : launch_join<float>(a, z, n_sm, s);
}

}  // namespace ice
