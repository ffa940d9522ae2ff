// Attention of a batch that shares a prefix: the fp32 kernel on the CUDA cores, the joining
// of the parts, and the choice of the parts.
#include <algorithm>
#include <cstring>

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
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float sum = l[j];
#pragma unroll
            for (int d = 8; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            const int r = rg * 4 + j, tok = it.tok0 + r / a.G;
            if (r >= nrow || (it.direct && tok >= valid_tok)) continue;
            const float inv = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);
            const long long R = ((long long)it.slot * a.H + it.h) * a.RP + it.tok0 * a.G + r;
            float* dst = it.direct ? (float*)a.out + ((long long)tok * a.H * a.G + it.h * a.G + r % a.G) * kD
                                   : a.part_o + R * kD;
#pragma unroll
            for (int k = 0; k < 2; ++k)
                *reinterpret_cast<float4*>(dst + 64 * k + kg * 4) =
                    make_float4(o[j][4 * k] * inv, o[j][4 * k + 1] * inv, o[j][4 * k + 2] * inv, o[j][4 * k + 3] * inv);
            if (kg == 0 && !it.direct) a.part_ml[R] = make_float2(m[j], sum);
        }
    }
}

// ---------------------------------------------------------------------------
// Joining: PW warps for a row of a KV head, four dimensions a lane. With parts (m_i, l_i,
// o_i), M = max m_i and w_i = l_i 2^(m_i - M): out = sum w_i o_i / sum w_i, zeros where
// nothing was seen. Rows with one part were written by the attention kernel. Bound by the
// parts' bytes, read once, where there are many rows (PW = 1), and by the latency of
// a chain of loads where there are few: the warps of a row then take every PW-th part.
// ---------------------------------------------------------------------------
constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;

template <typename T>
__device__ __forceinline__ void store4(T* p, float4 v) {
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(p) = v;
    } else {
        __nv_bfloat162 x = __floats2bfloat162_rn(v.x, v.y), y = __floats2bfloat162_rn(v.z, v.w);
        uint2 u;
        memcpy(&u.x, &x, 4);
        memcpy(&u.y, &y, 4);
        *reinterpret_cast<uint2*>(p) = u;
    }
}

template <typename T, int PW>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(PagedAttn a, PagedTiles z) {
    __shared__ float4 red[kJoinWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int group = warp / PW, pw = warp % PW, h = blockIdx.y, G = a.G;
    const int R = blockIdx.x * (kJoinWarps / PW) + group, tok = R / G;
    // Before the wait: q_start and seq_len were complete when the attention kernel's blocks let
    // this one be scheduled (they wait for the kernels before them first).
    int req = 0, nq = -1, own = 0, blk = 0;
    if (tok < a.q_start[a.n_req]) {
        int lo = 0, hi = a.n_req;  // q_start[lo] <= tok < q_start[hi]; 32 probes a step
        while (hi - lo > 1) {
            const int w = (hi - lo + 31) / 32, probe = lo + lane * w;
            const unsigned le = __ballot_sync(0xffffffffu, probe < hi && a.q_start[min(probe, a.n_req)] <= tok);
            const int k = 31 - __clz(le);  // lane 0 always holds
            hi = min(hi, lo + (k + 1) * w);
            lo = lo + k * w;
        }
        const int b = a.q_start[lo];
        req = lo, nq = a.q_start[lo + 1] - b, own = a.seq_len[lo], blk = (tok - b) / z.TB;
    }
    pdl_wait_then_release();
    if (!a.plan[kPlanOk]) return;
    int parts = -1, first = 0;  // -1: nothing to write
    if (nq > z.TS) {
        const PagedLong f = {a.plan[kPlanWhole], a.plan[kPlanSplit]};
        const int blocks = long_blocks(nq, own, z);
        first = a.prefix_splits;
        const bool whole = f.whole == INT_MAX || a.first_long[req] + h * blocks + blk < f.whole;
        parts = blocks == 0 ? 0 : whole || f.split == 1 ? -1 : f.split;
    } else if (nq > 0) {
        const int n = plan_parts(own, a.H, z, a.plan[kPlanChunk]);
        parts = (a.prefix_splits == 0 && n == 1) || a.plan[kPlanDirect] ? -1 : a.prefix_splits + n;
    }
    if (PW == 1 && parts < 0) return;
    const long long step = (long long)a.H * a.RP, row = (long long)first * step + (long long)h * a.RP + R;
    float2 ml[kPagedMaxSlots / 32];  // lane p: parts p, p + 32, ...
    float M = -INFINITY, W = 0.0f;
#pragma unroll
    for (int k = 0; k < kPagedMaxSlots / 32; ++k) {
        const int p = lane + 32 * k;
        ml[k] = p < parts ? a.part_ml[row + p * step] : make_float2(-INFINITY, 0.0f);
        M = fmaxf(M, ml[k].x);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (M == -INFINITY) M = 0.0f;
#pragma unroll
    for (int k = 0; k < kPagedMaxSlots / 32; ++k) {
        ml[k].y *= exp2_approx(ml[k].x - M);
        W += ml[k].y;
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) W += __shfl_xor_sync(0xffffffffu, W, o);
    const float4* src = reinterpret_cast<const float4*>(a.part_o + row * kD) + lane;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < kPagedMaxSlots / 32; ++k) {
        const int end = min(parts - 32 * k, 32);
#pragma unroll 4
        for (int p = pw; p < end; p += PW) {
            const float w = __shfl_sync(0xffffffffu, ml[k].y, p);
            const float4 v = src[(32 * k + p) * step * (kD / 4)];
            acc.x = fmaf(w, v.x, acc.x);
            acc.y = fmaf(w, v.y, acc.y);
            acc.z = fmaf(w, v.z, acc.z);
            acc.w = fmaf(w, v.w, acc.w);
        }
    }
    if (PW > 1) {
        red[warp][lane] = acc;
        __syncthreads();
        if (pw > 0 || parts < 0) return;
#pragma unroll
        for (int k = 1; k < PW; ++k) {
            const float4 v = red[warp + k][lane];
            acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
        }
    }
    const float inv = W > 0.0f ? 1.0f / W : (W == 0.0f ? 0.0f : W);
    store4<T>((T*)a.out + ((long long)tok * a.H * G + h * G + R % G) * kD + lane * 4,
              make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
}

template <typename T>
static cudaError_t launch_join(const PagedAttn& a, const PagedTiles& z, int n_sm, cudaStream_t s) {
    // warps that share a row's parts: as many as bring the warps near 32 a SM
    const long long rows = (long long)a.RP * a.H;
    const dim3 block(kJoinThreads);
    auto grid = [&](int pw) {
        const int per = kJoinWarps / pw;
        return dim3((unsigned)((a.RP + per - 1) / per), (unsigned)a.H);
    };
    if (rows >= 16 * n_sm) return launch_pdl(paged_join_kernel<T, 1>, grid(1), block, 0, s, a, z);
    if (rows >= 4 * n_sm) return launch_pdl(paged_join_kernel<T, 4>, grid(4), block, 0, s, a, z);
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
    a.RP = a.n_tokens * a.G;
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
