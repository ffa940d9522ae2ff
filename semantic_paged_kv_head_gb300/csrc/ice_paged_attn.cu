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

__global__ void __launch_bounds__(kSimtThreads) paged_simt_kernel(PagedAttn a) {
    extern __shared__ __align__(16) float simt_smem[];
    __shared__ PlanShared sh;
    float* sQ = simt_smem;
    float* sK = sQ + kSimtRows * kSimtStrideK;
    float* sV = sK + kSimtKeys * kSimtStrideK;
    float* sP = sV + kSimtKeys * kD;
    int* cum = reinterpret_cast<int*>(sP + kSimtRows * kSimtStrideP);
    const int tid = threadIdx.x, rg = tid >> 4, kg = tid & 15;
    const int TB = kSimtRows / a.G;
    pdl_wait_then_release();
    make_plan<kSimtThreads>(a, kSimtKeys, TB, cum, sh);
    if (!sh.ok) return;
    const long long rows_all = (long long)a.n_tokens * a.H * a.G;
    const int valid_tok = a.q_start[a.n_req];
    PagedItem it;
    for (long long i = blockIdx.x; get_item(a, kSimtKeys, TB, cum, sh, i, it); i += gridDim.x) {
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
            lim[j] = r < nrow ? min(it.kv_len, it.tok0 + r / a.G + it.lim_off) : 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) o[j][k] = 0.0f;
        }
        for (int kt = it.kt0; kt < it.kt1; ++kt) {
            const int key0 = kt * kSimtKeys;
            __syncthreads();
            for (int x = tid; x < kSimtKeys * (kD / 4); x += kSimtThreads) {
                const int r = x / (kD / 4), c = (x % (kD / 4)) * 4, key = key0 + r;
                float vk[4] = {0.0f, 0.0f, 0.0f, 0.0f}, vv[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                if (key < it.kv_len) {
                    const int page = it.table[key / a.P];
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
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    s[j][k] = key0 + kg + 16 * k < lim[j] ? s[j][k] * a.scale_log2 : -INFINITY;
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
            for (int t = 0; t < kSimtKeys; t += 4) {
                float4 pv[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    pv[j] = *reinterpret_cast<const float4*>(sP + (rg * 4 + j) * kSimtStrideP + t);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const float4 v0 = *reinterpret_cast<const float4*>(sV + (t + u) * kD + kg * 4);
                    const float4 v1 = *reinterpret_cast<const float4*>(sV + (t + u) * kD + 64 + kg * 4);
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
            const int r = rg * 4 + j;
            if (r >= nrow) continue;
            const int tok = it.tok0 + r / a.G;
            const long long row = (long long)tok * a.H * a.G + it.h * a.G + r % a.G;
            const float inv = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);
            if (it.direct) {
                if (tok >= valid_tok) continue;
                float* dst = (float*)a.out + row * kD;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    dst[kg * 4 + k] = o[j][k] * inv;
                    dst[64 + kg * 4 + k] = o[j][4 + k] * inv;
                }
            } else {
                float* dst = a.part_o + (it.slot * rows_all + row) * kD;
                *reinterpret_cast<float4*>(dst + kg * 4) =
                    make_float4(o[j][0] * inv, o[j][1] * inv, o[j][2] * inv, o[j][3] * inv);
                *reinterpret_cast<float4*>(dst + 64 + kg * 4) =
                    make_float4(o[j][4] * inv, o[j][5] * inv, o[j][6] * inv, o[j][7] * inv);
                if (kg == 0) a.part_ml[it.slot * rows_all + row] = make_float2(m[j], sum);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Joining: a warp per row. With parts (m_i, l_i, o_i), M = max m_i and
// w_i = l_i 2^(m_i - M): out = sum w_i o_i / sum w_i, zeros where nothing was
// seen. Rows with one part were written by the attention kernel.
// ---------------------------------------------------------------------------
constexpr int kJoinThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(PagedAttn a, int KT) {
    pdl_wait_then_release();
    if (!a.plan[kPlanOk]) return;
    const int lane = threadIdx.x & 31, Hq = a.H * a.G;
    const long long row = (long long)blockIdx.x * (kJoinThreads / 32) + (threadIdx.x >> 5);
    const long long rows_all = (long long)a.n_tokens * Hq;
    if (row >= rows_all) return;
    const int tok = (int)(row / Hq);
    // the request of the token: 32 probes a step
    if (tok >= a.q_start[a.n_req]) return;
    int lo = 0, hi = a.n_req;  // q_start[lo] <= tok < q_start[hi]
    while (hi - lo > 1) {
        const int w = (hi - lo + 31) / 32;
        const int probe = lo + lane * w;
        const unsigned le = __ballot_sync(0xffffffffu, probe < hi && a.q_start[min(probe, a.n_req)] <= tok);
        const int k = 31 - __clz(le);  // lane 0 always holds
        hi = min(hi, lo + (k + 1) * w);
        lo = lo + k * w;
    }
    const int own = plan_splits(a.q_start[lo + 1] - a.q_start[lo], a.seq_len[lo], KT, a.plan[kPlanChunk]);
    const int n = a.prefix_splits + own;
    if (n == 1 && (a.prefix_splits == 0 || a.plan[kPlanOwn] == 0)) return;
    float M = -INFINITY;
    for (int i = lane; i < n; i += 32) M = fmaxf(M, a.part_ml[i * rows_all + row].x);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (M == -INFINITY) M = 0.0f;
    float W = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int i = 0; i < n; ++i) {
        const float2 ml = a.part_ml[i * rows_all + row];
        const float w = ml.y * exp2_approx(ml.x - M);
        float v[4];
        load4(a.part_o + (i * rows_all + row) * kD + lane * 4, v);
        W += w;
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[k] = fmaf(w, v[k], acc[k]);
    }
    const float inv = W > 0.0f ? 1.0f / W : (W == 0.0f ? 0.0f : W);
    T* dst = (T*)a.out + row * kD + lane * 4;
#pragma unroll
    for (int k = 0; k < 4; ++k) dst[k] = from_f<T>(acc[k] * inv);
}

static int simt_bytes(int n_req) { return kSimtSmem + (n_req + 1) * 4; }

cudaError_t paged_tables_prepare();
cudaError_t paged_tc_prepare();
int paged_tc_keys(int P);
int paged_tc_tokens(int G);
cudaError_t launch_paged_tc(const PagedAttn& a, int n_sm, cudaStream_t s);

cudaError_t paged_prepare() {
    cudaError_t e = paged_tables_prepare();
    if (e != cudaSuccess) return e;
    e = paged_tc_prepare();
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(paged_simt_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                simt_bytes(kPagedMaxRequests));
}

// Parts of the prefix: n_base row blocks x heads, each part a wave's share of
// tiles. The time of s parts is taken as waves x (tiles of a part + the fixed cost of
// an item, in tiles); the least wins, the fewest parts among equals.
static int prefix_parts(long long n_base, int tiles, int limit, int n_sm) {
    constexpr int kItemCost = 3;
    int best = 1;
    long long best_t = -1;
    for (int s = 1; s <= std::min(std::min(limit, tiles), kPagedMaxPrefixSplits); ++s) {
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
    const long long rows = (long long)a.n_tokens * a.H * a.G;
    const int slots = (int)std::min<long long>(rows_cap / rows, 1 << 20);  // >= 2
    const bool tc = dtype == ICE_BF16;
    const int KT = tc ? paged_tc_keys(a.P) : kSimtKeys, TB = tc ? paged_tc_tokens(a.G) : kSimtRows / a.G;
    const long long n_base = (long long)((a.n_tokens + TB - 1) / TB) * a.H;
    a.prefix_splits =
        a.prefix_len > 0 ? prefix_parts(n_base, (a.prefix_len + KT - 1) / KT, slots - 1, n_sm) : 0;
    a.max_splits = slots - a.prefix_splits;
    a.target_items = 2 * n_sm;
    cudaError_t e;
    if (tc)
        e = launch_paged_tc(a, n_sm, s);
    else
        e = launch_pdl(paged_simt_kernel, dim3(n_sm), dim3(kSimtThreads), (size_t)simt_bytes(a.n_req), s, a);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)((rows + kJoinThreads / 32 - 1) / (kJoinThreads / 32)));
    if (dtype == ICE_BF16)
        return launch_pdl(paged_join_kernel<__nv_bfloat16>, grid, dim3(kJoinThreads), 0, s, a, KT);
    return launch_pdl(paged_join_kernel<float>, grid, dim3(kJoinThreads), 0, s, a, KT);
}

}  // namespace ice
