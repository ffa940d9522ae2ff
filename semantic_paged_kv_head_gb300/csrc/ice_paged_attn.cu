// Attention of a batch that shares a prefix: the fp32 kernel on the CUDA cores, the joining
// of the parts, and the choice of the parts.
#include <algorithm>
#include <cstring>

#include "ice_paged.cuh"
#include "ice_paged_search.h"

namespace ice {

// ---------------------------------------------------------------------------
// One block takes items in turn: rows (new tokens x G heads) against a range of tiles of 64
// keys, in one pass with a running maximum m and sum l a row: m' = max(m, max_t s_t),
// l' = l 2^(m - m') + sum_t 2^(s_t - m'), and the same factor on the output, with
// s_t = q . k_t log2(e) / sqrt(d). On the CUDA cores: a tensor-core form that keeps fp32's 24 bits takes three
// bf16 terms a value and six products.
//
// More than kFewRows rows (up to 64): the next tile is copied into shared memory while one is worked
// on, and the page ids of the one after are read. A warp has RW rows: a lane makes the scores of
// two keys, and then four dimensions of the output, so that the statistics need shuffles only, and
// the rows' operands are read once a warp. 4 requests of up to 512 tokens on 4k: 1.29 ms, 40 TFLOP/s,
// half of what the fp32 units give; neither they (56 %) nor shared memory (about half, by count) are full. 16 warps
// of half the rows were slower (1.51 ms, spills), operands one step ahead in registers no faster.
//
// Few rows (a decode step's own tokens): bound by memory. The warps take groups of 4 keys in
// turn, 8 lanes a key for the scores and 4 dimensions a lane for the output, straight from
// global memory, the next group's loads under way; their parts meet in shared memory at the end.
// 24 requests of up to 777 own tokens: 14.4 us, of which about 11 us are the call's fixed part
// (plan, first loads, joining).
// ---------------------------------------------------------------------------
constexpr int kSimtThreads = 256;
constexpr int kSimtWarps = kSimtThreads / 32;
constexpr int kSimtRows = 64;
constexpr int kSimtKeys = 64;
constexpr int kFewRows = 8;
constexpr int kSimtStrideK = kD + 4;          // floats a row: consecutive rows 4 banks apart
constexpr int kSimtStrideP = kSimtKeys + 4;
constexpr int kSimtStage = kSimtKeys * (kSimtStrideK + kD);  // floats of a K and a V tile
constexpr int kSimtSmem = 4 * (kSimtRows * kSimtStrideK + 2 * kSimtStage + kSimtRows * kSimtStrideP);
constexpr int kFewFold = 16;  // groups of 4 keys after which a warp's sums are added to those of the groups before
static_assert(kFewRows * kD + kSimtWarps * kFewRows * (kD + 2 + 32 * 12) <= kSimtSmem / 4, "queries, the warps' parts and folds fit");

// Row of the pool of a key of the page list, -1 for a key past its end, -2 for a bad page.
__device__ __forceinline__ int key_row(const PagedAttn& a, const PagedTile& t, int h, int key) {
    if (key >= t.len) return -1;
    const int page = t.table[key / a.P];
    if (page >= 0 && page < a.n_pages) return (page * a.H + h) * a.P + key % a.P;
    set_status(a.status, ICE_ERR_BOUNDS);
    return -2;  // reads as zeros
}

__device__ __forceinline__ void copy16(void* smem, const void* gmem, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((unsigned)__cvta_generic_to_shared(smem)), "l"(gmem),
                 "r"(there ? 16 : 0)
                 : "memory");
}

// Where the output of row r of the item goes; null for a row that is not to be written.
__device__ __forceinline__ float* row_dst(const PagedAttn& a, const PagedStream& it, int r, int valid_tok, float2** ml) {
    const int tok = it.tok0 + r / a.G;
    if (r >= it.ntok * a.G || (it.direct && tok >= valid_tok)) return nullptr;
    const long long R = ((long long)it.slot * a.H + it.h) * a.RP + it.tok0 * a.G + r;
    *ml = it.direct ? nullptr : a.part_ml + R;
    return it.direct ? (float*)a.out + ((long long)tok * a.H * a.G + it.h * a.G + r % a.G) * kD : a.part_o + R * kD;
}

// A row's weight sum as a factor: zeros where nothing was seen.
__device__ __forceinline__ float inverse(float sum) { return sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum); }

__device__ __forceinline__ float4 load_or_zero(const float* base, int row, int off) {
    return row >= 0 ? __ldg(reinterpret_cast<const float4*>(base + (long long)row * kD + off)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n add.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}\n"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float f) {
    float2 d;
    asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %4};\n mul.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}\n"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(f));
    return d;
}
// sum += x with what the rounding cuts off carried in c (Kahan 1965): with plain additions, sums of one sign
// over a million keys of equal weight were off by 0.7 %. Plain ones only within 64 keys.
__device__ __forceinline__ void add_carried(float2& sum, float2& c, float2 x) {
    const float2 y = add2(x, c), t = add2(sum, y);
    c = add2(y, fma2(t, make_float2(-1.0f, -1.0f), sum));
    sum = t;
}
__device__ __forceinline__ void add_carried(float& sum, float& c, float x) {
    const float y = __fadd_rn(x, c), t = __fadd_rn(sum, y);
    c = __fadd_rn(y, __fsub_rn(sum, t));
    sum = t;
}

template <int R>
__device__ __forceinline__ void few_rows(const PagedAttn& a, const PagedTiles& z, const PagedStream& it, int valid_tok,
                                         float* smem) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, kk = lane >> 3, dd = lane & 7;
    const int nrow = it.ntok * a.G;
    float4 acc[R];
    float m[R], l[R];
    float* sq = smem;             // the rows' queries
    float* parts = smem + R * kD; // the warps' parts: [warp][row][d], then m and l
    float4* folds = reinterpret_cast<float4*>(parts + kSimtWarps * R * (kD + 2)) + (warp * R * 32 + lane) * 3;  // [row][32][3]
    bool folded = false;
    // acc, l and what the carried sums of the folds before lack; those refer to the maximum f[2].z
    auto fold = [&](bool last) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float4* f = folds + r * 96;
            float2 lo = make_float2(0.0f, 0.0f), hi = lo, c_lo = lo, c_hi = lo;
            float ls = 0.0f, lc = 0.0f;
            if (folded) {
                const float4 a4 = f[0], c4 = f[1], s4 = f[2];
                const float g = m[r] > -INFINITY ? exp2_approx(s4.z - m[r]) : 0.0f;
                lo = mul2(make_float2(a4.x, a4.y), g), hi = mul2(make_float2(a4.z, a4.w), g);
                c_lo = mul2(make_float2(c4.x, c4.y), g), c_hi = mul2(make_float2(c4.z, c4.w), g);
                ls = s4.x * g, lc = s4.y * g;
            }
            add_carried(lo, c_lo, make_float2(acc[r].x, acc[r].y));
            add_carried(hi, c_hi, make_float2(acc[r].z, acc[r].w));
            add_carried(ls, lc, l[r]);
            if (last) {
                acc[r] = make_float4(lo.x, lo.y, hi.x, hi.y);
                l[r] = ls;
            } else {
                f[0] = make_float4(lo.x, lo.y, hi.x, hi.y);
                f[1] = make_float4(c_lo.x, c_lo.y, c_hi.x, c_hi.y);
                f[2] = make_float4(ls, lc, m[r], 0.0f);
                acc[r] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                l[r] = 0.0f;
            }
        }
        folded = true;
    };
    int lim[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int tok = it.tok0 + r / a.G;
        lim[r] = r < nrow ? min(it.own_len, tok + it.lim_off) : 0;
        m[r] = -INFINITY;
        l[r] = 0.0f;
        acc[r] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    for (int x = threadIdx.x; x < R * (kD / 4); x += kSimtThreads) {
        const int r = x / (kD / 4), c = (x % (kD / 4)) * 4;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (r < nrow)
            v = *reinterpret_cast<const float4*>((const float*)a.q + (it.tok0 + r / a.G) * a.q_stride +
                                                 (it.h * a.G + r % a.G) * kD + c);
        *reinterpret_cast<float4*>(sq + r * kD + c) = v;
    }
    __syncthreads();
    // groups of 4 keys: 16 a tile; the warp takes every kSimtWarps-th
    const int g_end = it.n * (kSimtKeys / 4);
    float4 kv[4] = {}, vv[4] = {};
    int row = -1, key1 = 0, end1 = 0, key = 0, end = 0;  // located group; loaded group
    bool own1 = false, own = false;
    auto locate = [&](int g) {
        const PagedTile t = tile_of(a, z, it, it.kt0 + g / (kSimtKeys / 4));
        key1 = t.key0 + (g % (kSimtKeys / 4)) * 4 + kk;
        own1 = t.own;
        end1 = t.len;
        row = key_row(a, t, it.h, key1);
    };
    auto load = [&]() {
        key = key1, own = own1, end = end1;
#pragma unroll
        for (int i = 0; i < 4; ++i) kv[i] = load_or_zero((const float*)a.k_pages, row, 4 * dd + 32 * i);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            vv[i] = load_or_zero((const float*)a.v_pages, __shfl_sync(0xffffffffu, row, 8 * i), 4 * lane);
    };
    // while a group is worked on, the next one's rows and the page ids of the one after are under way
#pragma unroll 1
    for (int g = warp - 2 * kSimtWarps; g < g_end; g += kSimtWarps) {
        float4 k_now[4], v_now[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) k_now[i] = kv[i], v_now[i] = vv[i];
        const int key_now = key, len_now = end;
        const bool own_now = own;
        if (g + kSimtWarps >= 0 && g + kSimtWarps < g_end) load();
        if (g + 2 * kSimtWarps < g_end) locate(g + 2 * kSimtWarps);
        if (g < 0) continue;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float2 s2 = make_float2(0.0f, 0.0f);  // even and odd dimensions
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 q = *reinterpret_cast<const float4*>(sq + r * kD + 4 * dd + 32 * i);
                s2 = fma2(make_float2(q.x, q.y), make_float2(k_now[i].x, k_now[i].y), s2);
                s2 = fma2(make_float2(q.z, q.w), make_float2(k_now[i].z, k_now[i].w), s2);
            }
            float s = s2.x + s2.y;
#pragma unroll
            for (int o = 4; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            s = key_now < (own_now ? lim[r] : len_now) ? s * a.scale_log2 : -INFINITY;
            float mx = fmaxf(m[r], s);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            const float mu = mx == -INFINITY ? 0.0f : mx;  // nothing seen yet: all weights 0
            const float f = exp2_approx(m[r] - mu), p = exp2_approx(s - mu);
            m[r] = mx;
            l[r] = l[r] * f + p;  // of this lane's key
            float2 lo = make_float2(acc[r].x * f, acc[r].y * f), hi = make_float2(acc[r].z * f, acc[r].w * f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float w = __shfl_sync(0xffffffffu, p, 8 * i);
                lo = fma2(make_float2(w, w), make_float2(v_now[i].x, v_now[i].y), lo);
                hi = fma2(make_float2(w, w), make_float2(v_now[i].z, v_now[i].w), hi);
            }
            acc[r] = make_float4(lo.x, lo.y, hi.x, hi.y);
        }
        if (g / kSimtWarps % kFewFold == kFewFold - 1 && g + kSimtWarps < g_end) fold(false);
    }
    if (folded) fold(true);
    float* sm = parts + kSimtWarps * R * kD;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float sum = l[r];
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        *reinterpret_cast<float4*>(parts + (warp * R + r) * kD + 4 * lane) = acc[r];
        if (lane == 0) {
            sm[(warp * R + r) * 2] = m[r];
            sm[(warp * R + r) * 2 + 1] = sum;
        }
    }
    __syncthreads();
    for (int r = warp; r < R; r += kSimtWarps) {
        float M = -INFINITY, W = 0.0f;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kSimtWarps; ++w) M = fmaxf(M, sm[(w * R + r) * 2]);
        const float mu = M == -INFINITY ? 0.0f : M;
#pragma unroll
        for (int w = 0; w < kSimtWarps; ++w) {
            const float f = exp2_approx(sm[(w * R + r) * 2] - mu);
            const float4 x = *reinterpret_cast<const float4*>(parts + (w * R + r) * kD + 4 * lane);
            W = fmaf(f, sm[(w * R + r) * 2 + 1], W);
            o.x = fmaf(f, x.x, o.x), o.y = fmaf(f, x.y, o.y), o.z = fmaf(f, x.z, o.z), o.w = fmaf(f, x.w, o.w);
        }
        float2* ml;
        float* dst = row_dst(a, it, r, valid_tok, &ml);
        if (dst == nullptr) continue;
        const float inv = inverse(W);
        *reinterpret_cast<float4*>(dst + 4 * lane) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
        if (ml != nullptr && lane == 0) *ml = make_float2(M, W);
    }
}

template <int RW>  // rows a warp: 8 RW rows a block
__device__ __forceinline__ void many_rows(const PagedAttn& a, const PagedTiles& z, const PagedStream& it, int valid_tok,
                                          float* smem) {
    float* sQ = smem;
    float* sKV = sQ + kSimtRows * kSimtStrideK;
    float* sP = sKV + 2 * kSimtStage;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nrow = it.ntok * a.G;
    // a warp copies a row of K and of V at a time; lane i finds its i-th row a tile ahead
    int rows = -1;
    auto locate = [&](int kt) {
        const PagedTile t = tile_of(a, z, it, kt);
        if (lane < kSimtKeys / kSimtWarps) rows = key_row(a, t, it.h, t.key0 + warp + kSimtWarps * lane);
    };
    auto copy_tile = [&](int stage) {
        float* k = sKV + stage * kSimtStage;
        float* v = k + kSimtKeys * kSimtStrideK;
#pragma unroll
        for (int i = 0; i < kSimtKeys / kSimtWarps; ++i) {
            const int r = warp + kSimtWarps * i, row = __shfl_sync(0xffffffffu, rows, i);
            const long long off = (long long)max(row, 0) * kD + 4 * lane;
            copy16(k + r * kSimtStrideK + 4 * lane, (const float*)a.k_pages + off, row >= 0);
            copy16(v + r * kD + 4 * lane, (const float*)a.v_pages + off, row >= 0);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // row r: token tok0 + r / G, head h G + r % G; rows past the item's are zero
    for (int x = tid; x < kSimtWarps * RW * (kD / 4); x += kSimtThreads) {
        const int r = x / (kD / 4), c = (x % (kD / 4)) * 4;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (r < nrow)
            v = *reinterpret_cast<const float4*>((const float*)a.q + (it.tok0 + r / a.G) * a.q_stride +
                                                 (it.h * a.G + r % a.G) * kD + c);
        *reinterpret_cast<float4*>(sQ + r * kSimtStrideK + c) = v;
    }
    float m[RW], l[RW], lc[RW];
    float2 o[RW][2], oc[RW][2];  // dimensions 4 lane .. + 3; oc, lc: what the sums lack
    int lim[RW];
#pragma unroll
    for (int j = 0; j < RW; ++j) {
        m[j] = -INFINITY;
        l[j] = lc[j] = 0.0f;
        const int r = warp * RW + j;
        lim[j] = r < nrow ? min(it.own_len, it.tok0 + r / a.G + it.lim_off) : 0;  // of own tokens
#pragma unroll
        for (int k = 0; k < 2; ++k) o[j][k] = oc[j][k] = make_float2(0.0f, 0.0f);
    }
#pragma unroll 1
    for (int i = -2; i < it.n; ++i) {
        if (i >= -1 && i + 1 < it.n) copy_tile((i + 1) & 1);
        if (i + 2 < it.n) locate(it.kt0 + i + 2);
        if (i < 0) continue;
        const PagedTile tile = tile_of(a, z, it, it.kt0 + i);
        const int key0 = tile.key0;
        const float* sK = sKV + (i & 1) * kSimtStage;
        const float* sV = sK + kSimtKeys * kSimtStrideK;
        if (i + 1 < it.n) asm volatile("cp.async.wait_group 1;" ::: "memory");
        else asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();
        float2 s2[RW][2];  // even and odd dimensions
#pragma unroll
        for (int j = 0; j < RW; ++j)
#pragma unroll
            for (int k = 0; k < 2; ++k) s2[j][k] = make_float2(0.0f, 0.0f);
#pragma unroll 4
        for (int c = 0; c < kD; c += 4) {
            float4 qv[RW], kv[2];
#pragma unroll
            for (int j = 0; j < RW; ++j) qv[j] = *reinterpret_cast<const float4*>(sQ + (warp * RW + j) * kSimtStrideK + c);
#pragma unroll
            for (int k = 0; k < 2; ++k) kv[k] = *reinterpret_cast<const float4*>(sK + (lane + 32 * k) * kSimtStrideK + c);
#pragma unroll
            for (int j = 0; j < RW; ++j)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    s2[j][k] = fma2(make_float2(qv[j].x, qv[j].y), make_float2(kv[k].x, kv[k].y), s2[j][k]);
                    s2[j][k] = fma2(make_float2(qv[j].z, qv[j].w), make_float2(kv[k].z, kv[k].w), s2[j][k]);
                }
        }
#pragma unroll
        for (int j = 0; j < RW; ++j) {
            float mx = m[j];
            const int end = tile.own ? lim[j] : tile.len;
            float s[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                s[k] = key0 + lane + 32 * k < end ? (s2[j][k].x + s2[j][k].y) * a.scale_log2 : -INFINITY;
                mx = fmaxf(mx, s[k]);
            }
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
            const float mu = mx == -INFINITY ? 0.0f : mx;  // nothing seen yet: all weights 0
            const float f = exp2_approx(m[j] - mu);
            m[j] = mx;
            l[j] *= f, lc[j] *= f;
#pragma unroll
            for (int k = 0; k < 2; ++k) o[j][k] = mul2(o[j][k], f), oc[j][k] = mul2(oc[j][k], f);
            float p[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                p[k] = exp2_approx(s[k] - mu);
                sP[(warp * RW + j) * kSimtStrideP + lane + 32 * k] = p[k];
            }
            add_carried(l[j], lc[j], p[0] + p[1]);
        }
        __syncwarp();  // a row's weights are written and read by one warp
        float2 t[RW][2];  // the tile's sums
#pragma unroll
        for (int j = 0; j < RW; ++j) t[j][0] = t[j][1] = make_float2(0.0f, 0.0f);
#pragma unroll 2
        for (int k0 = 0; k0 < kSimtKeys; k0 += 4) {
            float4 pv[RW];
#pragma unroll
            for (int j = 0; j < RW; ++j) pv[j] = *reinterpret_cast<const float4*>(sP + (warp * RW + j) * kSimtStrideP + k0);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float4 v0 = *reinterpret_cast<const float4*>(sV + (k0 + u) * kD + lane * 4);
#pragma unroll
                for (int j = 0; j < RW; ++j) {
                    const float p = u == 0 ? pv[j].x : u == 1 ? pv[j].y : u == 2 ? pv[j].z : pv[j].w;
                    const float2 p2 = make_float2(p, p);
                    t[j][0] = fma2(p2, make_float2(v0.x, v0.y), t[j][0]);
                    t[j][1] = fma2(p2, make_float2(v0.z, v0.w), t[j][1]);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < RW; ++j)
#pragma unroll
            for (int k = 0; k < 2; ++k) add_carried(o[j][k], oc[j][k], t[j][k]);
        __syncthreads();  // the tile's memory is free for the copy after the next
    }
#pragma unroll
    for (int j = 0; j < RW; ++j) {
        float sum = l[j];
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        float2* ml;
        float* dst = row_dst(a, it, warp * RW + j, valid_tok, &ml);
        if (dst == nullptr) continue;
        const float inv = inverse(sum);
        *reinterpret_cast<float4*>(dst + lane * 4) = make_float4(o[j][0].x * inv, o[j][0].y * inv, o[j][1].x * inv, o[j][1].y * inv);
        if (ml != nullptr && lane == 0) *ml = make_float2(m[j], sum);
    }
}

// 208 registers (246 if left to the compiler): the blocks of the joining kernel, 256 threads of 40, then fit beside
// this one and are in place when it ends (24 requests on 4k: 26.0 -> 24.3 us).
__global__ void __maxnreg__(208) paged_simt_kernel(PagedAttn a, PagedTiles z) {
    extern __shared__ __align__(16) float simt_smem[];
    __shared__ PlanShared sh;
    __shared__ PagedItem item;
    __shared__ int s_next;
    int* cum = reinterpret_cast<int*>(simt_smem + kSimtSmem / 4);
    const int tid = threadIdx.x;
    pdl_wait_then_release();
    make_plan<kSimtThreads>(a, z, cum, sh);
    const int n_items = sh.ok ? sh.pre + sh.own : 0;
    const int valid_tok = a.q_start[a.n_req];
    // the block's first item is its own number, the others are handed out
    for (int i = blockIdx.x; i < n_items; i = s_next) {
        if (tid == 0) get_item(a, z, cum, sh, i, item);
        __syncthreads();
        if (tid == 0) s_next = gridDim.x + atomicAdd(&a.next[0], 1u);  // read after the item's last barrier
        const PagedStream it = item.st[0];
        if (item.ns > 0) {
            const int nrow = it.ntok * a.G;
            if (nrow > 32) many_rows<8>(a, z, it, valid_tok, simt_smem);
            else if (nrow > 16) many_rows<4>(a, z, it, valid_tok, simt_smem);
            else if (nrow > kFewRows) many_rows<2>(a, z, it, valid_tok, simt_smem);
            else if (nrow > 2) few_rows<8>(a, z, it, valid_tok, simt_smem);
            else few_rows<2>(a, z, it, valid_tok, simt_smem);
        }
        __syncthreads();
    }
    if (tid == 0) {  // the last block to end leaves the counters at zero
        __threadfence();
        if (atomicAdd(&a.next[1], 1u) == gridDim.x - 1) {
            a.next[0] = 0;
            a.next[1] = 0;
        }
    }
}

// ---------------------------------------------------------------------------
// Joining: PW warps for a row of a KV head, four dimensions a lane. With parts (m_i, l_i,
// o_i), M = max m_i and w_i = l_i 2^(m_i - M): out = sum w_i o_i / sum w_i, zeros where
// nothing was seen. Rows with one part were written by the attention kernel. Bound by the
// parts' bytes, read once, where there are many rows (PW = 1), and by the latency of
// a chain of loads where there are few: the warps of a row then take every PW-th part. 4 requests
// of up to 400 tokens on 8k: 24.2 us cold for 52 MB of parts; decode steps 7 to 14 us cold.
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
    // Nothing is read before the wait, not even q_start and seq_len: that the attention kernel waited for
    // their writer is promised to that kernel's threads only.
    pdl_wait_then_release();
    const int ok = a.plan[kPlanOk], chunk = a.plan[kPlanChunk], direct = a.plan[kPlanDirect];
    const PagedLong f = {a.plan[kPlanWhole], a.plan[kPlanSplit]};
    int req = 0, nq = -1, own = 0, blk = 0;
    if (tok < a.q_start[a.n_req]) {
        RowSearch r(a.n_req);  // beside the load of the verdict, which may be that the lists are out of range
        while (r.open())
            r.narrow(__ballot_sync(0xffffffffu, r.has_probe(lane) && a.q_start[r.probe(lane)] <= tok));
        const int b = a.q_start[r.lo];
        req = r.lo, nq = a.q_start[r.lo + 1] - b, own = a.seq_len[r.lo], blk = (tok - b) / z.TB;
    }
    if (!ok) return;
    int parts = -1, first = 0;  // -1: nothing to write
    if (nq > z.TS) {
        const int blocks = long_blocks(nq, own, z);
        first = a.prefix_splits;
        const bool whole = f.whole == INT_MAX || a.first_long[req] + h * blocks + blk < f.whole;
        parts = blocks == 0 ? 0 : whole || f.split == 1 ? -1 : f.split;
    } else if (nq > 0) {
        const int n = plan_parts(own, a.H, z, chunk);
        parts = (a.prefix_splits == 0 && n == 1) || direct ? -1 : a.prefix_splits + n;
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

// Ranges of the prefix: n_base row blocks x heads, each range a wave's share of tiles, `streams` of
// them side by side. The time of s ranges, in half steps, is taken as waves x (steps of a range +
// the fixed cost of an item), and that of the own items (own_cost each: their lengths are on the
// GPU) that do not fit beside the last wave; the least wins, the fewest ranges among equals.
// Without the own items in the model 16 requests of 500 own tokens at most on 36864 took 48 us (19
// ranges, a full wave), with them 45 us (16).
static int prefix_ranges(long long n_base, int tiles, int limit, int n_sm, int streams, int item_cost, long long own,
                         int own_cost) {
    int best = 1;
    long long best_t = -1;
    for (int s = 1; s <= std::min(limit, tiles); ++s) {
        const long long waves = (n_base * s + n_sm - 1) / n_sm, item = 2 * ((tiles + streams * s - 1) / (streams * s)) + item_cost;
        const long long beside = (waves * n_sm - n_base * s) * (item / own_cost), rest = std::max(0LL, own - beside);
        const long long t = waves * item + (rest + n_sm - 1) / n_sm * own_cost;
        if (best_t < 0 || t < best_t) {
            best_t = t;
            best = s;
        }
    }
    return best;
}

// f32 blocks of 64 rows, or of 32 or 16 while that many more prefix items still fit one wave
// (24 requests of 2 heads on 4k: 64 rows 34 us, 32 rows 24 us; 64 rows a head on 32k with 4 KV
// heads, where blocks of 64 fill the waves: 139 us, blocks of 8 over 400 us).
static PagedTiles simt_tiles(const PagedAttn& a, long long rows_cap, int n_sm) {
    const long long slots = std::min<long long>(rows_cap / ((long long)a.H * a.n_tokens * a.G), kPagedMaxSlots);
    const long long tiles = std::max(1, (a.prefix_len + kSimtKeys - 1) / kSimtKeys);
    const long long ranges = std::min<long long>(std::min<long long>(slots / 2, kPagedMaxPrefixSplits), tiles);
    int rows = kSimtRows;
    while (rows > 16) {
        const int t = rows / 2 / a.G;
        if ((long long)((a.n_tokens + t - 1) / t) * a.H * ranges > n_sm) break;
        rows /= 2;
    }
    return PagedTiles{kSimtKeys, rows / a.G, rows / a.G, 0, 0, 0};
}

cudaError_t launch_paged_attn(PagedAttn a, int dtype, long long rows_cap, int n_sm, cudaStream_t s) {
    const bool tc = dtype == ICE_BF16;
    PagedTiles z = tc ? paged_tc_tiles(a.P, a.G) : simt_tiles(a, rows_cap, n_sm);
    z.NP = (a.prefix_len + z.KT - 1) / z.KT;
    a.RP = a.n_tokens * a.G;
    const int slots = (int)std::min<long long>(rows_cap / ((long long)a.H * a.RP), kPagedMaxSlots);  // >= 3
    const long long n_base = (long long)((a.n_tokens + z.TB - 1) / z.TB) * a.H;
    a.prefix_splits = 0;
    if (a.prefix_len > 0) {
        const int tiles = z.NP, limit = std::min(slots / 2, kPagedMaxPrefixSplits);
        const bool twin = a.n_tokens <= z.TD;  // two parts a range
        // bf16: an item's end takes 7 us with two full row tiles, of 1.25 us a step, and an own item 5;
        // with two parts side by side a step takes 3 us. f32: own items are short beside a tile
        const long long own = tc ? (long long)std::min(a.n_req, a.n_tokens) * ((a.H + 1) / 2) : 0;
        a.prefix_splits = prefix_ranges(n_base, tiles, twin ? std::max(1, limit / 2) : limit, n_sm, twin ? 2 : 1,
                                        !tc ? 6 : twin ? 4 : 12, own, twin ? 5 : 8);
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
