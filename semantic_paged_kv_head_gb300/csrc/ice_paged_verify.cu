// Drafted tokens against the target model's probabilities, or its logits.
#include <algorithm>

#include "ice_paged_verify.cuh"

namespace ice {

// ---------------------------------------------------------------------------
// Speculative sampling (Leviathan et al. 2023, Chen et al. 2023): draft i with token x stays if u_i q_i(x) < p_i(x). The
// first that does not is replaced by a token drawn from max(p - q, 0); behind the last one that stays a token is drawn
// from p. Drawing is by the inverse of the cumulative sum: the first j with w_0 + ... + w_j > u W, W the sum of all.
// Greedy: draft i stays if it is the largest entry's index of row i; the token is that index of the first row where it is not.
//
// A border between two tokens may lie anywhere, so sums have to be near those of exact arithmetic: with 2^17 tokens of
// like weight fp32 sums would move one draw in ten. Sums therefore carry what each addition and each p - q cuts off (two-sum,
// Knuth 1969; within a tile the cheaper form of Dekker 1971): pairs of fp32, off by 2^-38 if every rounding went
// the same way, by 2^-42 as they come. The fp32 pipe and the
// entries' checks, not memory, would else bound short rows in bf16.
//
// No block waits for another in either case. Sampling: several blocks a request. Each finds the first rejected draft by
// itself (K gathers), so that only the one or two rows that decide are read; each warp sums a part of the vocabulary and leaves
// the sum in the handle's scratch, and the last block of a request to have done so draws the token: the part by the
// sums, then that part again, its tiles and at last the elements of a tile.
//
// Greedy: a row is cut into groups of tiles, a warp each; it leaves its group's best entry in the scratch and counts it; the
// warp that counts the last group of a request's last row ends the request. Groups are handed out row by row, all requests' first
// rows first; a warp skips its group when a draft before that row is known not to stay, which changes what is read but
// not the result.
//
// Measured: one request of four drafts on 128000 fp32 entries 7.6 us, three loads that depend on each other, the
// count, and the search. 64 requests of up to seven 16.7 us (57 MB: 3.4 TB/s): the same fixed parts around a warp's three or four
// tiles, each of which is loaded, added up and reduced before the next one's loads; 256 looked-up requests on 50001 bf16 entries
// (about three tiles a warp) 16.3 us, 1000 of them 38. At 64 registers, 1024 threads an SM, the bf16 forms spill 12 bytes. Greedy, 128 requests of up to four drafts on 150001 bf16
// entries 29.8 us, of which 136 MB are read where 94 are needed (rows of the next draft are under way before the verdict on this one); 512 of one draft 45 us, 5.8 TB/s.
// A thread-block cluster a request took as long for the 64 (16 us), but 22 us for the 256 looked-up ones and 61 for the
// greedy ones, whose rows it read one after the other.
// ---------------------------------------------------------------------------
constexpr int kSmpMost = 256;  // threads of a block: these, or half of them
constexpr int kGrdThreads = 128, kGrdWarps = kGrdThreads / 32;
constexpr int kVerVecs = 4;  // 16-byte words of a lane in a tile

template <typename T> constexpr int kVec = 16 / sizeof(T);               // elements of 16 bytes
template <typename T> constexpr int kTile = 32 * kVerVecs * kVec<T>;     // elements of a tile

// What an entry counts for: NaN, negative and huge ones nothing (2^22 of 2^100 have a sum in fp32). As an unsigned number each
// of those is above the bits of 2^100.
constexpr unsigned kMostBits = 0x71800000u;
__device__ __forceinline__ float clean(float x) { return __float_as_uint(x) <= kMostBits ? x : 0.0f; }

__device__ __forceinline__ float clamp_uniform(float u) { return fminf(fmaxf(u, 0.0f), 0.99999994f); }

// 16 bytes at p. Not ALIGNED: p is aligned to an element only, and the 16-byte words around it, which the caller has checked
// to lie in the row, are put together.
template <bool ALIGNED>
__device__ __forceinline__ uint4 load16(const char* p) {
    if (ALIGNED) return __ldcs(reinterpret_cast<const uint4*>(p));
    const unsigned sh = (unsigned)(uintptr_t)p & 15;
    const uint4* b = reinterpret_cast<const uint4*>(p - sh);
    const uint4 x = b[0], y = sh ? b[1] : x;
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

template <typename T> __device__ __forceinline__ void unpack(const uint4& w, float (&v)[kVec<T>]);
template <> __device__ __forceinline__ void unpack<float>(const uint4& w, float (&v)[4]) {
    v[0] = __uint_as_float(w.x), v[1] = __uint_as_float(w.y), v[2] = __uint_as_float(w.z), v[3] = __uint_as_float(w.w);
}
template <> __device__ __forceinline__ void unpack<__nv_bfloat16>(const uint4& w, float (&v)[8]) {
    const unsigned u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(u[i] << 16), v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
}

// A number as a sum of two of fp32, |lo| at most half a step of hi: 48 bits. The fp64 units would bound the kernel: they make two
// additions a cycle and SM.
struct Wide {
    float hi = 0.0f, lo = 0.0f;
};
__device__ __forceinline__ Wide wide_add(Wide a, Wide b) {
    const float s = a.hi + b.hi, t = s - a.hi;
    const float e = ((a.hi - (s - t)) + (b.hi - t)) + (a.lo + b.lo);
    Wide r;
    r.hi = s + e;
    r.lo = e - (r.hi - s);
    return r;
}
__device__ __forceinline__ Wide wide_sub(Wide a, Wide b) {
    b.hi = -b.hi, b.lo = -b.lo;
    return wide_add(a, b);
}
__device__ __forceinline__ Wide wide_mul(float u, Wide a) {
    float p = u * a.hi, e = fmaf(u, a.hi, -p) + u * a.lo;
    if (a.hi < 0x1p-90f) {
        // What the products cut off may lie below the least number, 2^-149. Sums are multiples of that, so the product down to the
        // next multiple has the same sums above it.
        const double x = (double)u * ((double)a.hi + (double)a.lo);
        p = (float)x;
        e = __double2float_rd(x - (double)p);
    }
    Wide r;
    r.hi = p + e;
    r.lo = e - (r.hi - p);
    return r;
}
__device__ __forceinline__ bool wide_less(Wide a, Wide b) { return a.hi < b.hi || (a.hi == b.hi && a.lo < b.lo); }
__device__ __forceinline__ Wide wide_xor(Wide a, int o) {
    Wide r;
    r.hi = __shfl_xor_sync(0xffffffffu, a.hi, o), r.lo = __shfl_xor_sync(0xffffffffu, a.lo, o);
    return r;
}
__device__ __forceinline__ Wide wide_at(Wide a, int lane) {
    Wide r;
    r.hi = __shfl_sync(0xffffffffu, a.hi, lane), r.lo = __shfl_sync(0xffffffffu, a.lo, lane);
    return r;
}
// Sum of the lanes up to each of the first LANES, and (before) up to the one before.
template <int LANES = 32>
__device__ __forceinline__ Wide wide_scan(Wide a, Wide& before) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) {
        Wide y;
        y.hi = __shfl_up_sync(0xffffffffu, a.hi, o), y.lo = __shfl_up_sync(0xffffffffu, a.lo, o);
        if (lane >= o) a = wide_add(y, a);
    }
    before.hi = __shfl_up_sync(0xffffffffu, a.hi, 1), before.lo = __shfl_up_sync(0xffffffffu, a.lo, 1);
    if (lane == 0) before.hi = before.lo = 0.0f;
    return a;
}
__device__ __forceinline__ Wide warp_sum(Wide x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = wide_add(x, wide_xor(x, o));
    return x;
}

// Two fp32 additions in one instruction.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n add.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}\n"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
// a - b, rounded once: b times -1 is exact.
__device__ __forceinline__ float2 sub2(float2 a, float2 b) { return fma2(b, make_float2(-1.0f, -1.0f), a); }

// Two sums of terms >= 0 with the parts that their additions cut off.
struct Sum2 {
    float2 hi = {0.0f, 0.0f}, lo = {0.0f, 0.0f};
    __device__ __forceinline__ void add(float2 d, float2 more) {
        const float2 s = add2(hi, d), t = sub2(s, hi);
        const float2 e = add2(sub2(hi, sub2(s, t)), sub2(d, t));
        hi = s;
        lo = add2(lo, add2(e, more));
    }
    __device__ __forceinline__ Wide value() const {
        Wide a, b, c, d;
        a.hi = hi.x, b.hi = lo.x, c.hi = hi.y, d.hi = lo.y;
        return wide_add(wide_add(a, b), wide_add(c, d));
    }
};

// The two sums of a tile. They begin at `base`, a power of two above every term: what an addition cuts off is then (d - (s - hi)),
// two operations instead of five (Dekker 1971), and base comes off exactly at the end.
struct TileSum {
    float2 hi, lo = {0.0f, 0.0f};
    float base;
    __device__ __forceinline__ explicit TileSum(unsigned most) {  // the largest term's bits, of 2^100 at most
        base = __uint_as_float((most & 0x7f800000u) + 0x00800000u);
        hi = make_float2(base, base);
    }
    __device__ __forceinline__ float2 cut(float2 d) {
        const float2 s = add2(hi, d), e = sub2(d, sub2(s, hi));
        hi = s;
        return e;
    }
    __device__ __forceinline__ void add(float2 p) { lo = add2(lo, cut(p)); }
    // max(p - q, 0) for p, q >= 0, exactly: the difference's own error is (p - d) - q where p >= q
    __device__ __forceinline__ void add_above(float2 p, float2 q) {
        p.x = fmaxf(p.x, q.x), p.y = fmaxf(p.y, q.y);
        const float2 d = sub2(p, q), e = sub2(sub2(p, d), q);
        lo = add2(lo, add2(cut(d), e));
    }
    __device__ __forceinline__ void end(Sum2& s) const { s.add(sub2(hi, make_float2(base, base)), lo); }
};

__device__ __forceinline__ Wide above(float p, float q) {
    p = fmaxf(p, q);
    Wide w;
    w.hi = p - q, w.lo = (p - w.hi) - q;
    return w;
}

template <typename T>
__device__ __forceinline__ Wide weight(const T* p, const T* q, int sure, int j) {
    return above(clean(to_f<T>(p[j])), q != nullptr ? clean(to_f<T>(q[j])) : j == sure ? 1.0f : 0.0f);
}

// The tiles of a row begin at a 16-byte boundary of p, at or before the row's first element: tile t is elements
// t kTile - s and on.
template <typename T>
__device__ __forceinline__ int row_shift(const T* p) { return (int)(((uintptr_t)p & 15) / sizeof(T)); }

// What is taken off the target's entries: nothing, a draft's row, or 1 at the token that the draft was certain of.
enum { kOffNone = 0, kOffRow = 1, kOffSure = 2 };

// 16 bytes of entries from element `at` on, where some of them may lie outside the row: those are `fill`.
template <typename T>
__device__ __forceinline__ uint4 load_end(const T* p, int at, int V, unsigned fill) {
    if (at >= 0 && at + kVec<T> <= V && ((uintptr_t)(p + at) & 15) == 0) return load16<true>(reinterpret_cast<const char*>(p + at));
    unsigned w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i] = fill;
#pragma unroll
        for (int j = 0; j < kVec<T> / 4; ++j) {
            const int k = at + i * (kVec<T> / 4) + j;
            if (k < 0 || k >= V) continue;
            if (sizeof(T) == 4) {
                w[i] = reinterpret_cast<const unsigned*>(p)[k];
            } else {
                const unsigned x = reinterpret_cast<const unsigned short*>(p)[k];
                w[i] = j ? (w[i] & 0xffffu) | x << 16 : (w[i] & 0xffff0000u) | x;
            }
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// What `clean` keeps of 16 bytes of entries.
template <typename T> __device__ __forceinline__ uint4 clean_words(uint4 w);
template <> __device__ __forceinline__ uint4 clean_words<float>(uint4 w) {
    auto f = [](unsigned x) { return x <= kMostBits ? x : 0u; };
    return make_uint4(f(w.x), f(w.y), f(w.z), f(w.w));
}
template <> __device__ __forceinline__ uint4 clean_words<__nv_bfloat16>(uint4 w) {
    auto f = [](unsigned x) { return ((x & 0xffffu) <= kMostBits >> 16 ? x & 0xffffu : 0u) | ((x >> 16) <= kMostBits >> 16 ? x & 0xffff0000u : 0u); };
    return make_uint4(f(w.x), f(w.y), f(w.z), f(w.w));
}

// The entries of a lane's part of a tile, cleaned. Returns the bits of the largest: most tiles hold nothing to be cleaned,
// which that tells.
template <typename T>
__device__ __forceinline__ unsigned most_bits(const uint4 (&x)[kVerVecs]) {
    unsigned m = 0;
#pragma unroll
    for (int i = 0; i < kVerVecs; ++i)
        m = sizeof(T) == 4 ? __vimax3_u32(__vimax3_u32(m, x[i].x, x[i].y), x[i].z, x[i].w)
                           : __vimax3_u16x2(__vimax3_u16x2(m, x[i].x, x[i].y), x[i].z, x[i].w);
    return sizeof(T) == 4 ? m : max(m << 16, m & 0xffff0000u);
}
template <typename T>
__device__ __forceinline__ unsigned clean_tile(uint4 (&x)[kVerVecs]) {
    unsigned m = most_bits<T>(x);
    if (m > kMostBits) {
#pragma unroll
        for (int i = 0; i < kVerVecs; ++i) x[i] = clean_words<T>(x[i]);
        m = most_bits<T>(x);
    }
    return m;
}

// How a tile's entries are loaded: whole tiles, of which the draft's row may begin at another offset of 16 bytes, and a row's ends.
enum { kTileAligned = 0, kTileShifted = 1, kTileEnd = 2 };

template <typename T, int OFF, int HOW>
__device__ __forceinline__ void add_tile_as(const T* p, const T* q, int sure, int V, int e0, Sum2& sum) {
    const int at = e0 + (threadIdx.x & 31) * kVec<T>;
    uint4 x[kVerVecs], y[OFF == kOffRow ? kVerVecs : 1];
#pragma unroll
    for (int i = 0; i < kVerVecs; ++i) {
        const int k = at + i * 32 * kVec<T>;
        if (HOW == kTileEnd) {
            x[i] = load_end<T>(p, k, V, 0u);
            if (OFF == kOffRow) y[i] = load_end<T>(q, k, V, 0u);
        } else {
            x[i] = load16<true>(reinterpret_cast<const char*>(p + k));
            if (OFF == kOffRow) y[i] = load16<HOW == kTileAligned>(reinterpret_cast<const char*>(q + k));
        }
    }
    TileSum s(clean_tile<T>(x));
    if constexpr (OFF == kOffRow) clean_tile<T>(y);
#pragma unroll
    for (int i = 0; i < kVerVecs; ++i) {
        float a[kVec<T>], b[kVec<T>];
        unpack<T>(x[i], a);
        if (OFF == kOffRow) unpack<T>(y[i], b);
#pragma unroll
        for (int j = 0; j < kVec<T>; j += 2) {
            const float2 v = make_float2(a[j], a[j + 1]);
            const int k = at + i * 32 * kVec<T> + j;
            if (OFF == kOffRow) s.add_above(v, make_float2(b[j], b[j + 1]));
            else if (OFF == kOffSure) s.add_above(v, make_float2(k == sure ? 1.0f : 0.0f, k + 1 == sure ? 1.0f : 0.0f));
            else s.add(v);
        }
    }
    s.end(sum);
}

// Adds the lane's weights of a tile.
template <typename T>
__device__ __forceinline__ void add_tile(const T* p, const T* q, int sure, int V, int e0, Sum2& s) {
    const bool inside = e0 >= 0 && e0 + kTile<T> <= V;
    if (q != nullptr) {
        if (inside && ((uintptr_t)(q + e0) & 15) == 0) return add_tile_as<T, kOffRow, kTileAligned>(p, q, sure, V, e0, s);
        if (e0 >= kVec<T> && e0 + kTile<T> + kVec<T> <= V) return add_tile_as<T, kOffRow, kTileShifted>(p, q, sure, V, e0, s);
        return add_tile_as<T, kOffRow, kTileEnd>(p, q, sure, V, e0, s);
    }
    if (inside && !(sure >= e0 && sure < e0 + kTile<T>)) return add_tile_as<T, kOffNone, kTileAligned>(p, q, sure, V, e0, s);
    add_tile_as<T, kOffSure, kTileEnd>(p, q, sure, V, e0, s);
}

// Tiles of part g of a row.
__device__ __forceinline__ void part_of(int tiles, int g, int parts, int& t0, int& t1) {
    t0 = (int)((long long)tiles * g / parts);
    t1 = (int)((long long)tiles * (g + 1) / parts);
}

// The tokens, counts and lengths of a request that has ended, by a warp.
__device__ __forceinline__ void write_request(const Verify& a, int r, int nd, int kept, int token) {
    const int K = a.K;
    const bool part = nd >= 0 && nd <= K;
    for (int i = threadIdx.x & 31; i <= K; i += 32)
        a.out[(long long)r * (K + 1) + i] = !part || i > kept ? -1 : i < kept ? a.tokens[(long long)r * K + i] : token;
    if ((threadIdx.x & 31) == 0) {
        a.accepted[r] = part ? kept : 0;
        a.n_new[r] = part ? kept - nd : 0;
        if (part ? token < 0 : nd != -1) set_status(a.status, ICE_ERR_BOUNDS);
    }
}

struct SampleShared {
    float2 warp[kSmpMost / 32];  // sums, as two numbers
    unsigned some[kSmpMost / 32], over[kSmpMost / 32];
    unsigned keep[2];
    int last;
};

// Over the block: the first thread whose sum reaches beyond x, else the last that has any weight; -1: none has. `before`
// becomes the sum up to that thread, and `all` of all.
struct BlockFind {
    int at;
    Wide before, all;
};
template <int kSmpWarps, typename X>
__device__ __forceinline__ BlockFind block_find(Wide w, X want, SampleShared& sh) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Wide before, base;
    const Wide end = wide_scan(w, before);
    __syncthreads();
    if (lane == 31) sh.warp[warp] = make_float2(end.hi, end.lo);
    __syncthreads();
    BlockFind f;
    Wide of_warp;
    if (lane < kSmpWarps) of_warp.hi = sh.warp[lane].x, of_warp.lo = sh.warp[lane].y;
    const Wide upto = wide_scan<kSmpWarps>(of_warp, base);
    f.all = wide_at(upto, kSmpWarps - 1);
    base = wide_at(base, warp);
    const Wide x = want(f.all);
    const unsigned some = __ballot_sync(0xffffffffu, w.hi > 0.0f);
    const unsigned over = some & __ballot_sync(0xffffffffu, wide_less(x, wide_add(base, end)));
    if (lane == 0) sh.some[warp] = some, sh.over[warp] = over;
    __syncthreads();
    f.at = -1;
    for (int k = kSmpWarps - 1; k >= 0; --k)
        if (f.at < 0 && sh.some[k]) f.at = 32 * k + 31 - __clz(sh.some[k]);
    for (int k = kSmpWarps - 1; k >= 0; --k)
        if (sh.over[k]) f.at = 32 * k + __ffs(sh.over[k]) - 1;
    before = wide_add(base, before);
    if ((int)threadIdx.x == f.at) sh.warp[0] = make_float2(before.hi, before.lo);
    __syncthreads();
    f.before.hi = sh.warp[0].x, f.before.lo = sh.warp[0].y;
    return f;
}

template <typename T, int kSmpThreads>
__global__ void __launch_bounds__(kSmpThreads, 1024 / kSmpThreads) verify_sample_kernel(Verify a) {
    constexpr int kSmpWarps = kSmpThreads / 32;
    __shared__ SampleShared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int blocks = a.blocks, r = blockIdx.x / blocks, chunk = blockIdx.x - r * blocks;
    pdl_wait_then_release();
    const int K = a.K, V = a.V, nd = a.n_draft[r];
    const float* const uniform = a.uniform + (long long)r * (K + 1);
    // asked for together with n_draft
    const int my_token = tid < K ? a.tokens[(long long)r * K + tid] : 0;
    const float my_u = tid < K ? uniform[tid] : 0.0f, u = clamp_uniform(uniform[K]);
    if (nd < 0 || nd > K) {  // a request that takes no part
        if (chunk == 0 && warp == 0) write_request(a, r, nd, 0, -1);
        return;
    }
    const T *const target = (const T*)a.target + r * a.t_req, *const draft = (const T*)a.draft + r * a.d_req;
    if (warp < 2) {  // the drafts that stay: one a lane
        bool stays = false;
        if (tid < nd) {
            const int x = my_token;
            if (x >= 0 && x < V) {
                const float px = clean(to_f<T>(target[tid * a.t_row + x]));
                const float qx = a.draft ? clean(to_f<T>(draft[tid * a.d_row + x])) : 1.0f;
                stays = (double)clamp_uniform(my_u) * (double)qx < (double)px;  // 48 bits: exact
            } else if (chunk == 0) {
                set_status(a.status, ICE_ERR_BOUNDS);
            }
        }
        const unsigned m = __ballot_sync(0xffffffffu, stays);
        if (lane == 0) sh.keep[warp] = m;
    }
    __syncthreads();
    const int kept = __ffsll((long long)~((unsigned long long)sh.keep[1] << 32 | sh.keep[0])) - 1;  // bit 63 is never set
    const T *const p = target + kept * a.t_row, *q = nullptr;
    int sure = -1;
    if (kept < nd) {
        if (a.draft) q = draft + kept * a.d_row;
        else sure = a.tokens[(long long)r * K + kept];
    }
    const int shift = row_shift(p), tiles = (V + shift + kTile<T> - 1) / kTile<T>;
    VerifyScratch* const w = a.scratch + r;
    auto part_sum = [&](int g) {
        int t0, t1;
        part_of(tiles, g, a.groups, t0, t1);
        Sum2 s;
        for (int t = t0; t < t1; ++t) add_tile(p, q, sure, V, t * kTile<T> - shift, s);
        const Wide x = warp_sum(s.value());
        if (lane == 0) __stcg(&w->sum[g], make_float2(x.hi, x.lo));
    };
    {
        int g0, g1;  // this warp's parts
        part_of(a.groups, chunk * kSmpWarps + warp, blocks * kSmpWarps, g0, g1);
        for (int g = g0; g < g1; ++g) part_sum(g);
    }
    __syncthreads();
    if (tid == 0) {
        __threadfence();
        sh.last = atomicAdd(&w->count[0], 1) == blocks - 1;
        __threadfence();
    }
    __syncthreads();
    if (!sh.last) return;
    // the last block of the request. At most twice: where the target is nowhere above the draft, a token of the target's own
    int token = -1;
    for (;;) {
        Wide mine;  // a part a thread
        if (tid < a.groups) {
            const float2 x = __ldcg(&w->sum[tid]);
            mine.hi = x.x, mine.lo = x.y;
        }
        Wide x;
        BlockFind f = block_find<kSmpWarps>(mine, [&](Wide all) { return x = wide_mul(u, all); }, sh);
        if (f.at >= 0) {
            x = wide_sub(x, f.before);
            int t0, t1;
            part_of(tiles, f.at, a.groups, t0, t1);
            // the part's tiles, a warp each
            while (t1 - t0 > 1) {
                const int n = min(t1 - t0, kSmpWarps);
                Wide s;
                if (warp < n) {
                    Sum2 c;
                    add_tile(p, q, sure, V, (t0 + warp) * kTile<T> - shift, c);
                    s = warp_sum(c.value());
                    if (lane != 0) s = Wide();
                }
                f = block_find<kSmpWarps>(s, [&](Wide) { return x; }, sh);
                if (t1 - t0 == n || wide_less(x, f.all)) {
                    if (f.at >= 0) {
                        x = wide_sub(x, f.before);
                        t0 += f.at / 32;
                    }
                    t1 = t0 + 1;
                } else {
                    x = wide_sub(x, f.all);
                    t0 += n;
                }
            }
            // The tile's elements, neighbouring ones a thread. The tiles' sums, added up in another order than the part's, may end just
            // below it, and so lead on to tiles without any weight: the last weight before those is then meant.
            constexpr int E = kTile<T> / kSmpThreads;
            Wide e[E];
            int j;
            for (;;) {
                j = t0 * kTile<T> - shift + E * tid;
                Wide c;
#pragma unroll
                for (int k = 0; k < E; ++k) {
                    e[k] = Wide();
                    if (j + k >= 0 && j + k < V) e[k] = weight(p, q, sure, j + k);
                    c = wide_add(c, e[k]);
                }
                f = block_find<kSmpWarps>(c, [&](Wide) { return x; }, sh);
                if (f.at >= 0 || t0 == 0) break;
                --t0;
                x.hi = INFINITY;
            }
            if (tid == f.at) {
                Wide low = f.before;
#pragma unroll
                for (int k = 0; k < E; ++k) {
                    if (e[k].hi > 0.0f && !(token >= 0 && wide_less(x, low))) {
                        token = j + k;
                        low = wide_add(low, e[k]);
                    }
                }
                sh.last = token;
            }
            if (f.at < 0 && tid == 0) sh.last = -1;
            __syncthreads();
            token = sh.last;
            break;
        }
        if (q == nullptr && sure < 0) break;
        q = nullptr, sure = -1;
        for (int g = warp; g < a.groups; g += kSmpWarps) part_sum(g);
        __threadfence_block();
        __syncthreads();
    }
    if (warp == 0) write_request(a, r, nd, kept, token);
    if (tid == 0) w->count[0] = 0;
}

// Order of the greedy comparison: larger is better, -0 is 0, 0 is nothing (NaN).
__device__ __forceinline__ unsigned greedy_order(float x) {
    const unsigned b = __float_as_uint(x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// The largest of 16 bytes of entries; a NaN is passed over.
template <typename T> __device__ __forceinline__ float largest(const uint4& w);
template <> __device__ __forceinline__ float largest<float>(const uint4& w) {
    return fmaxf(fmaxf(__uint_as_float(w.x), __uint_as_float(w.y)), fmaxf(__uint_as_float(w.z), __uint_as_float(w.w)));
}
template <> __device__ __forceinline__ float largest<__nv_bfloat16>(const uint4& w) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&w);
    const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    return fmaxf(__low2float(m), __high2float(m));
}

// A lane's best entry of the tiles that it has seen, and the first 16 bytes that hold it.
struct Best {
    float x = -INFINITY;
    int word = INT_MIN;  // none yet
};

constexpr unsigned kNothing = 0x7fff7fffu;  // NaN, of either type

template <typename T, bool INSIDE>
__device__ __forceinline__ void best_of_tile(const T* p, int V, int e0, Best& best) {
    const int at = e0 + (threadIdx.x & 31) * kVec<T>;
    uint4 w[kVerVecs];
#pragma unroll
    for (int i = 0; i < kVerVecs; ++i) {
        const int k = at + i * 32 * kVec<T>;
        w[i] = INSIDE ? load16<true>(reinterpret_cast<const char*>(p + k)) : load_end(p, k, V, kNothing);
    }
#pragma unroll
    for (int i = 0; i < kVerVecs; ++i) {
        const float m = largest<T>(w[i]);
        if (m > best.x || (best.word == INT_MIN && m == best.x)) best.x = m, best.word = at + i * 32 * kVec<T>;
    }
}

// The warp's best entry, order and index (the lower is the larger), 0: none. The words that hold it are looked at again for the
// index: most words are not, and a comparison for each entry would cost more than the loads.
template <typename T>
__device__ __forceinline__ unsigned long long warp_best(const T* p, int V, const Best& best) {
    const unsigned x = best.word == INT_MIN ? 0u : greedy_order(best.x), top = __reduce_max_sync(0xffffffffu, x);
    if (top == 0) return 0;
    unsigned j = 0xffffffffu;
    if (x == top) {
        float v[kVec<T>];
        unpack<T>(load_end(p, best.word, V, kNothing), v);
#pragma unroll
        for (int i = kVec<T> - 1; i >= 0; --i)
            if (v[i] == best.x) j = (unsigned)(best.word + i);
    }
    j = __reduce_min_sync(0xffffffffu, j);
    return (unsigned long long)top << 32 | (0xffffffffu - j);
}

template <typename T>
__global__ void __launch_bounds__(kGrdThreads, sizeof(T) == 2 ? 12 : 8) verify_greedy_kernel(Verify a) {
    const int lane = threadIdx.x & 31, K = a.K, V = a.V, G = a.groups;
    const long long warps = (long long)gridDim.x * kGrdWarps, level = (long long)a.n_req * G, items = level * (K + 1);
    pdl_wait_then_release();
    for (long long item = (long long)blockIdx.x * kGrdWarps + (threadIdx.x >> 5); item < items; item += warps) {
        const int i = (int)(item / level);
        const long long rest = item - i * level;
        const int r = (int)(rest / G), g = (int)(rest - (long long)r * G);
        VerifyScratch* const w = a.scratch + r;
        const int nd = a.n_draft[r];
        // Other warps raise `wrong` meanwhile, so its loads may differ by lane: a vote, since the way taken has reductions over the whole
        // warp in it.
        const bool open = __any_sync(0xffffffffu, i <= kVerMaxDrafts + 1 - *(volatile int*)&w->wrong);
        const bool part = nd >= 0 && nd <= K && i <= nd;
        if (part && open) {
            const T* p = (const T*)a.target + r * a.t_req + i * a.t_row;
            Best best;
            int t0, t1;
            const int shift = row_shift(p);
            part_of((V + shift + kTile<T> - 1) / kTile<T>, g, G, t0, t1);
            for (int t = t0; t < t1; ++t) {
                const int e0 = t * kTile<T> - shift;
                if (e0 >= 0 && e0 + kTile<T> <= V) best_of_tile<T, true>(p, V, e0, best);
                else best_of_tile<T, false>(p, V, e0, best);
            }
            const unsigned long long k = warp_best(p, V, best);
            if (lane == 0 && k) atomicMax(&w->best[i], k);
        }
        int last = 0;
        if (lane == 0) {
            __threadfence();
            if (atomicAdd(&w->count[i], 1) == G - 1) {  // the row is complete, or does not matter
                __threadfence();
                if (part) {
                    const unsigned long long k = __ldcg(&w->best[i]);
                    const int x = i < nd ? a.tokens[(long long)r * K + i] : -1;
                    if (i < nd && (x < 0 || x >= V)) set_status(a.status, ICE_ERR_BOUNDS);
                    // a row that some of whose groups were skipped lies behind a wrong one: that stays the first
                    if (k == 0 || x != (int)(0xffffffffu - (unsigned)k)) atomicMax(&w->wrong, kVerMaxDrafts + 1 - i);
                }
                __threadfence();
                last = atomicAdd(&w->rows, 1) == K;
                __threadfence();
            }
        }
        if (!__shfl_sync(0xffffffffu, last, 0)) continue;
        const int kept = kVerMaxDrafts + 1 - __ldcg(&w->wrong);
        const unsigned long long k = nd >= 0 && nd <= K ? __ldcg(&w->best[kept]) : 0ull;
        write_request(a, r, nd, kept, k ? (int)(0xffffffffu - (unsigned)k) : -1);
        __syncwarp();
        for (int x = lane; x <= K; x += 32) w->best[x] = 0, w->count[x] = 0;
        if (lane == 0) w->wrong = w->rows = 0;
    }
}

// Blocks of a request, and whether those of all run at once (1024 threads an SM). With a tile a warp at least the blocks that run
// at once share the requests, where that leaves a warp no more than six tiles (100 requests of 128000 fp32 entries 21.2 us, in waves
// 25.2); else a warp has four, and in several waves one's ends lie beside another's loads (256 of 128000 bf16 entries 29.6 us, in one wave
// 33.3).
template <typename T, int kSmpThreads>
static bool sample_in_one_wave(Verify& a) {
    constexpr int kSmpWarps = kSmpThreads / 32;
    const int tiles = (a.V + kTile<T> - 1) / kTile<T>;
    const int once = 152 * (1024 / kSmpThreads) / a.n_req, want = (tiles + 4 * kSmpWarps - 1) / (4 * kSmpWarps);
    const bool one = 3 * once >= 2 * want;
    a.blocks = std::min(32, one ? std::max(1, std::min(once, (tiles + kSmpWarps - 1) / kSmpWarps)) : want);
    // In one wave each tile is a part of its own (a part a thread of the last block), so that the drawn part needs no search by tiles:
    // 64 requests of 128000 entries 18.7 -> 18.2 us. In more waves the time is that of the sums, and a warp's tiles are one part: 200
    // requests 40.2 -> 37.8.
    const bool parts = a.n_req * a.blocks <= 152 * (1024 / kSmpThreads);
    a.groups = parts ? std::min(kSmpThreads, tiles) : a.blocks * kSmpWarps;
    return one;
}

// Blocks of 256 threads where they run at once and a smaller block's threads would be fewer than the tiles: one request of 128000
// fp32 entries 7.3 us (8.4 with 128). Else of 128: the requests' ends are chains of loads, and more of them are under way (1000
// requests of 50001 bf16 entries 38.3 us, 44.2 with 256; 4000 of 5000 fp32 entries 42.8 and 65.8; 256 looked-up 16.2 and 16.8).
template <typename T>
static cudaError_t launch_sample(Verify a, cudaStream_t s) {
    if (a.V > 128 * kTile<T> && sample_in_one_wave<T, 256>(a))
        return launch_pdl(verify_sample_kernel<T, 256>, dim3(a.n_req * a.blocks), dim3(256), 0, s, a);
    sample_in_one_wave<T, 128>(a);
    return launch_pdl(verify_sample_kernel<T, 128>, dim3(a.n_req * a.blocks), dim3(128), 0, s, a);
}

template <typename T>
static cudaError_t launch_greedy(Verify a, cudaStream_t s) {
    const int tiles = (a.V + kTile<T> - 1) / kTile<T>;
    // groups of four tiles where they are many; the shortest way for few
    const int per = (long long)a.n_req * (a.K + 1) * tiles > 152 * 64 ? 4 : 1;
    a.groups = (tiles + per - 1) / per;
    const long long items = (long long)a.n_req * a.groups * (a.K + 1);
    // a block in turn for each group: what is handed out late can still be skipped
    const dim3 grid((unsigned)std::min<long long>((items + kGrdWarps - 1) / kGrdWarps, 0x7FFFFFFF));
    return launch_pdl(verify_greedy_kernel<T>, grid, dim3(kGrdThreads), 0, s, a);
}

cudaError_t launch_verify(const Verify& a, int dtype, cudaStream_t s) {
    if (dtype == ICE_BF16) return a.uniform ? launch_sample<__nv_bfloat16>(a, s) : launch_greedy<__nv_bfloat16>(a, s);
    return a.uniform ? launch_sample<float>(a, s) : launch_greedy<float>(a, s);
}

}  // namespace ice
