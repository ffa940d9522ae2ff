// New tokens' queries and keys rotated by their positions, keys and values written into the pages.
#include <algorithm>

#include "ice_paged_rope.cuh"
#include "ice_paged_turns.h"

namespace ice {

// ---------------------------------------------------------------------------
// Pair i of a head, (a, b), turns by the angle w_i p, with p the token's position on the pair's axis:
// (a cos - b sin, b cos + a sin). An angle counts modulo whole turns, so w_i / 2 pi is held as a 64-bit
// fraction of a turn and multiplied by p in whole numbers modulo 2^64: the product is right to 2^-65 |p| turns at
// every position of 32 bits (in fp32 an angle of 2^20 radians would be off by 1/16). Of its first 32 bits two, rounded, are the
// quadrant, and the rest, at most an eighth of a turn either way, goes to sincospi in fp32: off by 2^-28 turns at most, less
// near a quadrant's axes, where the sine or the cosine is small (the whole angle in fp32 would be off by 2^-26 there too).
//
// A warp works on one token: its lanes make the 64 pairs' sines and cosines, once for all heads, and pass
// them through shared memory. Then eight lanes take a row (a head's 128 elements of q, k or v), each the two
// pieces of eight elements that its pairs lie in, so that every access is 16 bytes and a row is read and
// written once; six groups of four rows are under way together with bf16, two with fp32. Where tokens are few, `parts` warps share
// the rows of a token.
//
// Bound by memory: 32768 tokens of 32 query and 8 KV heads in bf16 121.5 us, 6.6 TB/s of read and write (98 % of the measured copy
// rate; three groups under way and blocks of 256 threads: 127); 30000 tokens of 8 + 4 heads in fp32 79.0 us (92 %); 64 tokens
// 3.1 us, the launch and two dependent loads.
// ---------------------------------------------------------------------------
constexpr int kRopeThreads = 64, kRopeWarps = kRopeThreads / 32;  // small blocks: an SM that has ended one takes another
constexpr int kRopePairs = 64;

template <typename T> constexpr int kRopeBatch = sizeof(T) == 2 ? 6 : 2;  // groups of four rows under way together

template <typename T> struct RopePiece;  // eight elements as 16-byte words
template <> struct RopePiece<__nv_bfloat16> {
    uint4 w[1];
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const unsigned u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(u[i] << 16);
            v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ void set(const float (&v)[8]) {
        unsigned u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            u[i] = *reinterpret_cast<const unsigned*>(&h);
        }
        w[0] = make_uint4(u[0], u[1], u[2], u[3]);
    }
};
template <> struct RopePiece<float> {
    uint4 w[2];
    __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            v[4 * i] = __uint_as_float(w[i].x);
            v[4 * i + 1] = __uint_as_float(w[i].y);
            v[4 * i + 2] = __uint_as_float(w[i].z);
            v[4 * i + 3] = __uint_as_float(w[i].w);
        }
    }
    __device__ __forceinline__ void set(const float (&v)[8]) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            w[i] = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                              __float_as_uint(v[4 * i + 3]));
    }
};

// Cosine and sine of f / 2^64 turns.
__device__ __forceinline__ float2 cos_sin(unsigned long long f) {
    const unsigned u = (unsigned)((f + 0x80000000ull) >> 32), quadrant = (u + 0x20000000u) >> 30;
    float s, c;
    sincospif((float)(int)(u - (quadrant << 30)) * 0x1p-31f, &s, &c);  // 2^-31: half turns
    const float x = quadrant & 1 ? s : c, y = quadrant & 1 ? c : s;
    return make_float2(quadrant == 1 || quadrant == 2 ? -x : x, quadrant & 2 ? -y : y);
}

template <typename T, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(RopeAppend a) {
    constexpr int W = sizeof(T) == 2 ? 1 : 2;   // 16-byte words of a piece
    constexpr int U = kRopeBatch<T>;
    __shared__ float2 s_cs[kRopeWarps][kRopePairs];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane >> 3, l = lane & 7;
    float2* cs = s_cs[warp];
    // the lane's two pairs
    const unsigned long long turn0 = a.turn[lane], turn1 = a.turn[lane + 32];
    const long long ax0 = a.axis[lane] * a.pos_stride, ax1 = a.axis[lane + 32] * a.pos_stride;
    // the lane's pieces of a row and the pairs in them
    int pa, pb, ia, ib;
    bool rot_a, rot_b;
    const int N = a.n_pairs;
    if (INTER) {  // pair i: elements 2i, 2i + 1
        pa = l, pb = l + 8;
        ia = 4 * pa, ib = 4 * pb;
        rot_a = ia < N, rot_b = ib < N;
    } else {  // pair i: elements i, i + N
        const int n8 = N >> 3;
        rot_a = rot_b = l < n8;
        pa = rot_a ? l : 2 * l;  // the pieces behind the pairs: 2 n8 + 2 (l - n8), and the one after
        pb = rot_a ? l + n8 : pa + 1;
        ia = ib = rot_a ? 8 * l : 0;
    }
    const int rows = a.Hq + 2 * a.H, groups = (rows + 3) >> 2;
    pdl_wait_then_release();
    const int nw = gridDim.x * kRopeWarps / a.parts;  // warps that a part of the tokens' rows has
    const int w = blockIdx.x * kRopeWarps + warp;
    const int part = w % a.parts;
    if (w / a.parts >= nw) return;  // a rest of warps that makes no whole token
    for (long long t = w / a.parts; t < a.n_tokens; t += nw) {
        const long long slot = a.slot_map[t];
        if (slot < 0 || slot >= a.n_slots) {  // the same for the whole warp
            if (slot != -1 && lane == 0) set_status(a.status, ICE_ERR_BOUNDS);
            continue;
        }
        const int p0 = a.positions[ax0 + t], p1 = a.positions[ax1 + t];
        const unsigned page = (unsigned)slot / (unsigned)a.P;  // n_slots < 2^31
        const int off = (int)((unsigned)slot - page * (unsigned)a.P);
        RopePiece<T> x[U][2];
        T* dst[U];
        bool rot[U];
        auto load = [&](int g0) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int r = ((g0 + u * a.parts) << 2) + sub;
                dst[u] = nullptr;
                rot[u] = false;
                if (r >= rows) continue;
                const T* src;
                if (r < a.Hq) {
                    src = (const T*)a.q + t * a.q_stride + r * kD;
                    dst[u] = (T*)a.q_out + t * a.q_out_stride + r * kD;
                    rot[u] = true;
                } else {
                    const bool is_k = r < a.Hq + a.H;
                    const int h = is_k ? r - a.Hq : r - a.Hq - a.H;
                    src = (is_k ? (const T*)a.k + t * a.k_stride : (const T*)a.v + t * a.v_stride) + h * kD;
                    dst[u] = (T*)(is_k ? a.k_pages : a.v_pages) + (((long long)page * a.H + h) * a.P + off) * kD;
                    rot[u] = is_k;
                }
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    x[u][0].w[i] = __ldcs(reinterpret_cast<const uint4*>(src + 8 * pa) + i);
                    x[u][1].w[i] = __ldcs(reinterpret_cast<const uint4*>(src + 8 * pb) + i);
                }
            }
        };
        load(part);
        // the token's sines and cosines
        const unsigned long long f0 = (unsigned long long)((long long)p0 + a.pos_offset) * turn0;
        const unsigned long long f1 = (unsigned long long)((long long)p1 + a.pos_offset) * turn1;
        const float2 c0 = cos_sin(f0), c1 = cos_sin(f1);
        __syncwarp();
        cs[lane] = c0;
        cs[lane + 32] = c1;
        __syncwarp();
        float2 c[8];
        if (INTER) {
#pragma unroll
            for (int i = 0; i < 4; ++i) c[i] = cs[ia + i], c[4 + i] = cs[ib + i];
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) c[i] = cs[ia + i];
        }
        for (int g0 = part; g0 < groups; g0 += U * a.parts) {
            if (g0 != part) load(g0);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (dst[u] == nullptr) continue;
                if (rot[u] && (rot_a || rot_b)) {
                    float va[8], vb[8];
                    x[u][0].get(va);
                    x[u][1].get(vb);
                    if (INTER) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float y = va[2 * i], z = va[2 * i + 1], y2 = vb[2 * i], z2 = vb[2 * i + 1];
                            va[2 * i] = fmaf(y, c[i].x, -z * c[i].y);
                            va[2 * i + 1] = fmaf(z, c[i].x, y * c[i].y);
                            vb[2 * i] = fmaf(y2, c[4 + i].x, -z2 * c[4 + i].y);
                            vb[2 * i + 1] = fmaf(z2, c[4 + i].x, y2 * c[4 + i].y);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float y = va[i], z = vb[i];
                            va[i] = fmaf(y, c[i].x, -z * c[i].y);
                            vb[i] = fmaf(z, c[i].x, y * c[i].y);
                        }
                    }
                    if (rot_a) x[u][0].set(va);
                    if (rot_b) x[u][1].set(vb);
                }
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    reinterpret_cast<uint4*>(dst[u] + 8 * pa)[i] = x[u][0].w[i];
                    reinterpret_cast<uint4*>(dst[u] + 8 * pb)[i] = x[u][1].w[i];
                }
            }
        }
    }
}

cudaError_t launch_rope_append(RopeAppend a, const ice_rope& r, int dtype, cudaStream_t s) {
    for (int i = 0; i < kRopePairs; ++i) {
        a.turn[i] = i < r.n_pairs ? turns(r.freq[i]) : 0;
        a.axis[i] = i < r.n_pairs ? (unsigned char)r.axis[i] : 0;
    }
    a.n_pairs = r.n_pairs;
    // Warps of a token: 16 warps an SM in all while tokens are fewer (each warp makes the token's sines again: 1000 tokens in bf16
    // 6.2 us with 2 warps each, 17.5 with 12; 100 tokens 3.3 with 12, 4.1 with 4)
    const int groups = (a.Hq + 2 * a.H + 3) / 4;
    a.parts = (int)std::max<long long>(1, std::min<long long>(groups, 152LL * 16 / a.n_tokens));
    const long long warps = (long long)a.n_tokens * a.parts;
    const long long most = std::max(152 * 64, (a.parts + kRopeWarps - 1) / kRopeWarps);
    const int blocks = (int)std::min((warps + kRopeWarps - 1) / kRopeWarps, most);
    const dim3 grid(blocks), block(kRopeThreads);
    if (dtype == ICE_BF16)
        return launch_pdl(r.interleaved ? rope_append_kernel<__nv_bfloat16, true> : rope_append_kernel<__nv_bfloat16, false>, grid,
                          block, 0, s, a);
    return launch_pdl(r.interleaved ? rope_append_kernel<float, true> : rope_append_kernel<float, false>, grid, block, 0, s, a);
}

}  // namespace ice
