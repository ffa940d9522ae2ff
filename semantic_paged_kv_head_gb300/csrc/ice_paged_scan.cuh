// Sums over the requests and searches in them, shared by the kernels of block tables.
#pragma once

#include "ice_paged.cuh"

namespace ice {

struct TabSums {
    unsigned v[3][32];
    float f[3][32];
};

// Exclusive block scan of three values below 2^31 per thread and their totals. The sums are
// modulo 2^32; those in fp32 tell whether one has wrapped (every bound that they are held to is below 2^31).
template <int NT>
__device__ __forceinline__ void scan3(unsigned (&x)[3], unsigned (&tot)[3], bool& wrapped, TabSums& sh) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float f[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        const unsigned mine = x[k];
        f[k] = (float)mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned y = __shfl_up_sync(0xffffffffu, x[k], o);
            if (lane >= o) x[k] += y;
            f[k] += __shfl_xor_sync(0xffffffffu, f[k], o);
        }
        if (lane == 31) {
            sh.v[k][warp] = x[k];
            sh.f[k][warp] = f[k];
        }
        x[k] -= mine;
    }
    __syncthreads();
    wrapped = false;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        const unsigned y = lane < NT / 32 ? sh.v[k][lane] : 0u;
        tot[k] = __reduce_add_sync(0xffffffffu, y);
        x[k] += __reduce_add_sync(0xffffffffu, lane < warp ? y : 0u);
        float g = lane < NT / 32 ? sh.f[k][lane] : 0.0f;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) g += __shfl_xor_sync(0xffffffffu, g, o);
        wrapped |= g > 4.0e9f;
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

}  // namespace ice
