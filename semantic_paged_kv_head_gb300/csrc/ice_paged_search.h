// The request of a row: r with q_start[r] <= tok < q_start[r + 1], searched by a warp with 32
// probes a step. Plain arithmetic, so that it also compiles and is tested on the host.
#pragma once

#ifdef __CUDACC__
#define ICE_HD __host__ __device__ __forceinline__
#else
#define ICE_HD inline
#endif

namespace ice {

// 0 <= lo < hi <= n at every step, whatever q_start holds: the lists are read before (or while) they
// are found to be out of range, so no index may depend on their being in order.
struct RowSearch {
    int lo, hi;
    ICE_HD explicit RowSearch(int n) : lo(0), hi(n) {}
    ICE_HD bool open() const { return hi - lo > 1; }
    ICE_HD int width() const { return (hi - lo + 31) / 32; }
    // The entry that a lane compares with tok; a lane past the interval has none.
    ICE_HD int probe(int lane) const { return lo + lane * width(); }
    ICE_HD bool has_probe(int lane) const { return probe(lane) < hi; }
    // le: bit of each lane with a probe whose entry is <= tok. Lane 0's holds for every list that is in
    // order; where it does not, the search goes on in the first interval.
    ICE_HD void narrow(unsigned le) {
        const int w = width();
#ifdef __CUDA_ARCH__
        const int k = 31 - __clz((int)(le | 1u));
#else
        const int k = 31 - __builtin_clz(le | 1u);
#endif
        const int end = lo + (k + 1) * w;
        hi = end < hi ? end : hi;
        lo += k * w;
    }
};

}  // namespace ice
