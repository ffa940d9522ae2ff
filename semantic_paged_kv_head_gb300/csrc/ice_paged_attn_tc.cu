// Attention of a batch that shares a prefix, bf16, on the fifth-generation tensor cores.
#include <algorithm>
#include <climits>
#include <mutex>

#include <cuda.h>

#include "ice_paged.cuh"
#include "ice_select_common.cuh"

namespace ice {

// ---------------------------------------------------------------------------
// One block per SM takes items in turn: one or two streams, each a tile of 128 rows (new
// tokens x G heads) against a range of tiles of KT keys (KT = the whole pages in 128
// keys). For each row tile and key tile
//   S = Q K^T      tcgen05.mma 128 x 128 x 128, accumulator S in tensor memory
//   P = 2^(S c - m) one thread a row: S read back, maximum, weights rounded to
//                  bf16 and written over S
//   O += P V       tcgen05.mma with A = P from tensor memory, V [key][d] as the
//                  N-major operand, accumulator O in tensor memory
// Warps 0-3 and 4-7 do the softmax of stream 0 and 1, warps 8 and 10 issue the
// copies, one thread of warp 9 the matrix products, one of warp 11 hands out the items. The
// products of one thread run in order: a stream's next scores may follow its
// last weights into their columns without a wait. Tensor memory is full: S0 S1 O0 O1,
// 128 columns each.
//
// The two streams are two row tiles of one block (they share the key tile, which is read
// once), or two KV heads, or two halves of a range, so that one's products run while the
// other's weights are made.
//
// The maximum m that the weights refer to moves only when a row's true maximum
// has grown by more than 8 (weights stay below 2^8; bf16 rounds them by 2^-8 of
// themselves at most, whatever their size); only then O is read back and rescaled. The sum
// l is of the rounded weights, the ones that meet V, in fp32. (The product takes both operands in one type, and V is
// bf16; weights in two terms would double it. Error of the output against 64 bits, as norms: 2.3e-3, with
// fp32 weights 1.7e-3, the output's own rounding.)
//
// A product's addition to O cuts off what does not fit O's 24 bits, and the cuts of sums of one sign add up:
// with equal weights O lost 0.4 % over a million keys, 3 % over four. So every kFaFold tiles O and l are
// added, rounded, to sums of their own in the item's rows of the parts, and begin at zero. Between two folds lie
// 8192 products of 16 keys, each of which cuts less than 2^-23: 2^-10 of sum p |v| at most, however long
// the item is.
//
// Pages are read by the tensor memory accelerator, a box of P rows x 64 dimensions
// (128-byte swizzle, the layout that the operand descriptors name), into rings of
// 32 KB stages. Key tiles end where pages do; rows of a stage behind the last key
// are zeroed before they meet weights of zero, whatever the page's free slots hold.
//
// Every wait is bounded (kWaitNs; those for a next item, kWaitNs without progress); when one runs out the block's roles leave their loops,
// what is in flight ends, and the status word says ICE_ERR_TIMEOUT.
//
// Bound by memory with few rows: 4 requests on 250k tokens, 167 us, 6.17 TB/s (91 % of the
// measured copy rate); 16 requests with 16k own tokens each, 178 us, 6.03 TB/s. With 256
// rows or more a key tile is bound by the softmax of its two streams (2500 cycles for 16.8 MFLOP,
// of which the products take 2048): chunks of up to 1021 tokens on 8k, 421 us, 1.24 PFLOP/s (66 %
// of the measured rate). Tried and not kept: key tiles of 64 with two score buffers a stream (twice
// the commits, 1.6 times the time), part of the exponentials as polynomials (the issue slots are
// what is short), weights made before the maximum is known (spills).
// ---------------------------------------------------------------------------
constexpr int kFaThreads = 384;
// registers a thread: 168 at launch, moved from the copy and product warps to the softmax warps.
// 128 x 80 + 256 x 208 = 63488 of the launch's 384 x 168 = 64512.
constexpr int kFaRegsIssue = 80, kFaRegsSoftmax = 208;
static_assert(128 * kFaRegsIssue + 256 * kFaRegsSoftmax <= kFaThreads * 168, "the shares fit the launch's registers");
constexpr int kFaRows = 128;              // rows of a tile (the MMA's M)
constexpr int kFaKeys = 128;              // key rows of a stage (N of S, K of O)
constexpr int kFaTileB = kFaRows * kD * 2;  // 32 KB: Q tile, K or V stage
constexpr int kFaHalfB = kFaTileB / 2;    // 64 dimensions
constexpr int kFaStagesK = 2, kFaStagesV = 2;  // two each: the matrix thread counts in bits
constexpr int kFaStages = kFaStagesK + kFaStagesV;
constexpr float kFaSlack = 8.0f;          // growth of the maximum (log2) that is let pass
constexpr int kFaFold = 1024;             // tiles after which O and l are added to the sums of the tiles before

// What every wait of the block watches: whether one has run out, and the key tiles copied so far.
struct FaWatch {
    int abort;
    unsigned tiles;
};
struct FaShared {
    unsigned long long q_full[4], q_empty[4], k_full[kFaStagesK], k_empty[kFaStagesK], v_full[kFaStagesV], v_empty[kFaStagesV];
    unsigned long long s_full[2], p_ready[2][2], o_done[2], drain;  // p_ready: portions of a tile's weights
    unsigned long long item_full[2], item_empty[2], item_want;
    unsigned tmem;
    FaWatch watch;
    int left[2];  // whether the item exists
    PagedItem item[2];
    PlanShared plan;
};

__host__ __device__ constexpr int fa_smem(int n_req) {
    return 1024 + (2 + kFaStages) * kFaTileB + plan_ints(n_req) * 4;  // with slack for the 1 KB alignment
}

// Shared-memory operand descriptors, 128-byte swizzle: the upper words are constants (1024 B
// between groups of 8 rows, the fixed bit 46, the swizzle), the lower word holds the address / 16
// and the leading offset / 16. K-major (Q, K: rows of 128 B): unused, 1. N-major (V: 64
// dimensions are a row of 128 B): kFaHalfB between the two halves.
#define FA_DESC_HI "0x40004040"
__device__ __forceinline__ unsigned fa_desc_k(unsigned saddr) { return (saddr >> 4) | (1u << 16); }
__device__ __forceinline__ unsigned fa_desc_v(unsigned saddr) { return (saddr >> 4) | ((unsigned)(kFaHalfB >> 4) << 16); }
// fp32 accumulator, bf16 A and B, M = N = 128; bit 16: B is N-major.
constexpr unsigned kFaIdescS = (1u << 4) | (1u << 7) | (1u << 10) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
constexpr unsigned kFaIdescO = kFaIdescS | (1u << 16);

__device__ __forceinline__ void fa_bar_init(unsigned long long* bar, int count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void fa_arrive(unsigned long long* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void fa_expect(unsigned long long* bar, unsigned bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool fa_try(unsigned bar, unsigned parity) {
    unsigned done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}
// Waits for phase `parity`, at most kWaitNs; false if it ran out here or elsewhere in the block
// (then every role leaves its loop). The wall clock is slow to read (a handover between
// warps would wait for it), so it is read every 64th try only.
// item: a wait for the next item or for room for one. A stream without rows and the thread that hands the items
// out wait for as long as an item takes (0.4 s with 30 million keys), so kWaitNs counts from the key tile that
// the block copied last. All others are handovers within a few tiles.
template <bool item>
__device__ __forceinline__ bool fa_wait_long(unsigned bar, unsigned parity, volatile FaWatch* watch) {
    unsigned long long t0 = 0;
    unsigned tiles = 0;
    for (unsigned k = 1;; ++k) {
        if (fa_try(bar, parity)) return true;
        if (k % 64) continue;
        if (watch->abort) return false;
        const unsigned long long t = global_ns();
        if (t0 == 0 || (item && watch->tiles != tiles)) {
            t0 = t;
            if (item) tiles = watch->tiles;
        }
        if (t - t0 > kWaitNs) {
            watch->abort = 1;
            return false;
        }
    }
}
__device__ __forceinline__ bool fa_wait(unsigned long long* b, unsigned parity, volatile FaWatch* watch) {
    return fa_try(smem_u32(b), parity) || fa_wait_long<false>(smem_u32(b), parity, watch);
}
__device__ __forceinline__ bool fa_wait_item(unsigned long long* b, unsigned parity, volatile FaWatch* watch) {
    return fa_try(smem_u32(b), parity) || fa_wait_long<true>(smem_u32(b), parity, watch);
}
__device__ __forceinline__ void fa_commit(unsigned long long* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void fa_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fa_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }

// True in one thread of the (converged) warp. The compiler knows that at most one thread
// passes it, so the product instructions, whose operands are warp-wide registers, need no
// loop over the active threads (with lane == 0 instead, a product took 105 cycles to issue).
__device__ __forceinline__ bool fa_elect() {
    unsigned one;
    asm volatile(
        "{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(one));
    return one != 0;
}

// S = Q K^T of one row tile: 8 steps of 16 dimensions, 32 B along the swizzled rows, the second
// 64 dimensions half a tile on. One statement, so that the operands become warp-wide registers
// once and not at each product.
__device__ __forceinline__ void fa_mma_s(unsigned tmem, unsigned sq, unsigned sk) {
    static_assert(kFaHalfB == 16384, "the offsets below");
    asm volatile(
        "{\n .reg .pred n, p;\n .reg .b32 q, k;\n .reg .b64 dq, dk;\n setp.ne.b32 n, 0, 0;\n setp.eq.b32 p, 0, 0;\n"
        " add.u32 q, %1, 0;\n add.u32 k, %2, 0;\n mov.b64 dq, {q, " FA_DESC_HI "};\n mov.b64 dk, {k, " FA_DESC_HI "};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], dq, dk, %3, n;\n"
        " add.u32 q, %1, 2;\n add.u32 k, %2, 2;\n mov.b64 dq, {q, " FA_DESC_HI "};\n mov.b64 dk, {k, " FA_DESC_HI "};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], dq, dk, %3, p;\n"
        " add.u32 q, %1, 4;\n add.u32 k, %2, 4;\n mov.b64 dq, {q, " FA_DESC_HI "};\n mov.b64 dk, {k, " FA_DESC_HI "};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], dq, dk, %3, p;\n"
        " add.u32 q, %1, 6;\n add.u32 k, %2, 6;\n mov.b64 dq, {q, " FA_DESC_HI "};\n mov.b64 dk, {k, " FA_DESC_HI "};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], dq, dk, %3, p;\n"
        " add.u32 q, %1, 1024;\n add.u32 k, %2, 1024;\n mov.b64 dq, {q, " FA_DESC_HI "};\n mov.b64 dk, {k, " FA_DESC_HI "};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], dq, dk, %3, p;\n"
        " add.u32 q, %1, 1026;\n add.u32 k, %2, 1026;\n mov.b64 dq, {q, " FA_DESC_HI "};\n mov.b64 dk, {k, " FA_DESC_HI "};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], dq, dk, %3, p;\n"
        " add.u32 q, %1, 1028;\n add.u32 k, %2, 1028;\n mov.b64 dq, {q, " FA_DESC_HI "};\n mov.b64 dk, {k, " FA_DESC_HI "};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], dq, dk, %3, p;\n"
        " add.u32 q, %1, 1030;\n add.u32 k, %2, 1030;\n mov.b64 dq, {q, " FA_DESC_HI "};\n mov.b64 dk, {k, " FA_DESC_HI "};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], dq, dk, %3, p;\n"
        "}\n" ::"r"(tmem),
        "r"(fa_desc_k(sq)), "r"(fa_desc_k(sk)), "r"(kFaIdescS)
        : "memory");
}
// O (+)= P V over keys 0 .. 95 and 96 .. 127 of a tile: steps of 16 keys, each 8 columns of packed
// weights and 2048 B of V rows.
__device__ __forceinline__ void fa_mma_o_first(unsigned tmem_o, unsigned tmem_p, unsigned sv, bool add) {
    asm volatile(
        "{\n .reg .pred n, p;\n .reg .b32 v, w;\n .reg .b64 dv;\n setp.ne.b32 n, %4, 0;\n setp.eq.b32 p, 0, 0;\n"
        " add.u32 v, %2, 0;\n add.u32 w, %1, 0;\n mov.b64 dv, {v, " FA_DESC_HI "};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [w], dv, %3, n;\n"
        " add.u32 v, %2, 128;\n add.u32 w, %1, 8;\n mov.b64 dv, {v, " FA_DESC_HI "};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [w], dv, %3, p;\n"
        " add.u32 v, %2, 256;\n add.u32 w, %1, 16;\n mov.b64 dv, {v, " FA_DESC_HI "};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [w], dv, %3, p;\n"
        " add.u32 v, %2, 384;\n add.u32 w, %1, 24;\n mov.b64 dv, {v, " FA_DESC_HI "};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [w], dv, %3, p;\n"
        " add.u32 v, %2, 512;\n add.u32 w, %1, 32;\n mov.b64 dv, {v, " FA_DESC_HI "};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [w], dv, %3, p;\n"
        " add.u32 v, %2, 640;\n add.u32 w, %1, 40;\n mov.b64 dv, {v, " FA_DESC_HI "};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [w], dv, %3, p;\n"
        "}\n" ::"r"(tmem_o),
        "r"(tmem_p), "r"(fa_desc_v(sv)), "r"(kFaIdescO), "r"(add ? 1u : 0u)
        : "memory");
}
__device__ __forceinline__ void fa_mma_o_rest(unsigned tmem_o, unsigned tmem_p, unsigned sv, bool add) {
    asm volatile(
        "{\n .reg .pred n, p;\n .reg .b32 v, w;\n .reg .b64 dv;\n setp.ne.b32 n, %4, 0;\n setp.eq.b32 p, 0, 0;\n"
        " add.u32 v, %2, 768;\n add.u32 w, %1, 48;\n mov.b64 dv, {v, " FA_DESC_HI "};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [w], dv, %3, n;\n"
        " add.u32 v, %2, 896;\n add.u32 w, %1, 56;\n mov.b64 dv, {v, " FA_DESC_HI "};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [w], dv, %3, p;\n"
        "}\n" ::"r"(tmem_o),
        "r"(tmem_p), "r"(fa_desc_v(sv)), "r"(kFaIdescO), "r"(add ? 1u : 0u)
        : "memory");
}

// fa_mma_o_rest, then the stream's next scores (their columns hold the weights until then) and the
// commit of them: the stretch that a stream waits for, in one statement.
__device__ __forceinline__ void fa_mma_o_rest_s(unsigned tmem_o, unsigned tmem_s, unsigned sv, unsigned sq, unsigned sk,
                                                unsigned long long* bar) {
    asm volatile(
        "{\n .reg .pred n, p;\n .reg .b32 v, w, q, k;\n .reg .b64 dv, dq, dk;\n setp.ne.b32 n, 0, 0;\n setp.eq.b32 p, 0, 0;\n"
        " add.u32 v, %2, 768;\n add.u32 w, %1, 48;\n mov.b64 dv, {v, " FA_DESC_HI "};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [w], dv, %3, p;\n"
        " add.u32 v, %2, 896;\n add.u32 w, %1, 56;\n mov.b64 dv, {v, " FA_DESC_HI "};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [w], dv, %3, p;\n"
        " add.u32 q, %4, 0;\n add.u32 k, %5, 0;\n mov.b64 dq, {q, " FA_DESC_HI "};\n mov.b64 dk, {k, " FA_DESC_HI "};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%1], dq, dk, %6, n;\n"
        " add.u32 q, %4, 2;\n add.u32 k, %5, 2;\n mov.b64 dq, {q, " FA_DESC_HI "};\n mov.b64 dk, {k, " FA_DESC_HI "};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%1], dq, dk, %6, p;\n"
        " add.u32 q, %4, 4;\n add.u32 k, %5, 4;\n mov.b64 dq, {q, " FA_DESC_HI "};\n mov.b64 dk, {k, " FA_DESC_HI "};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%1], dq, dk, %6, p;\n"
        " add.u32 q, %4, 6;\n add.u32 k, %5, 6;\n mov.b64 dq, {q, " FA_DESC_HI "};\n mov.b64 dk, {k, " FA_DESC_HI "};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%1], dq, dk, %6, p;\n"
        " add.u32 q, %4, 1024;\n add.u32 k, %5, 1024;\n mov.b64 dq, {q, " FA_DESC_HI "};\n mov.b64 dk, {k, " FA_DESC_HI "};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%1], dq, dk, %6, p;\n"
        " add.u32 q, %4, 1026;\n add.u32 k, %5, 1026;\n mov.b64 dq, {q, " FA_DESC_HI "};\n mov.b64 dk, {k, " FA_DESC_HI "};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%1], dq, dk, %6, p;\n"
        " add.u32 q, %4, 1028;\n add.u32 k, %5, 1028;\n mov.b64 dq, {q, " FA_DESC_HI "};\n mov.b64 dk, {k, " FA_DESC_HI "};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%1], dq, dk, %6, p;\n"
        " add.u32 q, %4, 1030;\n add.u32 k, %5, 1030;\n mov.b64 dq, {q, " FA_DESC_HI "};\n mov.b64 dk, {k, " FA_DESC_HI "};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%1], dq, dk, %6, p;\n"
        " tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%7];\n}\n" ::"r"(tmem_o),
        "r"(tmem_s), "r"(fa_desc_v(sv)), "r"(kFaIdescO), "r"(fa_desc_k(sq)), "r"(fa_desc_k(sk)), "r"(kFaIdescS), "r"(smem_u32(bar))
        : "memory");
}

// N columns of the warp's 32 lanes of tensor memory, as register bits.
__device__ __forceinline__ void fa_ld(unsigned addr, unsigned (&u)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
                 "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15"
                 "}, [%16];"
                 : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
                   "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void fa_st(unsigned addr, const unsigned (&u)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {"
                 "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15"
                 "};" ::"r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
                 "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]),
                 "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void fa_ld(unsigned addr, unsigned (&u)[32]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
                 "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31"
                 "}, [%32];"
                 : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
                   "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]),
                   "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]),
                   "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void fa_st(unsigned addr, const unsigned (&u)[32]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {"
                 "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31"
                 "};" ::"r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
                 "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]), "r"(u[16]), "r"(u[17]), "r"(u[18]),
                 "r"(u[19]), "r"(u[20]), "r"(u[21]), "r"(u[22]), "r"(u[23]), "r"(u[24]), "r"(u[25]), "r"(u[26]), "r"(u[27]),
                 "r"(u[28]), "r"(u[29]), "r"(u[30]), "r"(u[31]),
                 "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void fa_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fa_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ unsigned fa_pack(float lo, float hi) {
    unsigned u;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u) : "f"(hi), "f"(lo));
    return u;
}

__device__ __forceinline__ float fa_max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// Adds the two bf16 values of u to x and y in fp32.
__device__ __forceinline__ void fa_add_pair(float& x, float& y, unsigned u) {
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n add.rn.f32.bf16 %0, a, %0;\n add.rn.f32.bf16 %1, b, %1;\n}\n"
        : "+f"(x), "+f"(y)
        : "r"(u));
}

// The pages of a key tile as rows of the pool's tensor map, page p in lane p % 32.
struct FaPages {
    int n, row[4];
    __device__ __forceinline__ void fetch(const PagedAttn& a, const PagedTiles& z, const int* own_table, int own_len,
                                          int head, int x, int lane) {
        const bool own = x >= z.NP;
        const int* table = own ? own_table : a.prefix_table;
        const int page0 = (own ? x - z.NP : x) * z.pages;
        n = min(z.pages, ceil_div(own ? own_len : a.prefix_len, a.P) - page0);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int p = lane + 32 * u;
            row[u] = (int)(a.n_pages * a.H * a.P);  // past the pool: reads as zeros
            if (p < n) {
                const int id = table[page0 + p];
                if (id >= 0 && id < a.n_pages) row[u] = (id * a.H + head) * a.P;
                else set_status(a.status, ICE_ERR_BOUNDS);
            }
        }
    }
};

// Adds O and l of a warp's rows to the sums of the folds before. Those, and the maximum that they refer to, are
// the row's part (a row that writes its output itself has one too, in a slot that no other item uses).
// The last fold's sums become O and the returned l as well. By way of O, not in the output's loop: the
// code is small then, and the calls that never fold lose 0.2 us (1.2 us with 16 requests on 36864 otherwise).
__device__ __forceinline__ float fa_fold(unsigned t_o, float* part_o, float2* part_ml, bool mine, bool first, bool last, float m, float l) {
    float f = 0.0f;
    if (mine) {
        if (!first) {
            const float2 x = *part_ml;
            f = m > -INFINITY ? exp2_approx(x.x - m) : 0.0f;
            l = fmaf(x.y, f, l);
        }
        *part_ml = make_float2(m, l);
    }
#pragma unroll 1
    for (int k = 0; k < kD; k += 16) {
        unsigned u[16];
        fa_ld(t_o + k, u);
        fa_wait_ld();
        if (mine) {
            float4* sum = reinterpret_cast<float4*>(part_o + k);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (!first) x = sum[c];
                x.x = fmaf(x.x, f, __uint_as_float(u[4 * c])), x.y = fmaf(x.y, f, __uint_as_float(u[4 * c + 1]));
                x.z = fmaf(x.z, f, __uint_as_float(u[4 * c + 2])), x.w = fmaf(x.w, f, __uint_as_float(u[4 * c + 3]));
                sum[c] = x;
                u[4 * c] = __float_as_uint(x.x), u[4 * c + 1] = __float_as_uint(x.y);
                u[4 * c + 2] = __float_as_uint(x.z), u[4 * c + 3] = __float_as_uint(x.w);
            }
        }
        __syncwarp();  // the next columns are read by the whole warp
        if (last) fa_st(t_o + k, u);
    }
    if (last) fa_wait_st();
    return l;
}

// Query tiles, one a stream: the p-th has slot p % 2. A tile of kFaFew rows or less is read as a
// box of kFaFew rows; the product reads 128 rows from it on, of which the others do
// not matter. Two of them in a slot lie 1 KB apart, so that the next item's queries arrive
// while this one's are in use.
constexpr int kFaFew = 8;
__device__ __forceinline__ unsigned fa_q_off(unsigned p, bool few) {
    return (p & 1) * kFaTileB + (few ? ((p >> 1) & 1) * 1024 : 0);
}

// The items of a block, read by its warps from a ring of two that warp 11 fills. An item is
// taken when kFaAhead tiles of the one before are left to copy, not earlier: a block in a
// long item would keep a second one waiting that another block could have begun.
constexpr int kFaAhead = 4;
constexpr int kFaReaders = 11;  // warps 0 .. 10
struct FaItems {
    unsigned cnt = 0;
    // One warp, or its one active thread (whole = false). False at the end or when a wait ran out (ok = false).
    __device__ __forceinline__ bool next(FaShared& sh, PagedItem& it, bool& ok, bool whole) {
        const unsigned k = cnt & 1;
        bool got = fa_wait_item(&sh.item_full[k], (cnt >> 1) & 1, &sh.watch);
        if (whole) got = __all_sync(0xffffffffu, got);
        if (!got) {
            ok = false;
            return false;
        }
        ++cnt;
        const bool left = sh.left[k] != 0;
        it = sh.item[k];
        if (whole) __syncwarp();
        if (!whole || (threadIdx.x & 31) == 0) fa_arrive(&sh.item_empty[k]);
        return left;
    }
};

__global__ void __launch_bounds__(kFaThreads, 1)
    paged_tc_kernel(PagedAttn a, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mf,
                    const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, PagedTiles z) {
    extern __shared__ unsigned char fa_raw[];
    __shared__ __align__(8) FaShared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const unsigned raw0 = smem_u32(fa_raw);
    const unsigned base = (raw0 + 1023u) & ~1023u;  // the swizzle's pattern repeats every 1024 B
    unsigned char* mem = fa_raw + (base - raw0);
    const unsigned s_q = base, s_k = base + 2 * kFaTileB, s_v = s_k + kFaStagesK * kFaTileB;
    int* cum = reinterpret_cast<int*>(mem + (2 + kFaStages) * kFaTileB);
    const int KT = z.KT;
    if (tid == 0) {
        sh.watch.abort = 0;
        sh.watch.tiles = 0;
        for (int k = 0; k < 4; ++k) {
            fa_bar_init(&sh.q_full[k], 1);
            fa_bar_init(&sh.q_empty[k], 1);
        }
        for (int k = 0; k < kFaStagesK; ++k) {
            fa_bar_init(&sh.k_full[k], 1);
            fa_bar_init(&sh.k_empty[k], 1);
        }
        for (int k = 0; k < kFaStagesV; ++k) {
            fa_bar_init(&sh.v_full[k], 1);
            fa_bar_init(&sh.v_empty[k], 1);
        }
        for (int k = 0; k < 2; ++k) {
            fa_bar_init(&sh.s_full[k], 1);
            for (int h = 0; h < 2; ++h) fa_bar_init(&sh.p_ready[k][h], 4);
            fa_bar_init(&sh.o_done[k], 1);
            fa_bar_init(&sh.item_full[k], 1);
            fa_bar_init(&sh.item_empty[k], kFaReaders);
        }
        fa_bar_init(&sh.item_want, 1);
        fa_bar_init(&sh.drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sh.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // rows of a stage that no page reaches (P does not divide 128) stay zero
    for (int x = tid; x < (kFaKeys - KT) * 8 * 2 * kFaStages; x += kFaThreads) {
        const int c = x & 7, half = (x >> 3) % (2 * kFaStages), row = KT + (x >> 3) / (2 * kFaStages);
        *reinterpret_cast<uint4*>(mem + 2 * kFaTileB + half * kFaHalfB + row * 128 + c * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    fa_before();
    pdl_wait_then_release();
    make_plan<kFaThreads>(a, z, cum, sh.plan);  // its barriers also publish the setup
    fa_after();
    const unsigned tmem = sh.tmem;
    volatile FaWatch* watch = &sh.watch;
    PagedItem it;
    FaItems items;
    bool ok = true;
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFaRegsIssue));
        if (warp == 8 || warp == 10) {
            // ---- copies: warp 8 queries and keys, warp 10 values ----
            const bool is_k = warp == 8;
            const int stages = is_k ? kFaStagesK : kFaStagesV;
            unsigned long long* full = is_k ? sh.k_full : sh.v_full;
            unsigned long long* empty = is_k ? sh.k_empty : sh.v_empty;
            const unsigned dst0 = is_k ? s_k : s_v;
            const unsigned long long map = reinterpret_cast<unsigned long long>(is_k ? &mk : &mv);
            unsigned cnt = 0, qcnt = 0;  // key or value tiles and query tiles issued
            unsigned last_few = 0;       // bit k: the query tile k + 1 before was of few rows
            while (ok && items.next(sh, it, ok, true)) {
                const int n1 = it.ns == 2 && !it.shared ? it.st[1].n : 0;
                const int n = it.ns > 0 ? it.st[0].n + n1 : 0;  // tiles to copy
                if (is_k && n <= kFaAhead && lane == 0) fa_arrive(&sh.item_want);
                if (n == 0) continue;
                // the x-th tile in the order of use: two lists take turns
                const int turns = 2 * min(it.st[0].n, n1);
                FaPages next;  // of the next tile, fetched a tile ahead
                auto fetch = [&](int x) {
                    int j = x;
                    bool second = false;
                    if (n1 > 0) {
                        j = x < turns ? x >> 1 : x - (turns >> 1);
                        second = x < turns ? (x & 1) : n1 > it.st[0].n;
                    }
                    next.fetch(a, z, second ? it.st[1].own_table : it.st[0].own_table,
                               second ? it.st[1].own_len : it.st[0].own_len, second ? it.st[1].h : it.st[0].h,
                               (second ? it.st[1].kt0 : it.st[0].kt0) + j, lane);
                };
#pragma unroll 1
                for (int x = -1; x < n; ++x) {
                    const FaPages cur = next;
                    if (x + 1 < n) fetch(x + 1);
                    if (x < 0) {
                        if (is_k) {
                            for (int t = 0; ok && t < (it.same_q ? 1 : it.ns); ++t) {
                                const PagedStream st = t ? it.st[1] : it.st[0];
                                if (st.n == 0) continue;
                                // free once the tile before in the slot is used up, or the one before that
                                // where those in between and this one are of few rows
                                const bool few = st.ntok * a.G <= kFaFew;
                                const unsigned back = few && (last_few & 2) ? 4 : 2;
                                if (qcnt >= back) {
                                    const unsigned w = qcnt - back;
                                    ok = __all_sync(0xffffffffu, fa_wait(&sh.q_empty[w & 3], (w >> 2) & 1, watch));
                                }
                                if (ok && fa_elect()) {
                                    unsigned long long* bar = &sh.q_full[qcnt & 3];
                                    fa_expect(bar, few ? kFaFew * kD * 2 : kFaTileB);
                                    for (int h = 0; h < 2; ++h)
                                        asm volatile(
                                            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
                                                s_q + fa_q_off(qcnt, few) + h * kFaHalfB),
                                            "l"(few ? reinterpret_cast<unsigned long long>(&mf) : reinterpret_cast<unsigned long long>(&mq)),
                                            "r"(h * 64), "r"(st.h * a.G), "r"(st.tok0), "r"(smem_u32(bar))
                                            : "memory");
                                }
                                __syncwarp();
                                ++qcnt;
                                last_few = (last_few << 1) | (few ? 1 : 0);
                            }
                            if (!ok) break;
                        }
                        continue;
                    }
                    if (is_k && n > kFaAhead && x == n - kFaAhead && lane == 0) fa_arrive(&sh.item_want);
                    const unsigned st = cnt % stages;
                    ok = __all_sync(0xffffffffu, fa_wait(&empty[st], ((cnt / stages) & 1) ^ 1, watch));
                    if (!ok) break;
                    const unsigned bar = smem_u32(&full[st]), dst = dst0 + st * kFaTileB;
                    if (lane == 0) {
                        // ICE_DEBUG_STALL_ATTN: the last key tile of the first block's first item with any expects 16 bytes that no
                        // copy delivers, so that the waits for it run out
                        const bool stall = a.debug && is_k && blockIdx.x == 0 && x == n - 1 && cnt == (unsigned)x;
                        fa_expect(&full[st], (unsigned)(cur.n * a.P * kD * 2) + (stall ? 16u : 0u));
                        if (is_k) watch->tiles = cnt + 1;
                    }
                    __syncwarp();
                    // one thread issues all boxes
#pragma unroll 1
                    for (int p = 0; p < cur.n; ++p) {
                        const int mine = p < 32 ? cur.row[0] : p < 64 ? cur.row[1] : p < 96 ? cur.row[2] : cur.row[3];
                        const int row = __shfl_sync(0xffffffffu, mine, p & 31);
                        if (fa_elect()) {
                            const unsigned to = dst + p * a.P * 128;
                            asm volatile(
                                "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(to),
                                "l"(map), "r"(0), "r"(row), "r"(bar)
                                : "memory");
                            asm volatile(
                                "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(to + kFaHalfB),
                                "l"(map), "r"(64), "r"(row), "r"(bar)
                                : "memory");
                        }
                    }
                    __syncwarp();
                    ++cnt;
                }
            }
            // copies in flight land (bounded) before the block ends, whatever ended the loop
            if (lane == 0) {
                if (!ok) set_status(a.status, ICE_ERR_TIMEOUT);
                for (unsigned k = qcnt > 4 ? qcnt - 4 : 0; k < qcnt; ++k)
                    mbar_wait_bounded(smem_u32(&sh.q_full[k & 3]), (k >> 2) & 1);
                for (unsigned k = cnt > (unsigned)stages ? cnt - stages : 0; k < cnt; ++k)
                    mbar_wait_bounded(smem_u32(&full[k % stages]), (k / stages) & 1);
            }
        } else if (warp == 11) {
            // ---- items: the block's first is its own number, the others are handed out ----
            if (fa_elect()) {
                const int n_items = sh.plan.ok ? sh.plan.pre + sh.plan.own : 0;
                int i = blockIdx.x;
                for (unsigned c = 0;; ++c) {
                    const unsigned k = c & 1;
                    if ((c > 0 && !fa_wait_item(&sh.item_want, (c - 1) & 1, watch)) ||
                        !fa_wait_item(&sh.item_empty[k], ((c >> 1) & 1) ^ 1, watch)) {
                        set_status(a.status, ICE_ERR_TIMEOUT);
                        break;
                    }
                    if (c > 0) i = gridDim.x + atomicAdd(&a.next[0], 1u);
                    const bool left = i < n_items;
                    if (left) get_item(a, z, cum, sh.plan, i, sh.item[k]);
                    sh.left[k] = left;
                    fa_arrive(&sh.item_full[k]);
                    if (!left) break;
                }
            }
            __syncwarp();
        } else if (fa_elect()) {
            // ---- matrix products (one thread of warp 9) ----
            unsigned kn = 0, vn = 0, qn = 0, pn0 = 0, pn1 = 0;  // tiles used, weights used by stream
            while (ok && items.next(sh, it, ok, false)) {
                const int ns = it.ns, n0 = ns > 0 ? it.st[0].n : 0, n1 = ns > 1 ? it.st[1].n : 0;
                const int n = max(n0, n1);
                if (n == 0) continue;
                // query tiles: number, address
                const unsigned q0 = qn, q1 = it.same_q || n0 == 0 ? qn : qn + 1;
                const unsigned sq0 = s_q + fa_q_off(q0, it.st[0].ntok * a.G <= kFaFew);
                const unsigned sq1 = s_q + fa_q_off(q1, it.st[1].ntok * a.G <= kFaFew);
                qn = n1 > 0 ? q1 + 1 : q0 + 1;
                if (it.shared) {
                    // two row tiles on the same key tiles: this thread's own instructions are on the
                    // path, so a round is written out (rounds of the loop below: 3 % slower)
                    const unsigned t0 = tmem, t1 = tmem + 128, o0 = tmem + 256, o1 = tmem + 384;
                    unsigned ks = kn & 1, sk = s_k + ks * kFaTileB;
                    ok = fa_wait(&sh.q_full[q0 & 3], (q0 >> 2) & 1, watch) &&
                         fa_wait(&sh.q_full[q1 & 3], (q1 >> 2) & 1, watch) && fa_wait(&sh.k_full[ks], (kn >> 1) & 1, watch);
                    if (!ok) break;
                    fa_after();
                    fa_mma_s(t0, sq0, sk);
                    fa_commit(&sh.s_full[0]);
                    fa_mma_s(t1, sq1, sk);
                    fa_commit(&sh.s_full[1]);
                    fa_commit(&sh.k_empty[ks]);
                    ++kn;
#pragma unroll 1
                    for (int left = n - 1; left > 0; --left) {
                        const unsigned vs = vn & 1, sv = s_v + vs * kFaTileB;
                        ks = kn & 1, sk = s_k + ks * kFaTileB;
                        if (!fa_wait(&sh.v_full[vs], (vn >> 1) & 1, watch) || !fa_wait(&sh.k_full[ks], (kn >> 1) & 1, watch) ||
                            !fa_wait(&sh.p_ready[0][0], pn0 & 1, watch))
                            break;
                        fa_after();
                        fa_mma_o_first(o0, t0, sv, (n - 1 - left) % kFaFold != 0);
                        if (!fa_wait(&sh.p_ready[0][1], pn0 & 1, watch)) break;
                        fa_after();
                        fa_mma_o_rest_s(o0, t0, sv, sq0, sk, &sh.s_full[0]);
                        ++pn0;
                        if (!fa_wait(&sh.p_ready[1][0], pn1 & 1, watch)) break;
                        fa_after();
                        fa_mma_o_first(o1, t1, sv, (n - 1 - left) % kFaFold != 0);
                        if (!fa_wait(&sh.p_ready[1][1], pn1 & 1, watch)) break;
                        fa_after();
                        fa_mma_o_rest_s(o1, t1, sv, sq1, sk, &sh.s_full[1]);
                        ++pn1;
                        fa_commit(&sh.k_empty[ks]);
                        fa_commit(&sh.v_empty[vs]);
                        ++kn;
                        ++vn;
                    }
                    ok = !watch->abort;
                    if (!ok) break;
                    // the last scores are issued; the last value tile
                    fa_commit(&sh.q_empty[q0 & 3]);
                    fa_commit(&sh.q_empty[q1 & 3]);
                    const unsigned vs = vn & 1, sv = s_v + vs * kFaTileB;
                    ok = fa_wait(&sh.v_full[vs], (vn >> 1) & 1, watch) && fa_wait(&sh.p_ready[0][0], pn0 & 1, watch) &&
                         fa_wait(&sh.p_ready[0][1], pn0 & 1, watch);
                    if (!ok) break;
                    fa_after();
                    fa_mma_o_first(o0, t0, sv, (n - 1) % kFaFold != 0);
                    fa_mma_o_rest(o0, t0, sv, true);
                    fa_commit(&sh.o_done[0]);
                    ++pn0;
                    ok = fa_wait(&sh.p_ready[1][0], pn1 & 1, watch) && fa_wait(&sh.p_ready[1][1], pn1 & 1, watch);
                    if (!ok) break;
                    fa_after();
                    fa_mma_o_first(o1, t1, sv, (n - 1) % kFaFold != 0);
                    fa_mma_o_rest(o1, t1, sv, true);
                    fa_commit(&sh.o_done[1]);
                    ++pn1;
                    fa_commit(&sh.v_empty[vs]);
                    ++vn;
                    continue;
                }
                // round j: each stream's products with its j-th value tile, then its scores against
                // key tile j + 1 (round -1: the first scores)
#pragma unroll 1
                for (int j = -1; ok && j < n; ++j)
#pragma unroll 1
                    for (int s = 0; ok && s < ns; ++s) {
                        const int ne = s ? n1 : n0;
                        const unsigned t_p = tmem + 128 * s, vs = vn % kFaStagesV, ks = kn % kFaStagesK;
                        bool k_here = false;
                        if (j >= ne) continue;
                        if (j >= 0) {
                            const unsigned t_o = t_p + 256, sv = s_v + vs * kFaTileB, np = s ? pn1 : pn0;
                            ok = fa_wait(&sh.v_full[vs], (vn / kFaStagesV) & 1, watch);
                            // the weights come in two portions: the first one's products run
                            // while the second is made
                            ok = ok && fa_wait(&sh.p_ready[s][0], np & 1, watch);
                            if (!ok) break;
                            fa_after();
                            fa_mma_o_first(t_o, t_p, sv, j % kFaFold != 0);
                            if (j + 1 < ne)  // off the path of the last weights
                                k_here = fa_try(smem_u32(&sh.k_full[ks]), (kn / kFaStagesK) & 1);
                            ok = fa_wait(&sh.p_ready[s][1], np & 1, watch);
                            if (!ok) break;
                            fa_after();
                            fa_mma_o_rest(t_o, t_p, sv, true);
                            if (s) ++pn1;
                            else ++pn0;
                            if (j + 1 == ne) fa_commit(&sh.o_done[s]);
                        }
                        if (j + 1 < ne) {
                            const unsigned q = s ? q1 : q0;
                            if (j < 0) ok = fa_wait(&sh.q_full[q & 3], (q >> 2) & 1, watch);
                            if (!k_here) ok = ok && fa_wait(&sh.k_full[ks], (kn / kFaStagesK) & 1, watch);
                            if (!ok) break;
                            fa_after();
                            fa_mma_s(t_p, s ? sq1 : sq0, s_k + ks * kFaTileB);
                            fa_commit(&sh.s_full[s]);  // the stream waits for it
                            fa_commit(&sh.k_empty[ks]);
                            ++kn;
                            // a query tile of both is done with the last scores of the two
                            if (it.same_q ? j + 2 == n && (s ? n1 >= n0 : n0 > n1) : j + 2 == ne)
                                fa_commit(&sh.q_empty[q & 3]);
                        }
                        if (j >= 0) {
                            fa_commit(&sh.v_empty[vs]);
                            ++vn;
                        }
                    }
            }
            // products in flight end (bounded) before the tensor memory is given back
            if (!ok) set_status(a.status, ICE_ERR_TIMEOUT);
            if (qn) {
                fa_commit(&sh.drain);
                mbar_wait_bounded(smem_u32(&sh.drain), 0);
            }
        }
        __syncwarp();
    } else {
        // ---- softmax and output: thread = row of stream s ----
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kFaRegsSoftmax));
        const int s = warp >> 2, wq = warp & 3, row = 32 * wq + lane;
        const unsigned t_s = tmem + 128 * s + ((unsigned)(32 * wq) << 16), t_o = t_s + 256;
        const int valid_tok = a.q_start[a.n_req];
        unsigned sn = 0, on = 0, vn = 0;
        while (ok && items.next(sh, it, ok, true)) {
            if (it.ns == 0) continue;
            const bool apart = !it.shared;
            const int n0 = it.st[0].n, n1 = it.ns > 1 ? it.st[1].n : 0;
            const unsigned vn0 = vn;
            vn += apart ? n0 + n1 : n0;
            if (s >= it.ns) continue;
            const PagedStream st = s ? it.st[1] : it.st[0];
            const int n = st.n, nrow = st.ntok * a.G;
            const bool busy = 32 * wq < nrow;  // a warp without rows only keeps the barriers going
            const int tok = st.tok0 + row / a.G;
            // own tokens that the row sees, and that every row of the warp sees (the first sees the fewest)
            const int lim = min(st.own_len, tok + st.lim_off);
            const int lim_all = min(st.own_len, st.tok0 + 32 * wq / a.G + st.lim_off);
            // the row's place among the parts
            auto part = [&]() { return ((long long)st.slot * a.H + st.h) * a.RP + st.tok0 * a.G + row; };
            float m = -INFINITY, l = 0.0f;
            for (int j = 0; j < n; ++j) {
                ok = __all_sync(0xffffffffu, fa_wait(&sh.s_full[s], sn & 1, watch));
                if (!ok) break;
                ++sn;
                const PagedTile t = tile_of(a, z, st, st.kt0 + j);
                if (t.key0 + KT > t.len) {  // the last tile of a list: rows behind the last key
                    const unsigned v = vn0 + (!apart ? j : s ? j + min(n0, j + 1) : j + min(n1, j)), vs = v % kFaStagesV;
                    ok = __all_sync(0xffffffffu, fa_wait(&sh.v_full[vs], (v / kFaStagesV) & 1, watch));
                    if (!ok) break;
                    const int r0 = t.len - t.key0;
                    unsigned char* v_st = mem + (2 + kFaStagesK + vs) * kFaTileB;
                    for (int x = row; x < (KT - r0) * 16; x += kFaRows)
                        *reinterpret_cast<uint4*>(v_st + ((x >> 3) & 1) * kFaHalfB + (r0 + (x >> 4)) * 128 + (x & 7) * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
                if (!busy) {
                    __syncwarp();
                    if (lane == 0) fa_arrive(&sh.p_ready[s][0]), fa_arrive(&sh.p_ready[s][1]);
                    continue;
                }
                fa_after();
                if (j > 0 && j % kFaFold == 0) {  // O of the tiles before is complete: its products precede S in the pipe
                    fa_fold(t_o, a.part_o + part() * kD, a.part_ml + part(), row < nrow, j == kFaFold, false, m, l);
                    l = 0.0f;
                }
                unsigned v[4][32];  // scores, as bits
#pragma unroll
                for (int k = 0; k < 4; ++k) fa_ld(t_s + 32 * k, v[k]);
                fa_wait_ld();
                // some key is hidden from some row
                if (t.key0 + kFaKeys > (t.own ? lim_all : t.len) || KT < kFaKeys) {
                    const int c_lim = min((t.own ? lim : t.len) - t.key0, KT);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            if (32 * k + c >= c_lim) v[k][c] = 0xFF800000u;  // -inf
                }
                float mx[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    mx[k] = fmaxf(__uint_as_float(v[k][0]), __uint_as_float(v[k][1]));
#pragma unroll
                    for (int c = 2; c < 32; c += 2)
                        mx[k] = fa_max3(mx[k], __uint_as_float(v[k][c]), __uint_as_float(v[k][c + 1]));
                }
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2;
                const bool grow = top > m + kFaSlack;  // also the first finite one
                if (__any_sync(0xffffffffu, grow)) {
                    const float f = grow ? exp2_approx(m - top) : 1.0f;
                    if (grow) m = top;
                    l *= f;
                    if (j % kFaFold != 0) {  // O of the tiles before is complete
#pragma unroll 1
                        for (int k = 0; k < kD; k += 16) {
                            unsigned u[16];
                            fa_ld(t_o + k, u);
                            fa_wait_ld();
#pragma unroll
                            for (int c = 0; c < 16; ++c) u[c] = __float_as_uint(__uint_as_float(u[c]) * f);
                            fa_st(t_o + k, u);
                        }
                    }
                }
                const float nm = m == -INFINITY ? 0.0f : -m;
                const float2 c2 = make_float2(a.scale_log2, a.scale_log2), nm2 = make_float2(nm, nm);
                float ls[2] = {l, 0.0f};
                auto ready = [&](int h) {  // portion h of the weights is written
                    fa_wait_st();
                    fa_before();
                    __syncwarp();
                    if (lane == 0) fa_arrive(&sh.p_ready[s][h]);
                };
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    unsigned u[16];
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        const float2 x = fma2(make_float2(__uint_as_float(v[k][2 * c]), __uint_as_float(v[k][2 * c + 1])), c2, nm2);
                        u[c] = fa_pack(exp2_approx(x.x), exp2_approx(x.y));
                        fa_add_pair(ls[0], ls[1], u[c]);
                    }
                    if (k == 3) ready(0);  // keys 0 .. 95, stored while these were made
                    fa_st(t_s + 16 * k, u);
                }
                ready(1);
                l = ls[0] + ls[1];
            }
            if (!ok) break;
            if (n > 0) {
                ok = __all_sync(0xffffffffu, fa_wait(&sh.o_done[s], on & 1, watch));
                if (!ok) break;
                ++on;
            }
            if (!busy) continue;
            fa_after();
            const bool mine = row < nrow;
            const long long R = part();
            if (n > kFaFold) l = fa_fold(t_o, a.part_o + R * kD, a.part_ml + R, mine, false, true, m, l);
            const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
            const float f = l > 0.0f || l != l ? inv : 0.0f;  // zeros where nothing was seen
#pragma unroll 1
            for (int k = 0; k < kD; k += 32) {
                unsigned u[32];
                if (n > 0) {
                    fa_ld(t_o + k, u);
                    fa_wait_ld();
                }
                if (n == 0 || f == 0.0f) {  // O was not written where n = 0
#pragma unroll
                    for (int c = 0; c < 32; ++c) u[c] = 0;
                }
#pragma unroll
                for (int c = 0; c < 32; ++c) u[c] = __float_as_uint(__uint_as_float(u[c]) * f);
                if (mine && st.direct && tok < valid_tok) {
                    uint4* dst = reinterpret_cast<uint4*>((__nv_bfloat16*)a.out +
                                                          ((long long)tok * a.H * a.G + st.h * a.G + row % a.G) * kD + k);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        unsigned w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            w[e] = fa_pack(__uint_as_float(u[8 * c + 2 * e]), __uint_as_float(u[8 * c + 2 * e + 1]));
                        dst[c] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                } else if (mine && !st.direct) {
                    float* dst = a.part_o + R * kD + k;
#pragma unroll
                    for (int c = 0; c < 32; c += 8)  // whole sectors of 32 B
                        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + c), "r"(u[c]),
                                     "r"(u[c + 1]), "r"(u[c + 2]), "r"(u[c + 3]), "r"(u[c + 4]), "r"(u[c + 5]), "r"(u[c + 6]),
                                     "r"(u[c + 7])
                                     : "memory");
                }
                __syncwarp();  // the next columns are read by the whole warp
            }
            if (mine && !st.direct) a.part_ml[R] = make_float2(m, l);
            fa_before();
        }
    }
    fa_before();
    __syncthreads();
    fa_after();
    if (warp == 9)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    if (tid == 0) {  // the last block to end leaves the counters at zero
        __threadfence();
        if (atomicAdd(&a.next[1], 1u) == gridDim.x - 1) {
            a.next[0] = 0;
            a.next[1] = 0;
        }
    }
}

typedef CUresult (*FaEncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                               const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                               CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static FaEncodeFn fa_encoder() {
    static FaEncodeFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<FaEncodeFn>(p);
        cudaGetLastError();
    });
    return fn;
}

static bool fa_map(CUtensorMap* m, const void* p, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                   const cuuint32_t* box) {
    const cuuint32_t estr[3] = {1, 1, 1};
    FaEncodeFn enc = fa_encoder();
    return enc != nullptr &&
           enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(p), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

PagedTiles paged_tc_tiles(int P, int G) { return {kFaKeys / P * P, 2 * kFaRows / G, kFaRows / G, kFaRows / G, 0, kFaKeys / P}; }

cudaError_t launch_paged_tc(const PagedAttn& a, const PagedTiles& z, int n_sm, cudaStream_t s) {
    CUtensorMap mq, mf, mk, mv;
    const cuuint64_t qd[3] = {kD, (cuuint64_t)(a.H * a.G), (cuuint64_t)a.n_tokens};
    const cuuint64_t qs[2] = {kD * 2, (cuuint64_t)a.q_stride * 2};
    const cuuint32_t qb[3] = {64, (cuuint32_t)a.G, (cuuint32_t)(kFaRows / a.G)};
    const cuuint32_t fb[3] = {64, (cuuint32_t)a.G, (cuuint32_t)(kFaFew / a.G)};
    const cuuint64_t kd[2] = {kD, (cuuint64_t)(a.n_pages * a.H * a.P)};
    const cuuint64_t ks[1] = {kD * 2};
    const cuuint32_t kb[2] = {64, (cuuint32_t)a.P};
    if (!fa_map(&mq, a.q, 3, qd, qs, qb) || !fa_map(&mf, a.q, 3, qd, qs, fb) || !fa_map(&mk, a.k_pages, 2, kd, ks, kb) || !fa_map(&mv, a.v_pages, 2, kd, ks, kb))
        return cudaErrorNotSupported;
    return launch_pdl(paged_tc_kernel, dim3(n_sm), dim3(kFaThreads), (size_t)fa_smem(a.n_req), s, a, mq, mf, mk, mv, z);
}

cudaError_t paged_tc_prepare() {
    return cudaFuncSetAttribute(paged_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                1024 + (2 + kFaStages) * kFaTileB + (kPagedMaxRequests + 1) * 4);
}

}  // namespace ice
