// What the grouped products share: tcgen05 products of 128-row tiles with
// operands in shared memory and fp32 sums in TMEM, the rings that feed them,
// and the walk over the groups of a CSR.
//
// Operand boxes.  Every operand tile is made of boxes of rows of 64 (or 32)
// contiguous 16-bit elements, eight rows to an atom whose 16-byte pieces are
// permuted by the 128-byte (64-byte) swizzle: piece c of row r sits at piece
// c ^ (r & 7), or c ^ (r / 2 & 3).  Where the contiguous direction is the one
// summed over, a box holds all of the tile's rows (K-major); where it is not, a
// box holds summed-over rows and the tile takes a box for every 64 of its own
// (MN-major; boxes of 32 columns were read a third slower that way).  Either
// way a box is the plain image of a piece of a row-major matrix, so TMA, or
// warps that copy rows, write it.
//
// fp32 operands are cut into three bf16 planes, each the rest rounded to
// nearest, 8 + 8 + 8 bits of the 24, which loses nothing; the six products of
// planes whose weights reach 2^-16 are summed, at a sixth of the bf16 rate, about
// four times fp32's on the CUDA cores.  What is left out is below 2^-24 of a
// term, of either sign (planes cut off instead of rounded left out up to 2^-21,
// always of the term's sign, in the same time: 8192 rows, 1024 -> 1024, 240 us).
// The right operand's planes lie side by side, so one instruction multiplies a
// plane of the left one by three, two or one of them, and the products sum up
// by weight: 1, 2^-8 and 2^-16.  The tensor cores truncate as they add (a sum
// over n steps comes out about n 2^-24 low, as measured), which only the first
// of the three sums feels; all leave TMEM every kChunk summed-over elements to
// be added, rounded to nearest, in registers.
//
// Every wait is bounded (zs_wait.cuh).  A wait that runs out marks the CTA
// dead: every role leaves its loop, the copies and products in flight are
// waited for (with a limit), TMEM is freed, and the outputs are undefined.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "zs_tma.cuh"
#include "zs_types.cuh"

namespace zs {

constexpr int kTileM = 128;                    // rows of a product's tile: TMEM lanes
// Summed-over elements of a stage: a K-major box's columns, an MN-major box's
// rows.  The three planes of fp32 take more room, so its stages are shorter.
template <typename T>
constexpr int kStageK = sizeof(T) == 4 ? 32 : 64;
constexpr int kBoxMN = 64;                     // columns of an MN-major box
template <int kCols>
__host__ __device__ constexpr uint32_t box_bytes(int rows) { return (uint32_t)rows * kCols * 2; }
constexpr uint32_t kDrainSpins = 1u << 16;

constexpr int kEpilogueWarps = 8;              // two for each 32 TMEM lanes
constexpr int kLoaderWarps = 8;                // of each of the two groups that take stages in turn
constexpr int kChunk = 128;                    // elements summed in TMEM at a time for fp32 operands
// Of 16-bit operands.  128 additions that truncate leave a sum of one sign up to
// 2^-16 low (1.3e-5 as measured), a thirtieth of half an ulp of fp16; a sum of
// 65536 in one piece came out 4.3e-4 low, of 262144 1.7e-3.  Longer sums pass to
// the epilogue every kLongSum elements, which adds them up in TMEM (32768 rows,
// 1024 -> 4096 bf16, us of dx and dw with 8192: 185 and 237; 2048: 186 and 242;
// 1024: 191 and 248).
constexpr int kLongSum = 2048;
template <typename T>
constexpr int kPlanes = sizeof(T) == 4 ? 3 : 1;
template <typename T>
constexpr int kSums = sizeof(T) == 4 ? 3 : 1;  // sums of a tile in TMEM
__host__ __device__ constexpr uint32_t tmem_cols(int n) { return n <= 32 ? 32 : n <= 64 ? 64 : n <= 128 ? 128 : n <= 256 ? 256 : 512; }

// ---------------------------------------------------------------- barriers

__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}

// Whole warps.  dead: set by the first wait of the CTA that runs out; the
// others give up soon after.  Every lane gets the same answer.
__device__ __forceinline__ bool bounded_wait(uint32_t bar, uint32_t parity, volatile int* dead) {
    bool ok = false;
    for (uint32_t i = 0; i < kMaxSpins && !ok; ++i) {
        ok = mbar_try_wait(bar, parity);
        if (!ok && (i & 63) == 63 && *dead) break;
        if (!ok && i == kMaxSpins - 1) {
            note_timeout();
            *dead = 1;
        }
    }
    return __all_sync(0xffffffffu, ok);
}
// The same without a vote, for the warps that issue copies and products: where
// it runs out the warp carries on (outputs are then undefined) and finds the CTA
// dead later.  A vote at each stage would cost them a tenth of the tensor cores'
// time.  kCluster: the other CTA of a pair arrives at this barrier too.
template <bool kCluster = false>
__device__ __forceinline__ void bounded_wait_on(uint32_t bar, uint32_t parity, volatile int* dead) {
    if (!(kCluster ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity))) {
#pragma unroll 1
        for (uint32_t i = 0; i < kMaxSpins; ++i) {
            if (kCluster ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)) break;
            if ((i & 63) == 63 && *dead) break;
            if (i == kMaxSpins - 1) {
                note_timeout();
                *dead = 1;
            }
        }
    }
    __syncwarp();
}
__device__ __forceinline__ bool is_dead(volatile int* dead) { return __any_sync(0xffffffffu, *dead != 0); }

// Whether the phase is over, without waiting.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(bar) : "memory");
}
// The same address in the first CTA of the cluster.
__device__ __forceinline__ uint32_t in_first(uint32_t at) {
    uint32_t there;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(there) : "r"(at));
    return there;
}
// At a barrier of the cluster.  (What is told of has been read from TMEM, nothing
// written; released to the whole cluster, an arrival took about 700 cycles.)
__device__ __forceinline__ void mbar_arrive_there(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" :: "r"(bar) : "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void pair_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// A position in a ring of S stages.
template <int S>
struct RingPos {
    int stage = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
        if (++stage == S) stage = 0, phase ^= 1;
    }
};

// ---------------------------------------------------------------- tcgen05

// kPair: both CTAs of a cluster of two take part (a warp of each allocates and
// frees; the first one's products are of both).
template <bool kPair>
__device__ __forceinline__ void tmem_alloc(uint32_t dst_smem, uint32_t cols) {
    if constexpr (kPair) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(dst_smem), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(dst_smem), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
}
template <bool kPair>
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
    if constexpr (kPair) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" :: "r"(addr), "r"(cols) : "memory");
    else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(addr), "r"(cols) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// Products and their commits are issued by one lane that the warp elects, always
// the same, with the warp in step: from inside a branch on the lane number each
// instruction took 143 cycles to issue, more than a 128 x 256 product's 128.
//
// An arrival at the barrier (of a pair: at both CTAs') once the products issued so far are done.
template <bool kPair>
__device__ __forceinline__ void tc_commit(uint32_t bar) {
    if constexpr (kPair)
        asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
                     "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}"
                     :: "r"(bar), "h"((unsigned short)3) : "memory");
    else
        asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
                     "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" :: "r"(bar) : "memory");
}
template <bool kPair>
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    if constexpr (kPair)
        asm volatile("{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                     :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate) : "memory");
    else
        asm volatile("{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                     :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate) : "memory");
}
// Four products one after the other, and an arrival at `bar` when they are done.
template <bool kPair, uint32_t kStepA, uint32_t kStepB>
__device__ __forceinline__ void tc_mma4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate, uint32_t bar) {
    if constexpr (kPair)
        asm volatile("{\n\t.reg .pred p, t, e;\n\t.reg .b64 a, b;\n\t"
                     "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
                     "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t"
                     "add.s64 a, %1, %6;\n\tadd.s64 b, %2, %7;\n\t"
                     "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, t;\n\t"
                     "add.s64 a, a, %6;\n\tadd.s64 b, b, %7;\n\t"
                     "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, t;\n\t"
                     "add.s64 a, a, %6;\n\tadd.s64 b, b, %7;\n\t"
                     "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, t;\n\t"
                     "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%5], %8;\n\t}"
                     :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate), "r"(bar), "n"(kStepA), "n"(kStepB),
                        "h"((unsigned short)3) : "memory");
    else
        asm volatile("{\n\t.reg .pred p, t, e;\n\t.reg .b64 a, b;\n\t"
                     "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
                     "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
                     "add.s64 a, %1, %6;\n\tadd.s64 b, %2, %7;\n\t"
                     "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
                     "add.s64 a, a, %6;\n\tadd.s64 b, b, %7;\n\t"
                     "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
                     "add.s64 a, a, %6;\n\tadd.s64 b, b, %7;\n\t"
                     "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
                     "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%5];\n\t}"
                     :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate), "r"(bar), "n"(kStepA), "n"(kStepB) : "memory");
}
// 32 columns of this warp's 32 TMEM lanes: lane l gets row l.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
                   "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
                   "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(addr) : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(addr) : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 "
                 "[%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
                 :: "r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
                    "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]) : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Where 16-byte piece c of row r sits in a box.
template <int kCols>
__device__ __forceinline__ uint32_t piece_at(int r, int c) {
    return r * (kCols * 2) + ((c ^ (kCols == 64 ? r & 7 : (r >> 1) & 3)) << 4);
}
// Shared-memory operand descriptor of boxes.  Both forms step one atom (sbo)
// per 8 box rows; lbo is the distance between the boxes of an MN-major tile
// (unused by a K-major one).
template <int kCols>
__device__ __forceinline__ uint64_t box_desc(uint32_t addr, uint32_t lbo) {
    constexpr uint64_t sbo = 8 * kCols * 2, swizzle = kCols == 64 ? 2 : 4;
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)((lbo & 0x3FFFFu) >> 4) << 16) | ((sbo >> 4) << 32) |
           (uint64_t(1) << 46) | (swizzle << 61);
}
// Descriptor address steps of one product's 16 summed-over elements: 32 bytes
// along a K-major row, 16 rows of an MN-major box.
template <int kCols, bool kMN>
constexpr uint32_t kDescStep = (kMN ? 16 * kCols * 2 : 32) >> 4;

// Instruction descriptor: 16-bit operands, fp32 sums, m x n tile.
template <typename T>
__device__ __forceinline__ uint32_t instr_desc(bool a_mn, bool b_mn, int n, int m = kTileM) {
    constexpr uint32_t type = sizeof(T) == 4 || std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;   // bf16 (planes too) or f16
    return (1u << 4) | (type << 7) | (type << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// The products of one stage: `steps` times 16 summed-over elements, into a tile
// of BN columns (fp32: three of them), and an arrival at `bar` when they are
// done.  Planes of the left operand are a_plane bytes apart, those of the right
// one follow each other.  Of a pair, each CTA holds 128 rows of the left operand
// and half the columns of the right one, at the same addresses, and gets its
// rows' sums.
template <typename T, bool kAMN, bool kBMN, int BN, bool kPair = false>
__device__ __forceinline__ void issue_stage(uint32_t d, uint32_t a, uint32_t a_plane, uint32_t a_lbo, uint32_t b, uint32_t b_lbo,
                                            int steps, bool accumulate, uint32_t bar) {
    constexpr int kACols = kAMN ? kBoxMN : kStageK<T>, kBCols = kBMN ? kBoxMN : kStageK<T>;
    constexpr uint32_t kStepA = kDescStep<kACols, kAMN>, kStepB = kDescStep<kBCols, kBMN>;
    constexpr int kMost = kStageK<T> / 16;
    const uint64_t a0 = box_desc<kACols>(a, a_lbo), b0 = box_desc<kBCols>(b, b_lbo);
    if constexpr (kPlanes<T> == 1) {
        static_assert(kMost == 4, "a whole stage's products in one block");
        const uint32_t idesc = instr_desc<T>(kAMN, kBMN, BN, kPair ? 2 * kTileM : kTileM);
        if (steps == kMost) {
            tc_mma4<kPair, kStepA, kStepB>(d, a0, b0, idesc, accumulate, bar);
            return;
        }
        for (int k = 0; k < steps; ++k) tc_mma<kPair>(d, a0 + k * kStepA, b0 + k * kStepB, idesc, accumulate || k > 0);
    } else {
        static_assert(!kPair, "fp32 tiles are a CTA's own");
#pragma unroll
        for (int k = 0; k < kMost; ++k) {
            if (k >= steps) break;
            const uint64_t ak = a0 + k * kStepA, bk = b0 + k * kStepB;
            const uint32_t ap = a_plane >> 4;
            tc_mma<false>(d, ak, bk, instr_desc<T>(kAMN, kBMN, 3 * BN), accumulate || k > 0);
            tc_mma<false>(d + BN, ak + ap, bk, instr_desc<T>(kAMN, kBMN, 2 * BN), true);
            tc_mma<false>(d + 2 * BN, ak + 2 * ap, bk, instr_desc<T>(kAMN, kBMN, BN), true);
        }
    }
    tc_commit<kPair>(bar);
}

// ---------------------------------------------------------------- TMA

// By a warp in step, as the products are.  kPair: the barrier is the first CTA's.
template <bool kPair = false>
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    if constexpr (kPair)
        asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
                     "@e cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
                     "[%0], [%1, {%2, %3}], [%4];\n\t}" :: "r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
    else
        asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
                     "@e cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                     "[%0], [%1, {%2, %3}], [%4];\n\t}" :: "r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
}
template <bool kPair = false>
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
    if constexpr (kPair)
        asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
                     "@e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
                     "[%0], [%1, {%2, %3, %4}], [%5];\n\t}" :: "r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
    else
        asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
                     "@e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                     "[%0], [%1, {%2, %3, %4}], [%5];\n\t}" :: "r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}
__device__ __forceinline__ void expect_bytes(uint32_t bar, uint32_t bytes) {
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
                 "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" :: "r"(bar), "r"(bytes) : "memory");
}
// ---------------------------------------------------------------- rows copied by warps

// How a matrix is read: rows `ld` elements apart, `cols` wide; aligned: every
// row starts on a 16-byte boundary.
struct Matrix {
    const void* p;
    int64_t ld;
    int cols;
    bool aligned;
};

// 16 bytes to shared memory, of which the first n are read and the others zero.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int n) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(n) : "memory");
}
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// a and b rounded to bf16 and left with what that takes from them.  kFirst: a
// finite one that would overflow is cut to the largest bf16 (an infinity too,
// which makes the plane after it infinite and the one after that NaN).
template <bool kFirst>
__device__ __forceinline__ uint32_t take_plane(float& a, float& b) {
    uint32_t u;
    if constexpr (kFirst) asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(u) : "f"(b), "f"(a));
    else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u) : "f"(b), "f"(a));
    a -= __uint_as_float(u << 16);
    b -= __uint_as_float(u & 0xffff0000u);
    return u;
}

// kRows rows of a box of kCols columns, for operands that are cut into planes
// or whose rows are not aligned.  A group of kLoaderWarps warps copies them in
// parts of 16 bytes (of the matrix) into slots of shared memory that are each
// thread's own, and later turns each part into the box's pieces; nothing is
// held in registers meanwhile, and no barrier is needed between the two.  A
// part of an unaligned row is copied as the two aligned pieces that hold it.
// A lane of warp w holds in `rows` the matrix row of box row kPer w + (lane
// mod kPer) (negative: zeros, as are columns past the matrix).
template <typename T, int kRows, int kCols>
struct BoxParts {
    static constexpr int kElems = 16 / (int)sizeof(T);
    static constexpr int kPer = kRows / kLoaderWarps;
    static constexpr int kLanes = kCols / kElems;        // of a row
    static constexpr int kAtOnce = 32 / kLanes;          // rows a warp copies at once
    static constexpr int kSteps = kPer / kAtOnce;        // parts of a thread
    static_assert(kPer <= 32 && kPer % kAtOnce == 0, "whole rows");

    // offs: bits 4 i .. of this thread's part i say where it starts within its slot (unaligned rows)
    static __device__ __forceinline__ uint32_t copy(const Matrix& m, int rows, int c0, uint32_t slot, uint32_t stride, bool aligned,
                                                    int lane) {
        uint32_t offs = 0;
        const int c = c0 + kElems * (lane % kLanes);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int r = __shfl_sync(0xffffffffu, rows, i * kAtOnce + lane / kLanes);
            const bool in = r >= 0 && c < m.cols;
            const char* at = static_cast<const char*>(m.p) + (in ? (r * m.ld + c) * (int64_t)sizeof(T) : 0);
            const int left = in ? (m.cols - c) * (int)sizeof(T) : 0;   // bytes to the row's end
            if (aligned) {
                copy16(slot + i * stride, at, imin(left, 16));
            } else {
                const int off = in ? (int)(reinterpret_cast<uintptr_t>(at) & 15u) : 0;
                const char* base = reinterpret_cast<const char*>(reinterpret_cast<uintptr_t>(at) & ~uintptr_t(15));
                copy16(slot + i * stride, base, in ? imin(off + left, 16) : 0);
                const int more = imin(off + left - 16, 16);
                copy16(slot + i * stride + 16, more > 0 ? base + 16 : base, imax(more, 0));
                offs |= (uint32_t)off << (4 * i);
            }
        }
        return offs;
    }

    // fp32: x = plane 0 + plane 1 + plane 2 exactly, each what the ones before leave rounded to bf16 (a value that is not
    // finite leaves NaN).
    static __device__ __forceinline__ void turn(const unsigned char* slot, uint32_t stride, bool aligned, uint32_t offs,
                                                unsigned char* box, uint32_t plane, int w, int lane) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            uint4 q;
            if (aligned) {
                q = *reinterpret_cast<const uint4*>(slot + i * stride);
            } else {
                const int off = offs >> (4 * i) & 15;
                const uint32_t* from = reinterpret_cast<const uint32_t*>(slot + i * stride + (off & 12));
                uint32_t* qe = &q.x;
                if constexpr (sizeof(T) == 4) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) qe[j] = from[j];
                } else {
                    uint32_t u[5];
#pragma unroll
                    for (int j = 0; j < 4; ++j) u[j] = from[j];
                    u[4] = off & 2 ? from[4] : 0;
#pragma unroll
                    for (int j = 0; j < 4; ++j) qe[j] = __funnelshift_r(u[j], u[j + 1], 8 * (off & 2));
                }
            }
            const int row = kPer * w + i * kAtOnce + lane / kLanes, part = lane % kLanes;
            if constexpr (sizeof(T) == 4) {
                unsigned char* to = box + piece_at<kCols>(row, part >> 1) + ((part & 1) << 3);
                float x[4] = {__uint_as_float(q.x), __uint_as_float(q.y), __uint_as_float(q.z), __uint_as_float(q.w)};
                *reinterpret_cast<uint2*>(to) = make_uint2(take_plane<true>(x[0], x[1]), take_plane<true>(x[2], x[3]));
#pragma unroll
                for (int p = 1; p < 3; ++p)
                    *reinterpret_cast<uint2*>(to + p * plane) = make_uint2(take_plane<false>(x[0], x[1]), take_plane<false>(x[2], x[3]));
            } else {
                *reinterpret_cast<uint4*>(box + piece_at<kCols>(row, part)) = q;
            }
        }
    }
};

// kPer rows from row0 on of a box of 64 columns of a 16-bit matrix with aligned
// rows, copied straight to their places; lane i holds the number of the i-th.  (TMA gathers four rows in about 40 cycles,
// which is 12 bytes a cycle of an SM; this took 75 us where that took 104, for
// 262144 rows of 256 channels.)
template <int kPer>
__device__ __forceinline__ void copy_rows(uint32_t box, const Matrix& m, int rows, int c0, int row0, int lane) {
    static_assert(kPer <= 32 && kPer % 4 == 0, "a lane holds a row's number");
    const int piece = lane & 7;
    const int c = c0 + 8 * piece;
#pragma unroll
    for (int i = 0; i < kPer / 4; ++i) {
        const int at = 4 * i + (lane >> 3), r = __shfl_sync(0xffffffffu, rows, at), row = row0 + at;
        const bool in = r >= 0 && c < m.cols;
        copy16(box + piece_at<64>(row, piece), static_cast<const uint16_t*>(m.p) + (in ? r * m.ld + c : 0),
               in ? imin(m.cols - c, 8) * 2 : 0);
    }
}

// ---------------------------------------------------------------- groups of a CSR

// The positions of the groups, cut into slots of kRows positions: group g
// starts at slot floor(row_ptr[g] / kRows) + g * kExtra, which leaves room for
// each group's pieces without a prefix sum (kExtra >= 1).  Slots past a
// group's last piece are empty.  start(G + 1) is M: the positions of no group
// are "group" G.  The starts of up to kGroupsHeld groups are kept in shared
// memory (a search there takes 0.1 us, in global memory one or two).
constexpr int kGroupsHeld = 1022;
template <int kRows, int kExtra>
struct Groups {
    const int32_t* p;   // start(0 .. G + 1) in shared memory, or row_ptr
    int G, M;
    bool held;
    __device__ __forceinline__ static int clamped(const int32_t* row_ptr, int g, int M) {
        const int v = __ldg(row_ptr + g);
        return v < 0 ? 0 : v > M ? M : v;
    }
    // All threads of the CTA; a barrier has to follow.
    __device__ __forceinline__ void hold(const int32_t* row_ptr, int G_, int M_, int32_t* smem) {
        G = G_;
        M = M_;
        held = G <= kGroupsHeld;
        p = held ? smem : row_ptr;
        if (held)
            for (int g = threadIdx.x; g <= G + 1; g += blockDim.x) smem[g] = g > G ? M : clamped(row_ptr, g, M);
    }
    __device__ __forceinline__ int start(int g) const { return held ? p[g] : g > G ? M : clamped(p, g, M); }
    __device__ __forceinline__ int slot(int g) const { return start(g) / kRows + g * kExtra; }
    // The group in [0, last) whose slots hold s (slot(0) <= s < slot(last)), found by the whole warp: 32 samples a round.
    __device__ __forceinline__ int find(int s, int last) const {
        const int lane = threadIdx.x & 31;
        int lo = 0, n = last;   // the answer is in [lo, lo + n)
        while (n > 1) {
            const int step = (n + 31) / 32, g = lo + lane * step;
            const unsigned m = __ballot_sync(0xffffffffu, lane * step < n && slot(g) <= s);
            const int i = 31 - __clz(m | 1u);
            lo += i * step;
            n = imin(step, n - i * step);
        }
        return lo;
    }
};

// ---------------------------------------------------------------- epilogue

// A warp's 32 rows x 64 bytes of results pass through shared memory (rows 80
// bytes apart) so that they leave as whole row segments.
constexpr int kStageRow = 80;
constexpr int kStageWarp = 32 * kStageRow;

// Writes `left` (of 32) columns: lane l holds those of row l, which goes to
// `row` (NULL: nowhere), 16 bytes at a time where `wide`.
template <typename TO>
__device__ __forceinline__ void emit32(const float (&f)[32], int left, TO* row, bool wide, unsigned char* stage, int lane) {
    constexpr int kCols = 64 / (int)sizeof(TO);   // columns of a 64-byte segment
    const unsigned long long mine = reinterpret_cast<unsigned long long>(row);
#pragma unroll
    for (int part = 0; part < 32 / kCols; ++part) {
        const int here = left - part * kCols;
        if (here <= 0) break;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float q[kVec<TO>];
#pragma unroll
            for (int j = 0; j < kVec<TO>; ++j) q[j] = f[part * kCols + i * kVec<TO> + j];
            *reinterpret_cast<uint4*>(stage + lane * kStageRow + 16 * i) = pack<TO>(q);
        }
        __syncwarp();
        if (wide) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 8 * i + (lane >> 2), c = (lane & 3) * kVec<TO>;
                TO* dst = reinterpret_cast<TO*>(__shfl_sync(0xffffffffu, mine, r));
                if (dst && c < here)
                    st_piece(dst + part * kCols + c, *reinterpret_cast<const uint4*>(stage + r * kStageRow + c * sizeof(TO)));
            }
        } else {
            constexpr int kAtOnce = 32 / kCols;   // rows of a warp's store
            constexpr int kBatch = 8;             // stores on their way at once: one after the other is latency alone
            const int c = lane % kCols;
            const bool inside = c < here;
#pragma unroll 1
            for (int r0 = 0; r0 < 32; r0 += kAtOnce * kBatch) {
                TO v[kBatch];
                TO* dst[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int r = r0 + kAtOnce * i + lane / kCols;
                    dst[i] = reinterpret_cast<TO*>(__shfl_sync(0xffffffffu, mine, r));
                    v[i] = *reinterpret_cast<const TO*>(stage + r * kStageRow + c * sizeof(TO));
                }
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
                    if (dst[i] && inside) dst[i][part * kCols + c] = v[i];
            }
        }
    }
}

// Writes columns [c0, c1) of this warp's rows of a tile in TMEM (zeros where
// tmem is kNoTile); row: where column 0 of lane l's row goes.
constexpr uint32_t kNoTile = 0xffffffffu;
template <typename TO>
__device__ __forceinline__ void store_tile(uint32_t tmem, int c0, int c1, TO* row, bool wide, unsigned char* stage, int lane) {
    for (int c = c0; c < c1; c += 32) {
        uint32_t w[32];
        float f[32];
        if (tmem != kNoTile) {
            tmem_ld32(tmem + c, w);
            tmem_ld_wait();
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) w[i] = 0;
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(w[i]);
        emit32<TO>(f, imin(32, c1 - c), row ? row + c : nullptr, wide, stage, lane);
    }
}

// Columns [c0, c1) of the tile at `to` += those at `from`, rounded to nearest.
__device__ __forceinline__ void add_tile(uint32_t to, uint32_t from, int c0, int c1) {
#pragma unroll 1
    for (int c = c0; c < c1; c += 16) {
        uint32_t a[16], b[16];
        tmem_ld16(to + c, a);
        tmem_ld16(from + c, b);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) a[i] = __float_as_uint(__uint_as_float(a[i]) + __uint_as_float(b[i]));
        tmem_st16(to + c, a);
    }
    tmem_st_wait();
}

// The two buffers of a tile's sums in TMEM, as both sides go through them: the
// parity of the barriers of each one's fill.  fp32 operands take them in turn, a
// chunk each.  A 16-bit tile starts in the one that the tile before did not, and
// the other one takes what comes after kLongSum elements, over and over.
template <typename T>
struct Buffers {
    uint32_t parity = 0;   // bit b: of buffer b
    __device__ __forceinline__ uint32_t of(int b, int n) const { return (kSums<T> > 1 ? n >> 1 : parity >> b) & 1; }
    __device__ __forceinline__ void used(int b) {
        if (kSums<T> == 1) parity ^= 1u << b;
    }
};

// acc += the three sums, `apart` columns from each other, of 32 columns of an
// fp32 product's chunk, the smallest first; 16 columns at a time, for the
// registers.
__device__ __forceinline__ void add_chunk(uint32_t from, int apart, float (&acc)[32]) {
#pragma unroll
    for (int at = 0; at < 32; at += 16) {
        float sum[16];
#pragma unroll
        for (int i = 2; i >= 0; --i) {
            uint32_t w[16];
            tmem_ld16(from + i * apart + at, w);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) sum[j] = i == 2 ? __uint_as_float(w[j]) : sum[j] + __uint_as_float(w[j]);
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[at + j] += sum[j];
    }
}

// The copies of a loader warp that are on their way, told of (an arrival at the
// stage's full barrier) as they land.  kCopyGroups groups of warps take the
// stages in turn: waiting, fencing and telling of one stage takes longer than its
// products (32768 bf16 rows, 1024 -> 1024, us with one, two and four groups:
// 83, 72 and 66).
constexpr int kCopyGroups = 4, kCopyWarps = kLoaderWarps / kCopyGroups;
template <int S>
struct Copies {
    int next, told;     // stages, counted from the kernel's start
    int ahead = 0;      // stages copied and not told of
    __device__ __forceinline__ explicit Copies(int group) : next(group), told(group) {}
    __device__ __forceinline__ int stage() const { return next % S; }
    // Waits for the oldest stage and tells of it.
    __device__ __forceinline__ void tell(uint32_t full) {
        switch (--ahead) {   // as many newer ones may still be on their way
            case 0: copies_wait<0>(); break;
            case 1: copies_wait<1>(); break;
            case 2: copies_wait<2>(); break;
            default: copies_wait<3>(); break;
        }
        fence_async_smem();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(full + 8 * (told % S));
        told += kCopyGroups;
    }
    // The next stage is free; while it is not, older ones are told of.
    __device__ __forceinline__ bool acquire(uint32_t full, uint32_t empty, volatile int* dead) {
        const uint32_t bar = empty + 8 * stage(), parity = (uint32_t)(next / S & 1) ^ 1;
        while (ahead > 0 && !__all_sync(0xffffffffu, mbar_test(bar, parity))) tell(full);
        return bounded_wait(bar, parity, dead);
    }
    __device__ __forceinline__ void issued() {
        copies_commit();
        ++ahead;
        next += kCopyGroups;
    }
    __device__ __forceinline__ void finish(uint32_t full) {
        while (ahead > 0) tell(full);
    }
};

// What every grouped kernel sets up: barriers, TMEM, the groups' starts.  Of a
// pair, both CTAs' copies are told to the first CTA's full barriers and both
// epilogues to its tempty barriers.
template <int S, uint32_t kTmemCols, int kTile, int kExtra, bool kPair = false>
struct Setup {
    static constexpr int kBytes = (2 * S + 7) * 8 + (kGroupsHeld + 2) * 4;
    uint32_t full, empty, tfull, tempty, done, tmem;
    volatile int* dead;
    Groups<kTile, kExtra> groups;
    __device__ __forceinline__ void begin(unsigned char* smem, int full_count, int epilogue_warps, const int32_t* row_ptr, int G,
                                          int M) {
        uint64_t* bars = reinterpret_cast<uint64_t*>(smem);
        dead = reinterpret_cast<volatile int*>(bars + 2 * S + 5);
        uint32_t* slot = reinterpret_cast<uint32_t*>(bars + 2 * S + 6);
        full = smem_u32(bars), empty = full + 8 * S, tfull = empty + 8 * S, tempty = tfull + 16, done = tempty + 16;
        if (threadIdx.x == 0) {
            if (kPair) epilogue_warps *= 2;
            for (int i = 0; i < S; ++i) {
                mbar_init(full + 8 * i, full_count);
                mbar_init(empty + 8 * i, 1);
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(tfull + 8 * i, 1);
                mbar_init(tempty + 8 * i, epilogue_warps);
            }
            mbar_init(done, 1);
            *dead = 0;
            mbar_fence_init();
        }
        pdl_wait();
        pdl_trigger();
        groups.hold(row_ptr, G, M, reinterpret_cast<int32_t*>(bars + 2 * S + 7));
        if ((threadIdx.x >> 5) == 2) tmem_alloc<kPair>(smem_u32(slot), kTmemCols);
        tc_fence_before();
        __syncthreads();
        if (kPair) pair_barrier();   // the other CTA's barriers are there
        tc_fence_after();
        tmem = *slot;
    }
    __device__ __forceinline__ void end() {
        tc_fence_before();
        __syncthreads();
        if (kPair) pair_barrier();   // nothing reads, or arrives at, a CTA that has left
        tc_fence_after();
        if ((threadIdx.x >> 5) == 2) tmem_free<kPair>(tmem, kTmemCols);
    }
    // Where the CTA is dead: what was issued last on each stage has landed.
    __device__ __forceinline__ void drain_copies(int issued) const {
        for (int i = 0; i < imin(issued, S); ++i) {
            const int k = issued - 1 - i;
            for (uint32_t n = 0; n < kDrainSpins && !mbar_try_wait(full + 8 * (k % S), (uint32_t)(k / S) & 1); ++n) {}
        }
    }
    __device__ __forceinline__ void drain_products() const {
        tc_commit<kPair>(done);
        for (uint32_t i = 0; i < kDrainSpins && !mbar_try_wait(done, 0); ++i) {}
    }
};

// ---------------------------------------------------------------- host

// A row-major matrix of 16-bit elements as boxes of 64 columns; depth > 0: a
// stack of that many.  False when the driver refuses.
bool encode_boxes(CUtensorMap* map, bool bf16, const void* p, int64_t cols, int64_t rows, int64_t ld, int64_t depth,
                  int box_rows);

constexpr int kSmemMost = 227 * 1024;

}  // namespace zs
