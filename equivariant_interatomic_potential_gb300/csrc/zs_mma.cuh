// What the grouped products share: tcgen05 products of 128-row tiles with
// operands in shared memory and fp32 sums in TMEM, the rings that feed them,
// and the walk over the groups of a CSR.
//
// Operand boxes.  Every operand tile is made of boxes of rows of 64
// contiguous 16-bit elements (128 bytes), eight rows to a 1024-byte atom
// whose 16-byte pieces are permuted by the 128-byte swizzle (piece c of row r
// sits at piece c ^ (r & 7)).  Where the contiguous direction is the one
// summed over, a box holds all of the tile's rows (K-major); where it is not,
// a box holds 64 summed-over rows and the tile takes a box for every 64 of
// its own rows (MN-major).  Either way a box is the plain image of a piece of
// a row-major matrix, so TMA, or a warp that reads a row, writes it.
//
// fp32 operands are cut into three bf16 planes by truncation, 8 + 8 + 8 bits
// of the 24, which loses nothing; the six products of planes whose weights
// reach 2^-16 are summed (what is left out is below 2^-23 of a term).  That
// costs six bf16 products instead of fp32's rate on the CUDA cores, a factor
// of about four in time where the product is the bound.
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
constexpr int kBoxCols = 64;                   // elements of a box's row
constexpr int kBoxRow = 128;                   // bytes
constexpr uint32_t kDrainSpins = 1u << 16;

template <typename T>
constexpr int kPlanes = sizeof(T) == 4 ? 3 : 1;

// ---------------------------------------------------------------- barriers

// dead: set by the first wait of the CTA that runs out; the others give up
// soon after.
__device__ __forceinline__ bool bounded_wait(uint32_t bar, uint32_t parity, volatile int* dead) {
    for (uint32_t i = 0; i < kMaxSpins; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 63) == 63 && *dead) return false;
    }
    note_timeout();
    *dead = 1;
    return false;
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(bar) : "memory");
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

__device__ __forceinline__ void tmem_alloc(uint32_t dst_smem, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(dst_smem), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(addr), "r"(cols) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" :: "r"(bar) : "memory");
}
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate) : "memory");
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
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Shared-memory operand descriptor of boxes with the 128-byte swizzle.  Both
// forms step 1024 bytes (sbo) per 8 box rows; lbo is the distance between
// the boxes of an MN-major tile (unused by a K-major one).
__device__ __forceinline__ uint64_t box_desc(uint32_t addr, uint32_t lbo) {
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)((lbo & 0x3FFFFu) >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
// Descriptor address steps of one product's 16 summed-over elements: 32 bytes
// along a K-major row, 16 rows of an MN-major box.
template <bool kMN>
constexpr uint32_t kDescStep = (kMN ? 16 * kBoxRow : 32) >> 4;

// Instruction descriptor: 16-bit operands, fp32 sums, 128 x n tile.
template <typename T>
__device__ __forceinline__ uint32_t instr_desc(bool a_mn, bool b_mn, int n) {
    constexpr uint32_t type = sizeof(T) == 4 || std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;   // bf16 (planes too) or f16
    return (1u << 4) | (type << 7) | (type << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kTileM >> 4) << 24);
}

// The products of one stage: `steps` times 16 summed-over elements.
template <typename T, bool kAMN, bool kBMN>
__device__ __forceinline__ void issue_stage(uint32_t d, uint32_t a, uint32_t a_plane, uint32_t a_lbo, uint32_t b,
                                            uint32_t b_plane, uint32_t b_lbo, uint32_t idesc, int steps, bool accumulate) {
    const uint64_t a0 = box_desc(a, a_lbo), b0 = box_desc(b, b_lbo);
    for (int k = 0; k < steps; ++k) {
        const uint64_t ak = a0 + k * kDescStep<kAMN>, bk = b0 + k * kDescStep<kBMN>;
        if constexpr (kPlanes<T> == 1) {
            tc_mma(d, ak, bk, idesc, accumulate || k > 0);
        } else {
            // the small products first
            const uint32_t ap = a_plane >> 4, bp = b_plane >> 4;
            tc_mma(d, ak + 2 * ap, bk, idesc, accumulate || k > 0);
            tc_mma(d, ak + ap, bk + bp, idesc, true);
            tc_mma(d, ak, bk + 2 * bp, idesc, true);
            tc_mma(d, ak + ap, bk, idesc, true);
            tc_mma(d, ak, bk + bp, idesc, true);
            tc_mma(d, ak, bk, idesc, true);
        }
    }
}

// ---------------------------------------------------------------- TMA

__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
                 :: "r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
}
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
                 :: "r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}
// Four rows of a map whose box is one row high.
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap* map, int x, int4 rows, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];"
                 :: "r"(dst), "l"(map), "r"(x), "r"(rows.x), "r"(rows.y), "r"(rows.z), "r"(rows.w), "r"(bar) : "memory");
}

// ---------------------------------------------------------------- rows read by warps

// How a matrix is read: rows `ld` elements apart, `cols` wide; pairs: every
// pair of elements that starts at an even column is aligned to the pair.
struct Matrix {
    const void* p;
    int64_t ld;
    int cols;
    bool pairs;
};

// Elements 2 i and 2 i + 1 of a row from column c0 on, zeros past its end.
template <typename T>
struct alignas(2 * sizeof(T)) Pair {
    T a, b;
};
template <typename T>
__device__ __forceinline__ Pair<T> load_pair(const Matrix& m, int64_t row, int c) {
    const T* p = static_cast<const T*>(m.p) + row * m.ld + c;
    Pair<T> v;
    if (m.pairs && c + 1 < m.cols) {
        if constexpr (sizeof(T) == 4) {
            const float2 f = __ldg(reinterpret_cast<const float2*>(p));
            v.a = f.x, v.b = f.y;
        } else {
            const uint32_t w = __ldg(reinterpret_cast<const unsigned int*>(p));
            const unsigned short lo = (unsigned short)w, hi = (unsigned short)(w >> 16);
            v.a = *reinterpret_cast<const T*>(&lo), v.b = *reinterpret_cast<const T*>(&hi);
        }
    } else {
        v.a = c < m.cols ? p[0] : from_f32<T>(0.f);
        v.b = c + 1 < m.cols ? p[1] : from_f32<T>(0.f);
    }
    return v;
}

// The bf16 planes of a value: x = plane 0 + plane 1 + plane 2 exactly.  A
// value that is not finite stays whole in plane 0.
__device__ __forceinline__ void split3(float x, uint32_t (&b)[3]) {
    const uint32_t u = __float_as_uint(x);
    const bool fin = (u & 0x7f800000u) != 0x7f800000u;
    const float r1 = x - __uint_as_float(u & 0xffff0000u);
    const uint32_t u1 = __float_as_uint(r1) & 0xffff0000u;
    const float r2 = r1 - __uint_as_float(u1);
    const uint32_t quiet = (u & 0x007fffffu) ? 0x00400000u : 0u;   // a NaN keeps a bit of its payload
    b[0] = (fin ? u : u | quiet) >> 16;
    b[1] = fin ? u1 >> 16 : 0u;
    b[2] = fin ? __float_as_uint(r2) >> 16 : 0u;
}

// Writes the pair at (row r, elements 2 lane and 2 lane + 1) of a box.
template <typename T>
__device__ __forceinline__ void store_pair(unsigned char* box, uint32_t plane, int r, int lane, Pair<T> v) {
    const int at = r * kBoxRow + (((lane >> 2) ^ (r & 7)) << 4) + ((lane & 3) << 2);
    if constexpr (sizeof(T) == 4) {
        uint32_t x[3], y[3];
        split3(v.a, x);
        split3(v.b, y);
#pragma unroll
        for (int i = 0; i < 3; ++i) *reinterpret_cast<uint32_t*>(box + i * plane + at) = x[i] | (y[i] << 16);
    } else {
        *reinterpret_cast<Pair<T>*>(box + at) = v;
    }
}

// ---------------------------------------------------------------- groups of a CSR

// The positions of the groups, cut into slots of kRows positions: group g
// starts at slot floor(row_ptr[g] / kRows) + g, which leaves room for each
// group's pieces without a prefix sum.  A slot past its group's last piece is
// empty.  start(G + 1) is M: the positions of no group are "group" G.
template <int kRows>
struct Groups {
    const int32_t* row_ptr;
    int G, M;
    __device__ __forceinline__ int start(int g) const {
        if (g > G) return M;
        const int v = __ldg(row_ptr + g);
        return v < 0 ? 0 : v > M ? M : v;
    }
    __device__ __forceinline__ int64_t slot(int g) const { return (int64_t)(start(g) / kRows) + g; }
    // the group whose slots hold `s` (0 <= s < slot(last)), among groups [0, last)
    __device__ __forceinline__ int find(int64_t s, int last) const {
        int lo = 0, hi = last;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (slot(mid) <= s) lo = mid; else hi = mid;
        }
        return lo;
    }
};

// ---------------------------------------------------------------- epilogue

// A warp's 32 rows x 128 bytes of results pass through shared memory (rows
// 144 bytes apart) so that they leave as whole row segments.
constexpr int kStageRow = 144;
constexpr int kStageWarp = 32 * kStageRow;

// Writes columns [0, cols) of this warp's 32 rows of the TMEM tile at `tmem`
// (zeros where tmem is kNoTile): lane l's row goes to `row` (NULL: nowhere),
// 16 bytes at a time where `wide`.
constexpr uint32_t kNoTile = 0xffffffffu;
template <typename TO>
__device__ __forceinline__ void store_tile(uint32_t tmem, int cols, TO* row, bool wide, unsigned char* stage, int lane) {
    constexpr int kCols = 128 / (int)sizeof(TO);   // columns of a 128-byte segment
    for (int c0 = 0; c0 < cols; c0 += kCols) {
        uint32_t w[32];   // the segment, as 32-bit words
#pragma unroll
        for (int half = 0; half < kCols / 32; ++half) {
            uint32_t f[32];
            if (tmem != kNoTile) {
                if (c0 + 32 * half < cols) tmem_ld32(tmem + c0 + 32 * half, f);
                tmem_ld_wait();
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) f[i] = 0;
            }
            if constexpr (sizeof(TO) == 4) {
#pragma unroll
                for (int i = 0; i < 32; ++i) w[i] = f[i];
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    Pair<TO> v;
                    v.a = from_f32<TO>(__uint_as_float(f[2 * i]));
                    v.b = from_f32<TO>(__uint_as_float(f[2 * i + 1]));
                    w[16 * half + i] = *reinterpret_cast<uint32_t*>(&v);
                }
            }
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint4*>(stage + lane * kStageRow + 16 * i) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        __syncwarp();
        const int left = cols - c0 < kCols ? cols - c0 : kCols;
        const unsigned long long mine = reinterpret_cast<unsigned long long>(row);
        if (wide) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = 4 * i + (lane >> 3), c = (lane & 7) * kVec<TO>;
                TO* dst = reinterpret_cast<TO*>(__shfl_sync(0xffffffffu, mine, r));
                if (dst && c < left) st_piece(dst + c0 + c, *reinterpret_cast<const uint4*>(stage + r * kStageRow + c * sizeof(TO)));
            }
        } else {
            for (int r = 0; r < 32; ++r) {
                TO* dst = reinterpret_cast<TO*>(__shfl_sync(0xffffffffu, mine, r));
                if (!dst) continue;
                for (int c = lane; c < left; c += 32) dst[c0 + c] = *reinterpret_cast<const TO*>(stage + r * kStageRow + c * sizeof(TO));
            }
        }
    }
}

// ---------------------------------------------------------------- host

// A row-major matrix of 16-bit elements as boxes of 64 columns; depth > 0: a
// stack of that many.  False when the driver refuses.
bool encode_boxes(CUtensorMap* map, bool bf16, const void* p, int64_t cols, int64_t rows, int64_t ld, int64_t depth,
                  int box_rows);

constexpr int kSmemMost = 227 * 1024;

}  // namespace zs
