// Rows that do not start on 16-byte boundaries, or that a CSR gathers, laid out
// anew: on such boundaries, and in the groups' order.
//
// The tensor-core products take their operands in 16-byte pieces.  Rows of an
// odd number of elements can be brought into that form as they are loaded, but
// then once for every tile that reads them; a copy costs one read and one
// write.  (us with the copy and without, fp16: 32768 rows, 217 -> 1360: y 53 and
// 192, dx 37 and 251, dw 56 and 226; 1000 rows, 131 -> 131: y 8 and 13; bf16,
// 150000 rows, 41 -> 25: y 23 and 29, dw 27 and 38.  From 256 rows on it is
// therefore always made.)  A thread makes a 16-byte piece out of the two aligned
// ones that hold it, four at a time; 32768 rows of 1363 fp16, 180 MB, take 32 us.
#include "zs_grouped.cuh"
#include "zs_types.cuh"

namespace zs {

namespace {

struct PadMatrix {
    const char* src;
    char* dst;
    const int32_t* perm;     // row of each position, or NULL: in order
    int64_t ld, rows;        // source rows in bytes
    int cols, pieces;        // bytes of a row, 16-byte pieces of a padded one
    int per_block;           // rows of a CTA
    uint32_t inverse;        // of pieces, times 2^32, rounded up (0: one row a CTA)
};
struct PadArgs {
    PadMatrix m[2];
    int64_t blocks0;         // CTAs of the first matrix
};

constexpr int kThreads = 256;
constexpr int kPerThread = 4;   // pieces of a thread that are loaded together

// The piece at byte c of the row at `at`, `end` the matrix's end.
template <int kEs>
__device__ __forceinline__ uint4 unaligned_piece(const char* at, int left, const char* end) {
    const int off = (int)(reinterpret_cast<uintptr_t>(at) & 15u);
    uint4 q = make_uint4(0, 0, 0, 0);
    uint32_t* qe = &q.x;
    if (at - off + (off ? 32 : 16) <= end) {
        const uint4* base = reinterpret_cast<const uint4*>(at - off);
        const uint4 lo = __ldg(base), hi = off ? __ldg(base + 1) : make_uint4(0, 0, 0, 0);
        const uint32_t u[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        const int sh = 8 * (off & 3);
        uint32_t v[5], t[6];   // words (off / 4) .. + 4 of u
#pragma unroll
        for (int j = 0; j < 6; ++j) t[j] = off & 8 ? u[j + 2] : u[j];
#pragma unroll
        for (int j = 0; j < 5; ++j) v[j] = off & 4 ? t[j + 1] : t[j];
#pragma unroll
        for (int j = 0; j < 4; ++j) qe[j] = __funnelshift_r(v[j], v[j + 1], sh);
        if (left < 16) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int keep = left - 4 * j;
                qe[j] = keep >= 4 ? qe[j] : keep <= 0 ? 0u : qe[j] & ((1u << (8 * keep)) - 1u);
            }
        }
    } else {                              // the matrix's last pieces, element by element
        for (int j = 0; j < imin(left, 16); j += kEs) {
            const uint32_t v = kEs == 2 ? *reinterpret_cast<const uint16_t*>(at + j) : *reinterpret_cast<const uint32_t*>(at + j);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (j >> 2 == k) qe[k] |= v << (8 * (j & 3));
        }
    }
    return q;
}

template <int kEs>
__global__ void __launch_bounds__(kThreads) pad_rows(const __grid_constant__ PadArgs a) {
    pdl_wait();
    pdl_trigger();
    const bool second = blockIdx.x >= a.blocks0;
    const PadMatrix& m = a.m[second];
    const int64_t row0 = (blockIdx.x - (second ? a.blocks0 : 0)) * m.per_block;
    const int64_t here = m.rows - row0 < m.per_block ? m.rows - row0 : m.per_block;
    const int count = (int)here * m.pieces;
    char* dst = m.dst + row0 * m.pieces * 16;
    const char* end = m.src + (m.rows - 1) * m.ld + m.cols;
    for (int p0 = threadIdx.x; p0 < count; p0 += kThreads * kPerThread) {
        uint4 q[kPerThread];
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) {
            const int p = p0 + i * kThreads;
            if (p >= count) break;
            const int r = m.pieces == 1 ? p : (int)__umulhi((uint32_t)p, m.inverse), c = (p - r * m.pieces) * 16;
            int64_t row = row0 + r;
            if (m.perm) row = __ldg(m.perm + row);
            q[i] = make_uint4(0, 0, 0, 0);
            if ((uint64_t)row < (uint64_t)m.rows) q[i] = unaligned_piece<kEs>(m.src + row * m.ld + c, m.cols - c, end);
        }
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) {
            const int p = p0 + i * kThreads;
            if (p < count) *reinterpret_cast<uint4*>(dst + (int64_t)p * 16) = q[i];
        }
    }
}

}  // namespace

// Both matrices at once (rows 0: none).
zs_status grouped_pad(const char* fn, int32_t dtype, const Padding (&p)[2], cudaStream_t s) {
    PadArgs a = {};
    const int es = dtype_bytes(dtype);
    int64_t blocks[2];
    for (int i = 0; i < 2; ++i) {
        PadMatrix& m = a.m[i];
        blocks[i] = 0;
        if (p[i].rows == 0) continue;
        m.src = static_cast<const char*>(p[i].src);
        m.dst = static_cast<char*>(p[i].dst);
        m.perm = p[i].perm;
        m.ld = p[i].ld * es;
        m.rows = p[i].rows;
        m.cols = p[i].cols * es;
        m.pieces = (m.cols + 15) / 16;
        m.per_block = imax(1, kThreads * kPerThread / m.pieces);
        // exact for p < 1024: p pieces < 2^32
        m.inverse = m.per_block > 1 ? (uint32_t)(((uint64_t(1) << 32) + m.pieces - 1) / m.pieces) : 0;
        blocks[i] = (m.rows + m.per_block - 1) / m.per_block;
    }
    if (blocks[0] + blocks[1] == 0) return ZS_OK;
    if (blocks[0] + blocks[1] >= (int64_t(1) << 31)) return fail(ZS_ERR_INVALID_ARG, "%s: operands too large", fn);
    a.blocks0 = blocks[0];
    launch(es == 2 ? pad_rows<2> : pad_rows<4>, dim3((unsigned)(blocks[0] + blocks[1])), dim3(kThreads), 0, s, a);
    return check_launch(fn);
}

}  // namespace zs
