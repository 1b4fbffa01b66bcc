// Rows in pieces: what the operators that move rows (embedding, experts'
// exchange) share.
//
// A row of C elements is P pieces of VEC elements: 16 bytes where every base
// and row stride is on 16-byte boundaries, single elements elsewhere.  Pieces
// of several rows are numbered together, so that a CTA's threads are all busy
// whatever the width.
#pragma once

#include <initializer_list>

#include "zs_types.cuh"

namespace zs {

// n / d for n < 2^31, 1 <= d < 2^31, as a product's high half, a sum and a shift.
struct FastDiv {
    uint32_t d, mul, shift;
    FastDiv() = default;
    explicit FastDiv(uint32_t d_) : d(d_), mul(0), shift(0) {
        while (shift < 31 && (1u << shift) < d) ++shift;
        mul = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << shift) - d)) / d + 1);
    }
    __device__ __forceinline__ uint32_t quotient(uint32_t n) const { return (__umulhi(n, mul) + n) >> shift; }
};

template <typename T, int VEC>
struct Row {
    static_assert(VEC == kVec<T> || VEC == 1, "16-byte pieces or elements");
    using Raw = typename std::conditional<VEC == 1, T, uint4>::type;
    static __device__ __forceinline__ Raw load(const T* row, int64_t piece) {
        if constexpr (VEC == 1) return __ldg(row + piece);
        else return __ldg(reinterpret_cast<const uint4*>(row) + piece);
    }
    // Data that is read once.
    static __device__ __forceinline__ Raw load_once(const T* row, int64_t piece) {
        if constexpr (VEC == 1) return __ldg(row + piece);
        else return ld_piece(row + piece * VEC);
    }
    static __device__ __forceinline__ Raw zero() {
        if constexpr (VEC == 1) return from_f32<T>(0.f);
        else return make_uint4(0, 0, 0, 0);
    }
    static __device__ __forceinline__ void store(T* row, int64_t piece, Raw v) {
        if constexpr (VEC == 1) row[piece] = v;
        else st_piece(row + piece * VEC, v);
    }
    static __device__ __forceinline__ void floats(Raw v, float (&f)[VEC]) {
        if constexpr (VEC == 1) f[0] = to_f32(v);
        else unpack<T>(v, f);
    }
    static __device__ __forceinline__ Raw rounded(const float (&f)[VEC]) {
        if constexpr (VEC == 1) return from_f32<T>(f[0]);
        else return pack<T>(f);
    }
};

// Whether rows of C elements at these bases and strides (in elements) are whole 16-byte pieces.
struct RowsAt {
    const void* p;
    int64_t ld;
};
inline bool whole_pieces(int32_t dtype, int32_t C, std::initializer_list<RowsAt> rows) {
    const int s = dtype_bytes(dtype);
    if ((int64_t)C * s % 16) return false;
    for (const RowsAt& r : rows)
        if (!aligned16(r.p) || r.ld * s % 16) return false;
    return true;
}

// Calls f with the element type and the elements of a piece as template arguments: f<T, VEC>(args...).
#define ZS_ROWS_DISPATCH(F, dtype, whole, ...)                                                      \
    ((dtype) == ZS_F32    ? ((whole) ? F<float, 4>(__VA_ARGS__) : F<float, 1>(__VA_ARGS__))         \
     : (dtype) == ZS_BF16 ? ((whole) ? F<__nv_bfloat16, 8>(__VA_ARGS__) : F<__nv_bfloat16, 1>(__VA_ARGS__)) \
                          : ((whole) ? F<__half, 8>(__VA_ARGS__) : F<__half, 1>(__VA_ARGS__)))

// Checks that the entry points of these operators share.
inline zs_status check_rows(const char* fn, const char* name, int32_t dtype, const void* p, int64_t ld, int64_t rows, int32_t C) {
    if (rows > 0 && !p) return fail(ZS_ERR_INVALID_ARG, "%s: %s is NULL", fn, name);
    if (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(dtype_bytes(dtype) - 1))
        return fail(ZS_ERR_INVALID_ARG, "%s: %s is not aligned to its elements", fn, name);
    if (rows > 1 && ld < C) return fail(ZS_ERR_INVALID_ARG, "%s: a row stride of %s, %lld, is below C=%d", fn, name, (long long)ld, C);
    return ZS_OK;
}
inline zs_status check_words(const char* fn, const char* name, const void* p, int64_t n) {
    if (n > 0 && !p) return fail(ZS_ERR_INVALID_ARG, "%s: %s is NULL", fn, name);
    if (reinterpret_cast<uintptr_t>(p) & 3) return fail(ZS_ERR_INVALID_ARG, "%s: %s is not aligned to its elements", fn, name);
    return ZS_OK;
}
constexpr int64_t kMaxRows = ((int64_t)1 << 31) - (1 << 16);   // rows and columns of one call

// Rows copied from where `Source` says, times a factor.  A CTA takes `rows`
// rows of P pieces, or where a row is wider than its tile, a tile of a row.
constexpr int kMoveThreads = 256;

struct MoveShape {
    int64_t M;
    int32_t P, rows, tile;   // pieces of a row, rows of a CTA, pieces of a CTA's part of a row
    FastDiv per_row;         // by the pieces of a CTA's part of a row
    int32_t ctas_x, ctas_y;
};

// Threads take up to `each` pieces; fewer where that leaves SMs without a CTA.
inline MoveShape move_shape(int64_t M, int32_t P, int each) {
    MoveShape s = {};
    int64_t tile = (int64_t)kMoveThreads * each;
    while (tile > kMoveThreads && M * P < tile * num_sms()) tile /= 2;
    s.M = M;
    s.P = P;
    s.tile = (int32_t)imin<int64_t>(P, tile);
    s.rows = (int32_t)imax<int64_t>(1, tile / P);
    s.per_row = FastDiv((uint32_t)s.tile);
    s.ctas_x = (int32_t)((M + s.rows - 1) / s.rows);
    s.ctas_y = (int32_t)imin<int64_t>(65535, (P + s.tile - 1) / s.tile);
    return s;
}

template <typename T, int VEC, int U, typename Source>
__global__ void __launch_bounds__(kMoveThreads) move_rows(MoveShape s, Source src, const T* __restrict__ x, int64_t x_ld, float factor,
                                                          T* __restrict__ y, int64_t y_ld) {
    using R = Row<T, VEC>;
    pdl_wait();
    pdl_trigger();
    const int64_t r0 = (int64_t)blockIdx.x * s.rows;
    const int rows = (int)imin<int64_t>(s.rows, s.M - r0);
    for (int64_t c0 = (int64_t)blockIdx.y * s.tile; c0 < s.P; c0 += (int64_t)gridDim.y * s.tile) {
        const int cols = (int)imin<int64_t>(s.tile, s.P - c0);
        const int n = rows * s.tile;
        for (int t0 = threadIdx.x; t0 < n; t0 += U * kMoveThreads) {
            typename R::Raw v[U];
            int row[U], col[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int t = t0 + u * kMoveThreads;
                row[u] = (int)s.per_row.quotient((uint32_t)t);
                col[u] = t - row[u] * s.tile;
                v[u] = R::zero();
                if (t < n && col[u] < cols) {
                    const int64_t from = src.row(r0 + row[u], c0 + col[u] == 0);
                    if (from >= 0) v[u] = R::load(x + from * x_ld, c0 + col[u]);
                } else {
                    row[u] = -1;
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (row[u] < 0) continue;
                if (Source::kScaled) {
                    float f[VEC];
                    R::floats(v[u], f);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) f[i] *= factor;
                    v[u] = R::rounded(f);
                }
                R::store(y + (r0 + row[u]) * y_ld, c0 + col[u], v[u]);
            }
        }
    }
}

}  // namespace zs
