// Rows in pieces: what the operators that move rows (embedding, experts'
// exchange) share.
//
// A row is written in aligned pieces of 16 bytes.  Where every base and row
// stride is on 16-byte boundaries and the width is whole pieces (kWhole), those
// are the row's own.  Elsewhere (odd widths, views at odd offsets) each row of
// the result has its own phase: its first and last piece are written element by
// element, and a piece is read from another row's phase as two aligned 16-byte
// words that are shifted together (fp16 rows of 301 dispatched, 64 MB: 94 us
// element by element, 26 so).  Pieces of several rows are numbered together, so
// that a CTA's threads are all busy whatever the width.
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

__device__ __forceinline__ uint4 ld_cached(const void* p) { return __ldg(static_cast<const uint4*>(p)); }
__device__ __forceinline__ void st_once(void* p, uint4 v) {   // data that nothing reads again soon
    asm volatile("st.global.cs.v4.u32 [%0], {%1,%2,%3,%4};" :: "l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// The 16 bytes at offset o (0 < o < 16) of two words in a row.
__device__ __forceinline__ uint4 shifted(uint4 a, uint4 b, int o) {
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (o & 8) {
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    }
    if (o & 4) {
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
    const int s = 8 * (o & 3);
    return make_uint4(__funnelshift_r(w[0], w[1], s), __funnelshift_r(w[1], w[2], s), __funnelshift_r(w[2], w[3], s),
                      __funnelshift_r(w[3], w[4], s));
}

// A matrix that is read: rows ld apart, all of it in [p, end).  Around `inner` rows from row `margin` on there are three
// pieces and more of it on both sides.
template <typename T>
struct Rows {
    const T *p, *end;
    int64_t ld;
    int32_t margin;
    uint32_t inner;
    Rows(const void* p_, int64_t rows, int64_t ld_, int32_t C)
        : p(static_cast<const T*>(p_)), end(p + (rows > 0 ? (rows - 1) * ld_ + C : 0)), ld(ld_) {
        margin = (int32_t)((3 * kVec<T> + (int64_t)C - 1) / C);   // a row takes C and more
        inner = rows > 2 * (int64_t)margin ? (uint32_t)(rows - 2 * margin) : 0u;
    }
};

// Pieces of rows of C elements.  kCached: rows that are read again soon.
template <typename T, bool kWhole>
struct Row {
    static constexpr int N = kVec<T>;   // elements of a piece

    // Pieces that cover a row, whatever its phase.
    static int32_t pieces(int32_t C) { return kWhole ? C / N : (int32_t)(((int64_t)C + 2 * N - 2) / N); }
    // The column of the first element of piece c of a row of the result at `to`: below 0 where the row starts inside it.
    static __device__ __forceinline__ int32_t column(const T* to, int32_t c) {
        return c * N - (kWhole ? 0 : (int32_t)((uint32_t)reinterpret_cast<uintptr_t>(to) & 15u) / (int32_t)sizeof(T));
    }
    // Which of the columns [e, e + N) are in the row, as bits.
    static __device__ __forceinline__ uint32_t inside(int32_t e, int32_t C) {
        return ((1u << imin(imax(C - e, 0), N)) - 1u) & (~0u << imax(-e, 0));
    }
    // Columns [e, e + N) of a row of m; of those outside the row, whatever lies there (but nothing outside m is read).
    template <bool kCached>
    static __device__ __forceinline__ uint4 load(const Rows<T>& m, int64_t i, int32_t e, int32_t C) {
        const T* row = m.p + i * m.ld;
        if constexpr (kWhole) {
            return kCached ? ld_cached(row + e) : ld_piece(row + e);
        } else {
            const int o = (int)(reinterpret_cast<uintptr_t>(row + e) & 15u), back = o / (int)sizeof(T);
            const T *first = row + (e - back), *second = first + N;   // the aligned words that hold them
            if ((uint32_t)((int32_t)i - m.margin) < m.inner) {
                const uint4 v = ld_cached(first);
                return o ? shifted(v, ld_cached(second), o) : v;
            }
            const bool a = e - back + N > 0 && e - back < C, b = o && e - back + 2 * N > 0 && e - back + N < C;
            if ((a && (first < m.p || first + N > m.end)) || (b && (second < m.p || second + N > m.end))) {
                Piece<T> v;   // at the ends of m
#pragma unroll 1
                for (int q = 0; q < N; ++q) v.e[q] = e + q >= 0 && e + q < C ? __ldg(row + e + q) : from_f32<T>(0.f);
                return v.raw;
            }
            const uint4 v = a ? ld_cached(first) : zero();
            return o ? shifted(v, b ? ld_cached(second) : zero(), o) : v;
        }
    }
    // Their values, zeros outside the row.
    static __device__ __forceinline__ void floats(uint4 v, int32_t e, int32_t C, float (&f)[N]) {
        unpack<T>(v, f);
        if (!kWhole && (e < 0 || e + N > C)) {
            const uint32_t in = inside(e, C);
#pragma unroll
            for (int q = 0; q < N; ++q) f[q] = in >> q & 1u ? f[q] : 0.f;
        }
    }
    template <bool kCached>
    static __device__ __forceinline__ void load_floats(const Rows<T>& m, int64_t i, int32_t e, int32_t C, float (&f)[N]) {
        floats(load<kCached>(m, i, e, C), e, C, f);
    }
    // Columns [e, e + N) of a row of the result, as far as they are in it.  kInPhase: e is a column(), on a 16-byte boundary.
    template <bool kOnce, bool kInPhase = true>
    static __device__ __forceinline__ void store(T* row, int32_t e, int32_t C, uint4 v) {
        if (kWhole || (e >= 0 && e + N <= C && (kInPhase || aligned16(row + e)))) {
            if (kOnce) st_once(row + e, v);
            else st_piece(row + e, v);
        } else {
            const uint32_t in = inside(e, C);
            Piece<T> p;
            p.raw = v;
#pragma unroll
            for (int q = 0; q < N; ++q)
                if (in >> q & 1u) row[e + q] = p.e[q];
        }
    }
    static __device__ __forceinline__ uint4 zero() { return make_uint4(0, 0, 0, 0); }
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

// Calls F with the element type and whether rows are whole pieces as template arguments.
#define ZS_ROWS_DISPATCH(F, dtype, whole, ...)                                                                            \
    ((dtype) == ZS_F32    ? ((whole) ? F<float, true>(__VA_ARGS__) : F<float, false>(__VA_ARGS__))                        \
     : (dtype) == ZS_BF16 ? ((whole) ? F<__nv_bfloat16, true>(__VA_ARGS__) : F<__nv_bfloat16, false>(__VA_ARGS__))        \
                          : ((whole) ? F<__half, true>(__VA_ARGS__) : F<__half, false>(__VA_ARGS__)))

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

// Work on rows of pieces.  A CTA takes `rows` rows of P pieces, or where a row is wider than its tile, a tile of a row.
constexpr int kMoveThreads = 256;

struct MoveShape {
    int64_t M;
    int32_t P, C, rows, tile;   // pieces and elements of a row, rows of a CTA, pieces of a CTA's part of a row
    FastDiv per_row;            // by the pieces of a CTA's part of a row
    int32_t ctas_x, ctas_y;
};

// Threads take up to `each` pieces; fewer where that leaves SMs without a CTA.
inline MoveShape move_shape(int64_t M, int32_t P, int32_t C, int each) {
    MoveShape s = {};
    int64_t tile = (int64_t)kMoveThreads * each;
    while (tile > kMoveThreads && M * P < tile * num_sms()) tile /= 2;
    s.M = M;
    s.P = P;
    s.C = C;
    s.tile = (int32_t)imin<int64_t>(P, tile);
    s.rows = (int32_t)imax<int64_t>(1, tile / P);
    s.per_row = FastDiv((uint32_t)s.tile);
    s.ctas_x = (int32_t)((M + s.rows - 1) / s.rows);
    s.ctas_y = (int32_t)imin<int64_t>(65535, (P + s.tile - 1) / s.tile);
    return s;
}

// Calls f(rows, pieces) for this CTA's pieces, up to U of a thread at a time: row -1 where there is none.
template <int U, typename F>
__device__ __forceinline__ void for_pieces(const MoveShape& s, F&& f) {
    const int64_t r0 = (int64_t)blockIdx.x * s.rows;
    const int n = (int)imin<int64_t>(s.rows, s.M - r0) * s.tile;
    for (int64_t c0 = (int64_t)blockIdx.y * s.tile; c0 < s.P; c0 += (int64_t)gridDim.y * s.tile) {
        const int cols = (int)imin<int64_t>(s.tile, s.P - c0);
        for (int t0 = threadIdx.x; t0 < n; t0 += U * kMoveThreads) {
            int32_t row[U], piece[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int t = t0 + u * kMoveThreads;
                const int q = (int)s.per_row.quotient((uint32_t)t), col = t - q * s.tile;
                row[u] = t < n && col < cols ? (int32_t)(r0 + q) : -1;
                piece[u] = (int32_t)(c0 + col);
            }
            f(row, piece);
        }
    }
}

// Rows copied from where `Source` says, times a factor.
template <typename T, bool kWhole, int U, typename Source>
__global__ void __launch_bounds__(kMoveThreads) move_rows(MoveShape s, Source src, Rows<T> x, float factor, T* __restrict__ y,
                                                          int64_t y_ld) {
    using R = Row<T, kWhole>;
    pdl_wait();
    pdl_trigger();
    for_pieces<U>(s, [&](const int32_t(&row)[U], const int32_t(&piece)[U]) {
        uint4 v[U];
        int32_t from[U];
#pragma unroll
        for (int u = 0; u < U; ++u) from[u] = row[u] >= 0 ? src.row(row[u], piece[u] == 0) : -1;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            v[u] = R::zero();
            if (from[u] >= 0) v[u] = R::template load<Source::kAgain>(x, from[u], R::column(y + (int64_t)row[u] * y_ld, piece[u]), s.C);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (row[u] < 0) continue;
            if (Source::kScaled) {
                float f[R::N];
                unpack<T>(v[u], f);
#pragma unroll
                for (int i = 0; i < R::N; ++i) f[i] *= factor;
                v[u] = pack<T>(f);
            }
            T* to = y + (int64_t)row[u] * y_ld;
            R::template store<true>(to, R::column(to, piece[u]), s.C, v[u]);
        }
    });
}

}  // namespace zs
