// Rows in pieces: what the operators that move rows (embedding, experts'
// exchange) share.
//
// A row is written in aligned pieces of 16 bytes.  Where every base and row
// stride is on 16-byte boundaries and the width is whole pieces (kWhole), those
// are the row's own.  Elsewhere (odd widths, views at odd offsets) each row of
// the result has its own phase: its first and last piece are written element by
// element, and a piece is read from another row's phase as two aligned 16-byte
// words that are shifted together (fp16 rows of 301 dispatched, 64 MB: 94 us
// element by element, 25 so).  Pieces of several rows are numbered together, so
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
// The 16 bytes at offset o (below 16, whole elements) of two words in a row.
template <typename T>
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
    if constexpr (sizeof(T) == 4) return make_uint4(w[0], w[1], w[2], w[3]);
    const int s = 8 * (o & 2);
    return make_uint4(__funnelshift_r(w[0], w[1], s), __funnelshift_r(w[1], w[2], s), __funnelshift_r(w[2], w[3], s),
                      __funnelshift_r(w[3], w[4], s));
}

// A matrix that is read: rows ld apart.  Around `inner` rows from row `margin` on there are three pieces and more of it on both
// sides.
template <typename T>
struct Rows {
    const T* p;
    int64_t ld;
    int32_t margin;
    uint32_t inner;
    Rows(const void* p_, int64_t rows, int64_t ld_, int32_t C)
        : p(static_cast<const T*>(p_)), ld(ld_) {
        margin = (int32_t)((3 * kVec<T> + (int64_t)C - 1) / C);   // a row takes C and more
        inner = rows > 2 * (int64_t)margin ? (uint32_t)(rows - 2 * margin) : 0u;
    }
};

// Pieces of rows of C elements.  kCached: rows that are read again soon.  kLane: rows of fp32 that are not whole pieces, read
// and written element by element: of P pieces, piece c has the columns c, c + P, c + 2 P, ... in all rows.  It takes fewer
// instructions than two words that are shifted, but more traffic, of 128 bytes that lie across two lines: it is taken where
// instructions are the limit (647170 x 95 looked up 65 us against 78, their gradient 84 against 108; but 256 MB, dispatched
// to 8 slots at a time, 73 against 53, and combined 97 against 76).
template <typename T, bool kWhole, bool kLane = false>
struct Row {
    static constexpr int N = kVec<T>;                       // elements of a piece
    static constexpr bool kStrided = !kWhole && kLane;
    static constexpr bool kOnePhase = kWhole || kStrided;   // a piece has the same columns in all rows

    // Pieces that cover a row, whatever its phase.
    static __host__ __device__ __forceinline__ int32_t pieces(int32_t C) {
        return kWhole ? C / N : (int32_t)(((int64_t)C + (kStrided ? N - 1 : 2 * N - 2)) / N);
    }
    // The column of the first element of piece c of a row of the result at `to`: below 0 where the row starts inside it.
    static __device__ __forceinline__ int32_t column(const T* to, int32_t c) {
        if (kStrided) return c;
        return c * N - (kWhole ? 0 : (int32_t)((uint32_t)reinterpret_cast<uintptr_t>(to) & 15u) / (int32_t)sizeof(T));
    }
    // Which of the columns [e, e + N) are in the row, as bits.
    static __device__ __forceinline__ uint32_t inside(int32_t e, int32_t C) {
        return ((1u << imin(imax(C - e, 0), N)) - 1u) & (~0u << imax(-e, 0));
    }
    // The piece of a row of m at column e, in flight: the aligned words that hold it, and the offset in these.  Nothing waits
    // for the words before join(), so that a thread's loads are all on their way together.
    struct Loaded {
        uint4 a, b;
        int o;
    };
    template <bool kCached>
    static __device__ __forceinline__ Loaded load(const Rows<T>& m, int32_t i, int32_t e, int32_t C) {
        const T* row = m.p + i * m.ld;
        Loaded v;
        if constexpr (kWhole) {
            v.a = kCached ? ld_cached(row + e) : ld_piece(row + e);
        } else if constexpr (kStrided) {
            static_assert(sizeof(T) == 4, "32-bit elements");
            uint32_t w[N];
#pragma unroll
            for (int q = 0; q < N; ++q) {
                const int64_t at = e + (int64_t)q * pieces(C);
                w[q] = at < C ? __ldg(reinterpret_cast<const uint32_t*>(row) + at) : 0u;
            }
            v.a = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            v.o = (int)(reinterpret_cast<uintptr_t>(row + e) & 15u);
            v.b = zero();
            if ((uint32_t)(i - m.margin) < m.inner || (e >= N && e + 2 * N <= C)) {
                const T* first = row + (e - v.o / (int)sizeof(T));
                v.a = ld_cached(first);
                if (v.o) v.b = ld_cached(first + N);
            } else {   // at the ends of rows near those of m, where a word may reach out of it: element by element
                constexpr int kBits = 8 * sizeof(T);
                v.o = 0;
                v.a = zero();
#pragma unroll 1
                for (int q = N - 1; q >= 0; --q) {
                    Piece<T> one;
                    one.raw = zero();
                    if (e + q >= 0 && e + q < C) one.e[0] = __ldg(row + e + q);
                    v.a.w = __funnelshift_lc(v.a.z, v.a.w, kBits);
                    v.a.z = __funnelshift_lc(v.a.y, v.a.z, kBits);
                    v.a.y = __funnelshift_lc(v.a.x, v.a.y, kBits);
                    v.a.x = __funnelshift_lc(0, v.a.x, kBits) | one.raw.x;
                }
            }
        }
        return v;
    }
    // Its elements; those outside the row hold anything.  kOften: rows of the same phase are frequent, which need no shift.
    template <bool kOften = false>
    static __device__ __forceinline__ uint4 join(const Loaded& v) {
        if constexpr (kWhole || kStrided) return v.a;
        else if constexpr (kOften) return v.o ? shifted<T>(v.a, v.b, v.o) : v.a;
        else return shifted<T>(v.a, v.b, v.o);
    }
    // Their values, zeros outside the row.
    static __device__ __forceinline__ void floats(uint4 v, int32_t e, int32_t C, float (&f)[N]) {
        unpack<T>(v, f);
        if (!kWhole && !kStrided && (e < 0 || e + N > C)) {
            const uint32_t in = inside(e, C);
#pragma unroll
            for (int q = 0; q < N; ++q) f[q] = in >> q & 1u ? f[q] : 0.f;
        }
    }
    // The piece of a row of the result at column e, as far as it is in it.  kInPhase: e is a column(), on a 16-byte boundary.
    template <bool kOnce, bool kInPhase = true>
    static __device__ __forceinline__ void store(T* row, int32_t e, int32_t C, uint4 v) {
        if constexpr (kStrided) {
            const uint32_t w[N] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int q = 0; q < N; ++q) {
                const int64_t at = e + (int64_t)q * pieces(C);
                if (at < C) reinterpret_cast<uint32_t*>(row)[at] = w[q];
            }
        } else if (kWhole || (e >= 0 && e + N <= C && (kInPhase || aligned16(row + e)))) {
            if (kOnce) st_once(row + e, v);
            else st_piece(row + e, v);
        } else if (!kInPhase && sizeof(T) == 2 && e >= 0 && e + N <= C) {   // two elements at a time where they are on a boundary
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            if (reinterpret_cast<uintptr_t>(row + e) & 2u) {
                Piece<T> p;
                p.raw = v;
                row[e] = p.e[0];
#pragma unroll
                for (int q = 0; q < 3; ++q) *reinterpret_cast<uint32_t*>(row + e + 1 + 2 * q) = __funnelshift_r(w[q], w[q + 1], 16);
                row[e + N - 1] = p.e[N - 1];
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q) *reinterpret_cast<uint32_t*>(row + e + 2 * q) = w[q];
            }
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
    using R = Row<T, kWhole, sizeof(T) == 4>;
    pdl_wait();
    pdl_trigger();
    for_pieces<U>(s, [&](const int32_t(&row)[U], const int32_t(&piece)[U]) {
        typename R::Loaded in[U];
        int32_t from[U];
#pragma unroll
        for (int u = 0; u < U; ++u) from[u] = row[u] >= 0 ? src.row(row[u], piece[u] == 0) : -1;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            in[u] = {};
            if (from[u] >= 0) in[u] = R::template load<Source::kAgain>(x, from[u], R::column(y + (int64_t)row[u] * y_ld, piece[u]), s.C);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (row[u] < 0) continue;
            uint4 v = R::join(in[u]);
            if (Source::kScaled) {
                float f[R::N];
                unpack<T>(v, f);
#pragma unroll
                for (int i = 0; i < R::N; ++i) f[i] *= factor;
                v = pack<T>(f);
            }
            T* to = y + (int64_t)row[u] * y_ld;
            R::template store<true>(to, R::column(to, piece[u]), s.C, v);
        }
    });
}
template <typename T, bool kWhole>
inline MoveShape move_rows_shape(int64_t M, int32_t C, int U) {
    return move_shape(M, Row<T, kWhole, sizeof(T) == 4>::pieces(C), C, U);
}

}  // namespace zs
