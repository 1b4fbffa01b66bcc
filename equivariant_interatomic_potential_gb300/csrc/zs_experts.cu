// The way of rows to several groups (experts) and back: an assignment is a row
// i and one of its k choices j, a = i k + j; the CSR of the assignments' groups
// puts them in the groups' order.
//
//   dispatch   xs[p] = x[perm[p] / k], slot[perm[p]] = p
//   combine    y[i] = sum_j weights[i,j] h[slot[i,j]]
//   backward   dh[slot[i,j]] = weights[i,j] dy[i], dweights[i,j] = <dy[i], h[slot[i,j]]>
//
// All three are bound by memory: (1 + k) rows for each row of x, in and out.  32768
// rows of 1024 bf16, 8 choices: 94, 97 and 176 us, 6.4, 6.2 and 6.5 TB/s.
#include "zs_rows.cuh"

namespace zs {
namespace {

constexpr int kChoices = 8;   // rows that a thread has in flight

struct AssignmentSource {
    static constexpr bool kScaled = false, kAgain = false;
    const int32_t *row_ptr, *perm;
    int32_t G, R;             // R assignments
    FastDiv by_k;
    int32_t* slot;
    __device__ __forceinline__ int32_t row(int32_t p, bool first) const {
        const int32_t a = __ldg(perm + p);
        if ((uint32_t)a >= (uint32_t)R) return -1;
        const bool held = p < __ldg(row_ptr + G);
        if (first) slot[a] = held ? p : -1;
        return held ? (int32_t)by_k.quotient((uint32_t)a) : -1;
    }
};

// slot alone, from perm.
__global__ void __launch_bounds__(kMoveThreads) invert(int32_t R, const int32_t* __restrict__ end, const int32_t* __restrict__ perm,
                                                       int32_t* __restrict__ slot) {
    pdl_wait();
    pdl_trigger();
    const int64_t p = (int64_t)blockIdx.x * kMoveThreads + threadIdx.x;
    if (p >= R) return;
    const int32_t a = __ldg(perm + p);
    if ((uint32_t)a < (uint32_t)R) slot[a] = p < __ldg(end) ? (int32_t)p : -1;
}

// Zeros in the rows of the result from row_ptr[G] on.
template <typename R, typename T>
__device__ __forceinline__ void clear_rows_behind(const int32_t* __restrict__ end, int32_t rows, T* to, int64_t ld, int32_t P, int32_t C) {
    if (blockIdx.y != 0) return;
    for (int64_t p = (int64_t)imax(__ldg(end), 0) + blockIdx.x; p < rows; p += gridDim.x)
        for (int c = threadIdx.x; c < P; c += blockDim.x) R::template store<true>(to + p * ld, R::column(to + p * ld, c), C, R::zero());
}

// Each row of x to its slots: x is read once, whatever k.
template <typename T, bool kWhole>
__global__ void __launch_bounds__(kMoveThreads) spread_rows(MoveShape s, int32_t k, int32_t R, Rows<T> x,
                                                            const int32_t* __restrict__ slot, const int32_t* __restrict__ end,
                                                            T* __restrict__ xs) {
    using Rw = Row<T, kWhole>;
    pdl_wait();
    pdl_trigger();
    for_pieces<1>(s, [&](const int32_t(&row)[1], const int32_t(&piece)[1]) {
        if (row[0] < 0) return;
        const int32_t* at = slot + (int64_t)row[0] * k;
        uint4 v = Rw::zero();
        if (kWhole) v = Rw::join(Rw::template load<false>(x, row[0], piece[0] * Rw::N, s.C));
        for (int j0 = 0; j0 < k; j0 += kChoices) {
            int32_t p[kChoices];
#pragma unroll
            for (int j = 0; j < kChoices; ++j) p[j] = j0 + j < k ? __ldg(at + j0 + j) : -1;
#pragma unroll
            for (int j = 0; j < kChoices; ++j) {
                if ((uint32_t)p[j] >= (uint32_t)R) continue;
                T* to = xs + (int64_t)p[j] * s.C;
                const int32_t e = Rw::column(to, piece[0]);
                if (!kWhole) v = Rw::template join<true>(Rw::template load<true>(x, row[0], e, s.C));   // to each slot's phase, from L1
                Rw::template store<true>(to, e, s.C, v);
            }
        }
    });
    clear_rows_behind<Rw>(end, R, xs, s.C, s.P, s.C);
}

template <typename T, bool kWhole>
zs_status dispatch(const void* x, int64_t x_ld, const int32_t* row_ptr, const int32_t* perm, int32_t R, int32_t k, int32_t G, int32_t C,
                   void* xs, int32_t* slot, cudaStream_t s) {
    using Rw = Row<T, kWhole>;
    const Rows<T> from(x, R / k, x_ld, C);
    T* to = static_cast<T*>(xs);
    // One kernel that reads a row of x for each of xs; from 8 MB of xs on two, the second of which reads x once (8 choices
    // of 1024 bf16: 1 MB 1.8 against 2.9 us, 8 MB 3.8 and 3.8, 64 MB 14.6 and 11.3, 512 MB 156 and 93).
    if (k > 1 && (int64_t)R * C * (int64_t)sizeof(T) >= 8 << 20) {
        launch(invert, dim3((R + kMoveThreads - 1) / kMoveThreads), dim3(kMoveThreads), 0, s, R, row_ptr + G, perm, slot);
        const MoveShape shape = move_shape(R / k, Rw::pieces(C), C, 1);
        launch(spread_rows<T, kWhole>, dim3(shape.ctas_x, shape.ctas_y), dim3(kMoveThreads), 0, s, shape, k, R, from,
               (const int32_t*)slot, row_ptr + G, to);
    } else {
        constexpr int U = 4;
        const MoveShape shape = move_rows_shape<T, kWhole>(R, C, U);
        launch(move_rows<T, kWhole, U, AssignmentSource>, dim3(shape.ctas_x, shape.ctas_y), dim3(kMoveThreads), 0, s, shape,
               AssignmentSource{row_ptr, perm, G, R, FastDiv((uint32_t)k), slot}, from, 1.f, to, (int64_t)C);
    }
    return check_launch("dispatch");
}

// U pieces of a thread at a time and KJ choices of each: four or eight loads in flight and four or five CTAs an SM.  More
// loads and fewer CTAs are slower (8 choices of 1024 bf16, 32768 rows: 106 us at 3 CTAs, 97 at 4; 2 choices of 256, 256 MB:
// 8 loads at 3 CTAs 111, 4 at 5 84), staging slots in shared memory too (115 to 188): the read of rows in any order is the
// limit, 0.93 of the copy rate.  (Two choices of two 16-bit pieces do not fit the 48 registers of five CTAs: 56 bytes of
// stores and 76 of loads are spilled; four CTAs have not been measured.)  Where rows have phases of their own a load is of
// two words, and two choices at a time are the most that five CTAs' registers hold (8 choices of 301 fp16, 256 MB: 79 us;
// four at four CTAs 87, eight at three 90).
template <typename T, bool kWhole, int KJ, int U>
__global__ void __launch_bounds__(kMoveThreads, KJ == kChoices ? 4 : 5) combine_rows(
    MoveShape s, int32_t k, int32_t R, Rows<T> h, const int32_t* __restrict__ slot, const float* __restrict__ weights, T* __restrict__ y,
    int64_t y_ld) {
    using Rw = Row<T, kWhole>;
    constexpr int N = Rw::N;
    pdl_wait();
    pdl_trigger();
    for_pieces<U>(s, [&](const int32_t(&row)[U], const int32_t(&piece)[U]) {
        float sum[U][N] = {};
        for (int j0 = 0; j0 < k; j0 += KJ) {
            typename Rw::Loaded v[U][KJ];
            float w[U][KJ];
            bool held[U][KJ];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int j = 0; j < KJ; ++j) {
                    held[u][j] = false;
                    if (row[u] < 0 || j0 + j >= k) continue;
                    const int64_t a = (int64_t)row[u] * k + j0 + j;
                    const int32_t p = __ldg(slot + a);
                    held[u][j] = (uint32_t)p < (uint32_t)R;
                    if (!held[u][j]) continue;
                    v[u][j] = Rw::template load<false>(h, p, Rw::column(y + (int64_t)row[u] * y_ld, piece[u]), s.C);
                    w[u][j] = weights ? __ldg(weights + a) : 1.f;
                }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int j = 0; j < KJ; ++j) {
                    if (!held[u][j]) continue;
                    float f[N];
                    unpack<T>(Rw::join(v[u][j]), f);
#pragma unroll
                    for (int i = 0; i < N; ++i) sum[u][i] = fmaf(w[u][j], f[i], sum[u][i]);
                }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (row[u] < 0) continue;
            T* to = y + (int64_t)row[u] * y_ld;
            Rw::template store<false>(to, Rw::column(to, piece[u]), s.C, pack<T>(sum[u]));
        }
    });
}

template <typename T, bool kWhole>
zs_status combine(const void* h, int64_t h_ld, const int32_t* slot, const float* weights, int64_t M, int32_t k, int32_t R, int32_t C,
                  void* y, int64_t y_ld, cudaStream_t s) {
    auto go = [&](auto choices, auto pieces) {
        constexpr int KJ = decltype(choices)::value, U = decltype(pieces)::value;
        const MoveShape shape = move_shape(M, Row<T, kWhole>::pieces(C), C, U);
        launch(combine_rows<T, kWhole, KJ, U>, dim3(shape.ctas_x, shape.ctas_y), dim3(kMoveThreads), 0, s, shape, k, R,
               Rows<T>(h, R, h_ld, C), slot, weights, static_cast<T*>(y), y_ld);
    };
    using std::integral_constant;
    if (k <= 2 || !kWhole) go(integral_constant<int, 2>(), integral_constant<int, kWhole ? 2 : 1>());
    else if constexpr (kWhole) {
        if (k <= 4) go(integral_constant<int, 4>(), integral_constant<int, 1>());
        else go(integral_constant<int, kChoices>(), integral_constant<int, 1>());
    }
    return check_launch("combine");
}

// The sums of the `lanes` threads (a power of two) of a row, at its first one.
constexpr int kBackThreads = 256;
template <int KJ>
__device__ __forceinline__ void sum_of_row(float (&dot)[KJ], int lanes, int lane, float (*part)[KJ]) {
#pragma unroll
    for (int j = 0; j < KJ; ++j)
        for (int o = imin(lanes, 32) >> 1; o > 0; o >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
    if (lanes > 32) {
        const int warp = threadIdx.x >> 5;
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int j = 0; j < KJ; ++j) part[warp][j] = dot[j];
        __syncthreads();
        if (lane == 0)
#pragma unroll
            for (int j = 0; j < KJ; ++j)
                for (int q = 1; q < lanes / 32; ++q) dot[j] += part[warp + q][j];
        __syncthreads();
    }
}

// `lanes` threads for a row i of dy, which they read once for each KJ of its choices: their rows of h in flight together, the
// products with dy in fp32 registers until the row's end (of 80 registers, of which eight choices spill 8 to 36 bytes).
// Memory: 32768 rows, 8 choices of 1024 bf16: 176 us, 0.95 of the copy rate.
template <typename T, bool kWhole, int KJ>
__global__ void __launch_bounds__(kBackThreads, 3) combine_rows_backward(
    int64_t M, int32_t k, int32_t R, int32_t P, int32_t C, int lane_bits, Rows<T> dy, Rows<T> h, const int32_t* __restrict__ slot,
    const float* __restrict__ weights, const int32_t* __restrict__ end, T* __restrict__ dh, float* __restrict__ dweights) {
    using Rw = Row<T, kWhole, sizeof(T) == 4>;
    constexpr int N = Rw::N;
    __shared__ float part[kBackThreads / 32][KJ];
    pdl_wait();
    pdl_trigger();
    const int lanes = 1 << lane_bits, lane = threadIdx.x & (lanes - 1);
    const int64_t i = (int64_t)blockIdx.x * (kBackThreads >> lane_bits) + (threadIdx.x >> lane_bits);
    const bool live = i < M;
    for (int j0 = 0; j0 < k; j0 += KJ) {
        float dot[KJ] = {}, w[KJ];
        int32_t at[KJ];
#pragma unroll
        for (int j = 0; j < KJ; ++j) {
            at[j] = -1;
            w[j] = 0.f;
            if (!live || j0 + j >= k) continue;
            const int32_t p = __ldg(slot + i * k + j0 + j);
            if ((uint32_t)p >= (uint32_t)R) continue;
            at[j] = p;
            w[j] = __ldg(weights + i * k + j0 + j);
        }
        if (live) {
            for (int c = lane; c < P; c += lanes) {
                const int32_t e = Rw::column(dh, c);
                float g[N];
                unpack<T>(Rw::join(Rw::template load<true>(dy, i, e, C)), g);
                uint4 v[KJ];
#pragma unroll
                for (int j = 0; j < KJ; ++j)
                    if (at[j] >= 0) v[j] = Rw::join(Rw::template load<false>(h, at[j], e, C));
#pragma unroll
                for (int j = 0; j < KJ; ++j) {
                    if (at[j] < 0) continue;
                    float f[N], scaled[N];
                    unpack<T>(v[j], f);
#pragma unroll
                    for (int q = 0; q < N; ++q) {
                        dot[j] = fmaf(g[q], f[q], dot[j]);
                        scaled[q] = w[j] * g[q];
                    }
                    Rw::template store<true>(dh + (int64_t)at[j] * C, e, C, pack<T>(scaled));
                }
            }
        }
        sum_of_row(dot, lanes, lane, part);
        if (live && lane == 0)
#pragma unroll
            for (int j = 0; j < KJ; ++j)
                if (j0 + j < k) dweights[i * k + j0 + j] = at[j] >= 0 ? dot[j] : 0.f;
    }
    clear_rows_behind<Rw>(end, R, dh, C, P, C);
}

// The same where rows have phases of their own: dy is shifted to each slot's (from L1), so that nothing is gained by a
// thread that takes a piece of all choices.  The threads go through the pieces of all choices instead (`chunk` pieces of a
// row at a time, all of it but for the widest rows), and no more of them idle than the last round leaves: fp16, 3 choices
// of 301, 256 MB: 208 us, where a thread for a piece of all choices took 378; two pieces of a thread at a time no less.
// What bounds it is issue slots.
template <typename T, int KJ>
__global__ void __launch_bounds__(kBackThreads, KJ == kChoices ? 4 : 5) combine_rows_backward_any(
    int64_t M, int32_t k, int32_t R, int32_t P, int32_t C, int lane_bits, int32_t chunk, FastDiv by_chunk, Rows<T> dy, Rows<T> h,
    const int32_t* __restrict__ slot, const float* __restrict__ weights, const int32_t* __restrict__ end, T* __restrict__ dh,
    float* __restrict__ dweights) {
    using Rw = Row<T, false>;
    constexpr int N = Rw::N;
    __shared__ float part[kBackThreads / 32][KJ];
    pdl_wait();
    pdl_trigger();
    const int lanes = 1 << lane_bits, lane = threadIdx.x & (lanes - 1);
    const int64_t i = (int64_t)blockIdx.x * (kBackThreads >> lane_bits) + (threadIdx.x >> lane_bits);
    const bool live = i < M;
    for (int j0 = 0; j0 < k; j0 += KJ) {
        float dot[KJ] = {};
        const int64_t a = i * k + j0;
        const int items = live ? imin(KJ, k - j0) * chunk : 0;
        for (int64_t c0 = 0; c0 < P; c0 += chunk)
            for (int t = lane; t < items; t += lanes) {
                const int j = (int)by_chunk.quotient((uint32_t)t);
                const int64_t c = c0 + (t - j * chunk);
                const int32_t p = c < P ? __ldg(slot + a + j) : -1;
                if ((uint32_t)p >= (uint32_t)R) continue;
                T* to = dh + (int64_t)p * C;
                const int32_t e = Rw::column(to, (int32_t)c);
                const typename Rw::Loaded v = Rw::template load<false>(h, p, e, C), d = Rw::template load<true>(dy, i, e, C);
                const float w = __ldg(weights + a + j);
                float f[N], g[N], product = 0.f;
                Rw::floats(Rw::template join<true>(v), e, C, f);
                Rw::floats(Rw::join(d), e, C, g);
#pragma unroll
                for (int q = 0; q < N; ++q) {
                    product = fmaf(g[q], f[q], product);
                    g[q] *= w;
                }
                Rw::template store<true>(to, e, C, pack<T>(g));
#pragma unroll
                for (int q = 0; q < KJ; ++q) dot[q] += q == j ? product : 0.f;
            }
        sum_of_row(dot, lanes, lane, part);
        if (live && lane == 0)
#pragma unroll
            for (int q = 0; q < KJ; ++q)   // 0 without a slot
                if (j0 + q < k) dweights[a + q] = dot[q];
    }
    clear_rows_behind<Rw>(end, R, dh, C, P, C);
}

template <typename T, bool kWhole>
zs_status combine_backward(const void* dy, int64_t dy_ld, const void* h, int64_t h_ld, const int32_t* slot, const float* weights,
                           const int32_t* end, int64_t M, int32_t k, int32_t C, void* dh, float* dweights, cudaStream_t s) {
    using Rw = Row<T, kWhole, sizeof(T) == 4>;
    const int32_t P = Rw::pieces(C), chunk = imin(P, 1 << 20);
    const int KJ = k <= 4 ? 4 : kChoices;
    const int64_t items = Rw::kOnePhase ? P : (int64_t)chunk * imin(k, KJ);
    // enough threads a row that no one takes more than one piece, or so many that every SM has work
    int lane_bits = 0;
    while (lane_bits < 5 && 1 << lane_bits < items) ++lane_bits;
    while (1 << lane_bits < kBackThreads && 1 << lane_bits < items && M << lane_bits < (int64_t)num_sms() * 512) ++lane_bits;
    const int64_t rows = kBackThreads >> lane_bits;
    const dim3 grid((unsigned)((M + rows - 1) / rows)), block(kBackThreads);
    const int32_t R = (int32_t)(M * k);
    const Rows<T> g(dy, M, dy_ld, C), v(h, R, h_ld, C);
    T* to = static_cast<T*>(dh);
    if constexpr (Rw::kOnePhase) {
        auto kernel = KJ == 4 ? combine_rows_backward<T, kWhole, 4> : combine_rows_backward<T, kWhole, kChoices>;
        launch(kernel, grid, block, 0, s, M, k, R, P, C, lane_bits, g, v, slot, weights, end, to, dweights);
    } else {
        auto kernel = KJ == 4 ? combine_rows_backward_any<T, 4> : combine_rows_backward_any<T, kChoices>;
        launch(kernel, grid, block, 0, s, M, k, R, P, C, lane_bits, chunk, FastDiv((uint32_t)chunk), g, v, slot, weights, end, to, dweights);
    }
    return check_launch("combine gradient");
}

zs_status check(const char* fn, int32_t dtype, int64_t M, int32_t k, int32_t G, int32_t C) {
    if (!known_dtype(dtype)) return fail(ZS_ERR_UNSUPPORTED, "%s: dtype %d is not a zs_dtype", fn, dtype);
    if (M < 0 || k < 1 || G < 0 || C < 1) return fail(ZS_ERR_INVALID_ARG, "%s: M=%lld k=%d G=%d C=%d", fn, (long long)M, k, G, C);
    if (M > kMaxRows || M * k > kMaxRows || C > kMaxRows)
        return fail(ZS_ERR_INVALID_ARG, "%s: M * k=%lld or C=%d is above 2^31 - 2^16", fn, (long long)M * k, C);
    return ZS_OK;
}

}  // namespace
}  // namespace zs

extern "C" {

zs_status zs_dispatch(int32_t dtype, const void* x, int64_t x_ld, const int32_t* row_ptr, const int32_t* perm, int64_t M, int32_t k,
                      int32_t G, int32_t C, void* xs, int32_t* slot, zs_stream_t stream) {
    using namespace zs;
    const char* fn = "zs_dispatch";
    if (zs_status st = check(fn, dtype, M, k, G, C)) return st;
    if (M == 0) return ZS_OK;
    const int64_t R = M * k;
    if (zs_status st = check_rows(fn, "x", dtype, x, x_ld, M, C)) return st;
    if (zs_status st = check_rows(fn, "xs", dtype, xs, C, R, C)) return st;
    if (zs_status st = check_words(fn, "row_ptr", row_ptr, 1)) return st;
    if (zs_status st = check_words(fn, "perm", perm, R)) return st;
    if (zs_status st = check_words(fn, "slot", slot, R)) return st;
    if (M < 2) x_ld = C;
    const bool whole = whole_pieces(dtype, C, {{x, x_ld}, {xs, C}});
    return ZS_ROWS_DISPATCH(dispatch, dtype, whole, x, x_ld, row_ptr, perm, (int32_t)R, k, G, C, xs, slot,
                            reinterpret_cast<cudaStream_t>(stream));
}

zs_status zs_combine(int32_t dtype, const void* h, int64_t h_ld, const int32_t* slot, const float* weights, int64_t M, int32_t k,
                     int64_t R, int32_t C, void* y, int64_t y_ld, zs_stream_t stream) {
    using namespace zs;
    const char* fn = "zs_combine";
    if (zs_status st = check(fn, dtype, M, k, 0, C)) return st;
    if (R < 0 || R > kMaxRows) return fail(ZS_ERR_INVALID_ARG, "%s: R=%lld is outside [0, 2^31 - 2^16]", fn, (long long)R);
    if (M == 0) return ZS_OK;
    if (zs_status st = check_rows(fn, "h", dtype, h, h_ld, R, C)) return st;
    if (zs_status st = check_rows(fn, "y", dtype, y, y_ld, M, C)) return st;
    if (zs_status st = check_words(fn, "slot", slot, M)) return st;
    if (zs_status st = check_words(fn, "weights", weights, 0)) return st;
    if (R < 2) h_ld = C;
    if (M < 2) y_ld = C;
    const bool whole = whole_pieces(dtype, C, {{h, h_ld}, {y, y_ld}});
    return ZS_ROWS_DISPATCH(combine, dtype, whole, h, h_ld, slot, weights, M, k, (int32_t)R, C, y, y_ld,
                            reinterpret_cast<cudaStream_t>(stream));
}

zs_status zs_combine_backward(int32_t dtype, const void* dy, int64_t dy_ld, const void* h, int64_t h_ld, const int32_t* slot,
                              const float* weights, const int32_t* row_ptr, int64_t M, int32_t k, int32_t G, int32_t C, void* dh,
                              float* dweights, zs_stream_t stream) {
    using namespace zs;
    const char* fn = "zs_combine_backward";
    if (zs_status st = check(fn, dtype, M, k, G, C)) return st;
    if (M == 0) return ZS_OK;
    const int64_t R = M * k;
    if (zs_status st = check_rows(fn, "dy", dtype, dy, dy_ld, M, C)) return st;
    if (zs_status st = check_rows(fn, "h", dtype, h, h_ld, R, C)) return st;
    if (zs_status st = check_rows(fn, "dh", dtype, dh, C, R, C)) return st;
    if (zs_status st = check_words(fn, "slot", slot, R)) return st;
    if (zs_status st = check_words(fn, "weights", weights, R)) return st;
    if (zs_status st = check_words(fn, "row_ptr", row_ptr, 1)) return st;
    if (zs_status st = check_words(fn, "dweights", dweights, R)) return st;
    if (M < 2) dy_ld = C;
    if (R < 2) h_ld = C;
    const bool whole = whole_pieces(dtype, C, {{dy, dy_ld}, {h, h_ld}, {dh, C}});
    return ZS_ROWS_DISPATCH(combine_backward, dtype, whole, dy, dy_ld, h, h_ld, slot, weights, row_ptr + G, M, k, C, dh, dweights,
                            reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
