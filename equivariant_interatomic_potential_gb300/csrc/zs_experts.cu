// The way of rows to several groups (experts) and back: an assignment is a row
// i and one of its k choices j, a = i k + j; the CSR of the assignments' groups
// puts them in the groups' order.
//
//   dispatch   xs[p] = x[perm[p] / k], slot[perm[p]] = p
//   combine    y[i] = sum_j weights[i,j] h[slot[i,j]]
//   backward   dh[slot[i,j]] = weights[i,j] dy[i], dweights[i,j] = <dy[i], h[slot[i,j]]>
//
// All three are bound by memory: (1 + k) rows for each row of x, in and out.
#include "zs_rows.cuh"

namespace zs {
namespace {

constexpr int kChoices = 8;   // rows that a thread has in flight

struct AssignmentSource {
    static constexpr bool kScaled = false;
    const int32_t *row_ptr, *perm;
    int32_t G, R;             // R assignments
    FastDiv by_k;
    int32_t* slot;
    __device__ __forceinline__ int64_t row(int64_t p, bool first) const {
        const int32_t a = __ldg(perm + p);
        if ((uint32_t)a >= (uint32_t)R) return -1;
        const bool held = p < __ldg(row_ptr + G);
        if (first) slot[a] = held ? (int32_t)p : -1;
        return held ? (int64_t)by_k.quotient((uint32_t)a) : -1;
    }
};

template <typename T, int VEC>
zs_status dispatch(const void* x, int64_t x_ld, const int32_t* row_ptr, const int32_t* perm, int32_t R, int32_t k, int32_t G, int32_t C,
                   void* xs, int32_t* slot, cudaStream_t s) {
    constexpr int U = VEC == 1 ? 8 : 4;
    const MoveShape shape = move_shape(R, C / VEC, U);
    launch(move_rows<T, VEC, U, AssignmentSource>, dim3(shape.ctas_x, shape.ctas_y), dim3(kMoveThreads), 0, s, shape,
           AssignmentSource{row_ptr, perm, G, R, FastDiv((uint32_t)k), slot}, static_cast<const T*>(x), x_ld, 1.f, static_cast<T*>(xs),
           (int64_t)C);
    return check_launch("dispatch");
}

template <typename T, int VEC>
__global__ void __launch_bounds__(kMoveThreads) combine_rows(MoveShape s, int32_t k, int32_t R, const T* __restrict__ h, int64_t h_ld,
                                                             const int32_t* __restrict__ slot, const float* __restrict__ weights,
                                                             T* __restrict__ y, int64_t y_ld) {
    using Rw = Row<T, VEC>;
    pdl_wait();
    pdl_trigger();
    const int64_t r0 = (int64_t)blockIdx.x * s.rows;
    const int n = (int)imin<int64_t>(s.rows, s.M - r0) * s.tile;
    for (int64_t c0 = (int64_t)blockIdx.y * s.tile; c0 < s.P; c0 += (int64_t)gridDim.y * s.tile) {
        const int cols = (int)imin<int64_t>(s.tile, s.P - c0);
        for (int t = threadIdx.x; t < n; t += kMoveThreads) {
            const int row = (int)s.per_row.quotient((uint32_t)t), col = t - row * s.tile;
            if (col >= cols) continue;
            const int32_t* at = slot + (r0 + row) * k;
            float sum[VEC] = {};
            for (int j0 = 0; j0 < k; j0 += kChoices) {
                typename Rw::Raw v[kChoices];
                float w[kChoices];
                bool held[kChoices];
#pragma unroll
                for (int j = 0; j < kChoices; ++j) {
                    held[j] = false;
                    if (j0 + j >= k) continue;
                    const int32_t p = __ldg(at + j0 + j);
                    held[j] = (uint32_t)p < (uint32_t)R;
                    if (!held[j]) continue;
                    v[j] = Rw::load_once(h + p * h_ld, c0 + col);
                    w[j] = weights ? __ldg(weights + (r0 + row) * k + j0 + j) : 1.f;
                }
#pragma unroll
                for (int j = 0; j < kChoices; ++j) {
                    if (!held[j]) continue;
                    float f[VEC];
                    Rw::floats(v[j], f);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) sum[i] = fmaf(w[j], f[i], sum[i]);
                }
            }
            Rw::store(y + (r0 + row) * y_ld, c0 + col, Rw::rounded(sum));
        }
    }
}

template <typename T, int VEC>
zs_status combine(const void* h, int64_t h_ld, const int32_t* slot, const float* weights, int64_t M, int32_t k, int32_t R, int32_t C,
                  void* y, int64_t y_ld, cudaStream_t s) {
    const MoveShape shape = move_shape(M, C / VEC, 1);
    launch(combine_rows<T, VEC>, dim3(shape.ctas_x, shape.ctas_y), dim3(kMoveThreads), 0, s, shape, k, R, static_cast<const T*>(h), h_ld,
           slot, weights, static_cast<T*>(y), y_ld);
    return check_launch("combine");
}

// `lanes` threads (a power of two) for a row i of dy, which they read once for its k choices.
constexpr int kBackThreads = 256;
template <typename T, int VEC>
__global__ void __launch_bounds__(kBackThreads) combine_rows_backward(
    int64_t M, int32_t k, int32_t R, int32_t P, int lanes, const T* __restrict__ dy, int64_t dy_ld, const T* __restrict__ h,
    int64_t h_ld, const int32_t* __restrict__ slot, const float* __restrict__ weights, const int32_t* __restrict__ end,
    T* __restrict__ dh, int64_t dh_ld, float* __restrict__ dweights) {
    using Rw = Row<T, VEC>;
    __shared__ float part[kBackThreads / 32][kChoices];
    pdl_wait();
    pdl_trigger();
    const int group = threadIdx.x / lanes, lane = threadIdx.x - group * lanes;
    const int64_t i = (int64_t)blockIdx.x * (kBackThreads / lanes) + group;
    const bool live = i < M;
    for (int j0 = 0; j0 < k; j0 += kChoices) {
        float dot[kChoices] = {}, w[kChoices];
        int32_t at[kChoices];
#pragma unroll
        for (int j = 0; j < kChoices; ++j) {
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
                typename Rw::Raw v[kChoices];
                const typename Rw::Raw raw = Rw::load(dy + i * dy_ld, c);
#pragma unroll
                for (int j = 0; j < kChoices; ++j)
                    if (at[j] >= 0) v[j] = Rw::load_once(h + at[j] * h_ld, c);
                float g[VEC];
                Rw::floats(raw, g);
#pragma unroll
                for (int j = 0; j < kChoices; ++j) {
                    if (at[j] < 0) continue;
                    float f[VEC], d[VEC];
                    Rw::floats(v[j], f);
#pragma unroll
                    for (int q = 0; q < VEC; ++q) {
                        dot[j] = fmaf(g[q], f[q], dot[j]);
                        d[q] = w[j] * g[q];
                    }
                    Rw::store(dh + at[j] * dh_ld, c, Rw::rounded(d));
                }
            }
        }
#pragma unroll
        for (int j = 0; j < kChoices; ++j)
            for (int o = imin(lanes, 32) >> 1; o > 0; o >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
        if (lanes > 32) {
            const int warp = threadIdx.x >> 5;
            if ((threadIdx.x & 31) == 0)
#pragma unroll
                for (int j = 0; j < kChoices; ++j) part[warp][j] = dot[j];
            __syncthreads();
            if (lane == 0)
#pragma unroll
                for (int j = 0; j < kChoices; ++j)
                    for (int q = 1; q < lanes / 32; ++q) dot[j] += part[warp + q][j];
            __syncthreads();
        }
        if (live && lane == 0)
#pragma unroll
            for (int j = 0; j < kChoices; ++j)
                if (j0 + j < k) dweights[i * k + j0 + j] = at[j] >= 0 ? dot[j] : 0.f;
    }
    // rows of dh behind the last group's
    for (int64_t p = (int64_t)imax(__ldg(end), 0) + blockIdx.x; p < R; p += gridDim.x)
        for (int c = threadIdx.x; c < P; c += kBackThreads) Rw::store(dh + p * dh_ld, c, Rw::zero());
}

template <typename T, int VEC>
zs_status combine_backward(const void* dy, int64_t dy_ld, const void* h, int64_t h_ld, const int32_t* slot, const float* weights,
                           const int32_t* end, int64_t M, int32_t k, int32_t C, void* dh, float* dweights, cudaStream_t s) {
    const int32_t P = C / VEC;
    // enough threads a row that no one takes more than one piece, or so many that every SM has work
    int lanes = 1;
    while (lanes < 32 && lanes < P) lanes *= 2;
    while (lanes < kBackThreads && lanes < P && M * lanes < (int64_t)num_sms() * 1024) lanes *= 2;
    const int64_t rows = kBackThreads / lanes;
    launch(combine_rows_backward<T, VEC>, dim3((unsigned)((M + rows - 1) / rows)), dim3(kBackThreads), 0, s, M, k, (int32_t)(M * k), P,
           lanes, static_cast<const T*>(dy), dy_ld, static_cast<const T*>(h), h_ld, slot, weights, end, static_cast<T*>(dh), (int64_t)C,
           dweights);
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
