// Matrix products grouped by a CSR over rows: y[i] = w[g(i)] x[i], its
// gradient in x (w transposed) and its gradient in w (sums of outer
// products over a group's rows).
#include <initializer_list>

#include "zs_types.cuh"

namespace zs {

namespace {

constexpr int kTile = 64, kStep = 16, kThreads = 256;

struct Operand {
    const void* p;
    int64_t ld;
};

// Rows of a product are cut into tiles of kTile positions within a group.
// Group g starts at slot floor(row_ptr[g] / kTile) + g, which leaves room for
// each group's tiles without a prefix sum; the positions of no group follow
// as group G.  A slot past its group's last tile is empty.
struct Slot {
    int g, p0, p1;   // positions [p0, p1) of group g
};
__device__ __forceinline__ int group_start(const int32_t* row_ptr, int g, int G, int64_t M) {
    if (g > G) return (int)M;
    const int v = __ldg(row_ptr + g);
    return v < 0 ? 0 : v > M ? (int)M : v;
}
__device__ __forceinline__ Slot find_slot(const int32_t* row_ptr, int G, int64_t M, int slot) {
    int lo = 0, hi = G + 1;   // start(lo) <= slot < start(hi)
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (group_start(row_ptr, mid, G, M) / kTile + mid <= slot) lo = mid; else hi = mid;
    }
    Slot s;
    s.g = lo;
    const int b = group_start(row_ptr, lo, G, M), e = group_start(row_ptr, lo + 1, G, M);
    const int64_t p0 = b + (int64_t)(slot - (b / kTile + lo)) * kTile;
    s.p0 = (int)imin<int64_t>(p0, e);
    s.p1 = (int)imin<int64_t>(p0 + kTile, e);
    return s;
}
__device__ __forceinline__ int row_of(const int32_t* perm, int64_t M, int p, int p1) {
    if (p >= p1) return -1;
    const int r = perm ? __ldg(perm + p) : p;
    return (uint32_t)r < (uint64_t)M ? r : -1;
}

// acc += a (kStep x kTile) outer b (kStep x kTile), 4 x 4 a thread.
__device__ __forceinline__ void accumulate(const float (&a)[kStep][kTile + 4], const float (&b)[kStep][kTile + 4],
                                           float (&acc)[4][4]) {
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
#pragma unroll
    for (int k = 0; k < kStep; ++k) {
        float av[4], bv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) av[i] = a[k][ty * 4 + i], bv[i] = b[k][tx * 4 + i];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
    }
}

// out[row, n] = sum_k a[row, k] * w[g, n * sn + k * sk], n < Nout, k < Kred.
template <typename T>
__global__ void __launch_bounds__(kThreads) rows_simple(Operand a, const T* __restrict__ w, int64_t sn, int64_t sk,
                                                        const int32_t* __restrict__ row_ptr, const int32_t* __restrict__ perm,
                                                        int64_t M, int Kred, int Nout, int G, T* out, int64_t out_ld) {
    __shared__ float as[kStep][kTile + 4], bs[kStep][kTile + 4];
    __shared__ int rows[kTile];
    pdl_wait();
    pdl_trigger();
    const Slot s = find_slot(row_ptr, G, M, blockIdx.x);
    if (s.p0 >= s.p1) return;
    const int n0 = blockIdx.y * kTile;
    if (threadIdx.x < kTile) rows[threadIdx.x] = row_of(perm, M, s.p0 + threadIdx.x, s.p1);
    __syncthreads();
    float acc[4][4] = {};
    if (s.g < G) {
        const T* wg = w + (int64_t)s.g * Kred * Nout;
        for (int k0 = 0; k0 < Kred; k0 += kStep) {
            for (int i = threadIdx.x; i < kTile * kStep; i += kThreads) {
                const int k = i % kStep, r = i / kStep, row = rows[r], n = n0 + r;
                const bool kin = k0 + k < Kred;
                as[k][r] = kin && row >= 0 ? to_f32(static_cast<const T*>(a.p)[row * a.ld + k0 + k]) : 0.f;
                bs[k][r] = kin && n < Nout ? to_f32(wg[n * sn + (k0 + k) * sk]) : 0.f;
            }
            __syncthreads();
            accumulate(as, bs, acc);
            __syncthreads();
        }
    }
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = rows[ty * 4 + i];
        if (row < 0) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = n0 + tx * 4 + j;
            if (n < Nout) out[row * out_ld + n] = from_f32<T>(acc[i][j]);
        }
    }
}

// dw[g, n, k] = sum over the rows of g of dy[row, n] * x[row, k].
template <typename T>
__global__ void __launch_bounds__(kThreads) weights_simple(Operand dy, Operand x, const int32_t* __restrict__ row_ptr,
                                                           const int32_t* __restrict__ perm, int64_t M, int K, int N, int G,
                                                           T* dw) {
    __shared__ float as[kStep][kTile + 4], bs[kStep][kTile + 4];
    pdl_wait();
    pdl_trigger();
    const int ktiles = (K + kTile - 1) / kTile;
    const int g = blockIdx.x, n0 = blockIdx.y / ktiles * kTile, k0 = blockIdx.y % ktiles * kTile;
    const int b = group_start(row_ptr, g, G, M), e = group_start(row_ptr, g + 1, G, M);
    float acc[4][4] = {};
    for (int p = b; p < e; p += kStep) {
        for (int i = threadIdx.x; i < kTile * kStep; i += kThreads) {
            const int c = i % kTile, m = i / kTile, row = row_of(perm, M, p + m, e);
            as[m][c] = row >= 0 && n0 + c < N ? to_f32(static_cast<const T*>(dy.p)[row * dy.ld + n0 + c]) : 0.f;
            bs[m][c] = row >= 0 && k0 + c < K ? to_f32(static_cast<const T*>(x.p)[row * x.ld + k0 + c]) : 0.f;
        }
        __syncthreads();
        accumulate(as, bs, acc);
        __syncthreads();
    }
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = n0 + ty * 4 + i, k = k0 + tx * 4 + j;
            if (n < N && k < K) dw[((int64_t)g * N + n) * K + k] = from_f32<T>(acc[i][j]);
        }
}

template <typename T>
zs_status rows_product(const char* fn, Operand a, const void* w, int64_t sn, int64_t sk, const int32_t* row_ptr,
                       const int32_t* perm, int64_t M, int Kred, int Nout, int G, void* out, int64_t out_ld, cudaStream_t s) {
    const dim3 grid((unsigned)(M / kTile + G + 2), (unsigned)((Nout + kTile - 1) / kTile));
    launch(rows_simple<T>, grid, dim3(kThreads), 0, s, a, static_cast<const T*>(w), sn, sk, row_ptr, perm, M, Kred, Nout, G,
           static_cast<T*>(out), out_ld);
    return check_launch(fn);
}

template <typename T>
zs_status weights_product(const char* fn, Operand dy, Operand x, const int32_t* row_ptr, const int32_t* perm, int64_t M,
                          int K, int N, int G, void* dw, cudaStream_t s) {
    const dim3 grid((unsigned)G, (unsigned)(((K + kTile - 1) / kTile) * ((N + kTile - 1) / kTile)));
    launch(weights_simple<T>, grid, dim3(kThreads), 0, s, dy, x, row_ptr, perm, M, K, N, G, static_cast<T*>(dw));
    return check_launch(fn);
}

zs_status check(const char* fn, int32_t dtype, int64_t M, int32_t K, int32_t N, int32_t G, const int32_t* row_ptr,
                const int32_t* perm, std::initializer_list<const void*> arrays) {
    if (!known_dtype(dtype)) return fail(ZS_ERR_UNSUPPORTED, "%s: dtype %d is not a zs_dtype", fn, dtype);
    if (M < 0 || M >= (int64_t(1) << 31) || K < 1 || N < 1 || G < 0)
        return fail(ZS_ERR_INVALID_ARG, "%s: M=%lld K=%d N=%d G=%d", fn, (long long)M, K, N, G);
    if (!row_ptr) return fail(ZS_ERR_INVALID_ARG, "%s: row_ptr is NULL", fn);
    if ((reinterpret_cast<uintptr_t>(row_ptr) | reinterpret_cast<uintptr_t>(perm)) & 3)
        return fail(ZS_ERR_INVALID_ARG, "%s: row_ptr or perm is not 4-byte aligned", fn);
    for (const void* p : arrays) {
        if (!p) return fail(ZS_ERR_INVALID_ARG, "%s: a NULL array", fn);
        if (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(dtype_bytes(dtype) - 1))
            return fail(ZS_ERR_INVALID_ARG, "%s: an array is not aligned to its elements", fn);
    }
    return ZS_OK;
}

zs_status check_ld(const char* fn, const char* what, int64_t ld, int64_t cols, int64_t M) {
    if (ld < cols && M > 1)
        return fail(ZS_ERR_INVALID_ARG, "%s: %s=%lld is below the row length %lld", fn, what, (long long)ld, (long long)cols);
    return ZS_OK;
}

}  // namespace

}  // namespace zs

extern "C" {

zs_status zs_grouped_matmul(int32_t dtype, const void* x, int64_t x_ld, const void* w, const int32_t* row_ptr,
                            const int32_t* perm, int64_t M, int32_t K, int32_t N, int32_t G, void* y, int64_t y_ld,
                            zs_stream_t stream) {
    using namespace zs;
    const char* fn = "zs_grouped_matmul";
    const void* any = row_ptr;   // what is not read when a size is zero need not exist
    if (zs_status st = check(fn, dtype, M, K, N, G, row_ptr, perm, {M ? x : any, M && G ? w : any, M ? y : any})) return st;
    if (zs_status st = check_ld(fn, "x_ld", x_ld, K, M)) return st;
    if (zs_status st = check_ld(fn, "y_ld", y_ld, N, M)) return st;
    if (M == 0) return ZS_OK;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const Operand a{x, x_ld};
    switch (dtype) {
        case ZS_F32: return rows_product<float>(fn, a, w, K, 1, row_ptr, perm, M, K, N, G, y, y_ld, s);
        case ZS_BF16: return rows_product<__nv_bfloat16>(fn, a, w, K, 1, row_ptr, perm, M, K, N, G, y, y_ld, s);
        default: return rows_product<__half>(fn, a, w, K, 1, row_ptr, perm, M, K, N, G, y, y_ld, s);
    }
}

zs_status zs_grouped_matmul_dx(int32_t dtype, const void* dy, int64_t dy_ld, const void* w, const int32_t* row_ptr,
                               const int32_t* perm, int64_t M, int32_t K, int32_t N, int32_t G, void* dx, int64_t dx_ld,
                               zs_stream_t stream) {
    using namespace zs;
    const char* fn = "zs_grouped_matmul_dx";
    const void* any = row_ptr;
    if (zs_status st = check(fn, dtype, M, K, N, G, row_ptr, perm, {M ? dy : any, M && G ? w : any, M ? dx : any})) return st;
    if (zs_status st = check_ld(fn, "dy_ld", dy_ld, N, M)) return st;
    if (zs_status st = check_ld(fn, "dx_ld", dx_ld, K, M)) return st;
    if (M == 0) return ZS_OK;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const Operand a{dy, dy_ld};
    switch (dtype) {
        case ZS_F32: return rows_product<float>(fn, a, w, 1, K, row_ptr, perm, M, N, K, G, dx, dx_ld, s);
        case ZS_BF16: return rows_product<__nv_bfloat16>(fn, a, w, 1, K, row_ptr, perm, M, N, K, G, dx, dx_ld, s);
        default: return rows_product<__half>(fn, a, w, 1, K, row_ptr, perm, M, N, K, G, dx, dx_ld, s);
    }
}

size_t zs_grouped_matmul_dw_workspace_bytes(int32_t dtype, int64_t M, int32_t K, int32_t N, int32_t G) {
    (void)dtype, (void)M, (void)K, (void)N, (void)G;   // the simple kernel keeps its sums in registers
    return 0;
}

zs_status zs_grouped_matmul_dw(int32_t dtype, const void* dy, int64_t dy_ld, const void* x, int64_t x_ld,
                               const int32_t* row_ptr, const int32_t* perm, int64_t M, int32_t K, int32_t N, int32_t G,
                               void* dw, void* workspace, size_t workspace_bytes, zs_stream_t stream) {
    using namespace zs;
    const char* fn = "zs_grouped_matmul_dw";
    const void* any = row_ptr;
    if (zs_status st = check(fn, dtype, M, K, N, G, row_ptr, perm, {M && G ? dy : any, M && G ? x : any, G ? dw : any}))
        return st;
    if (zs_status st = check_ld(fn, "dy_ld", dy_ld, N, M)) return st;
    if (zs_status st = check_ld(fn, "x_ld", x_ld, K, M)) return st;
    const size_t need = zs_grouped_matmul_dw_workspace_bytes(dtype, M, K, N, G);
    if (workspace_bytes < need || (need && !workspace))
        return fail(ZS_ERR_INVALID_ARG, "%s: workspace of %zu bytes, %zu needed", fn, workspace_bytes, need);
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
        return fail(ZS_ERR_INVALID_ARG, "%s: workspace is not 256-byte aligned", fn);
    if (G == 0) return ZS_OK;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const Operand d{dy, dy_ld}, a{x, x_ld};
    switch (dtype) {
        case ZS_F32: return weights_product<float>(fn, d, a, row_ptr, perm, M, K, N, G, dw, s);
        case ZS_BF16: return weights_product<__nv_bfloat16>(fn, d, a, row_ptr, perm, M, K, N, G, dw, s);
        default: return weights_product<__half>(fn, d, a, row_ptr, perm, M, K, N, G, dw, s);
    }
}

}  // extern "C"
