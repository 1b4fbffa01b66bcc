// C entry points of the products grouped by a CSR over rows, and the tensor
// maps their kernels load through.
#include <cuda.h>

#include <initializer_list>

#include "zs_grouped.cuh"
#include "zs_mma.cuh"

namespace zs {

bool encode_boxes(CUtensorMap* map, bool bf16, const void* p, int64_t cols, int64_t rows, int64_t ld, int64_t depth,
                  int box_rows) {
    using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Encode encode = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        cudaGetLastError();
        return reinterpret_cast<Encode>(f);
    }();
    if (!encode) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)depth};
    const cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)ld * 2 * (cuuint64_t)rows};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1}, one[3] = {1, 1, 1};
    return encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, depth > 0 ? 3 : 2,
                  const_cast<void*>(p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

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
    if (grouped_is_few(dtype, 0, M, N, G)) return grouped_few(fn, dtype, 0, x, x_ld, w, K, row_ptr, perm, M, K, N, G, y, y_ld, s);
    if (grouped_is_small(K, N)) return grouped_small_rows(fn, dtype, 0, x, x_ld, w, row_ptr, perm, M, K, N, G, y, y_ld, s);
    return grouped_rows(fn, dtype, x, M > 1 ? x_ld : K, w, row_ptr, perm, M, K, N, G, y, y_ld, false, s);
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
    if (grouped_is_few(dtype, 1, M, N, G)) return grouped_few(fn, dtype, 1, dy, dy_ld, w, K, row_ptr, perm, M, K, N, G, dx, dx_ld, s);
    if (grouped_is_small(K, N)) return grouped_small_rows(fn, dtype, 1, dy, dy_ld, w, row_ptr, perm, M, K, N, G, dx, dx_ld, s);
    return grouped_rows(fn, dtype, dy, M > 1 ? dy_ld : N, w, row_ptr, perm, M, K, N, G, dx, dx_ld, true, s);
}

size_t zs_grouped_matmul_dw_workspace_bytes(int32_t dtype, int64_t M, int32_t K, int32_t N, int32_t G) {
    if (!zs::known_dtype(dtype) || M < 0 || M >= (int64_t(1) << 31) || K < 1 || N < 1 || G < 1) return 0;
    return zs::grouped_is_few(dtype, 2, M, N, G) ? 0 : zs::grouped_weights_workspace(dtype, M, K, N, G);
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
    if (grouped_is_few(dtype, 2, M, N, G))
        return grouped_few(fn, dtype, 2, dy, dy_ld, x, x_ld, row_ptr, perm, M, K, N, G, dw, K, reinterpret_cast<cudaStream_t>(stream));
    return grouped_weights(fn, dtype, dy, M > 1 ? dy_ld : N, x, M > 1 ? x_ld : K, row_ptr, perm, M, K, N, G, dw, workspace,
                           reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
