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

// Rows and columns a tile or a chunk past the last one are still numbers of 32 bits.
constexpr int64_t kMostSide = (int64_t(1) << 31) - (1 << 16);

zs_status check(const char* fn, int32_t dtype, int64_t M, int32_t K, int32_t N, int32_t G, const int32_t* row_ptr,
                const int32_t* perm, std::initializer_list<const void*> arrays) {
    if (!known_dtype(dtype)) return fail(ZS_ERR_UNSUPPORTED, "%s: dtype %d is not a zs_dtype", fn, dtype);
    if (M < 0 || M > kMostSide || K < 1 || K > kMostSide || N < 1 || N > kMostSide || G < 0)
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

// Rows of `cols` elements as whole 16-byte pieces.
int64_t padded(int32_t dtype, int64_t cols) {
    const int64_t per16 = 16 / dtype_bytes(dtype);
    return (cols + per16 - 1) / per16 * per16;
}
bool pieces(int32_t dtype, const void* p, int64_t ld) { return aligned16(p) && ld % (16 / dtype_bytes(dtype)) == 0; }

// Hands out a workspace's room for matrices that are laid out anew.
struct Padder {
    Padding list[2] = {};
    int n = 0;
    char* room;
    size_t left;
    int32_t dtype;
    // p and ld replaced by a place in the workspace; false where it does not fit, or there is nothing to do.
    bool lay_out(const void*& p, int64_t& ld, int64_t rows, int32_t cols, const int32_t* perm = nullptr) {
        const int64_t to = padded(dtype, cols);
        const size_t bytes = align_up((size_t)rows * to * dtype_bytes(dtype), 256);
        if (rows == 0 || !room || bytes > left) return false;
        list[n++] = {p, ld, rows, cols, perm, room};
        p = room;
        ld = to;
        room += bytes;
        left -= bytes;
        return true;
    }
};

// Gathered 16-bit rows are put in order first where many tiles read them again, and TMA brings them from then on (32768 bf16
// rows, us so and gathered by each tile): products of at least kOrderCols columns (216 -> 1360: 55 and 66; 512 -> 2048: 74 and
// 77; 1024 -> 4096: 200 and 238; but 256 -> 1024, 65536 rows: 67 and 58), weight gradients of at least kOrderTiles tiles
// (1024 -> 4096, 128 tiles: 350 and 447; 2048 -> 512, 32 tiles: 137 and 128).  fp32 takes its rows through registers either way.
constexpr int kOrderCols = 1280, kOrderTiles = 64;
bool order_rows(int32_t dtype, int32_t cols) { return dtype != ZS_F32 && cols >= kOrderCols; }
bool order_both(int32_t dtype, int32_t K, int32_t N) {
    return dtype != ZS_F32 && (int64_t)((N + 127) / 128) * ((K + 255) / 256) >= kOrderTiles;
}

// Fewer rows than this are not worth a copy.
constexpr int64_t kPadRows = 256;
size_t padded_bytes(int32_t dtype, int64_t rows, int32_t cols) {
    return align_up((size_t)rows * padded(dtype, cols) * dtype_bytes(dtype), 256);
}

zs_status product(const char* fn, int which, int32_t dtype, const void* a, int64_t a_ld, const void* w, const int32_t* row_ptr,
                  const int32_t* perm, int64_t M, int32_t K, int32_t N, int32_t G, void* out, int64_t out_ld, void* workspace,
                  size_t workspace_bytes, zs_stream_t stream) {
    const void* any = row_ptr;   // what is not read when a size is zero need not exist
    if (zs_status st = check(fn, dtype, M, K, N, G, row_ptr, perm, {M ? a : any, M && G ? w : any, M ? out : any})) return st;
    const int32_t in_cols = which ? N : K, out_cols = which ? K : N;
    if (zs_status st = check_ld(fn, which ? "dy_ld" : "x_ld", a_ld, in_cols, M)) return st;
    if (zs_status st = check_ld(fn, which ? "dx_ld" : "y_ld", out_ld, out_cols, M)) return st;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
        return fail(ZS_ERR_INVALID_ARG, "%s: workspace is not 256-byte aligned", fn);
    if (M == 0) return ZS_OK;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (M == 1) a_ld = in_cols;
    if (grouped_is_few(dtype, which, M, N, G)) return grouped_few(fn, dtype, which, a, a_ld, w, K, row_ptr, perm, M, K, N, G, out, out_ld, s);
    if (grouped_is_small(K, N)) return grouped_small_rows(fn, dtype, which, a, a_ld, w, row_ptr, perm, M, K, N, G, out, out_ld, s);
    int64_t w_ld = K;
    const int32_t* gather = perm;
    Padder pad{{}, 0, static_cast<char*>(workspace), workspace ? workspace_bytes : 0, dtype};
    if (M >= kPadRows) {
        if (!pieces(dtype, w, w_ld)) pad.lay_out(w, w_ld, (int64_t)G * N, K);
        const int32_t* order = dtype == ZS_F32 ? nullptr : perm;
        if ((!pieces(dtype, a, a_ld) || (order && order_rows(dtype, out_cols))) && pad.lay_out(a, a_ld, M, in_cols, order) && order)
            gather = nullptr;
        if (zs_status st = grouped_pad(fn, dtype, pad.list, s)) return st;
    }
    return grouped_rows(fn, dtype, a, a_ld, w, w_ld, row_ptr, perm, gather, M, K, N, G, out, out_ld, which != 0, s);
}

}  // namespace

}  // namespace zs

extern "C" {

zs_status zs_grouped_matmul(int32_t dtype, const void* x, int64_t x_ld, const void* w, const int32_t* row_ptr,
                            const int32_t* perm, int64_t M, int32_t K, int32_t N, int32_t G, void* y, int64_t y_ld,
                            zs_stream_t stream) {
    return zs::product("zs_grouped_matmul", 0, dtype, x, x_ld, w, row_ptr, perm, M, K, N, G, y, y_ld, nullptr, 0, stream);
}

zs_status zs_grouped_matmul_dx(int32_t dtype, const void* dy, int64_t dy_ld, const void* w, const int32_t* row_ptr,
                               const int32_t* perm, int64_t M, int32_t K, int32_t N, int32_t G, void* dx, int64_t dx_ld,
                               zs_stream_t stream) {
    return zs::product("zs_grouped_matmul_dx", 1, dtype, dy, dy_ld, w, row_ptr, perm, M, K, N, G, dx, dx_ld, nullptr, 0, stream);
}

size_t zs_grouped_matmul_workspace_bytes(int32_t dtype, int64_t M, int32_t K, int32_t N, int32_t G) {
    using namespace zs;
    if (!known_dtype(dtype) || M < kPadRows || M > kMostSide || K < 1 || N < 1 || G < 1 || grouped_is_small(K, N)) return 0;
    const bool k = padded(dtype, K) != K, n = padded(dtype, N) != N;
    return (k ? padded_bytes(dtype, (int64_t)G * N, K) : 0) +
           imax(k || order_rows(dtype, N) ? padded_bytes(dtype, M, K) : 0, n || order_rows(dtype, K) ? padded_bytes(dtype, M, N) : 0);
}

zs_status zs_grouped_matmul_ws(int32_t dtype, const void* x, int64_t x_ld, const void* w, const int32_t* row_ptr,
                               const int32_t* perm, int64_t M, int32_t K, int32_t N, int32_t G, void* y, int64_t y_ld,
                               void* workspace, size_t workspace_bytes, zs_stream_t stream) {
    return zs::product("zs_grouped_matmul_ws", 0, dtype, x, x_ld, w, row_ptr, perm, M, K, N, G, y, y_ld, workspace,
                       workspace_bytes, stream);
}

zs_status zs_grouped_matmul_dx_ws(int32_t dtype, const void* dy, int64_t dy_ld, const void* w, const int32_t* row_ptr,
                                  const int32_t* perm, int64_t M, int32_t K, int32_t N, int32_t G, void* dx, int64_t dx_ld,
                                  void* workspace, size_t workspace_bytes, zs_stream_t stream) {
    return zs::product("zs_grouped_matmul_dx_ws", 1, dtype, dy, dy_ld, w, row_ptr, perm, M, K, N, G, dx, dx_ld, workspace,
                       workspace_bytes, stream);
}

size_t zs_grouped_matmul_dw_workspace_bytes(int32_t dtype, int64_t M, int32_t K, int32_t N, int32_t G) {
    if (!zs::known_dtype(dtype) || M < 0 || M > zs::kMostSide || K < 1 || N < 1 || G < 1) return 0;
    using namespace zs;
    if (grouped_is_few(dtype, 2, M, N, G)) return 0;
    return grouped_weights_workspace(dtype, M, K, N, G);
}

size_t zs_grouped_matmul_dw_copy_bytes(int32_t dtype, int64_t M, int32_t K, int32_t N, int32_t G) {
    using namespace zs;
    if (!known_dtype(dtype) || M < kPadRows || M > kMostSide || K < 1 || N < 1 || G < 1 || grouped_is_small(K, N) ||
        grouped_is_few(dtype, 2, M, N, G))
        return 0;
    const bool both = order_both(dtype, K, N);
    return (both || padded(dtype, K) != K ? padded_bytes(dtype, M, K) : 0) + (both || padded(dtype, N) != N ? padded_bytes(dtype, M, N) : 0);
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
    if (M == 1) dy_ld = N, x_ld = K;
    // the partial sums first, then what is laid out anew; in the groups' order only both operands at once
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    Padder pad{{}, 0, static_cast<char*>(workspace) + need, workspace ? workspace_bytes - need : 0, dtype};
    if (M >= kPadRows && !grouped_is_small(K, N)) {
        const bool x_off = !pieces(dtype, x, x_ld), dy_off = !pieces(dtype, dy, dy_ld);
        if (perm && dtype != ZS_F32 && ((x_off && dy_off) || order_both(dtype, K, N)) && padded_bytes(dtype, M, K) + padded_bytes(dtype, M, N) <= pad.left &&
            pad.lay_out(x, x_ld, M, K, perm) && pad.lay_out(dy, dy_ld, M, N, perm)) {
            perm = nullptr;
        } else {
            if (x_off) pad.lay_out(x, x_ld, M, K);
            if (dy_off) pad.lay_out(dy, dy_ld, M, N);
        }
        if (zs_status st = grouped_pad(fn, dtype, pad.list, s)) return st;
    }
    return grouped_weights(fn, dtype, dy, dy_ld, x, x_ld, row_ptr, perm, M, K, N, G, dw, workspace, s);
}

}  // extern "C"
