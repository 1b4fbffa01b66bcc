// The grouped products behind the C entry points.
#pragma once

#include "zs_common.cuh"

namespace zs {

zs_status grouped_rows(const char* fn, int32_t dtype, const void* x, int64_t x_ld, const void* w, const int32_t* row_ptr,
                       const int32_t* perm, int64_t M, int32_t K, int32_t N, int32_t G, void* out, int64_t out_ld,
                       bool transposed, cudaStream_t s);
size_t grouped_weights_workspace(int32_t dtype, int64_t M, int32_t K, int32_t N, int32_t G);
zs_status grouped_weights(const char* fn, int32_t dtype, const void* dy, int64_t dy_ld, const void* x, int64_t x_ld,
                          const int32_t* row_ptr, const int32_t* perm, int64_t M, int32_t K, int32_t N, int32_t G, void* dw,
                          void* workspace, cudaStream_t s);

}  // namespace zs
