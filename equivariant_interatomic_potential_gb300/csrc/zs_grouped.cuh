// The grouped products behind the C entry points.
#pragma once

#include "zs_common.cuh"

namespace zs {

zs_status grouped_rows(const char* fn, int32_t dtype, const void* x, int64_t x_ld, const void* w, int64_t w_ld, const int32_t* row_ptr,
                       const int32_t* perm, const int32_t* gather, int64_t M, int32_t K, int32_t N, int32_t G, void* out, int64_t out_ld,
                       bool transposed, cudaStream_t s);
// Whether a row's operands are so short that the CUDA cores are the faster ones.
bool grouped_is_small(int32_t K, int32_t N);
// which: 0 y, 1 dx.
zs_status grouped_small_rows(const char* fn, int32_t dtype, int which, const void* a, int64_t a_ld, const void* w,
                             const int32_t* row_ptr, const int32_t* perm, int64_t M, int32_t K, int32_t N, int32_t G, void* out,
                             int64_t out_ld, cudaStream_t s);
size_t grouped_weights_workspace(int32_t dtype, int64_t M, int32_t K, int32_t N, int32_t G);
zs_status grouped_weights(const char* fn, int32_t dtype, const void* dy, int64_t dy_ld, const void* x, int64_t x_ld,
                          const int32_t* row_ptr, const int32_t* perm, int64_t M, int32_t K, int32_t N, int32_t G, void* dw,
                          void* workspace, cudaStream_t s);


// A matrix to be laid out with rows of whole 16-byte pieces, next to each other; with perm in its order (zeros for
// what is no row).
struct Padding {
    const void* src;
    int64_t ld, rows;
    int32_t cols;
    const int32_t* perm;
    void* dst;
};
zs_status grouped_pad(const char* fn, int32_t dtype, const Padding (&p)[2], cudaStream_t s);

// Whether the rows are so few that the kernels for few rows are the faster ones.
bool grouped_is_few(int32_t dtype, int which, int64_t M, int32_t N, int32_t G);
// which: 0 y (a x, b w), 1 dx (a dy, b w), 2 dw (a dy, b x).
zs_status grouped_few(const char* fn, int32_t dtype, int which, const void* a, int64_t a_ld, const void* b, int64_t b_ld,
                      const int32_t* row_ptr, const int32_t* perm, int64_t M, int32_t K, int32_t N, int32_t G, void* out,
                      int64_t out_ld, cudaStream_t s);

}  // namespace zs
