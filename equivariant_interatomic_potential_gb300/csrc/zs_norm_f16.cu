#include "zs_norm_kernels.cuh"

namespace zs {
template zs_status norm_forward<__half>(NormArgs& a, cudaStream_t s);
template zs_status norm_backward<__half>(NormArgs& a, cudaStream_t s);
}  // namespace zs
