#include "zs_norm_kernels.cuh"

namespace zs {
template zs_status norm_forward<float>(NormArgs& a, cudaStream_t s);
template zs_status norm_backward<float>(NormArgs& a, cudaStream_t s);
}  // namespace zs
