#include "zs_norm_kernels.cuh"

namespace zs {
template zs_status norm_forward<__nv_bfloat16>(NormArgs& a, cudaStream_t s);
template zs_status norm_backward<__nv_bfloat16>(NormArgs& a, cudaStream_t s);
}  // namespace zs
