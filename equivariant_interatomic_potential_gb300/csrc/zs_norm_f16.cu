#include "zs_norm_kernels.cuh"

namespace zs {
template zs_status norm_forward<__half>(NormArgs& a, cudaStream_t s);
template zs_status norm_backward<__half>(NormArgs& a, cudaStream_t s);
unsigned int take_timeouts_norm_f16() { return take_timeouts_local(); }
cudaError_t set_timeout_flag_norm_f16(unsigned int* flag) { return set_timeout_flag_local(flag); }
}  // namespace zs
