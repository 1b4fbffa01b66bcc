#include "zs_norm_kernels.cuh"

namespace zs {
template zs_status norm_forward<float>(NormArgs& a, cudaStream_t s);
template zs_status norm_backward<float>(NormArgs& a, cudaStream_t s);
unsigned int take_timeouts_norm_f32() { return take_timeouts_local(); }
cudaError_t set_timeout_flag_norm_f32(unsigned int* flag) { return set_timeout_flag_local(flag); }
}  // namespace zs
