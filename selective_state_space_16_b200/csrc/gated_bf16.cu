// gated_bf16.cu -- the gated linear recurrence for bf16 elements (gated_launch.cuh).
#include "gated_launch.cuh"

namespace ssmh {
template ssm_status_t launch_gated_fwd<__nv_bfloat16>(const ssm::GatedParams&, int, cudaStream_t);
template ssm_status_t launch_gated_bwd<__nv_bfloat16>(const ssm::GatedParams&, int, cudaStream_t);
template ssm_status_t launch_gated_step<__nv_bfloat16>(const ssm_gated_step_t&, int, cudaStream_t);
}  // namespace ssmh
