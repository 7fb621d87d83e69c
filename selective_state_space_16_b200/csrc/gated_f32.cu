// gated_f32.cu -- the gated linear recurrence for f32 elements (gated_launch.cuh).
#include "gated_launch.cuh"

namespace ssmh {
template ssm_status_t launch_gated_fwd<float>(const ssm::GatedParams&, int, cudaStream_t);
template ssm_status_t launch_gated_bwd<float>(const ssm::GatedParams&, int, cudaStream_t);
template ssm_status_t launch_gated_step<float>(const ssm_gated_step_t&, int, cudaStream_t);
}  // namespace ssmh
