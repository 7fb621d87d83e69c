// gated_host.h -- launchers of the gated linear recurrence, one translation unit per element type.
#pragma once

#include "../../include/ssm_gated.h"
#include "gated_math.cuh"

namespace ssmh {

template <typename IO> ssm_status_t launch_gated_fwd(const ssm::GatedParams& p, int sms, cudaStream_t stream);
template <typename IO> ssm_status_t launch_gated_bwd(const ssm::GatedParams& p, int sms, cudaStream_t stream);
template <typename IO> ssm_status_t launch_gated_step(const ssm_gated_step_t& a, int sms, cudaStream_t stream);

}  // namespace ssmh
