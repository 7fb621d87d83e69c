// gated_launch.cuh -- launch shapes of the gated recurrence's kernels.
#pragma once

#include "gated_host.h"
#include "gated_scan.cuh"
#include "gated_step.cuh"
#include "host_common.h"

namespace ssmh {

template <typename IO>
ssm_status_t launch_gated_fwd(const ssm::GatedParams& p, cudaStream_t stream) {
    const long long rows = static_cast<long long>(p.batch) * p.dim;
    const bool gate = p.z.p != nullptr, reset = p.reset != nullptr;
    auto kern = gate ? (reset ? ssm::gated_fwd_kernel<IO, true, true> : ssm::gated_fwd_kernel<IO, true, false>)
                     : (reset ? ssm::gated_fwd_kernel<IO, false, true> : ssm::gated_fwd_kernel<IO, false, false>);
    kern<<<static_cast<unsigned>((rows + ssm::kGatedWarps - 1) / ssm::kGatedWarps), ssm::kGatedWarps * 32, 0, stream>>>(p);
    return launch_status();
}

template <typename IO>
ssm_status_t launch_gated_bwd(const ssm::GatedParams& p, cudaStream_t stream) {
    const long long rows = static_cast<long long>(p.batch) * p.dim;
    const bool gate = p.z.p != nullptr, reset = p.reset != nullptr;
    auto kern = gate ? (reset ? ssm::gated_bwd_kernel<IO, true, true> : ssm::gated_bwd_kernel<IO, true, false>)
                     : (reset ? ssm::gated_bwd_kernel<IO, false, true> : ssm::gated_bwd_kernel<IO, false, false>);
    kern<<<static_cast<unsigned>((rows + ssm::kGatedWarps - 1) / ssm::kGatedWarps), ssm::kGatedWarps * 32, 0, stream>>>(p);
    return launch_status();
}

template <typename IO>
ssm_status_t launch_gated_step(const ssm_gated_step_t& a, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>((a.dim + ssm::kStepThreads - 1) / ssm::kStepThreads), static_cast<unsigned>(a.batch));
    ssm::gated_step_kernel<IO><<<grid, ssm::kStepThreads, 0, stream>>>(a);
    return launch_status();
}

}  // namespace ssmh
