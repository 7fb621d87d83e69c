// gated_launch.cuh -- launch shapes of the gated recurrence's kernels.
#pragma once

#include <algorithm>

#include "gated_host.h"
#include "gated_scan.cuh"
#include "gated_step.cuh"
#include "host_common.h"

namespace ssmh {

// How rows are laid on lanes, each of which holds `steps` steps.  Rows that fit in half a warp share one;
// few long rows are split over the warps of a block until the GPU has work for all its SMs.
struct GatedShape {
    int seg, split;
};

template <typename IO>
GatedShape gated_shape(long long rows, int L, int steps) {
    constexpr int kVec = 16 / sizeof(IO);
    const long long need = L % kVec ? L + static_cast<long long>(kVec) - 1 : L;  // (rows then start anywhere in a vector)
    int seg = 1, split = 1;
    while (seg < 32 && static_cast<long long>(seg) * steps < need) seg *= 2;
    if (seg == 32)
        while (split < ssm::kMaxSplit && rows * split < 148 * 10 && static_cast<long long>(split) * 32 * steps < L) split *= 2;
    return {seg, split};
}

using GatedKernel = void (*)(const ssm::GatedParams);

template <typename IO, bool GATE, bool RESET>
GatedKernel gated_kernel(GatedShape shape, bool backward) {
    if (shape.seg < 32) return backward ? ssm::gated_bwd_kernel<IO, GATE, RESET, 0, false> : ssm::gated_fwd_kernel<IO, GATE, RESET, 0, false>;
    if (shape.split > 1) return backward ? ssm::gated_bwd_kernel<IO, GATE, RESET, 32, true> : ssm::gated_fwd_kernel<IO, GATE, RESET, 32, true>;
    return backward ? ssm::gated_bwd_kernel<IO, GATE, RESET, 32, false> : ssm::gated_fwd_kernel<IO, GATE, RESET, 32, false>;
}

template <typename IO>
ssm_status_t launch_gated(ssm::GatedParams p, bool backward, cudaStream_t stream) {
    const long long rows = static_cast<long long>(p.batch) * p.dim;
    const GatedShape shape = gated_shape<IO>(rows, p.L, backward ? ssm::kBwdSteps : ssm::kFwdSteps<IO>);
    p.seg = shape.seg;
    p.split = shape.split;
    const bool gate = p.z.p != nullptr, reset = p.reset != nullptr;
    const GatedKernel kern = gate ? (reset ? gated_kernel<IO, true, true>(shape, backward) : gated_kernel<IO, true, false>(shape, backward))
                                  : (reset ? gated_kernel<IO, false, true>(shape, backward) : gated_kernel<IO, false, false>(shape, backward));
    const int block = shape.split > 1 ? shape.split * 32 : ssm::kGatedWarps * 32;
    const long long per_block = shape.split > 1 ? 1 : block / shape.seg;
    const int smem = backward ? ssm::bwd_smem<IO>(gate, block) : 0;
    if (smem > 46 * 1024 &&  // (with the static part of it, past the 48 KB that need no asking)
        !ensure_smem_attr(reinterpret_cast<const void*>(kern), smem)) return SSM_ERR_LAUNCH;
    kern<<<static_cast<unsigned>((rows + per_block - 1) / per_block), block, smem, stream>>>(p);
    return launch_status();
}

template <typename IO>
ssm_status_t launch_gated_fwd(const ssm::GatedParams& p, cudaStream_t stream) {
    return launch_gated<IO>(p, false, stream);
}

template <typename IO>
ssm_status_t launch_gated_bwd(const ssm::GatedParams& p, cudaStream_t stream) {
    return launch_gated<IO>(p, true, stream);
}

template <typename IO>
ssm_status_t launch_gated_step(const ssm_gated_step_t& a, int sms, cudaStream_t stream) {
    const unsigned mask = ssm::kStepChannels * sizeof(IO) - 1;
    const auto on = [](const void* p, long long stride, unsigned m) {
        return ((reinterpret_cast<uintptr_t>(p) | static_cast<unsigned long long>(stride)) & m) == 0;
    };
    const auto io = [&](const void* p, long long stride) { return on(p, stride * static_cast<long long>(sizeof(IO)), mask); };
    const bool vec = io(a.x, a.x_stride) && io(a.r, a.r_stride) && io(a.i, a.i_stride) && io(a.z, a.z ? a.z_stride : 0) &&
                     io(a.y, a.y_stride) && on(a.state, a.state_stride * 4, 15) && on(a.lam, 0, 15) && on(a.r_bias, 0, 15) &&
                     on(a.i_bias, 0, 15);
    const int per_block = ssm::kStepThreads * ssm::kStepChannels;
    const int chunks = (a.dim + per_block - 1) / per_block;
    // rows of a block: as few as fill the resident blocks
    const int rows = static_cast<int>(std::min<long long>(a.batch, std::max<long long>(1, STEP_BLOCKS * sms / chunks)));
    const dim3 grid(static_cast<unsigned>(chunks), static_cast<unsigned>(rows));
    const long long bitmap = (a.n_slots + 31LL) / 32 * 4;
    const bool small = bitmap <= 40 * 1024;
    const ssm::GatedStep g{a, vec, !small};
    auto kern = a.z ? ssm::gated_step_kernel<IO, true> : ssm::gated_step_kernel<IO, false>;
    kern<<<grid, ssm::kStepThreads, a.slots && a.batch > 1 && small ? static_cast<int>(bitmap) : 0, stream>>>(g);
    return launch_status();
}

}  // namespace ssmh
