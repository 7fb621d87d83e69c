// gated_launch.cuh -- launch shapes of the gated recurrence's kernels.
#pragma once

#include <algorithm>
#include <cmath>

#include "gated_host.h"
#include "gated_scan.cuh"
#include "gated_step.cuh"
#include "host_common.h"

namespace ssmh {

// How rows are laid on lanes, each of which holds `steps` steps: rows that fit in half a warp share one; a
// long row is split over `split` warps in `blocks` blocks of a cluster.
struct GatedShape {
    int seg, split, blocks;
};

// How full the waves of `resident` warps are, if each of `warps` is a warp's work.
inline double wave_fill(long long warps, long long resident) {
    const double waves = static_cast<double>(warps) / static_cast<double>(resident);
    return waves / std::ceil(waves);
}

// Splitting goes on, by twos, until the GPU has 8 warps per SM (16 are resident) or a round covers the row: up to
// 4 warps of one block, then with fewer rows than SMs up to 8 blocks, else up to 8 warps.  Forward and backward of
// bf16 rows with a gate, us: 64 x 32768 58 with 4 warps, 43 with 8, 32 with 4 x 4 blocks, 27 with 4 x 8; 128 x 32768 62,
// 46, 44 and 54; 200 x 16384 42 with 4, 38 with 8, 37 with 4 x 2 blocks; 300 x 16384 51 with 4, 55 with 8, 61 with
// 4 x 2; 768 x 16384 122, 93, 92 and 98 with 1, 2, 4 and 8; 1536 x 8192 85 and 90 with 1 and 2.  3 or 6 warps took
// longer than 2 and 4 throughout.
// Long rows in a few waves (`alone`: the warps of an SM with a row each; 16 with rows split) are split too where
// that fills the last wave better by enough to pay for the barriers:
// us with 1, 2 and 4 warps: fp32 forward 5120 x 16384 311, 293 and 287, bf16 3000 x 16384 107, 106 and 105, 2600 x 8192 53,
// 48 and 49, backward 87 with 1 and 2; but bf16 forward 5120 x 32768 332, 339 and 338, 12288 x 8192 197 and 206 with 1
// and 2.  Rows of 4 tiles lose: 12288 x 2048 56, 63 and 84.
// The fp32 backward, 12 warps alone, rows of 8192 steps with 1 and 2: 2000 rows 127 and 112, 2368 136 and 132, 2600 145
// and 146, 3003 157 and 164, 3300 164 and 173, 4000 217 and 209 (not taken, as 4700: 238 and 237).
inline GatedShape split_shape(long long rows, int L, int steps, int sms, bool backward, bool f32, int alone) {
    const long long tiles = (L + 32LL * steps - 1) / (32 * steps);
    int warps = 1, blocks = 1;
    while (rows * warps * blocks < 8LL * sms && warps * blocks < tiles) {
        if (warps < 4 || (rows >= sms && warps < 8))
            warps *= 2;
        else if (rows < sms && blocks < ssm::kMaxCluster)
            blocks *= 2;
        else
            break;
    }
    const long long split = 2LL * ssm::kMaxSplit * sms;
    if (rows > static_cast<long long>(alone) * sms)
        while (warps < (backward ? 2 : 4) && tiles >= (backward ? 16 : 8) * warps * warps &&
               wave_fill(rows * warps * 2, split) >
                   (f32 && !backward ? 1.06 : 1.3) * wave_fill(rows * warps, warps > 1 ? split : static_cast<long long>(alone) * sms))
            warps *= 2;
    return {32, warps * blocks, blocks};
}

// A row begins anywhere that its strides and address allow in a 16-byte vector; its lanes count from the vector's
// begin (bf16 forward of 16 x 5120 rows of 250 steps: 67 us on half warps, 114 on whole ones).
template <typename IO>
GatedShape gated_shape(long long rows, const ssm::GatedTensor& x, int L, int steps, int sms, bool backward) {
    const unsigned long long at = (reinterpret_cast<uintptr_t>(x.p) / sizeof(IO)) | x.bs | x.ds | (16 / sizeof(IO));
    const long long need = L + static_cast<long long>(16 / sizeof(IO) - (at & -at));  // (its first vector may begin before it)
    int seg = 1;
    while (seg < 32 && static_cast<long long>(seg) * steps < need) seg *= 2;
    if (seg < 32) return {seg, 1, 1};
    return split_shape(rows, L, steps, sms, backward, sizeof(IO) == 4, ssm::kGatedWarps * (backward ? ssm::kBwdBlocks<IO> : ssm::kFwdBlocks));
}

using GatedKernel = void (*)(const ssm::GatedParams);

template <typename IO, bool GATE, bool RESET>
GatedKernel gated_kernel(GatedShape shape, bool backward) {
    if (shape.seg < 32) return backward ? ssm::gated_bwd_kernel<IO, GATE, RESET, 0, false> : ssm::gated_fwd_kernel<IO, GATE, RESET, 0, false>;
    if (shape.split > 1) return backward ? ssm::gated_bwd_kernel<IO, GATE, RESET, 32, true> : ssm::gated_fwd_kernel<IO, GATE, RESET, 32, true>;
    return backward ? ssm::gated_bwd_kernel<IO, GATE, RESET, 32, false> : ssm::gated_fwd_kernel<IO, GATE, RESET, 32, false>;
}

template <typename IO>
ssm_status_t launch_gated(ssm::GatedParams p, bool backward, int sms, cudaStream_t stream) {
    const long long rows = static_cast<long long>(p.batch) * p.dim;
    const GatedShape shape = gated_shape<IO>(rows, p.x, p.L, backward ? ssm::kBwdSteps : ssm::kFwdSteps<IO>, sms, backward);
    p.seg = shape.seg;
    p.split = shape.split;
    p.blocks = shape.blocks;
    const bool gate = p.z.p != nullptr, reset = p.reset != nullptr;
    const auto alike = [](const ssm::GatedTensor& a, const ssm::GatedTensor& b) {
        return a.bs == b.bs && a.ds == b.ds && ((reinterpret_cast<uintptr_t>(a.p) ^ reinterpret_cast<uintptr_t>(b.p)) & 15) == 0;
    };
    p.alike_in = alike(p.x, p.r) && alike(p.x, p.i) && (!gate || alike(p.x, p.z)) && (!backward || alike(p.x, p.dy));
    p.alike_out = alike(p.dx, p.dr) && alike(p.dx, p.di) && (!gate || alike(p.dx, p.dz));
    // 2^(31 + shift) / dim rounded up, 2^shift >= dim: off by less than 2^shift in it, so by less than 1 / dim in a
    // quotient of rows below 2^31
    p.dim_shift = 0;
    while (1LL << p.dim_shift < p.dim) ++p.dim_shift;
    p.dim_mul = static_cast<unsigned>(((1ULL << (31 + p.dim_shift)) + p.dim - 1) / p.dim);
    const GatedKernel kern = gate ? (reset ? gated_kernel<IO, true, true>(shape, backward) : gated_kernel<IO, true, false>(shape, backward))
                                  : (reset ? gated_kernel<IO, false, true>(shape, backward) : gated_kernel<IO, false, false>(shape, backward));
    const int block = shape.split > 1 ? shape.split / shape.blocks * 32 : ssm::kGatedWarps * 32;
    const long long per_block = block / shape.seg;
    const int smem = backward ? ssm::bwd_smem<IO>(gate, reset, block) : 0;
    if (smem > 46 * 1024 &&  // (with the static part of it, past the 48 KB that need no asking)
        !ensure_smem_attr(reinterpret_cast<const void*>(kern), smem)) return SSM_ERR_LAUNCH;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(shape.split > 1 ? rows * shape.blocks : (rows + per_block - 1) / per_block));
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute cluster{};
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim.x = static_cast<unsigned>(shape.blocks);
    cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
    cfg.attrs = &cluster;
    cfg.numAttrs = shape.blocks > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? launch_status() : SSM_ERR_LAUNCH;
}

template <typename IO>
ssm_status_t launch_gated_fwd(const ssm::GatedParams& p, int sms, cudaStream_t stream) {
    return launch_gated<IO>(p, false, sms, stream);
}

template <typename IO>
ssm_status_t launch_gated_bwd(const ssm::GatedParams& p, int sms, cudaStream_t stream) {
    return launch_gated<IO>(p, true, sms, stream);
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
    const int rows = static_cast<int>(std::min<long long>(a.batch, std::max<long long>(1, ssm::kStepBlocks * sms / chunks)));
    const dim3 grid(static_cast<unsigned>(chunks), static_cast<unsigned>(rows));
    const long long bitmap = (a.n_slots + 31LL) / 32 * 4;
    const bool small = bitmap <= 40 * 1024;
    const ssm::GatedStep g{a, vec, !small};
    auto kern = a.z ? ssm::gated_step_kernel<IO, true> : ssm::gated_step_kernel<IO, false>;
    kern<<<grid, ssm::kStepThreads, a.slots && a.batch > 1 && small ? static_cast<int>(bitmap) : 0, stream>>>(g);
    return launch_status();
}

}  // namespace ssmh
