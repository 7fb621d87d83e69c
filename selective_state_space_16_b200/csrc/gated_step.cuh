// gated_step.cuh -- one token of the gated linear recurrence on states kept by slot.
#pragma once

#include "gated_math.cuh"
#include "../../include/ssm_gated.h"

namespace ssm {

constexpr int kStepThreads = 128;

// Thread = one channel of one batch row.  Rows that name the same slot are consecutive tokens of
// one sequence: the first of them applies them all in batch order, the others do nothing.
template <typename IO>
__global__ void __launch_bounds__(kStepThreads) gated_step_kernel(const ssm_gated_step_t p) {
    const int b = blockIdx.y, d = blockIdx.x * kStepThreads + threadIdx.x;
    const int slot = p.slots ? p.slots[b] : b;
    if (slot < 0 || slot >= p.n_slots || d >= p.dim) return;
    if (p.slots)
        for (int k = 0; k < b; ++k)
            if (p.slots[k] == slot) return;
    float* state = p.state + slot * p.state_stride + d;
    const float rate = -p.c * softplus_once(p.lam[d]) * kLog2e;
    const float rb = p.r_bias ? p.r_bias[d] : 0.f, ib = p.i_bias ? p.i_bias[d] : 0.f;
    float h = *state;
    for (int k = b; k < p.batch; ++k) {
        if (k > b && (!p.slots || p.slots[k] != slot)) continue;
        const float xv = IoTraits<IO>::to_f32(static_cast<const IO*>(p.x)[k * p.x_stride + d]);
        const float rv = IoTraits<IO>::to_f32(static_cast<const IO*>(p.r)[k * p.r_stride + d]);
        const float iv = IoTraits<IO>::to_f32(static_cast<const IO*>(p.i)[k * p.i_stride + d]);
        const float yv = rate * rcp_approx(1.f + ex2_mufu(-kLog2e * (rv + rb)));
        const float a = ex2_mufu(yv);
        const float m = sqrt_approx(one_minus_square(yv, a));
        h = fmaf(a, h, m * rcp_approx(1.f + ex2_mufu(-kLog2e * (iv + ib))) * xv);
        float out = h;
        if (p.z) out *= silu_f32(IoTraits<IO>::to_f32(static_cast<const IO*>(p.z)[k * p.z_stride + d]));
        static_cast<IO*>(p.y)[k * p.y_stride + d] = IoTraits<IO>::from_f32(out);
    }
    *state = h;
}

}  // namespace ssm
