// gated_step.cuh -- one token of the gated linear recurrence on states kept by slot.
#pragma once

#include "gated_math.cuh"
#include "../../include/ssm_gated.h"

namespace ssm {

constexpr int kStepThreads = 128;
constexpr int kStepChannels = 4;  // per thread

struct GatedStep {
    ssm_gated_step_t a;
    int vec;  // every row of every operand starts on a boundary of 4 elements
};

// Channels d .. d + 3 of a row (those below dim) as fp32.
template <typename T>
__device__ __forceinline__ void load4(const T* p, int d, int dim, bool vec, float (&v)[kStepChannels]) {
    if (vec && d + kStepChannels <= dim) {
        if constexpr (sizeof(T) == 2) {
            const uint2 w = *reinterpret_cast<const uint2*>(p + d);
            v[0] = __uint_as_float(w.x << 16), v[1] = __uint_as_float(w.x & 0xffff0000u);
            v[2] = __uint_as_float(w.y << 16), v[3] = __uint_as_float(w.y & 0xffff0000u);
        } else {
            const float4 w = *reinterpret_cast<const float4*>(p + d);
            v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
        }
    } else {
#pragma unroll
        for (int k = 0; k < kStepChannels; ++k) v[k] = d + k < dim ? IoTraits<T>::to_f32(p[d + k]) : 0.f;
    }
}

template <typename T>
__device__ __forceinline__ void store4(T* p, int d, int dim, bool vec, const float (&v)[kStepChannels]) {
    if (vec && d + kStepChannels <= dim) {
        if constexpr (sizeof(T) == 2)
            *reinterpret_cast<uint2*>(p + d) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
        else
            *reinterpret_cast<float4*>(p + d) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
        for (int k = 0; k < kStepChannels; ++k)
            if (d + k < dim) p[d + k] = IoTraits<T>::from_f32(v[k]);
    }
}

// Thread = four channels of one batch row.  Rows that name the same slot are consecutive tokens of one
// sequence: the first of them applies them all in batch order, the others do nothing.  The block
// looks for such rows while its loads are under way.
template <typename IO, bool GATE>
__global__ void __launch_bounds__(kStepThreads) gated_step_kernel(const GatedStep g) {
    const ssm_gated_step_t& p = g.a;
    const int b = blockIdx.y, d = (blockIdx.x * kStepThreads + threadIdx.x) * kStepChannels;
    const int slot = p.slots ? p.slots[b] : b;
    if (slot < 0 || slot >= p.n_slots) return;
    const bool vec = g.vec != 0;
    float* state = p.state + slot * p.state_stride;
    float h[kStepChannels], x[kStepChannels], r[kStepChannels], i[kStepChannels], z[kStepChannels], root[kStepChannels],
        rb[kStepChannels] = {}, ib[kStepChannels] = {};
    const auto load_row = [&](int k) {
        load4(static_cast<const IO*>(p.x) + k * p.x_stride, d, p.dim, vec, x);
        load4(static_cast<const IO*>(p.r) + k * p.r_stride, d, p.dim, vec, r);
        load4(static_cast<const IO*>(p.i) + k * p.i_stride, d, p.dim, vec, i);
        if (GATE) load4(static_cast<const IO*>(p.z) + k * p.z_stride, d, p.dim, vec, z);
    };
    load4(state, d, p.dim, vec, h);
    load_row(b);
    load4(p.lam, d, p.dim, vec, root);
    if (p.r_bias) load4(p.r_bias, d, p.dim, vec, rb);
    if (p.i_bias) load4(p.i_bias, d, p.dim, vec, ib);
    bool again = false;
    if (p.slots) {
        bool before = false, after = false;
        for (int k = threadIdx.x; k < p.batch; k += kStepThreads) {
            const bool same = p.slots[k] == slot;
            before |= same && k < b;
            after |= same && k > b;
        }
        if (__syncthreads_or(before)) return;
        again = __syncthreads_or(after);
    }
    if (d >= p.dim) return;
#pragma unroll
    for (int k = 0; k < kStepChannels; ++k) root[k] = sqrtf(2.f * p.c * softplus_lam(root[k]));
    for (int row = b;;) {
#pragma unroll
        for (int k = 0; k < kStepChannels; k += 2) {
            const float2 hv = make_float2(h[k], h[k + 1]), xv = make_float2(x[k], x[k + 1]);
            const Decay dec = decay_of<false, false>(make_float2(r[k] + rb[k], r[k + 1] + rb[k + 1]), 0.f, make_float2(root[k], root[k + 1]));
            const Gate gate = gate_of(make_float2(i[k] + ib[k], i[k + 1] + ib[k + 1]), 0.f);
            const float2 now = __ffma2_rn(dec.a, hv, __fmul2_rn(__fmul2_rn(dec.m, gate.sig), xv));
            h[k] = now.x, h[k + 1] = now.y;
            float2 out = now;
            if (GATE) {
                const float2 zv = make_float2(z[k], z[k + 1]);
                out = __fmul2_rn(now, gate_silu2<IO>(zv));
            }
            x[k] = out.x, x[k + 1] = out.y;
        }
        store4(static_cast<IO*>(p.y) + row * p.y_stride, d, p.dim, vec, x);
        if (!again) break;
        do ++row;
        while (row < p.batch && p.slots[row] != slot);
        if (row == p.batch) break;
        load_row(row);
    }
    store4(state, d, p.dim, vec, h);
}

}  // namespace ssm
