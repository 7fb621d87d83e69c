// gated_step.cuh -- one token of the gated linear recurrence on states kept by slot.
#pragma once

#include <type_traits>

#include "gated_math.cuh"
#include "../../include/ssm_gated.h"

namespace ssm {

constexpr int kStepThreads = 128;
// Resident blocks per SM (80 registers), which is also how many a launch has at most.  With the gate, graph of 60
// steps: bf16 256 x 5120 6.5 us and 2048 x 5120 36.8 us (74% of the copy rate), with 8 blocks 6.6 and 36.4 but fp32 512 x
// 8192 28.9 instead of 20.9 (spills), with 10 9.2 and 65.6; one row per block 9.0 and 89.9.  Channels that are not near
// cost 2% (2048 x 5120), one in a warp's 128 as much as all.
constexpr int kStepBlocks = 6;
constexpr int kStepChannels = 4;  // per thread

struct GatedStep {
    ssm_gated_step_t a;
    int vec;        // every row of every operand starts on a boundary of 4 elements
    int no_bitmap;  // the slots do not fit a bitmap in shared memory
};

// Channels d .. d + 3 of a row (those below dim, else 0) as they lie in memory, and as fp32.
template <typename T>
struct Four {
    uint32_t w[sizeof(T)];
};

template <typename T>
__device__ __forceinline__ Four<T> load4(const T* p, int d, int dim, bool vec) {
    Four<T> f{};
    if (vec && d + kStepChannels <= dim) {
        if constexpr (sizeof(T) == 2) {
            const uint2 v = *reinterpret_cast<const uint2*>(p + d);
            f.w[0] = v.x, f.w[1] = v.y;
        } else {
            const uint4 v = *reinterpret_cast<const uint4*>(p + d);
            f.w[0] = v.x, f.w[1] = v.y, f.w[2] = v.z, f.w[3] = v.w;
        }
    } else {
#pragma unroll
        for (int k = 0; k < kStepChannels; ++k) {
            if (d + k >= dim) continue;
            if constexpr (sizeof(T) == 2)
                f.w[k / 2] |= static_cast<uint32_t>(reinterpret_cast<const unsigned short*>(p)[d + k]) << (k % 2 * 16);
            else
                f.w[k] = reinterpret_cast<const uint32_t*>(p)[d + k];
        }
    }
    return f;
}

// Channels 2 k and 2 k + 1 of the four.
template <typename T>
__device__ __forceinline__ float2 two_of(const Four<T>& f, int k) {
    if constexpr (sizeof(T) == 2) return make_float2(__uint_as_float(f.w[k] << 16), __uint_as_float(f.w[k] & 0xffff0000u));
    else return make_float2(__uint_as_float(f.w[2 * k]), __uint_as_float(f.w[2 * k + 1]));
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

// Thread = four channels of every gridDim.y-th batch row, the next row's operands under way while one
// is computed; the channels' parameters are read and worked out once.
//
// Rows that name the same slot are consecutive tokens of one sequence: the first of them applies them
// all in batch order, the others do nothing.  Whether there are any, each block finds out by marking the
// slots in a bitmap while its first loads are under way; only if so does it search the list row by row
// (no_bitmap: more slots than shared memory has bits for, search at once).
template <typename IO, bool GATE>
__global__ void __launch_bounds__(kStepThreads, kStepBlocks) gated_step_kernel(const GatedStep g) {
    extern __shared__ unsigned seen[];
    const ssm_gated_step_t& p = g.a;
    const int d = (blockIdx.x * kStepThreads + threadIdx.x) * kStepChannels;
    const bool vec = g.vec != 0;
    struct Row {
        Four<float> h;
        Four<IO> x, r, i, z;
    };
    const auto slot_of = [&](int b) { return b < p.batch ? (p.slots ? p.slots[b] : b) : -1; };
    const auto in_pool = [&](int slot) { return slot >= 0 && slot < p.n_slots; };
    const auto load_inputs = [&](Row& w, int b) {
        w.x = load4(static_cast<const IO*>(p.x) + b * p.x_stride, d, p.dim, vec);
        w.r = load4(static_cast<const IO*>(p.r) + b * p.r_stride, d, p.dim, vec);
        w.i = load4(static_cast<const IO*>(p.i) + b * p.i_stride, d, p.dim, vec);
        if (GATE) w.z = load4(static_cast<const IO*>(p.z) + b * p.z_stride, d, p.dim, vec);
    };
    const auto load_row = [&](Row& w, int b, int slot) {
        if (!in_pool(slot)) return;
        w.h = load4(p.state + slot * p.state_stride, d, p.dim, vec);
        load_inputs(w, b);
    };
    Row row, next;
    int slot = slot_of(blockIdx.y), slot1 = slot_of(blockIdx.y + gridDim.y);  // of this row and the next
    load_row(row, blockIdx.y, slot);
    float2 root[2], rb[2] = {}, ib[2] = {};
    {
        const Four<float> lam = load4(p.lam, d, p.dim, vec);
        Four<float> r{}, i{};
        if (p.r_bias) r = load4(p.r_bias, d, p.dim, vec);
        if (p.i_bias) i = load4(p.i_bias, d, p.dim, vec);
#pragma unroll
        for (int k = 0; k < 2; ++k) root[k] = two_of(lam, k), rb[k] = two_of(r, k), ib[k] = two_of(i, k);
    }
    bool shared = p.slots && g.no_bitmap;
    if (p.slots && p.batch > 1 && !g.no_bitmap) {
        for (int k = threadIdx.x; k < (p.n_slots + 31) / 32; k += kStepThreads) seen[k] = 0;
        __syncthreads();
        bool twice = false;
        for (int k = threadIdx.x; k < p.batch; k += kStepThreads) {
            const int s = p.slots[k];
            if (in_pool(s)) twice |= (atomicOr(&seen[s >> 5], 1u << (s & 31)) >> (s & 31) & 1) != 0;
        }
        shared = __syncthreads_or(twice);
    }
    bool near = true;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        root[k] = make_float2(root_of(p.c, root[k].x), root_of(p.c, root[k].y));
        near &= root[k].x <= kNear && root[k].y <= kNear;
    }
    near = __all_sync(0xffffffffu, near);
    const auto apply = [&](Row& w, int b) {
        float2 y[2];
        const auto step = [&](auto near_tag) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const Decay dec = decay_of<decltype(near_tag)::value, false>(__fadd2_rn(two_of(w.r, k), rb[k]), 0.f, root[k]);
                const Gate gate = gate_of(__fadd2_rn(two_of(w.i, k), ib[k]), 0.f);
                y[k] = __ffma2_rn(dec.a, two_of(w.h, k), __fmul2_rn(__fmul2_rn(dec.m, gate.sig), two_of(w.x, k)));
                w.h.w[2 * k] = __float_as_uint(y[k].x), w.h.w[2 * k + 1] = __float_as_uint(y[k].y);
                if (GATE) y[k] = __fmul2_rn(y[k], silu2(two_of(w.z, k)));
            }
        };
        if (near)
            step(std::true_type{});
        else
            step(std::false_type{});
        const float out[kStepChannels] = {y[0].x, y[0].y, y[1].x, y[1].y};
        store4(static_cast<IO*>(p.y) + b * p.y_stride, d, p.dim, vec, out);
    };
    for (int b = blockIdx.y; b < p.batch; b += gridDim.y) {
        const int slot2 = slot_of(b + 2 * static_cast<int>(gridDim.y));
        load_row(next, b + gridDim.y, slot1);
        bool mine = in_pool(slot);
        if (shared && mine)
            for (int k = 0; k < b; ++k) mine &= p.slots[k] != slot;
        if (mine) {
            apply(row, b);
            if (shared)
                for (int k = b + 1; k < p.batch; ++k)
                    if (p.slots[k] == slot) load_inputs(row, k), apply(row, k);
            const float out[kStepChannels] = {__uint_as_float(row.h.w[0]), __uint_as_float(row.h.w[1]), __uint_as_float(row.h.w[2]),
                                              __uint_as_float(row.h.w[3])};
            store4(p.state + slot * p.state_stride, d, p.dim, vec, out);
        }
        row = next, slot = slot1, slot1 = slot2;
    }
}

}  // namespace ssm
