// gated_math.cuh -- the pieces shared by the kernels of the gated linear recurrence
//   h_t = a_t h_{t-1} + m_t iota_t x_t,   a = exp(-v),  v = c softplus(lam) sigmoid(r),
//   m = sqrt(1 - a^2),  iota = sigmoid(i)
// : its parameters, the coefficients of a step in fp32, and the tiles that a warp works on.
#pragma once

#include <cmath>

#include "common.cuh"
#include "scan_math.cuh"

namespace ssm {

// A (batch, dim, seqlen) operand; strides in elements, steps next to each other.
struct GatedTensor {
    const void* p;
    long long bs, ds;
};

struct GatedParams {
    GatedTensor x, r, i, z, y;  // z.p, y.p may be null
    const float *lam, *r_bias, *i_bias, *h0;
    float* last;
    const int* lengths;
    const unsigned char* reset;
    float* ckpt;  // (rows, ckpt_row): state before every group of kGroup steps, or null
    int batch, dim, L;
    long long ckpt_row;
    float c;
    // backward
    GatedTensor dy, dx, dr, di, dz;
    const float* dlast;
    float* dh0;
    float* part;  // (3, rows): sums of T, dr and di over a row's steps, or null
};

constexpr int kGroup = 8;           // steps that a lane holds at once, and between two checkpoints
constexpr int kTile = 32 * kGroup;  // steps of a warp's tile

__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rsqrt_approx(float x) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float sqrt_approx(float x) {
    float y;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// softplus(lam), once per row and so by the library functions: large lam return lam itself.
__device__ __forceinline__ float softplus_once(float lam) { return lam > 20.f ? lam : log1pf(expf(lam)); }

// 1 - a^2 = 1 - e^{-u} with u = 2 v >= 0, from y = -v log2(e) and a = 2^y.  Near a = 1 the
// difference cancels, so below u = 1/4 the series u (1 - u/2 + u^2/6 - ...) up to u^6 / 720 takes its
// place: the first term left out is 5e-8 of the sum there, and above the border the cancellation
// costs at most 2e-6.  For both element types: the state and the parameters' gradients are fp32.
__device__ __forceinline__ float one_minus_square(float y, float a) {
    const float u = y * (-2.f * kLn2);
    float p = fmaf(u, -1.f / 720, 1.f / 120);
    p = fmaf(u, p, -1.f / 24);
    p = fmaf(u, p, 1.f / 6);
    p = fmaf(u, p, -0.5f);
    p = u * fmaf(u, p, 1.f);
    return u < 0.25f ? p : fmaf(-a, a, 1.f);
}

// Two stretches of the recurrence, each (P, H): h -> P h + H, are composed by carry_on for H and
// join for P.  A reset has the coefficient kCut, whose sign marks it (decays are never negative):
// the mark stays with every product that spans it, and what lies before a marked stretch is
// dropped rather than multiplied by 0, so that an infinity or NaN cannot pass.  A product that
// merely underflows has no mark, and lets them pass as the steps one by one would.
constexpr float kCut = -0.f;

__device__ __forceinline__ bool is_cut(float P) { return __float_as_int(P) < 0; }

template <bool RESET>
__device__ __forceinline__ float carry_on(float P, float earlier, float H) {
    const float v = fmaf(P, earlier, H);
    if constexpr (RESET) return is_cut(P) ? H : v;
    return v;
}

template <bool RESET>
__device__ __forceinline__ float join(float P, float Q) {
    const float v = P * Q;
    if constexpr (RESET)
        return __int_as_float(__float_as_int(v) | ((__float_as_int(P) | __float_as_int(Q)) & 0x80000000));
    return v;
}

// Steps [t0, t0 + kGroup) of a row as fp32; steps outside [0, L) as 0.
template <typename IO>
__device__ __forceinline__ void load_group(const IO* row, int t0, int L, float (&v)[kGroup]) {
#pragma unroll
    for (int e = 0; e < kGroup; ++e) v[e] = (t0 + e >= 0 && t0 + e < L) ? IoTraits<IO>::to_f32(row[t0 + e]) : 0.f;
}

template <typename IO>
__device__ __forceinline__ void store_group(IO* row, int t0, int L, const float (&v)[kGroup]) {
#pragma unroll
    for (int e = 0; e < kGroup; ++e)
        if (t0 + e >= 0 && t0 + e < L) row[t0 + e] = IoTraits<IO>::from_f32(v[e]);
}

template <typename IO>
__device__ __forceinline__ IO* row_of(const GatedTensor& t, int b, int d) {
    return static_cast<IO*>(const_cast<void*>(t.p)) + b * t.bs + d * t.ds;
}

__device__ __forceinline__ int row_length(const GatedParams& p, int b) {
    return p.lengths ? min(max(p.lengths[b], 0), p.L) : p.L;
}

}  // namespace ssm
