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
    float* ckpt;  // CkptHeader, then (rows, ckpt_row): the state before every group of a row; or null
    int batch, dim, L;
    long long ckpt_row;
    float c;
    int split;  // warps that share a row (1: a row per warp or part of one)
    // backward
    GatedTensor dy, dx, dr, di, dz;
    const float* dlast;
    float* dh0;
    float* part;  // (3, rows): sums of T, dr and di over a row's steps, or null
};

// Where the groups of the checkpointed rows start (phase_of their x): row (b, d) has the phase
// (base + b * bs + d * ds) mod 16 bytes, in elements.  The backward goes by it, wherever its x is.
struct CkptHeader {
    unsigned base, bs, ds, pad;
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

// softplus(lam) = max(lam, 0) + log1p(e^{-|lam|}) as softplus_f32, with the exponent's product by
// log2(e) carried to twice the length: lam reaches far below 0, where its rounding alone would cost
// |lam| 2^-24 of the result.  About 2^-21 relative.
__device__ __forceinline__ float softplus_lam(float lam) {
    constexpr float c[] = SSM_LOG1P_POLY;
    constexpr float kLog2eLow = 1.925963033500e-8f;  // log2(e) - kLog2e
    const float x = -fabsf(lam), y = x * kLog2e;
    const float low = fmaf(x, kLog2eLow, fmaf(x, kLog2e, -y));
    float e = ex2_mufu(y);
    e = fmaf(e, low * kLn2, e);
    float p = c[8];
#pragma unroll
    for (int i = 7; i >= 0; --i) p = fmaf(p, e, c[i]);
    return fmaf(e, p, fmaxf(lam, 0.f));
}

// The decay a = e^{-v} and 1 - a^2 = -w (2 + w), w = a - 1, from y = -v log2(e).  Near a = 1 the
// difference w cancels, so below v = 1/8 the series w = -v (1 - v/2 + v^2/6 - ...) up to v^6 / 720
// takes its place (the first term left out is 1e-9 of the sum there; above the border the cancellation
// costs at most 2e-6 of w), and a = 1 + w is then good to half a step.  For both element types: the
// state and the parameters' gradients are fp32.
struct Decay {
    float a, m2;  // m2 = 1 - a^2
};

__device__ __forceinline__ Decay decay_of(float y) {
    const float e = ex2_mufu(y), x = y * kLn2;
    float p = fmaf(x, 1.f / 720, 1.f / 120);
    p = fmaf(x, p, 1.f / 24);
    p = fmaf(x, p, 1.f / 6);
    p = fmaf(x, p, 0.5f);
    p = fmaf(x * x, p, x);
    const bool near = x > -0.125f;
    const float w = near ? p : e - 1.f;
    return {near ? 1.f + w : e, -w * (2.f + w)};
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

// Steps [t0, t0 + kGroup) of a row as they lie in memory.  `vec`: the group starts on a 16-byte
// boundary.  Whole groups inside the row [0, L) are read as vectors, the row's ends and rows that lie
// otherwise element by element; steps outside [0, len) are 0 or anything, and never used.
template <typename IO>
struct RawGroup {
    uint4 v[sizeof(IO) / 2];
};

__device__ __forceinline__ uint4 ld_stream(const uint4* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

template <typename IO>
__device__ __forceinline__ RawGroup<IO> load_group(const IO* row, int t0, int len, int L, bool vec) {
    RawGroup<IO> g{};
    if (t0 >= len) return g;
    if (vec && t0 >= 0 && t0 + kGroup <= L) {
#pragma unroll
        for (int k = 0; k < static_cast<int>(sizeof(IO) / 2); ++k) g.v[k] = ld_stream(reinterpret_cast<const uint4*>(row + t0) + k);
    } else {
        uint32_t w[sizeof(IO) * 2] = {};
#pragma unroll
        for (int e = 0; e < kGroup; ++e) {
            if (t0 + e < 0 || t0 + e >= len) continue;
            if constexpr (sizeof(IO) == 2)
                w[e / 2] |= static_cast<uint32_t>(reinterpret_cast<const unsigned short*>(row)[t0 + e]) << (e % 2 * 16);
            else
                w[e] = reinterpret_cast<const uint32_t*>(row)[t0 + e];
        }
#pragma unroll
        for (int k = 0; k < static_cast<int>(sizeof(IO) / 2); ++k) g.v[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
    }
    return g;
}

template <typename IO>
__device__ __forceinline__ void unpack(const RawGroup<IO>& g, float (&v)[kGroup]) {
    constexpr int n = Group16<IO>::kN;
#pragma unroll
    for (int k = 0; k < kGroup / n; ++k) {
        float part[n];
        Group16<IO>::unpack(g.v[k], part);
#pragma unroll
        for (int e = 0; e < n; ++e) v[k * n + e] = part[e];
    }
}

// The steps of the group that lie in [0, n).
template <typename IO>
__device__ __forceinline__ void store_group(IO* row, int t0, int n, bool vec, const float (&v)[kGroup]) {
    if (vec && t0 >= 0 && t0 + kGroup <= n) {
        uint4* to = reinterpret_cast<uint4*>(row + t0);
        if constexpr (sizeof(IO) == 2) {
            *to = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
        } else {
            reinterpret_cast<float4*>(to)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4*>(to)[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < kGroup; ++e)
            if (t0 + e >= 0 && t0 + e < n) row[t0 + e] = IoTraits<IO>::from_f32(v[e]);
    }
}

// A row's groups are laid so that those of x start on 16-byte boundaries: group g holds the steps
// from g * kGroup - phase.  Operands that lie like x, which dense ones of one shape do, are read and
// written as vectors at any length of the rows; each operand is looked at by itself.
template <typename IO>
__device__ __forceinline__ int phase_of(const IO* row) {
    return static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(IO));
}

template <typename IO>
__device__ __forceinline__ IO* row_of(const GatedTensor& t, int b, int d) {
    return static_cast<IO*>(const_cast<void*>(t.p)) + b * t.bs + d * t.ds;
}

__device__ __forceinline__ int row_length(const GatedParams& p, int b) {
    return p.lengths ? min(max(p.lengths[b], 0), p.L) : p.L;
}

}  // namespace ssm
