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

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// min that keeps a NaN.
__device__ __forceinline__ float min_nan(float x, float limit) {
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(limit));
    return y;
}

// Both gates of two steps: rho = sigmoid(r + r_bias), iota = sigmoid(i + i_bias) from kr = -log2(e)
// r_bias and ki likewise, and Er = e^{-(r + r_bias)}, Ei (1 - rho = Er rho without cancellation).
// One reciprocal serves a step's two gates, 1 / ((1 + Er)(1 + Ei)), as the special-function unit is
// the scarcest.  So that the product stays finite a gate below 2^-63 counts as 2^-63.
struct Gates {
    float2 rho, iota, Er, Ei;
};

__device__ __forceinline__ Gates gates_of(float2 r, float2 i, float kr, float ki) {
    const float2 yr = __ffma2_rn(both(-kLog2e), r, both(kr)), yi = __ffma2_rn(both(-kLog2e), i, both(ki));
    Gates g;
    g.Er = make_float2(ex2_mufu(min_nan(yr.x, 63.f)), ex2_mufu(min_nan(yr.y, 63.f)));
    g.Ei = make_float2(ex2_mufu(min_nan(yi.x, 63.f)), ex2_mufu(min_nan(yi.y, 63.f)));
    const float2 dr = __fadd2_rn(both(1.f), g.Er), di = __fadd2_rn(both(1.f), g.Ei), d = __fmul2_rn(dr, di);
    const float2 inv = make_float2(rcp_approx(d.x), rcp_approx(d.y));
    g.rho = __fmul2_rn(inv, di);
    g.iota = __fmul2_rn(inv, dr);
    return g;
}

// The decay a = e^x and 1 - a^2 = -w (2 + w), w = a - 1, of two steps with x = -v <= 0.  Near a = 1 the
// difference w cancels, so for v < 1/8 the series w = x (1 + x/2 + x^2/6 + x^3/24 + x^4/120) takes its
// place (the first term left out is 4e-8 of the sum there; beyond it the cancellation costs at most
// 2e-6 of w), and a = 1 + w is then good to half a step.  For both element types: the state and the
// parameters' gradients are fp32.  NEAR: c softplus(lam) < 1/8, so that no step of the channel needs
// the exponential: channels with a memory of some ten steps or more.
constexpr float kNear = 0.125f;

struct Decay {
    float2 a, m2;  // m2 = 1 - a^2
};

template <bool NEAR>
__device__ __forceinline__ Decay decay_of(float2 x) {
    float2 p = __ffma2_rn(x, both(1.f / 120), both(1.f / 24));
    p = __ffma2_rn(x, p, both(1.f / 6));
    p = __ffma2_rn(x, p, both(0.5f));
    float2 w = __ffma2_rn(__fmul2_rn(x, x), p, x);
    Decay d;
    if constexpr (NEAR) {
        d.a = __fadd2_rn(both(1.f), w);
    } else {
        const float2 y = __fmul2_rn(x, both(kLog2e));
        const float2 e = make_float2(ex2_mufu(y.x), ex2_mufu(y.y)), f = __fadd2_rn(e, both(-1.f));
        w = make_float2(x.x > -kNear ? w.x : f.x, x.y > -kNear ? w.y : f.y);
        const float2 near = __fadd2_rn(both(1.f), w);
        d.a = make_float2(x.x > -kNear ? near.x : e.x, x.y > -kNear ? near.y : e.y);
    }
    d.m2 = __fmul2_rn(w, __ffma2_rn(both(-1.f), w, both(-2.f)));
    return d;
}

__device__ __forceinline__ float2 sigmoid2(float2 z) {
    const float2 y = __fmul2_rn(both(-kLog2e), z);
    const float2 d = __fadd2_rn(both(1.f), make_float2(ex2_mufu(y.x), ex2_mufu(y.y)));
    return make_float2(rcp_approx(d.x), rcp_approx(d.y));
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

constexpr int kPairs = kGroup / 2;

// Step e of a group kept as pairs of steps.
__device__ __forceinline__ float& step_of(float2 (&v)[kPairs], int e) { return e % 2 ? v[e / 2].y : v[e / 2].x; }

template <typename IO>
__device__ __forceinline__ void unpack(const RawGroup<IO>& g, float2 (&v)[kPairs]) {
    constexpr int n = Group16<IO>::kN;
#pragma unroll
    for (int k = 0; k < kGroup / n; ++k) {
        float part[n];
        Group16<IO>::unpack(g.v[k], part);
#pragma unroll
        for (int e = 0; e < n; e += 2) v[(k * n + e) / 2] = make_float2(part[e], part[e + 1]);
    }
}

// The steps of the group that lie in [0, n).
template <typename IO>
__device__ __forceinline__ void store_group(IO* row, int t0, int n, bool vec, float2 (&v)[kPairs]) {
    if (vec && t0 >= 0 && t0 + kGroup <= n) {
        uint4* to = reinterpret_cast<uint4*>(row + t0);
        if constexpr (sizeof(IO) == 2) {
            *to = make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y), pack_bf16x2(v[2].x, v[2].y), pack_bf16x2(v[3].x, v[3].y));
        } else {
            reinterpret_cast<float4*>(to)[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
            reinterpret_cast<float4*>(to)[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
        }
    } else {
#pragma unroll
        for (int e = 0; e < kGroup; ++e)
            if (t0 + e >= 0 && t0 + e < n) row[t0 + e] = IoTraits<IO>::from_f32(step_of(v, e));
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
