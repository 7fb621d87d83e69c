// gated_math.cuh -- the pieces shared by the kernels of the gated linear recurrence
//   h_t = a_t h_{t-1} + m_t iota_t x_t,   a = exp(-v),  v = c softplus(lam) sigmoid(r),
//   m = sqrt(1 - a^2),  iota = sigmoid(i)
// : its parameters, the coefficients of a step in fp32, and how a row's steps are read and written.
#pragma once

#include <cmath>

#include "common.cuh"
#include "gated_poly.cuh"
#include "scan_math.cuh"

namespace ssm {

// A (batch, dim, seqlen) operand; strides in elements, steps next to each other.
struct GatedTensor {
    const void* p;
    long long bs, ds;
    long long most;    // where the last row starts
    unsigned long long before;  // elements beside a row that may be read where the operand has them: 15, or 0 (rows backwards)
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
    int seg;     // lanes that share a row
    int split;   // warps that share a row (1: a row per warp or part of one)
    int blocks;  // blocks that those warps belong to, a cluster
    bool alike_in, alike_out;  // the inputs, and the gradients, have the same strides and the same place in a vector
    unsigned dim_mul;          // row / dim = row * dim_mul >> (31 + dim_shift)
    int dim_shift;
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

constexpr int kGroup = 8;  // steps between two checkpoints

// Steps that a lane holds at once.  bf16 forward: 16 (two 16-byte vectors of each operand) halve the shuffles
// and the tile's own work per step; 32768 steps of 5120 channels 408 us with 8, 331 with 16.
// fp32, and the backward with six values kept per step: 8.
template <typename IO> constexpr int kFwdSteps = sizeof(IO) == 2 ? 16 : 8;
constexpr int kBwdSteps = 8;

// Stages of the backward's ring.  Forward and backward, us: 8 x 1536 x 2048 bf16 153, 151 and 151 with 2, 3 and 4 (a tenth
// more without a ring, on an earlier form); fp32 253, 250 and 256, but 64 x 32768 fp32 40, 52 and 53 (shared memory for
// fewer blocks).
template <typename IO> constexpr int kBwdStages = sizeof(IO) == 2 ? 3 : 2;

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
    constexpr float kLog2eLow = 1.925963e-8f;  // log2(e) - kLog2e
    const float x = -fabsf(lam), y = x * kLog2e;
    const float low = x > -1e3f ? fmaf(x, kLog2eLow, fmaf(x, kLog2e, -y)) : 0.f;  // (-inf: 0, not NaN)
    float e = ex2_mufu(y);
    e = fmaf(e, low * kLn2, e);
    float p = c[8];
#pragma unroll
    for (int i = 7; i >= 0; --i) p = fmaf(p, e, c[i]);
    return fmaf(e, p, fmaxf(lam, 0.f));
}

// sqrt(2 c softplus(lam)), the root of twice a channel's largest decay exponent, as far as that is an fp32 number: a
// shut gate multiplies it by 0.  (At the bound a = 0 and m = 1 for any open gate.)
__device__ __forceinline__ float root_of(float c, float lam) {
    const float root = sqrtf(2.f * (c * softplus_lam(lam)));
    return root > 1.8e19f ? 1.8e19f : root;
}

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// 1 + y P(y) for the polynomials of gated_poly.cuh, for two steps.
template <int DEG>
__device__ __forceinline__ float2 poly2(float2 y, const float (&c)[DEG]) {
    float2 p = both(c[DEG - 1]);
#pragma unroll
    for (int k = DEG - 2; k >= 0; --k) p = __ffma2_rn(y, p, both(c[k]));
    return __ffma2_rn(y, p, both(1.f));
}

// The coefficients of two steps from their gates' pre-activations.  With E = e^{-(r + r_bias)} (kr is
// -log2(e) r_bias) and root = sqrt(2 c softplus(lam)): Q = root / sqrt(1 + E), so that Q^2 = 2 v.
// A shut gate, E = inf, gives Q = 0 and with it exactly a = 1 and m = 0.
//   a = e^{-v}, m = sqrt(1 - a^2), and v / m for the backward
// are polynomials in 2 v up to v = 1/8, where 1 - a^2 would cancel; beyond it the cancellation costs at
// most 2e-6 of it and they are formed as written.  NEAR: c softplus(lam) <= 1/8, so that no step of
// the channel is beyond it (channels with a memory of some ten steps or more), which saves an
// exponential and a root.  For both element types in fp32: so are the state and the parameters'
// gradients.
constexpr float kNear = 0.5f;  // root of a channel at the border, sqrt(2 / 8)

struct Decay {
    float2 a, m;
    float2 E, rho, v, v_over_m;  // (backward)
};

template <bool NEAR, bool BACKWARD>
__device__ __forceinline__ Decay decay_of(float2 r, float kr, float2 root) {
    constexpr float ca[] = SSM_GATED_DECAY_POLY, cg[] = SSM_GATED_WEIGHT_POLY, ci[] = SSM_GATED_WEIGHT_INV_POLY;
    Decay d;
    const float2 x = __ffma2_rn(both(-kLog2e), r, both(kr));
    d.E = make_float2(ex2_mufu(x.x), ex2_mufu(x.y));
    const float2 p = __fadd2_rn(both(1.f), d.E);
    const float2 R = make_float2(rsqrt_approx(p.x), rsqrt_approx(p.y)), Q = __fmul2_rn(root, R), y = __fmul2_rn(Q, Q);
    d.a = poly2(y, ca);
    d.m = __fmul2_rn(Q, poly2(y, cg));
    if constexpr (BACKWARD) {
        const float2 h = __fmul2_rn(both(0.5f), Q);
        d.rho = __fmul2_rn(R, R);
        d.v = __fmul2_rn(h, Q);
        d.v_over_m = __fmul2_rn(h, poly2(y, ci));
    }
    if constexpr (!NEAR) {
        const float2 half = __fmul2_rn(both(-0.5f * kLog2e), y);
        const float2 e = make_float2(ex2_mufu(half.x), ex2_mufu(half.y));
        const bool nx = y.x < 0.25f, ny = y.y < 0.25f;
        d.a = make_float2(nx ? d.a.x : e.x, ny ? d.a.y : e.y);
        const float2 m2 = __ffma2_rn(make_float2(-e.x, -e.y), e, both(1.f));
        if constexpr (BACKWARD) {
            const float2 rs = make_float2(rsqrt_approx(m2.x), rsqrt_approx(m2.y));
            d.m = make_float2(nx ? d.m.x : m2.x * rs.x, ny ? d.m.y : m2.y * rs.y);
            d.v_over_m = make_float2(nx ? d.v_over_m.x : d.v.x * rs.x, ny ? d.v_over_m.y : d.v.y * rs.y);
        } else {
            d.m = make_float2(nx ? d.m.x : sqrt_approx(m2.x), ny ? d.m.y : sqrt_approx(m2.y));
        }
    }
    return d;
}

// e^{-(i + i_bias)} and sigmoid(i + i_bias) of two steps (ki = -log2(e) i_bias).
struct Gate {
    float2 E, sig;
};

__device__ __forceinline__ Gate gate_of(float2 i, float ki) {
    const float2 x = __ffma2_rn(both(-kLog2e), i, both(ki));
    Gate g;
    g.E = make_float2(ex2_mufu(x.x), ex2_mufu(x.y));
    const float2 d = __fadd2_rn(both(1.f), g.E);
    g.sig = make_float2(rcp_approx(d.x), rcp_approx(d.y));
    return g;
}

// 1 - s of a sigmoid s = 1 / (1 + E) without cancellation.
__device__ __forceinline__ float2 rest_of(float2 E, float2 s) { return __fmul2_rn(make_float2(fminf(E.x, 1e38f), fminf(E.y, 1e38f)), s); }

__device__ __forceinline__ float2 sigmoid2(float2 z) {
    const float2 y = __fmul2_rn(both(-kLog2e), z);
    const float2 d = __fadd2_rn(both(1.f), make_float2(ex2_mufu(y.x), ex2_mufu(y.y)));
    return make_float2(rcp_approx(d.x), rcp_approx(d.y));
}

// silu(z) of two steps, for either type of y: the backward differentiates this gate.  (z (1 + tanh(z / 2)) / 2 with the
// approximate tanh is one special-function operation instead of two, but 2^-12 |z| off: 3.7% of y at z = -5.)
__device__ __forceinline__ float2 silu2(float2 z) { return __fmul2_rn(z, sigmoid2(z)); }

// Two stretches of the recurrence, each (P, H): h -> P h + H, are composed by carry_on for H and
// join for P.  A reset has the coefficient kCut = -0, and CUT = false multiplies by it: enough as
// long as all states are finite.  Infinities and NaNs stay with every state that follows, so a look at
// the last one tells.  Then CUT = true: the sign marks the reset (decays are never negative), the mark
// stays with every product that spans it, and what lies before a marked stretch is dropped, so
// that an infinity or NaN cannot pass.  A product that merely underflows has no mark, and lets them
// pass as the steps one by one would.
constexpr float kCut = -0.f;

__device__ __forceinline__ bool is_cut(float P) { return __float_as_int(P) < 0; }

template <bool CUT>
__device__ __forceinline__ float carry_on(float P, float earlier, float H) {
    const float v = fmaf(P, earlier, H);
    if constexpr (CUT) return is_cut(P) ? H : v;
    return v;
}

template <bool CUT>
__device__ __forceinline__ float join(float P, float Q) {
    const float v = P * Q;
    if constexpr (CUT)
        return __int_as_float(__float_as_int(v) | ((__float_as_int(P) | __float_as_int(Q)) & 0x80000000));
    return v;
}

// N consecutive steps of a row as they lie in memory.
template <typename IO, int N>
struct Raw {
    static constexpr int kVecs = N * sizeof(IO) / 16;
    uint4 v[kVecs];
};

__device__ __forceinline__ uint4 ld_stream(const uint4* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

template <typename IO, int N>
__device__ __forceinline__ void load_vectors(const IO* row, int t0, Raw<IO, N>& g) {
    const uint4* q = reinterpret_cast<const uint4*>(row + t0);
#pragma unroll
    for (int k = 0; k < Raw<IO, N>::kVecs; ++k) g.v[k] = ld_stream(q + k);
}

// The row's ends, and rows that lie otherwise than the groups do: element by element, 0 outside [0, len).
template <typename IO, int N>
__device__ __forceinline__ void load_elements(const IO* row, int t0, int len, Raw<IO, N>& g) {
    constexpr int kWords = N * sizeof(IO) / 4;
    uint32_t w[kWords] = {};
#pragma unroll
    for (int e = 0; e < N; ++e) {
        if (t0 + e < 0 || t0 + e >= len) continue;
        if constexpr (sizeof(IO) == 2)
            w[e / 2] |= static_cast<uint32_t>(reinterpret_cast<const unsigned short*>(row)[t0 + e]) << (e % 2 * 16);
        else
            w[e] = reinterpret_cast<const uint32_t*>(row)[t0 + e];
    }
#pragma unroll
    for (int k = 0; k < kWords / 4; ++k) g.v[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
}

// Which steps of a row may be read as whole vectors: up to 15 before and behind it, as far as that is
// inside every operand (a row's neighbours are).  So only the ends of an operand are read by elements.
struct Reach {
    int low, high;
};

__host__ __device__ __forceinline__ void narrow(Reach& reach, const GatedTensor& t, long long at) {
    // (unsigned, so that places before the address, where `before` is 0, do not wrap)
    reach.low = max(reach.low, -static_cast<int>(min(static_cast<unsigned long long>(at), t.before)));
    reach.high = min(reach.high, static_cast<int>(min(static_cast<unsigned long long>(t.most - at), t.before)));
}

__device__ __forceinline__ long long offset_of(const GatedTensor& t, int b, int d) { return b * t.bs + d * t.ds; }

// The row (b, d) of operands that are `alike` or not, which narrows the reach.  A row's own work is as many
// instructions as a tile, so what alike operands share is found once (with row / dim as a product: 2% of the backward
// of 16 x 5120 rows of 250 steps).
template <typename IO, int N, typename... T>
__device__ __forceinline__ void rows_of(bool alike, int b, int d, IO* (&row)[N], Reach& reach, const GatedTensor& t0, const T&... t) {
    static_assert(sizeof...(T) + 1 == N, "a tensor for each row");
    const long long at = offset_of(t0, b, d);
    int k = 0;
    if (alike) {
        narrow(reach, t0, at);
        row[0] = static_cast<IO*>(const_cast<void*>(t0.p)) + at;
        ((row[++k] = static_cast<IO*>(const_cast<void*>(t.p)) + at), ...);
    } else {
        narrow(reach, t0, at);
        row[0] = static_cast<IO*>(const_cast<void*>(t0.p)) + at;
        ((narrow(reach, t, offset_of(t, b, d)), row[++k] = static_cast<IO*>(const_cast<void*>(t.p)) + offset_of(t, b, d)), ...);
    }
}

// A row's groups are laid so that those of x start on 16-byte boundaries: group g holds the steps
// from g * kGroup - phase.  Operands that lie like x, which dense ones of one shape do, are read and
// written as vectors at any length of the rows; each operand is looked at by itself.
template <typename IO>
__device__ __forceinline__ int phase_of(const IO* row) {
    return static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(IO));
}

// Which rows have their vectors where the groups have them.
template <typename IO, int N>
__device__ __forceinline__ bool in_phase(bool alike, IO* const (&row)[N], int phase, bool (&vec)[N]) {
    bool all = phase_of(row[0]) == phase;
    vec[0] = all;
    if (alike) {
#pragma unroll
        for (int k = 1; k < N; ++k) vec[k] = vec[0];
    } else {
#pragma unroll
        for (int k = 1; k < N; ++k) all &= vec[k] = phase_of(row[k]) == phase;
    }
    return all;
}

// Steps [t0, t0 + N) of the operands, those of them inside [0, len); the others are anything.
template <typename IO, int N, int IN>
__device__ __forceinline__ void load_steps(const IO* const (&in)[IN], const bool (&vec)[IN], bool all_vec, int t0, int len, Reach reach,
                                           Raw<IO, N> (&g)[IN]) {
    const bool whole = t0 >= reach.low && t0 + N <= reach.high;
    if (all_vec && whole && t0 < len) {
#pragma unroll
        for (int k = 0; k < IN; ++k) load_vectors(in[k], t0, g[k]);
    } else if (t0 < len && t0 + N > 0) {
#pragma unroll
        for (int k = 0; k < IN; ++k) {
            if (vec[k] && whole)
                load_vectors(in[k], t0, g[k]);
            else
                load_elements(in[k], t0, len, g[k]);
        }
    }
}

// The same a few tiles ahead: the threads of a warp copy the steps of the tiles to come into slots of shared memory
// and read them from there when their turn comes.  Nothing outside the warp touches its slots, so there is
// nothing to wait for but its own copies; and the tiles under way take no registers.  A thread's slots lie
// next to each other, in pairs exchanged so that reading them has no bank conflicts; a warp whose tile is whole
// copies it in 512-byte pieces (COOP: a tile is one stretch of a row).
template <typename IO, int N, int IN, bool COOP>
struct Ring {
    static constexpr int kV = Raw<IO, N>::kVecs, kVecs = IN * kV;  // 16-byte slots of a thread for an operand, a stage
    __device__ static uint4* slot(uint4* ring, int stage, int k, int chunk) {  // chunk of the warp's 32 * kV
        if (kV == 2) chunk ^= chunk >> 3 & 1;
        return ring + (stage * kVecs + k * kV) * blockDim.x + (threadIdx.x & ~31u) * kV + chunk;
    }
    // One group of copies: steps [t0, t0 + N) of each thread.
    __device__ static void load(uint4* ring, int stage, const IO* const (&in)[IN], const bool (&vec)[IN], bool all_vec, int t0, int len,
                                Reach reach) {
        const int lane = threadIdx.x & 31;
        const bool whole = t0 >= reach.low && t0 + N <= reach.high, all = all_vec && whole && t0 < len;
        if (kV > 1 && COOP && __all_sync(0xffffffffu, all)) {
            constexpr int kChunk = 16 / sizeof(IO);
#pragma unroll
            for (int k = 0; k < IN; ++k)
#pragma unroll
                for (int j = 0; j < kV; ++j)
                    cp_async_16(slot(ring, stage, k, j * 32 + lane), in[k] + (t0 - lane * N) + (j * 32 + lane) * kChunk, 16);
        } else if (all) {
#pragma unroll
            for (int k = 0; k < IN; ++k) copy(ring, stage, k, in[k], t0);
        } else if (t0 < len && t0 + N > 0) {
#pragma unroll
            for (int k = 0; k < IN; ++k) {
                if (vec[k] && whole) {
                    copy(ring, stage, k, in[k], t0);
                } else {
                    Raw<IO, N> g;
                    load_elements(in[k], t0, len, g);
#pragma unroll
                    for (int j = 0; j < kV; ++j) *slot(ring, stage, k, lane * kV + j) = g.v[j];
                }
            }
        }
        cp_async_commit();
    }
    __device__ static void copy(uint4* ring, int stage, int k, const IO* row, int t0) {
        const uint4* q = reinterpret_cast<const uint4*>(row + t0);
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int j = 0; j < kV; ++j) cp_async_16(slot(ring, stage, k, lane * kV + j), q + j, 16);
    }
    // After it the oldest of STAGES - 1 groups has arrived.
    template <int STAGES>
    __device__ static void wait() {
        cp_async_wait<STAGES - 2>();
        if (kV > 1 && COOP) __syncwarp();
    }
    __device__ static Raw<IO, N> read(uint4* ring, int stage, int k) {
        Raw<IO, N> s;
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int j = 0; j < kV; ++j) s.v[j] = *slot(ring, stage, k, lane * kV + j);
        return s;
    }
};

__device__ __forceinline__ bool finite(float v) { return fabsf(v) < __int_as_float(0x7f800000); }

// Step e of steps kept as pairs.
template <int PAIRS>
__device__ __forceinline__ float& step_of(float2 (&v)[PAIRS], int e) {
    return e % 2 ? v[e / 2].y : v[e / 2].x;
}

template <typename IO, int N>
__device__ __forceinline__ void unpack(const Raw<IO, N>& g, float2 (&v)[N / 2]) {
    constexpr int n = Group16<IO>::kN;
#pragma unroll
    for (int k = 0; k < N / n; ++k) {
        float part[n];
        Group16<IO>::unpack(g.v[k], part);
#pragma unroll
        for (int e = 0; e < n; e += 2) v[(k * n + e) / 2] = make_float2(part[e], part[e + 1]);
    }
}

template <typename IO, int PAIRS>
__device__ __forceinline__ void store_vectors(IO* row, int t0, float2 (&v)[PAIRS]) {
    uint4* to = reinterpret_cast<uint4*>(row + t0);
    if constexpr (sizeof(IO) == 2) {
#pragma unroll
        for (int k = 0; k < PAIRS; k += 4)
            to[k / 4] = make_uint4(pack_bf16x2(v[k].x, v[k].y), pack_bf16x2(v[k + 1].x, v[k + 1].y), pack_bf16x2(v[k + 2].x, v[k + 2].y),
                                   pack_bf16x2(v[k + 3].x, v[k + 3].y));
    } else {
#pragma unroll
        for (int k = 0; k < PAIRS; k += 2) reinterpret_cast<float4*>(to)[k / 2] = make_float4(v[k].x, v[k].y, v[k + 1].x, v[k + 1].y);
    }
}

// Which of the steps [t0, t0 + N) lie in [0, n), a bit each.
template <int N> constexpr unsigned all_steps = (1u << N) - 1;

template <int N>
__device__ __forceinline__ unsigned steps_inside(int t0, int n) {
    unsigned bits = all_steps<N>;
    if (t0 + N > n) bits = n > t0 ? (1u << (n - t0)) - 1 : 0;  // (n - t0 < N)
    if (t0 < 0) bits &= t0 > -N ? ~((1u << -t0) - 1) : 0;
    return bits;
}

// The steps at the bits; `vec`: as a vector where that is all of them.  A row's ends: each word and element under its
// own bit, without a branch (a tenth of the backward of 16 x 5120 rows of 101 steps).
template <typename IO, int PAIRS>
__device__ __forceinline__ void store_steps(IO* row, int t0, unsigned bits, bool vec, float2 (&v)[PAIRS]) {
    if (vec && bits == all_steps<2 * PAIRS>) {
        store_vectors(row, t0, v);
    } else if (bits) {
        IO* to = row + t0;
        const unsigned words = sizeof(IO) == 2 && vec ? bits & bits >> 1 & 0x5555u : 0;  // pairs that are both inside
        const unsigned rest = bits & ~(words * 3);
#pragma unroll
        for (int k = 0; k < PAIRS; ++k) {
            if constexpr (sizeof(IO) == 2) {
                const uint32_t w = pack_bf16x2(v[k].x, v[k].y);
                unsigned short* half = reinterpret_cast<unsigned short*>(to) + 2 * k;
                if (words >> (2 * k) & 1) *reinterpret_cast<uint32_t*>(half) = w;
                if (rest >> (2 * k) & 1) half[0] = static_cast<unsigned short>(w);
                if (rest >> (2 * k) & 2) half[1] = static_cast<unsigned short>(w >> 16);
            } else {
                if (bits >> (2 * k) & 1) to[2 * k] = v[k].x;
                if (bits >> (2 * k) & 2) to[2 * k + 1] = v[k].y;
            }
        }
    }
}

// The steps outside the bits become `other`, given as a word of elements.  With the recurrence gate shut
// (-inf) a step has a = 1 and no input, and with the rest 0 no gradient: it passes the state through.
template <typename IO> constexpr uint32_t shut = sizeof(IO) == 2 ? 0xff80ff80u : 0xff800000u;

// (A bias of +inf must not meet that -inf.)
__device__ __forceinline__ float bounded(float v) { return v == v ? fminf(fmaxf(v, -3e38f), 3e38f) : v; }

template <typename IO, int N>
__device__ __forceinline__ void mask_steps(unsigned bits, Raw<IO, N>& g, uint32_t other) {
    uint32_t* w = reinterpret_cast<uint32_t*>(g.v);
    constexpr int kPer = 4 / sizeof(IO);
#pragma unroll
    for (int k = 0; k < N / kPer; ++k) {
        const unsigned b = bits >> (k * kPer);
        const uint32_t keep = kPer == 1 ? 0u - (b & 1) : (b & 1 ? 0xffffu : 0u) | (b & 2 ? 0xffff0000u : 0u);
        w[k] = (w[k] & keep) | (other & ~keep);
    }
}

// The reset flags of 8 steps, a byte each, 0 outside [0, len).  A row's flags lie at any alignment: two
// aligned words and a shift, or bytes where those words would reach out of the array [begin, end).
__device__ __forceinline__ unsigned long long reset_flags(const unsigned char* row, int t0, int len, const unsigned char* begin,
                                                          const unsigned char* end) {
    const unsigned char* q = row + t0;
    const unsigned off = static_cast<unsigned>(reinterpret_cast<uintptr_t>(q) & 7u);
    unsigned long long flags = 0;
    if (t0 >= len || t0 + 8 <= 0) return 0;
    if (t0 >= 0 && t0 + 8 <= len && q - off >= begin && q - off + 16 <= end) {
        const auto* w = reinterpret_cast<const unsigned long long*>(q - off);
        flags = w[0] >> (8 * off);
        if (off) flags |= w[1] << (64 - 8 * off);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (t0 + e >= 0 && t0 + e < len) flags |= static_cast<unsigned long long>(q[e]) << (8 * e);
    }
    return flags;
}

__device__ __forceinline__ bool flag_of(unsigned long long flags, int e) {
    return (static_cast<unsigned>(flags >> (e / 4 * 32)) & (0xffu << (e % 4 * 8))) != 0;
}

template <typename IO>
__device__ __forceinline__ IO* row_of(const GatedTensor& t, int b, int d) {
    return static_cast<IO*>(const_cast<void*>(t.p)) + offset_of(t, b, d);
}

__device__ __forceinline__ int batch_of(const GatedParams& p, unsigned row) {
    return static_cast<int>(static_cast<unsigned long long>(row) * p.dim_mul >> (31 + p.dim_shift));
}

__device__ __forceinline__ int row_length(const GatedParams& p, int b) {
    return p.lengths ? min(max(p.lengths[b], 0), p.L) : p.L;
}

}  // namespace ssm
