// gated_scan.cuh -- forward and backward of the gated linear recurrence over whole sequences.
//
// A warp walks one (b, d) row in tiles of 256 steps: lane k holds 8 consecutive steps.  The
// recurrence is composed of pairs (P, H), h -> P h + H: each lane forms its own 8 steps' pair,
// five rounds of shuffles give every lane the state before its first step, and the lane runs its
// steps again from there.  The backward does the same from the last tile to the first.
#pragma once

#include "gated_math.cuh"

namespace ssm {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kGatedWarps = 4;

template <typename IO, bool GATE, bool RESET>
__global__ void __launch_bounds__(kGatedWarps * 32) gated_fwd_kernel(const GatedParams p) {
    const int lane = threadIdx.x & 31;
    const long long row = static_cast<long long>(blockIdx.x) * kGatedWarps + threadIdx.x / 32;
    if (row >= static_cast<long long>(p.batch) * p.dim) return;
    const int b = static_cast<int>(row / p.dim), d = static_cast<int>(row % p.dim);
    const int len = row_length(p, b);
    const IO *x = row_of<IO>(p.x, b, d), *r = row_of<IO>(p.r, b, d), *i = row_of<IO>(p.i, b, d);
    const IO* z = GATE ? row_of<IO>(p.z, b, d) : nullptr;
    IO* y = p.y.p ? row_of<IO>(p.y, b, d) : nullptr;
    const unsigned char* reset = RESET ? p.reset + static_cast<long long>(b) * p.L : nullptr;
    const float rate = -p.c * softplus_once(p.lam[d]) * kLog2e;
    const float rb = p.r_bias ? p.r_bias[d] : 0.f, ib = p.i_bias ? p.i_bias[d] : 0.f;
    float carry = p.h0 ? p.h0[row] : 0.f;

    for (int t = 0; t < len; t += kTile) {
        const int t0 = t + lane * kGroup;
        float a[kGroup], u[kGroup], rv[kGroup], iv[kGroup];
        load_group(x, t0, len, u);
        load_group(r, t0, len, rv);
        load_group(i, t0, len, iv);
        float P = 1.f, H = 0.f;
#pragma unroll
        for (int e = 0; e < kGroup; ++e) {
            const float yv = rate * rcp_approx(1.f + ex2_mufu(-kLog2e * (rv[e] + rb)));
            a[e] = ex2_mufu(yv);
            float m = sqrt_approx(one_minus_square(yv, a[e]));
            if (RESET && t0 + e < len && reset[t0 + e]) a[e] = kCut, m = 1.f;
            u[e] *= m * rcp_approx(1.f + ex2_mufu(-kLog2e * (iv[e] + ib)));
            if (t0 + e >= len) a[e] = 1.f, u[e] = 0.f;
            H = carry_on<RESET>(a[e], H, u[e]);
            P = join<RESET>(P, a[e]);
        }
#pragma unroll
        for (int s = 1; s < 32; s *= 2) {
            const float Pe = __shfl_up_sync(kAll, P, s), He = __shfl_up_sync(kAll, H, s);
            if (lane >= s) H = carry_on<RESET>(P, He, H), P = join<RESET>(P, Pe);
        }
        const float all = carry_on<RESET>(P, carry, H);  // the state after this lane's steps
        float h = __shfl_up_sync(kAll, all, 1);
        if (lane == 0) h = carry;
        carry = __shfl_sync(kAll, all, 31);
        if (p.ckpt && t0 < len) p.ckpt[row * p.ckpt_row + t0 / kGroup] = h;
#pragma unroll
        for (int e = 0; e < kGroup; ++e) u[e] = h = carry_on<RESET>(a[e], h, u[e]);
        if (GATE) {
            load_group(z, t0, len, rv);
#pragma unroll
            for (int e = 0; e < kGroup; ++e) u[e] *= silu_f32(rv[e]);
        }
        if (y) store_group(y, t0, len, u);
    }
    if (p.last && lane == 0) p.last[row] = carry;
}

template <typename IO, bool GATE, bool RESET>
__global__ void __launch_bounds__(kGatedWarps * 32) gated_bwd_kernel(const GatedParams p) {
    const int lane = threadIdx.x & 31;
    const long long row = static_cast<long long>(blockIdx.x) * kGatedWarps + threadIdx.x / 32;
    const long long rows = static_cast<long long>(p.batch) * p.dim;
    if (row >= rows) return;
    const int b = static_cast<int>(row / p.dim), d = static_cast<int>(row % p.dim);
    const int len = row_length(p, b);
    const IO *x = row_of<IO>(p.x, b, d), *r = row_of<IO>(p.r, b, d), *i = row_of<IO>(p.i, b, d);
    const IO *z = GATE ? row_of<IO>(p.z, b, d) : nullptr, *dy = row_of<IO>(p.dy, b, d);
    const unsigned char* reset = RESET ? p.reset + static_cast<long long>(b) * p.L : nullptr;
    const float rate = -p.c * softplus_once(p.lam[d]) * kLog2e;
    const float rb = p.r_bias ? p.r_bias[d] : 0.f, ib = p.i_bias ? p.i_bias[d] : 0.f;
    float carry = p.dlast ? p.dlast[row] : 0.f;  // a_{t+1} g_{t+1}, the gradient from the steps after the tile
    float sumT = 0.f, sumr = 0.f, sumi = 0.f;

    for (int t = (p.L - 1) / kTile * kTile; t >= 0; t -= kTile) {
        const int t0 = t + lane * kGroup;
        float a[kGroup], g[kGroup], kx[kGroup], ki[kGroup], kT[kGroup], kr[kGroup], v[kGroup], w[kGroup];
        load_group(x, t0, len, kx);
        load_group(r, t0, len, kr);
        load_group(i, t0, len, ki);
        load_group(dy, t0, len, g);
        if (GATE) load_group(z, t0, len, w);
        float h = t0 < len ? p.ckpt[row * p.ckpt_row + t0 / kGroup] : 0.f;
        float P = 1.f, S = 0.f;
#pragma unroll
        for (int e = 0; e < kGroup; ++e) {
            const bool in = t0 + e < len;
            const bool cut = RESET && in && reset[t0 + e];
            const float Er = ex2_mufu(-kLog2e * (kr[e] + rb)), Ei = ex2_mufu(-kLog2e * (ki[e] + ib));
            const float rho = rcp_approx(1.f + Er), iota = rcp_approx(1.f + Ei);
            const float yv = rate * rho;
            a[e] = ex2_mufu(yv);
            const float m2 = one_minus_square(yv, a[e]);
            const float rs = rsqrt_approx(fmaxf(m2, 1e-30f));  // v -> 0: m and v / m go to 0
            float m = m2 * rs;
            const float vv = -kLn2 * yv, q = vv * rs;
            if (cut) a[e] = kCut, m = 1.f;
            const float ux = iota * kx[e];
            // what g_t is to be multiplied by, for each gradient
            const float T = cut ? 0.f : a[e] * (ux * a[e] * q - h * vv);
            kT[e] = T;
            kr[e] = T * (fminf(Er, 1e38f) * rho);              // 1 - rho = Er rho, without cancellation
            ki[e] = m * ux * (fminf(Ei, 1e38f) * iota);
            kx[e] = m * iota;
            h = carry_on<RESET>(a[e], h, m * ux);
            if (GATE) {
                const float sig = rcp_approx(1.f + ex2_mufu(-kLog2e * w[e]));
                v[e] = g[e] * h * sig * fmaf(w[e], 1.f - sig, 1.f);
                g[e] *= w[e] * sig;
            }
            if (!in) a[e] = 1.f, g[e] = 0.f, v[e] = kT[e] = kr[e] = ki[e] = kx[e] = 0.f;
        }
        if (GATE) store_group(row_of<IO>(p.dz, b, d), t0, p.L, v);
#pragma unroll
        for (int e = kGroup - 1; e >= 0; --e) {
            S = carry_on<RESET>(a[e], g[e] + S, 0.f);
            P = join<RESET>(P, a[e]);
        }
#pragma unroll
        for (int s = 1; s < 32; s *= 2) {
            const float Pl = __shfl_down_sync(kAll, P, s), Sl = __shfl_down_sync(kAll, S, s);
            if (lane + s < 32) S = carry_on<RESET>(P, Sl, S), P = join<RESET>(P, Pl);
        }
        const float all = carry_on<RESET>(P, carry, S);
        float s = __shfl_down_sync(kAll, all, 1);
        if (lane == 31) s = carry;
        carry = __shfl_sync(kAll, all, 0);
#pragma unroll
        for (int e = kGroup - 1; e >= 0; --e) {
            const float ge = g[e] + s;
            s = carry_on<RESET>(a[e], ge, 0.f);
            sumT = fmaf(ge, kT[e], sumT);
            kx[e] *= ge;
            kr[e] *= ge;
            ki[e] *= ge;
            sumr += kr[e];
            sumi += ki[e];
        }
        store_group(row_of<IO>(p.dx, b, d), t0, p.L, kx);
        store_group(row_of<IO>(p.dr, b, d), t0, p.L, kr);
        store_group(row_of<IO>(p.di, b, d), t0, p.L, ki);
    }
    if (p.dh0 && lane == 0) p.dh0[row] = carry;
    if (p.part) {
#pragma unroll
        for (int s = 16; s; s /= 2) {
            sumT += __shfl_xor_sync(kAll, sumT, s);
            sumr += __shfl_xor_sync(kAll, sumr, s);
            sumi += __shfl_xor_sync(kAll, sumi, s);
        }
        if (lane == 0) p.part[row] = sumT, p.part[rows + row] = sumr, p.part[2 * rows + row] = sumi;
    }
}

}  // namespace ssm
