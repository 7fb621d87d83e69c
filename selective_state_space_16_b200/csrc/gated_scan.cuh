// gated_scan.cuh -- forward and backward of the gated linear recurrence over whole sequences.
//
// A row (b, d) is walked in tiles: lane k of SEG lanes holds 8 consecutive steps (a group).  The
// recurrence is composed of pairs (P, H), h -> P h + H: each lane forms its group's pair, rounds of
// shuffles give every lane the state before its first step, and the lane runs its steps again from
// there.  The backward does the same from the last tile to the first; the states come from the
// checkpoints, one before every group, so it has to scan in one direction only.
//
// SEG = 32: a warp per row.  SEG = 8, 2: several short rows per warp, so that few lanes idle.
// SPLIT: p.split warps of a block share one row, each taking every p.split-th tile; a barrier a round
// joins their pairs.  That is for few long rows, which could not fill the GPU's warps otherwise.
#pragma once

#include "gated_math.cuh"

namespace ssm {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kGatedWarps = 4;  // warps of a block without SPLIT
constexpr int kMaxSplit = 16;
#ifndef FWD_MINB
#define FWD_MINB 6
#endif
#ifndef BWD_MINB
#define BWD_MINB 4
#endif

// The row of this lane, and where in it the lane works.
template <int SEG, bool SPLIT>
struct RowPlace {
    long long row;
    int lane;         // 0 .. SEG - 1
    int part, parts;  // which of the warps that share the row
    __device__ RowPlace(const GatedParams& p) {
        lane = threadIdx.x % SEG;
        part = SPLIT ? threadIdx.x / 32 : 0;
        parts = SPLIT ? p.split : 1;
        row = SPLIT ? blockIdx.x : static_cast<long long>(blockIdx.x) * (kGatedWarps * 32 / SEG) + threadIdx.x / SEG;
    }
};

// With SPLIT: from the pairs of the warps that share a row, in the order in which they follow each
// other, what enters this warp's tile and, in `carry`, what leaves the round.  One barrier a round:
// a buffer is written again two rounds later, behind the barrier that its readers have passed.
template <bool RESET>
__device__ __forceinline__ float join_parts(float2* pairs, int place, int parts, bool writer, float P, float H, float& carry) {
    if (writer) pairs[place] = make_float2(P, H);
    __syncthreads();
    float in = carry, mine = carry;
    for (int k = 0; k < parts; ++k) {
        if (k == place) mine = in;
        in = carry_on<RESET>(pairs[k].x, in, pairs[k].y);
    }
    carry = in;
    return mine;
}

template <typename IO, bool GATE, bool RESET, int SEG, bool SPLIT>
__global__ void __launch_bounds__(SPLIT ? kMaxSplit * 32 : kGatedWarps * 32, SPLIT ? 1 : FWD_MINB) gated_fwd_kernel(const GatedParams p) {
    constexpr int kStep = SEG * kGroup;
    __shared__ float2 pairs[SPLIT ? 2 : 1][SPLIT ? kMaxSplit : 1];
    const RowPlace<SEG, SPLIT> at(p);
    const long long row = at.row;
    const long long rows = static_cast<long long>(p.batch) * p.dim;
    const bool valid = row < rows;
    if (SEG == 32 && !valid) return;  // (a whole warp)
    const int b = valid ? static_cast<int>(row / p.dim) : 0, d = valid ? static_cast<int>(row % p.dim) : 0;
    const int len = valid ? row_length(p, b) : 0;
    const IO *x = row_of<IO>(p.x, b, d), *r = row_of<IO>(p.r, b, d), *i = row_of<IO>(p.i, b, d);
    const IO* z = GATE ? row_of<IO>(p.z, b, d) : nullptr;
    IO* y = p.y.p ? row_of<IO>(p.y, b, d) : nullptr;
    const int phase = phase_of(x);
    const bool vr = phase_of(r) == phase, vi = phase_of(i) == phase, vz = GATE && phase_of(z) == phase, vy = phase_of(y) == phase;
    const unsigned char* reset = RESET ? p.reset + static_cast<long long>(b) * p.L : nullptr;
    const float rate = -p.c * softplus_lam(p.lam[d]) * kLog2e;
    const float rb = -kLog2e * (p.r_bias ? p.r_bias[d] : 0.f), ib = -kLog2e * (p.i_bias ? p.i_bias[d] : 0.f);
    float carry = p.h0 && valid ? p.h0[row] : 0.f;
    float* ckpt = p.ckpt ? p.ckpt + sizeof(CkptHeader) / 4 + row * p.ckpt_row : nullptr;
    if (p.ckpt && blockIdx.x == 0 && threadIdx.x == 0) {
        constexpr unsigned n = 16 / sizeof(IO);
        *reinterpret_cast<CkptHeader*>(p.ckpt) = {static_cast<unsigned>(phase_of(static_cast<const IO*>(p.x.p))),
                                                  static_cast<unsigned>(p.x.bs) % n, static_cast<unsigned>(p.x.ds) % n, 0};
    }

    int t0 = (at.part * SEG + at.lane) * kGroup - phase;
    const int stride = at.parts * kStep;
    RawGroup<IO> nx = load_group(x, t0, len, p.L, true), nr = load_group(r, t0, len, p.L, vr), ni = load_group(i, t0, len, p.L, vi), nz;
    if (GATE) nz = load_group(z, t0, len, p.L, vz);
    int round = 0;
#pragma unroll 1
    for (int t = -phase; SEG == 32 ? t < len : __any_sync(kAll, t < len); t += stride, t0 += stride, ++round) {
        float a[kGroup], u[kGroup], v[kGroup], w[kGroup];
        unpack<IO>(nx, u);
        unpack<IO>(nr, v);
        unpack<IO>(ni, w);
        const RawGroup<IO> zc = nz;
        // the next tile's loads are under way while this one is computed
        nx = load_group(x, t0 + stride, len, p.L, true);
        nr = load_group(r, t0 + stride, len, p.L, vr);
        ni = load_group(i, t0 + stride, len, p.L, vi);
        if (GATE) nz = load_group(z, t0 + stride, len, p.L, vz);
        const bool whole = t0 >= 0 && t0 + kGroup <= len;
#pragma unroll
        for (int e = 0; e < kGroup; ++e) {
            const Decay dec = decay_of(rate * rcp_approx(1.f + ex2_mufu(fmaf(-kLog2e, v[e], rb))));
            a[e] = dec.a;
            float m = sqrt_approx(dec.m2);
            if (RESET && t0 + e >= 0 && t0 + e < len && reset[t0 + e]) a[e] = kCut, m = 1.f;
            u[e] *= m * rcp_approx(1.f + ex2_mufu(fmaf(-kLog2e, w[e], ib)));
        }
        if (!whole) {
#pragma unroll
            for (int e = 0; e < kGroup; ++e)
                if (t0 + e < 0 || t0 + e >= len) a[e] = 1.f, u[e] = 0.f;
        }
        float P = a[0], H = u[0];
#pragma unroll
        for (int e = 1; e < kGroup; ++e) {
            H = carry_on<RESET>(a[e], H, u[e]);
            P = join<RESET>(P, a[e]);
        }
#pragma unroll
        for (int s = 1; s < SEG; s *= 2) {
            const float Pe = __shfl_up_sync(kAll, P, s, SEG), He = __shfl_up_sync(kAll, H, s, SEG);
            if (at.lane >= s) H = carry_on<RESET>(P, He, H), P = join<RESET>(P, Pe);
        }
        float h;
        if constexpr (SPLIT) {
            const float in = join_parts<RESET>(pairs[round & 1], at.part, at.parts, at.lane == 31, P, H, carry);
            const float all = carry_on<RESET>(P, in, H);
            h = __shfl_up_sync(kAll, all, 1);
            if (at.lane == 0) h = in;
        } else {
            const float all = carry_on<RESET>(P, carry, H);  // the state after this lane's steps
            h = __shfl_up_sync(kAll, all, 1, SEG);
            if (at.lane == 0) h = carry;
            carry = __shfl_sync(kAll, all, SEG - 1, SEG);
        }
        if (ckpt && t0 < len) ckpt[(t0 + phase) / kGroup] = h;
#pragma unroll
        for (int e = 0; e < kGroup; ++e) u[e] = h = carry_on<RESET>(a[e], h, u[e]);
        if (GATE) {
            unpack<IO>(zc, w);
#pragma unroll
            for (int e = 0; e < kGroup; ++e) u[e] *= silu_f32(w[e]);
        }
        if (y) store_group(y, t0, len, vy, u);
    }
    if (p.last && valid && at.part == 0 && at.lane == 0) p.last[row] = carry;
}

template <typename IO, bool GATE, bool RESET, int SEG, bool SPLIT>
__global__ void __launch_bounds__(SPLIT ? kMaxSplit * 32 : kGatedWarps * 32, SPLIT ? 1 : BWD_MINB) gated_bwd_kernel(const GatedParams p) {
    constexpr int kStep = SEG * kGroup;
    __shared__ float2 pairs[SPLIT ? 2 : 1][SPLIT ? kMaxSplit : 1];
    __shared__ float part_sums[SPLIT ? 3 : 1][SPLIT ? kMaxSplit : 1];
    const RowPlace<SEG, SPLIT> at(p);
    const long long row = at.row;
    const long long rows = static_cast<long long>(p.batch) * p.dim;
    const bool valid = row < rows;
    if (SEG == 32 && !valid) return;
    const int b = valid ? static_cast<int>(row / p.dim) : 0, d = valid ? static_cast<int>(row % p.dim) : 0;
    const int len = valid ? row_length(p, b) : 0, L = valid ? p.L : 0;
    const IO *x = row_of<IO>(p.x, b, d), *r = row_of<IO>(p.r, b, d), *i = row_of<IO>(p.i, b, d);
    const IO *z = GATE ? row_of<IO>(p.z, b, d) : nullptr, *dy = row_of<IO>(p.dy, b, d);
    IO *dx = row_of<IO>(p.dx, b, d), *dr = row_of<IO>(p.dr, b, d), *di = row_of<IO>(p.di, b, d);
    IO* dz = GATE ? row_of<IO>(p.dz, b, d) : nullptr;
    const CkptHeader where = *reinterpret_cast<const CkptHeader*>(p.ckpt);
    const int phase = static_cast<int>((where.base + b * where.bs + d * where.ds) % (16 / sizeof(IO)));
    const bool vx = phase_of(x) == phase, vr = phase_of(r) == phase, vi = phase_of(i) == phase, vz = GATE && phase_of(z) == phase,
               vdy = phase_of(dy) == phase, vdx = phase_of(dx) == phase, vdr = phase_of(dr) == phase, vdi = phase_of(di) == phase,
               vdz = GATE && phase_of(dz) == phase;
    const unsigned char* reset = RESET ? p.reset + static_cast<long long>(b) * p.L : nullptr;
    const float* ckpt = p.ckpt + sizeof(CkptHeader) / 4 + row * p.ckpt_row;
    const float rate = -p.c * softplus_lam(p.lam[d]) * kLog2e;
    const float rb = -kLog2e * (p.r_bias ? p.r_bias[d] : 0.f), ib = -kLog2e * (p.i_bias ? p.i_bias[d] : 0.f);
    float carry = p.dlast && valid ? p.dlast[row] : 0.f;  // a_{t+1} g_{t+1}: what the steps after the tile send back
    float sumT = 0.f, sumr = 0.f, sumi = 0.f;

    const int stride = at.parts * kStep;
    int t = (len + phase + stride - 1) / stride * stride - phase;  // where the rounds with steps end
    for (int t0 = t + (at.part * SEG + at.lane) * kGroup; t0 < L; t0 += stride) {  // padding: zeros
        const float zero[kGroup] = {};
        store_group(dx, t0, L, vdx, zero);
        store_group(dr, t0, L, vdr, zero);
        store_group(di, t0, L, vdi, zero);
        if (GATE) store_group(dz, t0, L, vdz, zero);
    }
    int round = 0;
#pragma unroll 1
    for (t -= stride; SEG == 32 ? t >= -phase : __any_sync(kAll, t >= -phase); t -= stride, ++round) {
        const int t0 = t + (at.part * SEG + at.lane) * kGroup;
        // (a short row that is done while others of its warp go on: t0 below its first step, no steps inside)
        const int end = t >= -phase ? len : -phase;
        float a[kGroup], g[kGroup], kx[kGroup], ki[kGroup], kT[kGroup], kr[kGroup];
        const RawGroup<IO> rz = GATE ? load_group(z, t0, end, p.L, vz) : RawGroup<IO>{};
        {
            const RawGroup<IO> rx = load_group(x, t0, end, p.L, vx), rr = load_group(r, t0, end, p.L, vr),
                               ri = load_group(i, t0, end, p.L, vi), rg = load_group(dy, t0, end, p.L, vdy);
            unpack<IO>(rx, kx);
            unpack<IO>(rr, kr);
            unpack<IO>(ri, ki);
            unpack<IO>(rg, g);
        }
        float h = t0 >= -phase && t0 < end ? ckpt[(t0 + phase) / kGroup] : 0.f;
        float zv[kGroup], gz[kGroup];
        if (GATE) unpack<IO>(rz, zv);
#pragma unroll
        for (int e = 0; e < kGroup; ++e) {
            const bool cut = RESET && t0 + e >= 0 && t0 + e < end && reset[t0 + e];
            const float Er = ex2_mufu(fmaf(-kLog2e, kr[e], rb)), Ei = ex2_mufu(fmaf(-kLog2e, ki[e], ib));
            const float rho = rcp_approx(1.f + Er), iota = rcp_approx(1.f + Ei);
            const float yv = rate * rho;
            const Decay dec = decay_of(yv);
            a[e] = dec.a;
            const float rs = rsqrt_approx(fmaxf(dec.m2, 1e-30f));  // v -> 0: m and v / m go to 0
            float m = dec.m2 * rs;
            const float v = -kLn2 * yv, q = v * rs;
            if (cut) a[e] = kCut, m = 1.f;
            const float ux = iota * kx[e];
            // what g_t is to be multiplied by, for each gradient
            const float T = cut ? 0.f : a[e] * (ux * a[e] * q - h * v);
            const float before = h;
            h = carry_on<RESET>(a[e], h, m * ux);
            kT[e] = T;
            kr[e] = T * (fminf(Er, 1e38f) * rho);  // 1 - rho = Er rho, without cancellation
            ki[e] = m * ux * (fminf(Ei, 1e38f) * iota);
            kx[e] = m * iota;
            if (GATE) {
                const float sig = rcp_approx(1.f + ex2_mufu(-kLog2e * zv[e]));
                gz[e] = g[e] * h * sig * fmaf(zv[e], 1.f - sig, 1.f);
                g[e] *= zv[e] * sig;
            }
            if (t0 + e < 0) h = before;
        }
        const bool whole = t0 >= 0 && t0 + kGroup <= end;
        if (!whole) {
#pragma unroll
            for (int e = 0; e < kGroup; ++e)
                if (t0 + e < 0 || t0 + e >= end) {
                    a[e] = 1.f;
                    g[e] = kT[e] = kr[e] = ki[e] = kx[e] = 0.f;
                    if (GATE) gz[e] = 0.f;
                }
        }
        if (GATE && t >= -phase) store_group(dz, t0, L, vdz, gz);
        float P = 1.f, S = 0.f;
#pragma unroll
        for (int e = kGroup - 1; e >= 0; --e) {
            S = carry_on<RESET>(a[e], g[e] + S, 0.f);
            P = join<RESET>(P, a[e]);
        }
#pragma unroll
        for (int s = 1; s < SEG; s *= 2) {
            const float Pl = __shfl_down_sync(kAll, P, s, SEG), Sl = __shfl_down_sync(kAll, S, s, SEG);
            if (at.lane + s < SEG) S = carry_on<RESET>(P, Sl, S), P = join<RESET>(P, Pl);
        }
        float s;
        if constexpr (SPLIT) {
            const float in = join_parts<RESET>(pairs[round & 1], at.parts - 1 - at.part, at.parts, at.lane == 0, P, S, carry);
            const float all = carry_on<RESET>(P, in, S);
            s = __shfl_down_sync(kAll, all, 1);
            if (at.lane == 31) s = in;
        } else {
            const float all = carry_on<RESET>(P, carry, S);
            s = __shfl_down_sync(kAll, all, 1, SEG);
            if (at.lane == SEG - 1) s = carry;
            carry = __shfl_sync(kAll, all, 0, SEG);
        }
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
        if (!whole) {  // (0 times an infinite gradient of the last state)
#pragma unroll
            for (int e = 0; e < kGroup; ++e)
                if (t0 + e >= end) kx[e] = kr[e] = ki[e] = 0.f;
        }
        if (t >= -phase) {
            store_group(dx, t0, L, vdx, kx);
            store_group(dr, t0, L, vdr, kr);
            store_group(di, t0, L, vdi, ki);
        }
    }
    if (p.dh0 && valid && at.part == 0 && at.lane == 0) p.dh0[row] = carry;
    if (p.part) {
#pragma unroll
        for (int s = SEG / 2; s; s /= 2) {
            sumT += __shfl_xor_sync(kAll, sumT, s, SEG);
            sumr += __shfl_xor_sync(kAll, sumr, s, SEG);
            sumi += __shfl_xor_sync(kAll, sumi, s, SEG);
        }
        if constexpr (SPLIT) {
            if (at.lane == 0) part_sums[0][at.part] = sumT, part_sums[1][at.part] = sumr, part_sums[2][at.part] = sumi;
            __syncthreads();
            if (threadIdx.x < 3) {
                float s = 0.f;
                for (int k = 0; k < at.parts; ++k) s += part_sums[threadIdx.x][k];
                p.part[threadIdx.x * rows + row] = s;
            }
        } else if (valid && at.lane == 0) {
            p.part[row] = sumT, p.part[rows + row] = sumr, p.part[2 * rows + row] = sumi;
        }
    }
}

}  // namespace ssm
