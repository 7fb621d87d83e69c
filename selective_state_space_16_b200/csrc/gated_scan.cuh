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

#include <type_traits>

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
    const float rate = -p.c * softplus_lam(p.lam[d]);
    const bool near = rate > -kNear;
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
        float2 a[kPairs], u[kPairs], v[kPairs], w[kPairs];
        unpack<IO>(nx, u);
        unpack<IO>(nr, v);
        unpack<IO>(ni, w);
        const RawGroup<IO> zc = nz;
        // the next tile's loads are under way while this one is computed
        nx = load_group(x, t0 + stride, len, p.L, true);
        nr = load_group(r, t0 + stride, len, p.L, vr);
        ni = load_group(i, t0 + stride, len, p.L, vi);
        if (GATE) nz = load_group(z, t0 + stride, len, p.L, vz);
        const auto coefficients = [&](auto near_tag) {
#pragma unroll
            for (int k = 0; k < kPairs; ++k) {
                const Gates gt = gates_of(v[k], w[k], rb, ib);
                const Decay dec = decay_of<decltype(near_tag)::value>(__fmul2_rn(both(rate), gt.rho));
                a[k] = dec.a;
                v[k] = make_float2(sqrt_approx(dec.m2.x), sqrt_approx(dec.m2.y));
                u[k] = __fmul2_rn(u[k], gt.iota);
            }
        };
        if (near)
            coefficients(std::true_type{});
        else
            coefficients(std::false_type{});
        if (RESET && t0 < len) {
#pragma unroll
            for (int e = 0; e < kGroup; ++e)
                if (t0 + e >= 0 && t0 + e < len && reset[t0 + e]) step_of(a, e) = kCut, step_of(v, e) = 1.f;
        }
#pragma unroll
        for (int k = 0; k < kPairs; ++k) u[k] = __fmul2_rn(u[k], v[k]);
        if (t0 < 0 || t0 + kGroup > len) {
#pragma unroll
            for (int e = 0; e < kGroup; ++e)
                if (t0 + e < 0 || t0 + e >= len) step_of(a, e) = 1.f, step_of(u, e) = 0.f;
        }
        float P = a[0].x, H = u[0].x;
#pragma unroll
        for (int e = 1; e < kGroup; ++e) {
            H = carry_on<RESET>(step_of(a, e), H, step_of(u, e));
            P = join<RESET>(P, step_of(a, e));
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
        for (int e = 0; e < kGroup; ++e) step_of(u, e) = h = carry_on<RESET>(step_of(a, e), h, step_of(u, e));
        if (GATE) {
            unpack<IO>(zc, w);
#pragma unroll
            for (int k = 0; k < kPairs; ++k) u[k] = __fmul2_rn(u[k], __fmul2_rn(w[k], sigmoid2(w[k])));
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
    const float rate = -p.c * softplus_lam(p.lam[d]);
    const bool near = rate > -kNear;
    const float rb = -kLog2e * (p.r_bias ? p.r_bias[d] : 0.f), ib = -kLog2e * (p.i_bias ? p.i_bias[d] : 0.f);
    float carry = p.dlast && valid ? p.dlast[row] : 0.f;  // a_{t+1} g_{t+1}: what the steps after the tile send back
    float2 sumT = both(0.f), sumr = both(0.f), sumi = both(0.f);

    const int stride = at.parts * kStep;
    int t = (len + phase + stride - 1) / stride * stride - phase;  // where the rounds with steps end
    for (int t0 = t + (at.part * SEG + at.lane) * kGroup; t0 < L; t0 += stride) {  // padding: zeros
        float2 zero[kPairs] = {};
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
        float2 a[kPairs], g[kPairs], kx[kPairs], ki[kPairs], kT[kPairs], kr[kPairs], b[kPairs], ax[kPairs];
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
        // what g_t is to be multiplied by, for each gradient:
        //   dx  kx = m iota         di  ki = b (1 - iota), b = m iota x
        //   T   kT = a (iota x a v / m - h_{t-1} v), its first part here      dr  T kr, kr = 1 - rho
        const auto coefficients = [&](auto near_tag) {
#pragma unroll
            for (int k = 0; k < kPairs; ++k) {
                const Gates gt = gates_of(kr[k], ki[k], rb, ib);
                const float2 xv = __fmul2_rn(both(rate), gt.rho);  // -v
                const Decay dec = decay_of<decltype(near_tag)::value>(xv);
                // v -> 0: m and v / m go to 0
                const float2 rs = make_float2(rsqrt_approx(fmaxf(dec.m2.x, 1e-30f)), rsqrt_approx(fmaxf(dec.m2.y, 1e-30f)));
                const float2 ux = __fmul2_rn(gt.iota, kx[k]), m = __fmul2_rn(dec.m2, rs);
                a[k] = dec.a;
                ax[k] = __fmul2_rn(dec.a, xv);
                kT[k] = __fmul2_rn(__fmul2_rn(make_float2(-dec.a.x, -dec.a.y), __fmul2_rn(ax[k], rs)), ux);
                kr[k] = __fmul2_rn(gt.Er, gt.rho);
                kx[k] = __fmul2_rn(m, gt.iota);
                b[k] = __fmul2_rn(m, ux);
                ki[k] = __fmul2_rn(b[k], __fmul2_rn(gt.Ei, gt.iota));
                if constexpr (RESET) {
                    const int t = t0 + 2 * k;
                    const bool c0 = t >= 0 && t < end && reset[t], c1 = t + 1 >= 0 && t + 1 < end && reset[t + 1];
                    if (c0) a[k].x = kCut, ax[k].x = kT[k].x = 0.f, kx[k].x = gt.iota.x, b[k].x = ux.x, ki[k].x = ux.x * (gt.Ei.x * gt.iota.x);
                    if (c1) a[k].y = kCut, ax[k].y = kT[k].y = 0.f, kx[k].y = gt.iota.y, b[k].y = ux.y, ki[k].y = ux.y * (gt.Ei.y * gt.iota.y);
                }
            }
        };
        if (near)
            coefficients(std::true_type{});
        else
            coefficients(std::false_type{});
        const bool whole = t0 >= 0 && t0 + kGroup <= end;
        if (!whole) {
#pragma unroll
            for (int e = 0; e < kGroup; ++e)
                if (t0 + e < 0 || t0 + e >= end) {
                    step_of(a, e) = 1.f;
                    step_of(g, e) = step_of(kT, e) = step_of(ax, e) = step_of(kr, e) = step_of(ki, e) = step_of(kx, e) = step_of(b, e) = 0.f;
                }
        }
#pragma unroll
        for (int e = 0; e < kGroup; ++e) {  // b becomes the states
            const float term = fmaf(h, step_of(ax, e), step_of(kT, e));
            step_of(kT, e) = RESET && is_cut(step_of(a, e)) ? 0.f : term;
            step_of(b, e) = h = carry_on<RESET>(step_of(a, e), h, step_of(b, e));
        }
        if (GATE) {
            float2 zv[kPairs];
            unpack<IO>(rz, zv);
#pragma unroll
            for (int k = 0; k < kPairs; ++k) {
                const float2 sig = sigmoid2(zv[k]), zs = __fmul2_rn(zv[k], sig);
                // silu' = sig (1 + z (1 - sig)) = sig + z sig - z sig sig
                const float2 slope = __ffma2_rn(make_float2(-zs.x, -zs.y), sig, __fadd2_rn(sig, zs));
                b[k] = __fmul2_rn(__fmul2_rn(g[k], b[k]), slope);
                g[k] = __fmul2_rn(g[k], zs);
            }
            if (!whole) {
#pragma unroll
                for (int e = 0; e < kGroup; ++e)
                    if (t0 + e < 0 || t0 + e >= end) step_of(g, e) = step_of(b, e) = 0.f;
            }
            if (t >= -phase) store_group(dz, t0, L, vdz, b);
        }
        float P = 1.f, S = 0.f;
#pragma unroll
        for (int k = 0; k < kPairs; ++k) ax[k] = __fmul2_rn(a[k], g[k]);
#pragma unroll
        for (int e = kGroup - 1; e >= 0; --e) {
            S = carry_on<RESET>(step_of(a, e), S, step_of(ax, e));
            P = join<RESET>(P, step_of(a, e));
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
            step_of(g, e) += s;
            s = carry_on<RESET>(step_of(a, e), s, step_of(ax, e));
        }
#pragma unroll
        for (int k = 0; k < kPairs; ++k) {
            const float2 T = __fmul2_rn(g[k], kT[k]);
            kx[k] = __fmul2_rn(g[k], kx[k]);
            kr[k] = __fmul2_rn(T, kr[k]);
            ki[k] = __fmul2_rn(g[k], ki[k]);
            sumT = __fadd2_rn(sumT, T);
            sumr = __fadd2_rn(sumr, kr[k]);
            sumi = __fadd2_rn(sumi, ki[k]);
        }
        if (!whole) {  // (0 times an infinite gradient of the last state)
#pragma unroll
            for (int e = 0; e < kGroup; ++e)
                if (t0 + e >= end) step_of(kx, e) = step_of(kr, e) = step_of(ki, e) = 0.f;
        }
        if (t >= -phase) {
            store_group(dx, t0, L, vdx, kx);
            store_group(dr, t0, L, vdr, kr);
            store_group(di, t0, L, vdi, ki);
        }
    }
    if (p.dh0 && valid && at.part == 0 && at.lane == 0) p.dh0[row] = carry;
    if (p.part) {
        float sT = sumT.x + sumT.y, sr = sumr.x + sumr.y, si = sumi.x + sumi.y;
#pragma unroll
        for (int s = SEG / 2; s; s /= 2) {
            sT += __shfl_xor_sync(kAll, sT, s, SEG);
            sr += __shfl_xor_sync(kAll, sr, s, SEG);
            si += __shfl_xor_sync(kAll, si, s, SEG);
        }
        if constexpr (SPLIT) {
            if (at.lane == 0) part_sums[0][at.part] = sT, part_sums[1][at.part] = sr, part_sums[2][at.part] = si;
            __syncthreads();
            if (threadIdx.x < 3) {
                float s = 0.f;
                for (int k = 0; k < at.parts; ++k) s += part_sums[threadIdx.x][k];
                p.part[threadIdx.x * rows + row] = s;
            }
        } else if (valid && at.lane == 0) {
            p.part[row] = sT, p.part[rows + row] = sr, p.part[2 * rows + row] = si;
        }
    }
}

}  // namespace ssm
