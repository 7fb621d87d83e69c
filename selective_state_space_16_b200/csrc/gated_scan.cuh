// gated_scan.cuh -- forward and backward of the gated linear recurrence over whole sequences.
//
// A row (b, d) is walked in tiles: each of its lanes holds 8 or 16 consecutive steps.  The recurrence is composed
// of pairs (P, H), h -> P h + H: each lane forms its steps' pair, rounds of shuffles give every lane the state
// before its first step, and the lane runs its steps again from there.  The backward does the same from the
// last tile to the first; the states come from the checkpoints, one before every group of 8, so it has to
// scan in one direction only, and dx, dr, di, dz and the parameters' sums leave the same pass.
//
// SEG = 32: a warp per row.  SEG = 0: p.seg lanes per row, 1 to 16: several short rows per warp, so that few
// lanes idle (16 x 5120 rows of 100 steps, forward and backward: 127 us, 264 with a warp each).
// SPLIT: the warps of a block, or of a cluster of blocks, share one row: of p.split warps in all each takes
// every p.split-th tile, and a barrier a round joins their pairs, which every warp writes into the shared
// memory of all blocks of the cluster.  That is for few long rows, which could not fill the GPU's warps
// otherwise (64 rows of 32768 steps: 27 us, 58 with 4 warps of a block).
//
// Figures here and in gated_math.cuh and gated_launch.cuh: us of replayed graphs under a steady load (a cold call is up to
// 5% faster where the power bounds the clock, a few us slower where it is short), bf16 with the output gate unless said,
// every channel near (decay_of), the backward with the forward's checkpoints.  From box to box they differ by 3%.
//
// What bounds it: the special-function unit (forward: 6 operations a step, three exponentials, a reciprocal root, two
// reciprocals; 71 to 76% of its peak) and issue (about 31 instructions a step forward, 65 backward, packed fp32 pairs
// throughout, and some 300 and 400 a row; 50 to 66%) beside the bytes.  32768 steps of 5120 channels: 331 us, 77% of the copy
// rate; 2048 steps of 8 x 1536 channels, forward and backward, 151 us (71%), with resets 164 (66%), fp32 252 (85%).
// Channels beyond the near ones cost an exponential and a root more: 384 us instead of 343 for the former on one box, 164
// instead of 155 for the second.  What was slower on earlier forms: the forward's operands through the backward's ring
// (5% and more); warps that stay and take the next row's first tile under way (registers); reset flags a tile ahead
// (3%); a later row's first tile fetched into L2 by the warp before (no gain, or 2%).
#pragma once

#include <type_traits>

#include "cluster.cuh"
#include "gated_math.cuh"

namespace ssm {

constexpr unsigned kAll = 0xffffffffu;

// 4- and 8-byte asynchronous copies global -> shared.
__device__ __forceinline__ void cp_async_4(void* dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_8(void* dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

constexpr int kGatedWarps = 4;  // warps of a block without SPLIT
constexpr int kMaxSplit = 8;    // warps of a block with SPLIT (two such blocks per SM)
constexpr int kMaxParts = 32;   // warps that share a row
constexpr int kMaxCluster = 8;  // blocks that share a row
// Blocks per SM that the registers are held to, so 128 registers, or 168 for the fp32 backward (3 x 1001 x 2047
// forward and backward: 72 us with 3, 78 with 4).  More blocks spill: 5 took 384 us against 331 (forward, 5120 x
// 32768), 116 against 96 (backward, 8 x 1536 x 2048).
constexpr int kFwdBlocks = 4;
template <typename IO> constexpr int kBwdBlocks = sizeof(IO) == 2 ? 4 : 3;

// Dynamic shared memory of a block of the backward: the ring, and slots for the checkpoints and reset flags.
template <typename IO>
constexpr int bwd_smem(bool gate, bool reset, int threads) {
    return kBwdStages<IO> * ((gate ? Ring<IO, kBwdSteps, 5, true>::kVecs : Ring<IO, kBwdSteps, 4, true>::kVecs) * 16 + 4 + (reset ? 8 : 0)) * threads;
}

// The product of a lane's decays, as join.
template <bool CUT, int PAIRS>
__device__ __forceinline__ float product(float2 (&a)[PAIRS]) {
    if constexpr (CUT) {
        float P = a[0].x;
#pragma unroll
        for (int e = 1; e < 2 * PAIRS; ++e) P = join<true>(P, step_of(a, e));
        return P;
    } else {
        float2 q[PAIRS / 2];
#pragma unroll
        for (int k = 0; k < PAIRS / 2; ++k) q[k] = __fmul2_rn(a[2 * k], a[2 * k + 1]);
#pragma unroll
        for (int k = 1; k < PAIRS / 2; ++k) q[0] = __fmul2_rn(q[0], q[k]);
        return q[0].x * q[0].y;
    }
}

// What steps outside a row send on: nothing, not even 0 times an infinity or NaN of the state or gradient that passes
// through them or of the channel's parameters.  Where all of these are finite the products are zeros by themselves
// (clearing them always: backward of 16 x 5120 rows of 101 steps 92 -> 94 us).
template <int PAIRS>
__device__ __forceinline__ void clear_outside(unsigned inside, float2 (&v)[PAIRS]) {
#pragma unroll
    for (int e = 0; e < 2 * PAIRS; ++e)
        if (!(inside >> e & 1)) step_of(v, e) = 0.f;
}

// Writes two floats to the same place of block `rank`'s shared memory as `here` in this one's.
__device__ __forceinline__ void st_cluster(const float2* here, unsigned rank, float2 v) {
    unsigned to;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(smem_u32(here)), "r"(rank));
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(v.x), "f"(v.y) : "memory");
}

// The row of this lane, and where in it the lane works.
template <int SEG, bool SPLIT>
struct RowPlace {
    unsigned row;
    int seg, lane;    // lanes per row; 0 .. seg - 1
    int part, parts;  // which of the warps that share the row
    int blocks, rank; // of the cluster that shares the row
    __device__ RowPlace(const GatedParams& p) {
        seg = SEG ? SEG : p.seg;
        lane = threadIdx.x & (seg - 1);
        blocks = SPLIT ? p.blocks : 1;
        rank = blocks > 1 ? static_cast<int>(cluster_rank()) : 0;
        part = SPLIT ? rank * (blockDim.x / 32) + threadIdx.x / 32 : 0;
        parts = SPLIT ? p.split : 1;
        row = SPLIT ? blockIdx.x / blocks : blockIdx.x * (kGatedWarps * 32 / seg) + threadIdx.x / seg;
    }
};

// With SPLIT: from the pairs of the warps that share a row, in the order in which they follow each
// other, what enters this warp's tile and, in `carry`, what leaves the round.  One barrier a round:
// a buffer is written again two rounds later, behind the barrier that its readers have passed.
template <bool RESET>
__device__ __forceinline__ float join_parts(float2* pairs, int place, int parts, int blocks, int writer, float P, float H, float& carry) {
    const int lane = threadIdx.x & 31;
    if (blocks == 1) {
        if (lane == writer) pairs[place] = make_float2(P, H);
        __syncthreads();
    } else {
        const float2 v = make_float2(__shfl_sync(kAll, P, writer), __shfl_sync(kAll, H, writer));
        if (lane < blocks) st_cluster(pairs + place, lane, v);
        __syncwarp();
        cluster_arrive();
        cluster_wait();
    }
    float in = carry, mine = carry;
    for (int k = 0; k < parts; ++k) {
        if (k == place) mine = in;
        in = carry_on<RESET>(pairs[k].x, in, pairs[k].y);
    }
    carry = in;
    return mine;
}

template <typename IO, bool GATE, bool RESET, int SEG, bool SPLIT>
__global__ void __launch_bounds__(SPLIT ? kMaxSplit * 32 : kGatedWarps * 32, SPLIT ? 2 : kFwdBlocks)
    gated_fwd_kernel(const GatedParams p) {
    constexpr int N = kFwdSteps<IO>, kPairs = N / 2, kIn = 3;
    __shared__ float2 pairs[SPLIT ? 2 : 1][SPLIT ? kMaxParts : 1];
    const RowPlace<SEG, SPLIT> at(p);
    const long long row = at.row;
    const long long rows = static_cast<long long>(p.batch) * p.dim;
    const bool valid = at.row < static_cast<unsigned>(rows);
    if (SEG == 32 && !valid) return;  // (a whole warp)
    if (SPLIT && at.blocks > 1) cluster_arrive(), cluster_wait();  // every block has begun: its shared memory may be written
    const int b = valid ? batch_of(p, at.row) : 0, d = valid ? at.row - static_cast<unsigned>(b) * p.dim : 0;
    const int len = valid ? row_length(p, b) : 0;
    Reach reach{-15, 15};
    const IO* in[kIn];
    const IO* zrow[1];
    if constexpr (GATE) {
        const IO* row_in[kIn + 1];
        rows_of(p.alike_in, b, d, row_in, reach, p.x, p.r, p.i, p.z);
        in[0] = row_in[0], in[1] = row_in[1], in[2] = row_in[2], zrow[0] = row_in[3];
    } else {
        rows_of(p.alike_in, b, d, in, reach, p.x, p.r, p.i);
    }
    reach.high += p.L;
    IO* y = p.y.p ? row_of<IO>(p.y, b, d) : nullptr;
    const int phase = valid ? phase_of(in[0]) : 0;  // (lanes without a row, of length 0: no step lies before that)
    bool vec[kIn];
    const bool all_vec = in_phase(p.alike_in, in, phase, vec);
    const bool vy = phase_of(y) == phase, vz[1] = {GATE && (p.alike_in || phase_of(zrow[0]) == phase)};
    const unsigned char* reset = RESET ? p.reset + static_cast<long long>(b) * p.L : nullptr;
    const unsigned char* reset_end = RESET ? p.reset + static_cast<long long>(p.batch) * p.L : nullptr;
    const float root = root_of(p.c, p.lam[d]);
    const bool near = root <= kNear;
    const float rb = bounded(-kLog2e * (p.r_bias ? p.r_bias[d] : 0.f)), ib = -kLog2e * (p.i_bias ? p.i_bias[d] : 0.f);
    float carry = p.h0 && valid ? p.h0[row] : 0.f;
    const float first = carry;
    float* ckpt = p.ckpt ? p.ckpt + sizeof(CkptHeader) / 4 + row * p.ckpt_row : nullptr;
    if (p.ckpt && blockIdx.x == 0 && threadIdx.x == 0) {
        constexpr unsigned n = 16 / sizeof(IO);
        *reinterpret_cast<CkptHeader*>(p.ckpt) = {static_cast<unsigned>(phase_of(static_cast<const IO*>(p.x.p))),
                                                  static_cast<unsigned>(p.x.bs) % n, static_cast<unsigned>(p.x.ds) % n, 0};
    }

    int t0 = (at.part * at.seg + at.lane) * N - phase;
    const int stride = at.parts * at.seg * N;
    Raw<IO, N> next[kIn];
    load_steps(in, vec, all_vec, t0, valid ? p.L : 0, reach, next);  // (not waiting for len)
    int round = 0;
#pragma unroll 1
    for (int t = -phase; SEG == 32 ? t < len : __any_sync(kAll, t < len); t += stride, t0 += stride, ++round) {
        float2 a[kPairs], u[kPairs], v[kPairs], w[kPairs];
        const unsigned inside = steps_inside<N>(t0, len);
        if (inside != all_steps<N>) mask_steps<IO, N>(inside, next[0], 0), mask_steps<IO, N>(inside, next[1], shut<IO>), mask_steps<IO, N>(inside, next[2], 0);
        unpack<IO, N>(next[0], u);
        unpack<IO, N>(next[1], v);
        unpack<IO, N>(next[2], w);
        Raw<IO, N> zc[1];
        if (GATE) load_steps(zrow, vz, vz[0], t0, len, reach, zc);  // wanted last
        load_steps(in, vec, all_vec, t0 + stride, len, reach, next);  // under way while this tile is computed
        const auto coefficients = [&](auto near_tag) {
#pragma unroll
            for (int k = 0; k < kPairs; ++k) {
                const Decay dec = decay_of<decltype(near_tag)::value, false>(v[k], rb, both(root));
                a[k] = dec.a;
                u[k] = __fmul2_rn(u[k], gate_of(w[k], ib).sig);
                if (RESET) v[k] = u[k];  // (m_t = 1 at a reset)
                u[k] = __fmul2_rn(u[k], dec.m);
            }
        };
        if (near)
            coefficients(std::true_type{});
        else
            coefficients(std::false_type{});
        bool any_cut = false;
        if (RESET) {
            unsigned long long flags[N / 8], any = 0;
#pragma unroll
            for (int k = 0; k < N / 8; ++k) any |= flags[k] = reset_flags(reset, t0 + 8 * k, len, p.reset, reset_end);
            any_cut = __any_sync(kAll, any != 0);
            if (any_cut) {
#pragma unroll
                for (int e = 0; e < N; ++e)
                    if (flag_of(flags[e / 8], e % 8)) step_of(a, e) = kCut, step_of(u, e) = step_of(v, e);
            }
        }
        float P, H;
        const auto compose = [&](auto cut_tag) {  // (P, H) of the tile up to and with this lane's steps
            constexpr bool CUT = decltype(cut_tag)::value;
            H = u[0].x;
#pragma unroll
            for (int e = 1; e < N; ++e) H = carry_on<CUT>(step_of(a, e), H, step_of(u, e));
            P = product<CUT>(a);
#pragma unroll
            for (int s = 1; s < at.seg; s *= 2) {
                const float Pe = __shfl_up_sync(kAll, P, s, at.seg), He = __shfl_up_sync(kAll, H, s, at.seg);
                if (at.lane >= s) H = carry_on<CUT>(P, He, H), P = join<CUT>(P, Pe);
            }
        };
        compose(std::false_type{});
        bool careful = false;
        if (RESET && any_cut) {
            careful = __any_sync(kAll, !finite(H) || (!SPLIT && !finite(carry)));
            if (careful) compose(std::true_type{});
        }
        float enters = carry;
        if constexpr (SPLIT) {
            enters = join_parts<RESET>(pairs[round & 1], at.part, at.parts, at.blocks, 31, any_cut ? kCut : P, H, carry);
            if (RESET && any_cut && !careful && !finite(enters)) careful = true, compose(std::true_type{});
        }
        const auto states = [&](auto cut_tag) {
            constexpr bool CUT = decltype(cut_tag)::value;
            const float all = carry_on<CUT>(P, enters, H);  // the state after this lane's steps
            float h = __shfl_up_sync(kAll, all, 1, at.seg);
            if (at.lane == 0) h = enters;
            if (!SPLIT) carry = __shfl_sync(kAll, all, at.seg - 1, at.seg);
            if (ckpt && t0 < len) ckpt[(t0 + phase) / kGroup] = h;
#pragma unroll
            for (int e = 0; e < N; ++e) {
                if (e == kGroup && ckpt && t0 + kGroup < len) ckpt[(t0 + phase) / kGroup + 1] = h;
                step_of(u, e) = h = carry_on<CUT>(step_of(a, e), h, step_of(u, e));
            }
        };
        if (RESET && careful)
            states(std::true_type{});
        else
            states(std::false_type{});
        if (GATE) {
            unpack<IO, N>(zc[0], w);
#pragma unroll
            for (int k = 0; k < kPairs; ++k) u[k] = __fmul2_rn(u[k], silu2(w[k]));
        }
        if (y) store_steps(y, t0, inside, vy, u);
    }
    if (p.last && valid && at.part == 0 && at.lane == 0) p.last[row] = len > 0 ? carry : first;
}

template <typename IO, bool GATE, bool RESET, int SEG, bool SPLIT>
__global__ void __launch_bounds__(SPLIT ? kMaxSplit * 32 : kGatedWarps * 32, SPLIT ? 2 : kBwdBlocks<IO>)
    gated_bwd_kernel(const GatedParams p) {
    constexpr int N = kBwdSteps, kPairs = N / 2, kIn = GATE ? 5 : 4, kOut = GATE ? 4 : 3;
    __shared__ float2 pairs[SPLIT ? 2 : 1][SPLIT ? kMaxParts : 1];
    __shared__ float2 part_sums[SPLIT ? kMaxParts : 1][2];
    const RowPlace<SEG, SPLIT> at(p);
    const long long row = at.row;
    const long long rows = static_cast<long long>(p.batch) * p.dim;
    const bool valid = at.row < static_cast<unsigned>(rows);
    if (SEG == 32 && !valid) return;
    if (SPLIT && at.blocks > 1) cluster_arrive(), cluster_wait();
    const int b = valid ? batch_of(p, at.row) : 0, d = valid ? at.row - static_cast<unsigned>(b) * p.dim : 0;
    const int len = valid ? row_length(p, b) : 0, L = valid ? p.L : 0;
    Reach reach{-15, 15}, any{0, 0};
    const IO* in[kIn];
    IO* out[kOut];
    if constexpr (GATE) {
        rows_of(p.alike_in, b, d, in, reach, p.x, p.r, p.i, p.dy, p.z);
        rows_of(p.alike_out, b, d, out, any, p.dx, p.dr, p.di, p.dz);
    } else {
        rows_of(p.alike_in, b, d, in, reach, p.x, p.r, p.i, p.dy);
        rows_of(p.alike_out, b, d, out, any, p.dx, p.dr, p.di);
    }
    reach.high += p.L;
    const CkptHeader where = *reinterpret_cast<const CkptHeader*>(p.ckpt);
    const int phase = valid ? static_cast<int>((where.base + b * where.bs + d * where.ds) % (16 / sizeof(IO))) : 0;
    bool vin[kIn], vout[kOut];
    const bool in_vec = in_phase(p.alike_in, in, phase, vin), all_vec = in_phase(p.alike_out, out, phase, vout) && in_vec;
    const unsigned char* reset = RESET ? p.reset + static_cast<long long>(b) * p.L : nullptr;
    const unsigned char* reset_end = RESET ? p.reset + static_cast<long long>(p.batch) * p.L : nullptr;
    const float* ckpt = p.ckpt + sizeof(CkptHeader) / 4 + row * p.ckpt_row;
    const float root = root_of(p.c, p.lam[d]);
    const bool near = root <= kNear;
    const float rb = bounded(-kLog2e * (p.r_bias ? p.r_bias[d] : 0.f)), ib = -kLog2e * (p.i_bias ? p.i_bias[d] : 0.f);
    float carry = p.dlast && valid ? p.dlast[row] : 0.f;  // a_{t+1} g_{t+1}: what the steps after the tile send back
    const float first = carry;
    float2 sumT = both(0.f), sumr = both(0.f), sumi = both(0.f);
    const bool plain = finite(root + rb) && ib == ib;  // (a gate's bias of -inf, ib = inf, just shuts it)

    const int stride = at.parts * at.seg * N;
    int t = ((len + phase + stride - 1) & -stride) - phase;  // where the rounds with steps end (stride: a power of two)
    for (int t0 = t + (at.part * at.seg + at.lane) * N; t0 < L; t0 += stride) {  // padding: zeros
        float2 zero[kPairs] = {};
#pragma unroll
        for (int k = 0; k < kOut; ++k) store_steps(out[k], t0, steps_inside<N>(t0, L), vout[k], zero);
    }
    using In = Ring<IO, N, kIn, SEG == 32>;
    constexpr int kStages = kBwdStages<IO>;
    extern __shared__ uint4 ring[];
    auto* flags_in = reinterpret_cast<unsigned long long*>(ring + kStages * In::kVecs * blockDim.x) + threadIdx.x;
    float* states_in = reinterpret_cast<float*>(flags_in - threadIdx.x + (RESET ? kStages * blockDim.x : 0)) + threadIdx.x;
    const auto load = [&](int stage, int t) {
        const int t0 = t + (at.part * at.seg + at.lane) * N;
        const bool active = t >= -phase;
        if (RESET) {
            if (active && t0 >= 0 && t0 + 8 <= len && (reinterpret_cast<uintptr_t>(reset + t0) & 7) == 0)
                cp_async_8(flags_in + stage * blockDim.x, reset + t0);
            else
                flags_in[stage * blockDim.x] = reset_flags(reset, t0, active ? len : -N, p.reset, reset_end);
        }
        if (active && t0 < len) cp_async_4(states_in + stage * blockDim.x, ckpt + (t0 + phase) / kGroup);
        In::load(ring, stage, in, vin, all_vec, t0, active ? len : -N, reach);
    };
    int round = 0, stage = 0;
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) load(k, t - (k + 1) * stride);
#pragma unroll 1
    for (t -= stride; SEG == 32 ? t >= -phase : __any_sync(kAll, t >= -phase); t -= stride, ++round) {
        const int t0 = t + (at.part * at.seg + at.lane) * N;
        // (a short row that is done while others of its warp go on lies before its first step: no steps inside)
        const bool active = SEG == 32 || t >= -phase;
        const int end = active ? len : -phase;
        const unsigned inside = steps_inside<N>(t0, end);
        const bool whole = inside == all_steps<N>;
        float2 a[kPairs], g[kPairs], kx[kPairs], ki[kPairs], kT[kPairs], kr[kPairs], b[kPairs], ax[kPairs];
        Raw<IO, N> raw[kIn];
        unsigned long long flags = 0;
        float h = 0.f;
        In::template wait<kStages>();
#pragma unroll
        for (int k = 0; k < kIn; ++k) raw[k] = In::read(ring, stage, k);
        if (t0 < end && active) h = states_in[stage * blockDim.x];
        if (RESET) flags = flags_in[stage * blockDim.x];
        load(stage == 0 ? kStages - 1 : stage - 1, t - (kStages - 1) * stride);  // into the slots read a tile ago
        stage = stage == kStages - 1 ? 0 : stage + 1;
        if (!whole) {
#pragma unroll
            for (int k = 0; k < kIn; ++k) mask_steps<IO, N>(inside, raw[k], k == 1 ? shut<IO> : 0);
        }
        unpack<IO, N>(raw[0], kx);
        unpack<IO, N>(raw[1], kr);
        unpack<IO, N>(raw[2], ki);
        unpack<IO, N>(raw[3], g);
        const bool any_cut = RESET && __any_sync(kAll, flags != 0);
        // what g_t is to be multiplied by, for each gradient:
        //   dx  kx = m iota         di  ki = b (1 - iota), b = m iota x
        //   T = a (iota x a v / m - h_{t-1} v) = kT - h_{t-1} ax       dr  T kr, kr = 1 - rho
        const auto coefficients = [&](auto near_tag) {
#pragma unroll
            for (int k = 0; k < kPairs; ++k) {
                const Decay dec = decay_of<decltype(near_tag)::value, true>(kr[k], rb, both(root));
                const Gate gate = gate_of(ki[k], ib);
                const float2 ux = __fmul2_rn(gate.sig, kx[k]), qa = __fmul2_rn(dec.a, dec.v_over_m);
                float2 m = dec.m;
                a[k] = dec.a;
                ax[k] = __fmul2_rn(dec.a, dec.v);
                kT[k] = __fmul2_rn(__fmul2_rn(dec.a, qa), ux);
                kr[k] = rest_of(dec.E, dec.rho);
                if (RESET && any_cut) {
                    if (flag_of(flags, 2 * k)) a[k].x = kCut, m.x = 1.f, ax[k].x = kT[k].x = 0.f;
                    if (flag_of(flags, 2 * k + 1)) a[k].y = kCut, m.y = 1.f, ax[k].y = kT[k].y = 0.f;
                }
                kx[k] = __fmul2_rn(m, gate.sig);
                b[k] = __fmul2_rn(m, ux);
                ki[k] = __fmul2_rn(b[k], rest_of(gate.E, gate.sig));
            }
        };
        if (near)
            coefficients(std::true_type{});
        else
            coefficients(std::false_type{});
        const auto states = [&](auto cut_tag) {
            constexpr bool CUT = decltype(cut_tag)::value;
#pragma unroll
            for (int e = 0; e < N; ++e) {  // kT becomes T, b the states
                const float term = fmaf(-h, step_of(ax, e), step_of(kT, e));
                step_of(kT, e) = CUT && is_cut(step_of(a, e)) ? 0.f : term;
                step_of(b, e) = h = carry_on<CUT>(step_of(a, e), h, step_of(b, e));
            }
        };
        bool clear = !whole && !(plain && finite(h));  // (finite so far)
        bool careful = false;
        if (RESET && any_cut) {  // no state is larger than this sum
            float most = fabsf(h);
#pragma unroll
            for (int e = 0; e < N; ++e) most += fabsf(step_of(b, e));
            careful = __any_sync(kAll, !finite(most));
        }
        if (RESET && careful)
            states(std::true_type{});
        else
            states(std::false_type{});
        clear |= !whole && !finite(h);
        if (GATE) {
            float2 zv[kPairs];
            unpack<IO, N>(raw[kIn - 1], zv);
#pragma unroll
            for (int k = 0; k < kPairs; ++k) {
                const float2 sig = sigmoid2(zv[k]), zs = __fmul2_rn(zv[k], sig);
                // silu' = sig + z sig (1 - sig)
                const float2 slope = __ffma2_rn(zs, __ffma2_rn(both(-1.f), sig, both(1.f)), sig);
                b[k] = __fmul2_rn(__fmul2_rn(g[k], b[k]), slope);
                g[k] = __fmul2_rn(g[k], zs);
            }
            if (all_vec && whole) {
                store_vectors(out[kOut - 1], t0, b);
            } else if (active) {
                if (clear) clear_outside(inside, b);
                store_steps(out[kOut - 1], t0, steps_inside<N>(t0, L), vout[kOut - 1], b);
            }
        }
#pragma unroll
        for (int k = 0; k < kPairs; ++k) ax[k] = __fmul2_rn(a[k], g[k]);
        float P, S;
        const auto compose = [&](auto cut_tag) {  // (P, S) of the tile from this lane's steps on
            constexpr bool CUT = decltype(cut_tag)::value;
            S = ax[kPairs - 1].y;
#pragma unroll
            for (int e = N - 2; e >= 0; --e) S = carry_on<CUT>(step_of(a, e), S, step_of(ax, e));
            P = product<CUT>(a);
#pragma unroll
            for (int s = 1; s < at.seg; s *= 2) {
                const float Pl = __shfl_down_sync(kAll, P, s, at.seg), Sl = __shfl_down_sync(kAll, S, s, at.seg);
                if (at.lane + s < at.seg) S = carry_on<CUT>(P, Sl, S), P = join<CUT>(P, Pl);
            }
        };
        const auto drop = [&] {  // a reset's own gradient goes nowhere either, not even as 0 * inf
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (is_cut(step_of(a, e))) step_of(ax, e) = 0.f;
        };
        compose(std::false_type{});
        careful = false;
        if (RESET && any_cut) {
            careful = __any_sync(kAll, !finite(S) || (!SPLIT && !finite(carry)));
            if (careful) drop(), compose(std::true_type{});
        }
        float enters = carry;
        if constexpr (SPLIT) {
            enters = join_parts<RESET>(pairs[round & 1], at.parts - 1 - at.part, at.parts, at.blocks, 0, any_cut ? kCut : P, S, carry);
            if (RESET && any_cut && !careful && !finite(enters)) careful = true, drop(), compose(std::true_type{});
        }
        const auto gradients = [&](auto cut_tag) {
            constexpr bool CUT = decltype(cut_tag)::value;
            const float all = carry_on<CUT>(P, enters, S);
            float s = __shfl_down_sync(kAll, all, 1, at.seg);
            if (at.lane == at.seg - 1) s = enters;
            clear |= !whole && !finite(s);
            if (!SPLIT) carry = __shfl_sync(kAll, all, 0, at.seg);
#pragma unroll
            for (int e = N - 1; e >= 0; --e) {
                step_of(g, e) += s;
                s = carry_on<CUT>(step_of(a, e), s, step_of(ax, e));
            }
            clear |= !whole && !finite(s);
        };
        if (RESET && careful)
            gradients(std::true_type{});
        else
            gradients(std::false_type{});
        if (clear) clear_outside(inside, g), clear_outside(inside, kT), clear_outside(inside, kr), clear_outside(inside, kx), clear_outside(inside, ki);
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
        if (all_vec && whole) {
            store_vectors(out[0], t0, kx);
            store_vectors(out[1], t0, kr);
            store_vectors(out[2], t0, ki);
        } else if (active) {
            const unsigned to = steps_inside<N>(t0, L);
            store_steps(out[0], t0, to, vout[0], kx);
            store_steps(out[1], t0, to, vout[1], kr);
            store_steps(out[2], t0, to, vout[2], ki);
        }
    }
    if (p.dh0 && valid && at.part == 0 && at.lane == 0) p.dh0[row] = len > 0 ? carry : first;
    if (p.part) {
        float sT = sumT.x + sumT.y, sr = sumr.x + sumr.y, si = sumi.x + sumi.y;
#pragma unroll
        for (int s = at.seg / 2; s; s /= 2) {
            sT += __shfl_xor_sync(kAll, sT, s, at.seg);
            sr += __shfl_xor_sync(kAll, sr, s, at.seg);
            si += __shfl_xor_sync(kAll, si, s, at.seg);
        }
        if constexpr (SPLIT) {  // summed by the first block, in the order of the parts
            if (at.blocks == 1) {
                if (at.lane == 0) part_sums[at.part][0] = make_float2(sT, sr), part_sums[at.part][1] = make_float2(si, 0.f);
                __syncthreads();
            } else {
                if (at.lane == 0) st_cluster(&part_sums[at.part][0], 0, make_float2(sT, sr)), st_cluster(&part_sums[at.part][1], 0, make_float2(si, 0.f));
                __syncwarp();
                cluster_arrive();
                cluster_wait();
            }
            if (at.rank == 0 && threadIdx.x == 0) {
                float3 s = make_float3(0.f, 0.f, 0.f);
                for (int k = 0; k < at.parts; ++k) s.x += part_sums[k][0].x, s.y += part_sums[k][0].y, s.z += part_sums[k][1].x;
                p.part[row] = s.x, p.part[rows + row] = s.y, p.part[2 * rows + row] = s.z;
            }
        } else if (valid && at.lane == 0) {
            p.part[row] = sT, p.part[rows + row] = sr, p.part[2 * rows + row] = si;
        }
    }
}

}  // namespace ssm
