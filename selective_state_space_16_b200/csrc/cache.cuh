// cache.cuh -- device side of the state cache (ssm_cache.h).
//
// Every call is a plan and a move.  The plan, one block, reads the lists and `used` and decides
// which page goes where; the move copies or clears the pages of all layers and pools.  The move is
// a programmatic dependent of the plan: its blocks are resident when the plan ends.
#pragma once

#include "../../include/ssm_cache.h"
#include "cluster.cuh"
#include "common.cuh"

namespace ssm {

constexpr int kPlanThreads = 1024;
// Blocks of a move: 64 per SM, far more than are resident, so that the hardware levels out their ends.
// 8 copies and 12 forks of 25 MB pages (0.92 GB) took 162 us with 64 and 1000 blocks per SM, 178 with 8;
// 64 of 256 sequences of 2.8 MB pages 61, 66 and 66 us.  Blocks of 128 or 512 threads, 2 or 8 vectors
// per thread and streaming cache hints measured the same or slower.
constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 4;  // vectors in flight per thread
constexpr int kMoveBlocksPerSm = 64;

// The plan's result, in the workspace.
struct CachePlan {
    int count;     // pairs of the lists below
    int in_order;  // the pairs depend on each other: one after another
    int pad[62];
    // int src[n], dst[n], scratch[n] follow
};
static_assert(sizeof(CachePlan) == 256, "lists start 256-byte aligned");

constexpr int kClear = -1, kNone = -2;  // as a source: the page becomes zeros; nothing happens

struct CachePool {
    char* data;
    long long page, slot_stride, layer_stride;
    int layers, width;         // width: bytes of a vector that every page of the pool is aligned to
    unsigned chunks;           // of kMoveThreads * kMoveUnroll vectors in a page
    unsigned units_before;     // (layer, chunk) units of the pools before this one
};

struct CacheMove {
    CachePool pool[SSM_CACHE_MAX_POOLS];
    int n_pools, n_slots;
    unsigned units;      // (pool, layer, chunk) units of a page
    int n;               // pairs; -1: plan->count
    int may_clear;       // a source of kClear makes the page zeros (else it is skipped)
    const CachePlan* plan;  // null: no plan came before
    const int *src, *dst;   // src null: clear
};

// ------------------------------------------------------------------------------------- plans
// Exclusive prefix sum of a flag over the block, and its total.
__device__ __forceinline__ int block_rank(bool flag, int* warp_sums, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned votes = __ballot_sync(0xffffffffu, flag);
    __syncthreads();  // (the sums of the call before have been read)
    if (lane == 0) warp_sums[warp] = __popc(votes);
    __syncthreads();
    int before = 0;
    total = 0;
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        const int s = warp_sums[w];
        before += w < warp ? s : 0;
        total += s;
    }
    return before + __popc(votes & ((1u << lane) - 1));
}

__device__ __forceinline__ bool in_pool(int slot, int n_slots) { return slot >= 0 && slot < n_slots; }

// The plans, by one block.  They read the lists and `used` and leave those as they are; what they find goes to lists
// in global or shared memory.

// Whether the pairs depend on each other: a page is written twice, or both written and read.  `written`: one bit per
// slot, `clash`: one int, both in shared memory.
__device__ __forceinline__ bool plan_copy(const int* src, const int* dst, int n, int n_slots, unsigned* written, int* clash) {
    for (int w = threadIdx.x; w < (n_slots + 31) / 32; w += kPlanThreads) written[w] = 0;
    if (threadIdx.x == 0) *clash = 0;
    __syncthreads();
    for (int j = threadIdx.x; j < n; j += kPlanThreads) {
        const int s = src[j], d = dst[j];
        if (s == d || !in_pool(s, n_slots) || !in_pool(d, n_slots)) continue;
        if (atomicOr(&written[d >> 5], 1u << (d & 31)) & (1u << (d & 31))) *clash = 1;
    }
    __syncthreads();
    for (int j = threadIdx.x; j < n; j += kPlanThreads) {
        const int s = src[j], d = dst[j];
        if (s == d || !in_pool(s, n_slots) || !in_pool(d, n_slots)) continue;
        if (written[s >> 5] & (1u << (s & 31))) *clash = 1;
    }
    __syncthreads();
    return *clash != 0;
}

// child[j]: the j-th accepted request's free slot, or -1; src[j]: its parent, kClear or kNone.  free_list: n entries.
__device__ __forceinline__ void plan_fork(const int* used, const int* parents, int n, int n_slots, int* sums, int* free_list, int* src,
                                          int* child) {
    int free = 0;  // the first n free slots, in ascending order
    for (int base = 0; base < n_slots && free < n; base += kPlanThreads) {
        const int slot = base + threadIdx.x;
        const bool is_free = slot < n_slots && used[slot] == 0;
        int total;
        const int rank = free + block_rank(is_free, sums, total);
        if (is_free && rank < n) free_list[rank] = slot;
        free += total;
    }
    free = min(free, n);
    __syncthreads();
    int taken = 0;
    for (int base = 0; base < n; base += kPlanThreads) {
        const int j = base + threadIdx.x;
        const int parent = j < n ? parents[j] : kNone;
        const bool ok = parent == SSM_CACHE_NEW || (in_pool(parent, n_slots) && used[parent] != 0);
        int total;
        const int rank = taken + block_rank(ok, sums, total);
        if (j < n) {
            const int c = ok && rank < free ? free_list[rank] : -1;
            child[j] = c;
            src[j] = c < 0 ? kNone : parent == SSM_CACHE_NEW ? kClear : parent;
        }
        taken += total;
    }
    __syncthreads();
}

// The pages that move (src to dst, `movers` of them), the number of used slots, and every slot's new place.
__device__ __forceinline__ int plan_compact(const int* used, int n_slots, int* sums, int* src, int* dst, int* to, int& movers) {
    int live = 0;
    for (int base = 0; base < n_slots; base += kPlanThreads) {
        const int slot = base + threadIdx.x;
        int total;
        block_rank(slot < n_slots && used[slot] != 0, sums, total);
        live += total;
    }
    int holes = 0;
    movers = 0;
    for (int base = 0; base < n_slots; base += kPlanThreads) {
        const int slot = base + threadIdx.x;
        const bool is_live = slot < n_slots && used[slot] != 0;
        const bool hole = slot < live && !is_live, mover = slot >= live && is_live;
        int total;
        int rank = holes + block_rank(hole, sums, total);
        if (hole) dst[rank] = slot;
        holes += total;
        rank = movers + block_rank(mover, sums, total);
        if (mover) src[rank] = slot;
        movers += total;
        if (slot < n_slots && !mover) to[slot] = is_live ? slot : -1;
    }
    __syncthreads();
    for (int k = threadIdx.x; k < movers; k += kPlanThreads) to[src[k]] = dst[k];
    __syncthreads();
    return live;
}

// What the calls change besides the pages, by one block once nobody reads it any more.
__device__ __forceinline__ void commit_fork(const int* child, int n, int* used, int* children) {
    for (int j = threadIdx.x; j < n; j += kPlanThreads) {
        children[j] = child[j];
        if (child[j] >= 0) used[child[j]] = 1;
    }
}

__device__ __forceinline__ void commit_compact(const int* to, int live, int n_slots, int* used, int* table, int n_table, int* remap,
                                               int* count) {
    for (int slot = threadIdx.x; slot < n_slots; slot += kPlanThreads) {
        used[slot] = slot < live;
        if (remap) remap[slot] = to[slot];
    }
    for (int k = threadIdx.x; k < n_table; k += kPlanThreads) table[k] = in_pool(table[k], n_slots) ? to[table[k]] : -1;
    if (count && threadIdx.x == 0) *count = live;
}

__global__ void __launch_bounds__(kPlanThreads) cache_plan_copy_kernel(const int* src, const int* dst, int n, int n_slots, CachePlan* plan) {
    extern __shared__ unsigned written[];
    __shared__ int clash;
    pdl_launch_dependents();
    const bool in_order = plan_copy(src, dst, n, n_slots, written, &clash);
    if (threadIdx.x == 0) plan->count = n, plan->in_order = in_order;
}

__global__ void __launch_bounds__(kPlanThreads) cache_plan_fork_kernel(int* used, const int* parents, int* children, int n, int n_slots,
                                                                       CachePlan* plan, int* src, int* dst, int* scratch) {
    __shared__ int sums[kPlanThreads / 32];
    pdl_launch_dependents();
    plan_fork(used, parents, n, n_slots, sums, scratch, src, dst);
    commit_fork(dst, n, used, children);
    if (threadIdx.x == 0) plan->count = n, plan->in_order = 0;
}

__global__ void __launch_bounds__(kPlanThreads) cache_plan_compact_kernel(int* used, int n_slots, int* table, int n_table, int* remap,
                                                                          int* count, CachePlan* plan, int* src, int* dst, int* scratch) {
    __shared__ int sums[kPlanThreads / 32];
    pdl_launch_dependents();
    int movers;
    const int live = plan_compact(used, n_slots, sums, src, dst, scratch, movers);
    commit_compact(scratch, live, n_slots, used, table, n_table, remap, count);
    if (threadIdx.x == 0) plan->count = movers, plan->in_order = 0;
}

__global__ void __launch_bounds__(kMoveThreads) cache_free_kernel(int* used, const int* slots, int n, int n_slots) {
    const int j = blockIdx.x * kMoveThreads + threadIdx.x;
    if (j < n && in_pool(slots[j], n_slots)) used[slots[j]] = 0;
}

// ------------------------------------------------------------------------------------- move
// Vector `first` + k * kMoveThreads of a page, k < kMoveUnroll: all loads before the stores.
template <typename V>
__device__ __forceinline__ void move_chunk(char* to, const char* from, long long first, long long vectors) {
    V v[kMoveUnroll];
#pragma unroll
    for (int k = 0; k < kMoveUnroll; ++k) {
        const long long at = first + k * kMoveThreads;
        v[k] = V{};
        if (from && at < vectors) v[k] = reinterpret_cast<const V*>(from)[at];
    }
#pragma unroll
    for (int k = 0; k < kMoveUnroll; ++k) {
        const long long at = first + k * kMoveThreads;
        if (at < vectors) reinterpret_cast<V*>(to)[at] = v[k];
    }
}

__device__ __forceinline__ void move_unit(const CachePool& pl, unsigned layer, unsigned chunk, int src, int dst, int thread) {
    char* base = pl.data + layer * pl.layer_stride;
    char* to = base + dst * pl.slot_stride;
    const char* from = src >= 0 ? base + src * pl.slot_stride : nullptr;
    const long long first = static_cast<long long>(chunk) * (kMoveThreads * kMoveUnroll) + thread;
    switch (pl.width) {
        case 16: move_chunk<uint4>(to, from, first, pl.page / 16); break;
        case 8: move_chunk<uint2>(to, from, first, pl.page / 8); break;
        case 4: move_chunk<uint32_t>(to, from, first, pl.page / 4); break;
        case 2: move_chunk<uint16_t>(to, from, first, pl.page / 2); break;
        default: move_chunk<uint8_t>(to, from, first, pl.page); break;
    }
}

// Groups of kMoveThreads threads take (pair, pool, layer, chunk) units in turn: group `first`, then `step` further on.
// Pairs that depend on each other are taken by one group per (pool, layer, chunk), where every thread copies its own
// bytes of all pairs in order.  src null: clear.
__device__ __forceinline__ void move_pages(const CacheMove& m, const int* src, const int* dst, int n, bool in_order, long long first,
                                           long long step, int thread) {
    const long long total = static_cast<long long>(m.units) * (in_order ? 1 : n);
    for (long long u = first; u < total; u += step) {
        const int pair = static_cast<int>(u / m.units);
        unsigned rest = static_cast<unsigned>(u % m.units);
        int k = 0;
        while (k + 1 < m.n_pools && rest >= m.pool[k + 1].units_before) ++k;
        rest -= m.pool[k].units_before;
        const unsigned layer = rest / m.pool[k].chunks, chunk = rest % m.pool[k].chunks;
        for (int j = pair; j < (in_order ? n : pair + 1); ++j) {
            const int s = src ? src[j] : kClear, d = dst[j];
            if (s == d || !in_pool(d, m.n_slots) || !(in_pool(s, m.n_slots) || (s == kClear && m.may_clear))) continue;
            move_unit(m.pool[k], layer, chunk, s, d, thread);
        }
    }
}

__global__ void __launch_bounds__(kMoveThreads) cache_move_kernel(const __grid_constant__ CacheMove m) {
    if (m.plan) pdl_wait_primary();
    const int n = m.n >= 0 ? m.n : m.plan->count;
    move_pages(m, m.src, m.dst, n, m.plan && m.plan->in_order, blockIdx.x, gridDim.x, threadIdx.x);
}

// ------------------------------------------------------------------------------------- small calls
// Plan and move in one launch, by one cluster: every block makes the whole plan in its own shared memory; once all
// have (nobody reads the lists and `used` any more) the first block commits it, and all of them move pages.  For
// up to kSmallUnits units of 16 KB: 2 copies and 3 forks of 117 KB pages took 23.5 us of host time in four launches,
// 19 in two.
constexpr int kSmallBlocks = 8;
constexpr int kSmallUnits = 256;
constexpr int kSmallSlots = 2048;
constexpr int kSmallList = 1024;

enum class CacheOp { kCopy, kFork, kCompact };

struct CacheSmall {
    CacheMove m;  // copy: src and dst are the caller's
    int *used, *table, *remap, *count;
    const int* parents;
    int* children;
    int n_table;
};

template <CacheOp OP>
__global__ void __launch_bounds__(kPlanThreads) cache_small_kernel(const __grid_constant__ CacheSmall c) {
    __shared__ int sums[kPlanThreads / 32], clash;
    __shared__ unsigned written[OP == CacheOp::kCopy ? kSmallSlots / 32 : 1];
    __shared__ int src[OP == CacheOp::kCopy ? 1 : kSmallList], dst[OP == CacheOp::kCopy ? 1 : kSmallList];
    __shared__ int more[OP == CacheOp::kFork ? kSmallList : OP == CacheOp::kCompact ? kSmallSlots : 1];
    const int n_slots = c.m.n_slots;
    int n = c.m.n, live = 0;
    bool in_order = false;
    if constexpr (OP == CacheOp::kCopy) in_order = plan_copy(c.m.src, c.m.dst, n, n_slots, written, &clash);
    if constexpr (OP == CacheOp::kFork) plan_fork(c.used, c.parents, n, n_slots, sums, more, src, dst);
    if constexpr (OP == CacheOp::kCompact) live = plan_compact(c.used, n_slots, sums, src, dst, more, n);
    if constexpr (OP != CacheOp::kCopy) {
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        if (cluster_rank() == 0) {
            if constexpr (OP == CacheOp::kFork) commit_fork(dst, n, c.used, c.children);
            if constexpr (OP == CacheOp::kCompact) commit_compact(more, live, n_slots, c.used, c.table, c.n_table, c.remap, c.count);
        }
    }
    constexpr int kGroups = kPlanThreads / kMoveThreads;
    move_pages(c.m, OP == CacheOp::kCopy ? c.m.src : src, OP == CacheOp::kCopy ? c.m.dst : dst, n, in_order,
               cluster_rank() * kGroups + threadIdx.x / kMoveThreads, kSmallBlocks * kGroups, threadIdx.x % kMoveThreads);
}

}  // namespace ssm
