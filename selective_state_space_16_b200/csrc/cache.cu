// cache.cu -- the C ABI of the state cache (ssm_cache.h): argument checks and launches.
#include <algorithm>

#include "cache.cuh"
#include "host_common.h"

namespace {

using namespace ssmh;
using ssm::CacheMove;
using ssm::CachePlan;

bool int_aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Whether n_out blocks of n_in pieces of `page` bytes lie apart.
bool apart(long long n_out, long long s_out, long long n_in, long long s_in, long long page) {
    if (n_in > 1 && s_in < page) return false;
    const long long inner = (n_in > 1 ? (n_in - 1) * s_in : 0) + page;
    return n_out <= 1 || s_out >= inner;
}

// Checks the pools and fills the move's description of them.
ssm_status_t describe(const ssm_cache_pool_t* pools, int n_pools, int n_slots, CacheMove* m) {
    if (n_pools < 1 || n_pools > SSM_CACHE_MAX_POOLS || n_slots < 0 || !pools) return SSM_ERR_INVALID_ARG;
    if (n_slots > SSM_CACHE_MAX_SLOTS) return SSM_ERR_UNSUPPORTED;
    *m = CacheMove{};
    m->n_slots = n_slots;
    unsigned long long units = 0;
    for (int k = 0; k < n_pools; ++k) {
        const ssm_cache_pool_t& p = pools[k];
        if (p.layers < 0 || p.page_bytes < 0) return SSM_ERR_INVALID_ARG;
        if (p.layers == 0 || p.page_bytes == 0) continue;
        if (!p.data && n_slots > 0) return SSM_ERR_INVALID_ARG;
        if (!apart(p.layers, p.layer_stride, n_slots, p.slot_stride, p.page_bytes) &&
            !apart(n_slots, p.slot_stride, p.layers, p.layer_stride, p.page_bytes))
            return SSM_ERR_INVALID_ARG;
        ssm::CachePool& o = m->pool[m->n_pools++];
        o.data = static_cast<char*>(p.data);
        o.page = p.page_bytes;
        o.slot_stride = p.slot_stride;
        o.layer_stride = p.layer_stride;
        o.layers = p.layers;
        const unsigned long long bits = reinterpret_cast<uintptr_t>(p.data) | static_cast<unsigned long long>(p.page_bytes) |
                                        (n_slots > 1 ? static_cast<unsigned long long>(p.slot_stride) : 0) |
                                        (p.layers > 1 ? static_cast<unsigned long long>(p.layer_stride) : 0) | 16;
        o.width = static_cast<int>(bits & (~bits + 1));
        const unsigned long long chunk = static_cast<unsigned long long>(o.width) * ssm::kMoveThreads * ssm::kMoveUnroll;
        const unsigned long long chunks = (p.page_bytes + chunk - 1) / chunk;
        o.units_before = static_cast<unsigned>(units);
        units += chunks * p.layers;
        if (units >= (1ull << 31)) return SSM_ERR_UNSUPPORTED;
        o.chunks = static_cast<unsigned>(chunks);
    }
    m->units = static_cast<unsigned>(units);
    return SSM_OK;
}

struct Workspace {
    CachePlan* plan;
    int *src, *dst, *scratch;
};

// Three lists of as many entries as the workspace was sized for.
ssm_status_t lay_out(void* workspace, size_t bytes, int n_slots, int n, Workspace* w) {
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || bytes < ssm_cache_workspace_size(n_slots, n))
        return SSM_ERR_WORKSPACE;
    const size_t list = std::max(n_slots, n);
    w->plan = static_cast<CachePlan*>(workspace);
    w->src = reinterpret_cast<int*>(w->plan + 1);
    w->dst = w->src + list;
    w->scratch = w->dst + list;
    return SSM_OK;
}

// The pages' copies, after a plan (m.plan) or by themselves.  `pairs`: an upper bound of them.
ssm_status_t launch_move(const CacheMove& m, long long pairs, int sm_count, cudaStream_t s) {
    const long long total = m.units * pairs;
    if (total == 0) return SSM_OK;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(std::min<long long>(total, static_cast<long long>(ssm::kMoveBlocksPerSm) * sm_count)));
    cfg.blockDim = dim3(ssm::kMoveThreads);
    cfg.stream = s;
    cudaLaunchAttribute pdl{};
    pdl.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &pdl;
    cfg.numAttrs = m.plan ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, ssm::cache_move_kernel, m) == cudaSuccess ? launch_status() : SSM_ERR_LAUNCH;
}

bool is_small(const CacheMove& m, long long pairs, int n_list) {
    return m.units * pairs <= ssm::kSmallUnits && m.n_slots <= ssm::kSmallSlots && n_list <= ssm::kSmallList;
}

template <ssm::CacheOp OP>
ssm_status_t launch_small(const ssm::CacheSmall& c, cudaStream_t s) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ssm::kSmallBlocks);
    cfg.blockDim = dim3(ssm::kPlanThreads);
    cfg.stream = s;
    cudaLaunchAttribute cluster{};
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim.x = ssm::kSmallBlocks;
    cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
    cfg.attrs = &cluster;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, ssm::cache_small_kernel<OP>, c) == cudaSuccess ? launch_status() : SSM_ERR_LAUNCH;
}

}  // namespace

extern "C" {

size_t ssm_cache_workspace_size(int n_slots, int n) {
    if (n_slots < 0 || n < 0 || n_slots > SSM_CACHE_MAX_SLOTS) return 0;
    return round_up(sizeof(CachePlan) + 3 * static_cast<size_t>(std::max(n_slots, n)) * sizeof(int), 256);
}

ssm_status_t ssm_cache_copy(const ssm_cache_pool_t* pools, int n_pools, int n_slots, const int32_t* src, const int32_t* dst,
                            int n, void* workspace, size_t workspace_bytes, ssm_stream_t stream) {
    CacheMove m;
    Workspace w;
    ssm_status_t st = describe(pools, n_pools, n_slots, &m);
    if (st != SSM_OK) return st;
    if (n < 0 || (n > 0 && (!src || !dst)) || !int_aligned(src) || !int_aligned(dst)) return SSM_ERR_INVALID_ARG;
    if (n == 0 || n_slots == 0) return SSM_OK;
    st = lay_out(workspace, workspace_bytes, n_slots, n, &w);
    if (st != SSM_OK) return st;
    int sms = 0;
    st = check_device(&sms);
    if (st != SSM_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    m.n = n;
    m.src = src;
    m.dst = dst;
    if (is_small(m, n, n)) return launch_small<ssm::CacheOp::kCopy>({m}, s);
    const int bitmap = (n_slots + 31) / 32 * 4;
    if (!ensure_smem_attr(reinterpret_cast<const void*>(ssm::cache_plan_copy_kernel), bitmap)) return SSM_ERR_LAUNCH;
    ssm::cache_plan_copy_kernel<<<1, ssm::kPlanThreads, bitmap, s>>>(src, dst, n, n_slots, w.plan);
    st = launch_status();
    if (st != SSM_OK) return st;
    m.plan = w.plan;
    return launch_move(m, n, sms, s);
}

ssm_status_t ssm_cache_fork(const ssm_cache_pool_t* pools, int n_pools, int n_slots, int32_t* used, const int32_t* parents,
                            int32_t* children, int n, void* workspace, size_t workspace_bytes, ssm_stream_t stream) {
    CacheMove m;
    Workspace w;
    ssm_status_t st = describe(pools, n_pools, n_slots, &m);
    if (st != SSM_OK) return st;
    if (n < 0 || (n > 0 && (!parents || !children || (n_slots > 0 && !used)))) return SSM_ERR_INVALID_ARG;
    if (!int_aligned(used) || !int_aligned(parents) || !int_aligned(children)) return SSM_ERR_INVALID_ARG;
    if (n > 0 && parents < children + n && children < parents + n) return SSM_ERR_INVALID_ARG;
    if (n == 0) return SSM_OK;
    st = lay_out(workspace, workspace_bytes, n_slots, n, &w);
    if (st != SSM_OK) return st;
    int sms = 0;
    st = check_device(&sms);
    if (st != SSM_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    m.n = n;
    m.may_clear = 1;
    if (is_small(m, n, n)) return launch_small<ssm::CacheOp::kFork>({m, used, nullptr, nullptr, nullptr, parents, children, 0}, s);
    ssm::cache_plan_fork_kernel<<<1, ssm::kPlanThreads, 0, s>>>(used, parents, children, n, n_slots, w.plan, w.src, w.dst, w.scratch);
    st = launch_status();
    if (st != SSM_OK) return st;
    m.plan = w.plan;
    m.src = w.src;
    m.dst = w.dst;
    return launch_move(m, n, sms, s);
}

ssm_status_t ssm_cache_free(const ssm_cache_pool_t* pools, int n_pools, int n_slots, int32_t* used, const int32_t* slots, int n,
                            int zero_pages, ssm_stream_t stream) {
    CacheMove m;
    ssm_status_t st = describe(pools, n_pools, n_slots, &m);
    if (st != SSM_OK) return st;
    if (n < 0 || (n > 0 && (!slots || (n_slots > 0 && !used))) || !int_aligned(used) || !int_aligned(slots)) return SSM_ERR_INVALID_ARG;
    if (n == 0 || n_slots == 0) return SSM_OK;
    int sms = 0;
    st = check_device(&sms);
    if (st != SSM_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    ssm::cache_free_kernel<<<(n + ssm::kMoveThreads - 1) / ssm::kMoveThreads, ssm::kMoveThreads, 0, s>>>(used, slots, n, n_slots);
    st = launch_status();
    if (st != SSM_OK || !zero_pages) return st;
    m.n = n;
    m.may_clear = 1;
    m.dst = slots;
    return launch_move(m, n, sms, s);
}

ssm_status_t ssm_cache_compact(const ssm_cache_pool_t* pools, int n_pools, int n_slots, int32_t* used, int32_t* table,
                               int n_table, int32_t* remap, int32_t* count, void* workspace, size_t workspace_bytes,
                               ssm_stream_t stream) {
    CacheMove m;
    Workspace w;
    ssm_status_t st = describe(pools, n_pools, n_slots, &m);
    if (st != SSM_OK) return st;
    if (n_table < 0 || (n_slots > 0 && !used)) return SSM_ERR_INVALID_ARG;
    for (const void* q : {used, table, remap, count})
        if (!int_aligned(q)) return SSM_ERR_INVALID_ARG;
    if (!table) n_table = 0;
    st = lay_out(workspace, workspace_bytes, n_slots, 0, &w);
    if (st != SSM_OK) return st;
    int sms = 0;
    st = check_device(&sms);
    if (st != SSM_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (is_small(m, n_slots / 2, n_slots / 2))
        return launch_small<ssm::CacheOp::kCompact>({m, used, table, remap, count, nullptr, nullptr, n_table}, s);
    ssm::cache_plan_compact_kernel<<<1, ssm::kPlanThreads, 0, s>>>(used, n_slots, table, n_table, remap, count, w.plan, w.src, w.dst,
                                                                   w.scratch);
    st = launch_status();
    if (st != SSM_OK) return st;
    m.n = -1;
    m.plan = w.plan;
    m.src = w.src;
    m.dst = w.dst;
    return launch_move(m, n_slots / 2, sms, s);  // a page moves into a hole: at most half of them
}

}  // extern "C"
