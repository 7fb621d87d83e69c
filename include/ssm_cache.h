/*
 * ssm_cache.h -- C ABI of the state cache: copying, forking, compacting and freeing its pages.
 *
 * A server keeps the recurrent states of its sequences in pools of slots: the scan states and the
 * conv inputs that the decode entry points of ssm_scan.h and ssm_gated.h read and write, of all
 * layers.  A PAGE is what one sequence owns: one slot in every layer of every pool.  Decode takes
 * dense batch rows, so the live pages belong at the front: compact() puts them there.
 *
 * Conventions: those of ssm_scan.h (device pointers owned by the caller, no device memory
 * allocated, calls asynchronous on `stream`, status codes).  Lists of slots, `used` and `table` are
 * int32 on the device; they are read when the call runs, so nothing here waits for the host
 * and every call can be captured into a CUDA graph.  Entries outside 0 .. n_slots-1 touch nothing.
 *   used    (n_slots): nonzero where the slot holds a sequence.
 */
#ifndef SSM_CACHE_H
#define SSM_CACHE_H

#include "ssm_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

/* One pool: slot s of layer l is the page_bytes bytes at data + l * layer_stride + s * slot_stride. */
typedef struct {
    void* data;
    int64_t page_bytes, slot_stride, layer_stride; /* bytes; slots and layers must not overlap */
    int32_t layers;
} ssm_cache_pool_t;

#define SSM_CACHE_MAX_POOLS 8
#define SSM_CACHE_MAX_SLOTS (1 << 20)
#define SSM_CACHE_NEW (-1) /* as a parent: the page of a new sequence, all zeros */

/*
 * Bytes of device workspace of the calls below that take one, for lists of up to n entries (a
 * multiple of 256; 0 for invalid sizes).  256-byte aligned, not initialised, not to be used by two
 * calls that can overlap on the GPU.
 */
size_t ssm_cache_workspace_size(int n_slots, int n);

/*
 * Copy page src[j] to page dst[j] for j = 0 .. n-1, as if one after another: a page that an earlier pair
 * wrote is copied as written, and of two copies to one page the later one stays.  (Lists in which
 * no page is written twice, or both written and read, run in parallel.)
 */
ssm_status_t ssm_cache_copy(const ssm_cache_pool_t* pools, int n_pools, int n_slots, const int32_t* src, const int32_t* dst,
                            int n, void* workspace, size_t workspace_bytes, ssm_stream_t stream);

/*
 * Fork n sequences: children[j] receives the lowest slot that is still free, marked used, and its
 * page a copy of page parents[j] (a used slot before the call; several forks of one parent are
 * allowed) or zeros (SSM_CACHE_NEW).  children[j] = -1, and nothing is written, where the parent is
 * neither, or no slot is left.  `children` may not be `parents`.
 */
ssm_status_t ssm_cache_fork(const ssm_cache_pool_t* pools, int n_pools, int n_slots, int32_t* used, const int32_t* parents,
                            int32_t* children, int n, void* workspace, size_t workspace_bytes, ssm_stream_t stream);

/*
 * Free the listed slots: used = 0, and with zero_pages their pages are zeroed.  A slot may be listed
 * more than once, or be free already.
 */
ssm_status_t ssm_cache_free(const ssm_cache_pool_t* pools, int n_pools, int n_slots, int32_t* used, const int32_t* slots, int n,
                            int zero_pages, ssm_stream_t stream);

/*
 * Move the used pages to the slots 0 .. count-1.  Only pages outside that range move, in ascending
 * order into its free slots in ascending order; what their old slots hold stays.  `used` becomes 1
 * for the first count slots and 0 for the rest.
 *   table   NULL, or n_table slots that follow their pages (a sequence's entry of a batch);
 *           entries that name no used slot become -1.
 *   remap   NULL, or (n_slots): receives the new slot of every used slot, -1 for the others.
 *   count   NULL, or one int32: receives the number of used slots.
 * workspace: for n_slots entries.
 */
ssm_status_t ssm_cache_compact(const ssm_cache_pool_t* pools, int n_pools, int n_slots, int32_t* used, int32_t* table,
                               int n_table, int32_t* remap, int32_t* count, void* workspace, size_t workspace_bytes,
                               ssm_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SSM_CACHE_H */
