// cache_internal.h -- shared declarations of libhstu_cache_b200 (not part of the C ABI).
#pragma once
#include "../../../include/hstu_cache.h"
#include "../host_util.h"
#include "../internal.h"

namespace hstu {

constexpr int kStatusFull = 4;       // the pool had too few free pages
constexpr int kTreeMaxNodes = 8192;  // largest tree (its parents lie in shared memory)
constexpr int kPlanThreads = 1024;

// Host checks of a cache description: HSTU_OK, or what to return.
inline int check_cache(const hstu_page_cache* c) {
    if (!c || c->n_pages < 0 || c->n_slots < 0 || c->max_pages < 1 || c->row_elems < 1) return HSTU_ERR_INVALID_ARG;
    if (c->dtype != HSTU_BF16 && c->dtype != HSTU_F32) return HSTU_ERR_INVALID_ARG;
    if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128) return HSTU_ERR_UNSUPPORTED;
    const long long row_bytes = (long long)c->row_elems * (c->dtype == HSTU_F32 ? 4 : 2);
    if (row_bytes % 16 != 0 || row_bytes / 16 > (1 << 20)) return HSTU_ERR_UNSUPPORTED;
    // row numbers of the pool and of a slot are 32-bit
    if ((long long)c->n_pages * c->page_size > 0x7fffffffLL || (long long)c->max_pages * c->page_size > kMaxSeqLen)
        return HSTU_ERR_UNSUPPORTED;
    if ((c->n_pages > 0 && (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->ts, 8) || !aligned(c->ref, 4))) ||
        (c->n_slots > 0 && (!aligned(c->page_table, 4) || !aligned(c->lens, 4))))
        return HSTU_ERR_INVALID_ARG;
    return HSTU_OK;
}

DebugWait cache_debug_wait();

#ifdef __CUDACC__
// The launch before this one has completed, and its writes are visible.
__device__ __forceinline__ void wait_for_prior_launch() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The next launch may start: it waits by wait_for_prior_launch before it reads our results.
__device__ __forceinline__ void allow_next_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Launch that may start while the one before it in the stream ends.
template <typename... Args>
cudaError_t launch_early(void (*kernel)(Args...), int grid, int block, uint32_t smem, cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}
#endif

}  // namespace hstu
