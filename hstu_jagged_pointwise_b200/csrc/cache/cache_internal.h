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

}  // namespace hstu
