/*
 * hstu_cache.h -- C ABI of libhstu_cache_b200: a paged cache of user histories for
 * HSTU serving, and the scorer that reads it.  B200 (sm_100a).
 *
 * The cache generalises the contiguous one of hstu_mfalcon_cache_history /
 * hstu_mfalcon_score (HSTU blog, sections 4.2-4.3: a user's history keys and values
 * are computed once and reused by later candidates): a history lies in pages of a
 * common pool, so that it can grow by a few events, be shared by several candidates'
 * branches, be cut down, and be dropped without moving any other.  The scorer
 * generalises the M-FALCON candidate mask: candidates form trees (a candidate sees
 * its ancestors besides the history and itself), and the history may be seen through
 * the same sliding window with sinks as HSTU_MASK_WINDOW.
 *
 * Conventions are those of hstu.h: device pointers owned by the caller, host structs
 * read before return, no device allocation, all work asynchronous on `stream`,
 * argument errors returned before any launch.  What only the device can see is
 * recorded in the status word of `workspace` (read and cleared by
 * hstu_cache_check_device_error); the call then changes nothing, unless said otherwise.
 * Workspaces are 256-byte aligned; the first 256 bytes are zeroed once before the first
 * use, the rest may hold anything.  One workspace, large enough for each, may serve several
 * caches, and both the page operators and the scorer (but not the calls of hstu.h as well),
 * one stream at a time: calls that may overlap take one each, and calls that change one
 * cache are ordered by the caller.
 */
#ifndef HSTU_CACHE_B200_H
#define HSTU_CACHE_B200_H

#include "hstu.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The pool and its tables.  Slot s holds lens[s] rows; row r lies in row r % page_size
 * of page page_table[s][r / page_size].  ref[p] is the number of slots that hold page
 * p, 0 when it is free.  A new cache has lens = 0, ref = 0 and page_table = -1
 * everywhere.  Entries past a slot's pages are -1.  Rows of a page past its slot's
 * length hold anything, NaN included. */
typedef struct {
    int32_t n_pages;      /* pages of the pool */
    int32_t page_size;    /* rows of a page: 16, 32, 64 or 128 */
    int32_t n_slots;      /* histories the cache can hold */
    int32_t max_pages;    /* pages one slot can hold (columns of page_table) */
    int32_t row_elems;    /* elements of a key or value row (H*d); whole 16-byte vectors */
    int32_t dtype;        /* hstu_dtype of k and v */
    void* k;              /* [n_pages, page_size, row_elems] */
    void* v;              /* [n_pages, page_size, row_elems] */
    int64_t* ts;          /* [n_pages, page_size] event times */
    int32_t* page_table;  /* [n_slots, max_pages] */
    int32_t* lens;        /* [n_slots] */
    int32_t* ref;         /* [n_pages] */
} hstu_page_cache;

/* Bytes of workspace of the page operators on this cache; 0 when its description is
 * invalid. */
HSTU_API size_t hstu_cache_workspace_bytes(const hstu_page_cache* cache);

/* The page operators take n_req requests, each for a slot of its own: a slot named
 * twice, or outside [0, n_slots), sets HSTU_ERR_DEVICE_BOUNDS.  New pages are the
 * lowest-numbered free ones, in the order of the requests; when the pool has too few,
 * the status is HSTU_ERR_CACHE_FULL.  Either way nothing changes.  The search starts at
 * page 0, so append and compact take longer the more held pages lie below the first free
 * ones (about 0.23 us for each thousand).  Caches of either type are kept; the scorer
 * reads HSTU_BF16 ones. */

/* Appends rows row_offsets[i] .. row_offsets[i+1]-1 to slot slots[i].  Row r comes from
 * row src_rows[r] (r itself when src_rows is NULL) of k, v [n_src, row_elems] and
 * ts [n_src].  A shared last page that has room is copied first, and the copy written
 * (its other holders keep the page).  Whether it is shared is judged before the call: where
 * all holders of a page append in one call, each gets a copy and the page is released, so
 * that the pool needs one free page more than the rows do.
 * row_offsets int32 [n_req+1], from 0 to T, non-decreasing.  A slot that would pass
 * max_pages * page_size rows, or bad offsets, set HSTU_ERR_DEVICE_BOUNDS.  A source row
 * outside [0, n_src) sets it too, but the other rows are appended and that one is zero. */
HSTU_API int hstu_cache_append(const hstu_page_cache* cache, int32_t n_req, const int32_t* slots,
                  const int32_t* row_offsets, int32_t T, const int32_t* src_rows, int32_t n_src,
                  const void* k, const void* v, const int64_t* ts,
                  void* workspace, size_t workspace_bytes, void* stream);

/* Makes slot dst_slots[i] hold the rows of src_slots[i] without copying them: the
 * pages are shared.  Sources may repeat; a destination must be empty and no source. */
HSTU_API int hstu_cache_fork(const hstu_page_cache* cache, int32_t n_req, const int32_t* src_slots,
                  const int32_t* dst_slots, void* workspace, size_t workspace_bytes, void* stream);

/* Replaces the content of slot slots[i] by its rows keep_rows[keep_offsets[i]] ..
 * keep_rows[keep_offsets[i+1]-1], in that order, copied into fresh pages; the old
 * pages are released (the fresh ones must be free before that).  keep_offsets int32
 * [n_req+1], from 0 to K, non-decreasing.  A row outside the slot sets
 * HSTU_ERR_DEVICE_BOUNDS, but the others are kept and that one is zero. */
HSTU_API int hstu_cache_compact(const hstu_page_cache* cache, int32_t n_req, const int32_t* slots,
                  const int32_t* keep_offsets, int32_t K, const int32_t* keep_rows,
                  void* workspace, size_t workspace_bytes, void* stream);

/* Empties the slots and releases their pages. */
HSTU_API int hstu_cache_free(const hstu_page_cache* cache, int32_t n_req, const int32_t* slots,
                  void* workspace, size_t workspace_bytes, void* stream);

/* Trees of candidates over cached histories. */
typedef struct {
    int32_t B;            /* trees */
    int32_t T;            /* nodes of all trees = node_offsets[B] */
    int32_t H, d;         /* heads and head width (64 or 128); H*d = the cache's row_elems */
    int32_t n_pos, n_tbuckets;
    int32_t max_nodes;    /* upper bound on every tree's nodes (device-checked), <= 8192 */
    float alpha, ln_eps;
} hstu_tree_dims;

/* Bytes of workspace of hstu_tree_score; 0 when the arguments are invalid. */
HSTU_API size_t hstu_tree_workspace_bytes(const hstu_tree_dims* dims, const hstu_page_cache* cache);

/* Scores tree b over the history of slot slots[b], of n rows.  parent[t] (int32 [T]) is
 * the index, within the tree, of node t's parent, smaller than its own, or -1.  With
 * depth(c) ancestors, node c sits at position n + depth(c); history row j at j.  With
 * the rule  see(i, j): i - j < window[b] or j < n_sink[b]  on positions (every pair,
 * when both arrays are NULL),
 *   Y_c = (1/alpha) [ sum over history rows j with see(n + depth(c), j) of SiLU(z_cj) v_j
 *                     + the same over c and its ancestors ]
 *   z_cj = q_c . k_j + rab_pos[pidx] + rab_time[tb],  O_pre_c = (LayerNorm(Y_c) gamma + beta) (.) u_c
 * with pidx and tb as in hstu.h: the last row of a causal (or window) layer over the
 * history and c's path.  One-node trees are M-FALCON's candidates; a single node is
 * the decoding step of a user's next event.  Trees are meant to be shallow: each node walks
 * its ancestors one after another (a chain of 512 nodes takes 0.26 ms, one of 8192 12 ms).
 * In:  node_q, node_k, node_v, node_u [T, H*d] bf16 (the cache's dtype must be
 *      HSTU_BF16), node_ts int64 [T], node_offsets int32 [B+1], slots int32 [B] (a slot
 *      may serve several trees), n_sink and window int32 [B], both or neither.
 * Out: y, o_pre [T, H*d] bf16.  Deterministic.  y is not read back: o_pre comes from
 *      the unrounded Y.
 * HSTU_ERR_DEVICE_BOUNDS: a bad slot, offset, parent or negative rule, a tree past
 * max_nodes, or a page that is seen but not in the pool.  Rows past a history's end and
 * rows that no node may see are never used, whatever they hold; what one node of a tree
 * sees must be finite for the others. */
HSTU_API int hstu_tree_score(const hstu_tree_dims* dims, const hstu_page_cache* cache, const int32_t* slots,
                  const int32_t* node_offsets, const int32_t* parent, const int64_t* node_ts,
                  const void* node_q, const void* node_k, const void* node_v, const void* node_u,
                  const int32_t* n_sink, const int32_t* window, const float* rab_pos, const float* rab_time,
                  const float* ln_gamma, const float* ln_beta, void* y, void* o_pre,
                  void* workspace, size_t workspace_bytes, void* stream);

/* Synchronizes `stream`, reads and clears the status word of a workspace. */
HSTU_API int hstu_cache_check_device_error(void* workspace, void* stream);

/* hstu_debug_set_wait_fault for hstu_tree_score (a test hook). */
HSTU_API int hstu_cache_debug_set_wait_fault(int64_t wait_limit_cycles, int32_t withhold_first_load);

#ifdef __cplusplus
}
#endif

#endif /* HSTU_CACHE_B200_H */
