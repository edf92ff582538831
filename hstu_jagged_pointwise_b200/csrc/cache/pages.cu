// pages.cu -- page operators of the paged history cache: append, fork, compact, free.
//
// Every request is checked before anything changes.  append and compact plan in one CTA
// (each step needs the one before it for all requests) and copy with a grid of warps;
// fork and free, whose work is one table entry and one reference count a page, take a
// cluster of eight CTAs, which agree through distributed shared memory: 256 forks of 36
// pages take one SM 10 us, since its requests to L2 are that many separate sectors.
//   append   rows n .. n + c - 1 of a slot that held n; pages needed =
//            ceil((n + c) / ps) - ceil(n / ps), and one more where the last page has
//            room but is shared (copied, then written: copy-on-write)
//   compact  c rows of a slot into ceil(c / ps) fresh pages; the old ones are released
//   fork     the table row and length of another slot; ref + 1 on each page
//   free     ref - 1 on each page of a slot
// The k-th page needed (requests in order) is the k-th free page (ref == 0) of the
// pool, so the result does not depend on timing.  The reference counts change by
// integer atomics only.
#include <cooperative_groups.h>

#include <algorithm>

#include "cache_internal.h"

namespace hstu {
namespace {

constexpr int kCopyThreads = 256;
constexpr int kRowsPerWarp = 4;     // rows whose loads a warp keeps in flight together
constexpr unsigned kAll = 0xffffffffu;

// Workspace behind the control block.
struct PageWs {
    size_t claim, base, old_len, cow, free_list, old_table, total;
};

PageWs page_ws(const hstu_page_cache& c) {
    PageWs w;
    size_t off = sizeof(Control);
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = align_up(off + bytes, 256);
        return at;
    };
    w.claim = take((size_t)c.n_slots * 4);       // 1 where a request names the slot, of the slots that this call looks at
    w.base = take((size_t)c.n_slots * 4);        // request: its first place in the free list
    w.old_len = take((size_t)c.n_slots * 4);     // request: rows the slot held
    w.cow = take((size_t)c.n_slots * 4);         // request: the shared page to copy, or -1
    w.free_list = take((size_t)c.n_pages * 4);
    w.old_table = take((size_t)c.n_slots * c.max_pages * 4);   // compact: the table rows before
    w.total = off;
    return w;
}

struct PlanParams {
    hstu_page_cache c;
    Control* ctrl;
    int* claim;
    int* base;
    int* old_len;
    int* cow;
    int* free_list;
    int* old_table;
    int n_req;
    const int32_t* slots;      // append, compact, free: the slots; fork: the destinations
    const int32_t* src_slots;  // fork
    const int32_t* off;        // append: row_offsets; compact: keep_offsets
    int T;
};

// Sum of v over the threads before this one; *total gets the sum over all.
__device__ __forceinline__ int block_exclusive(int v, int* s_warp, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kAll, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        const int w = s_warp[lane];
        int wi = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kAll, wi, o);
            if (lane >= o) wi += y;
        }
        s_warp[lane] = wi - w;
        if (lane == 31) *total = wi;
    }
    __syncthreads();
    const int r = s_warp[warp] + inc - v;
    __syncthreads();
    return r;
}

__device__ __forceinline__ int pages_of(int rows, int ps) { return (rows + ps - 1) / ps; }

// Whatever lies in claim (the workspace may have served another cache, or the scorer), a call first
// clears the entries that it will look at.
__device__ __forceinline__ void clear_claim(const PlanParams& p, int s) {
    if (s >= 0 && s < p.c.n_slots) p.claim[s] = 0;
}

// Names a slot; false when it is out of range, named before, or of a length that the cache cannot hold.
__device__ __forceinline__ bool claim_slot(const PlanParams& p, int s, int* len) {
    *len = 0;
    if (s < 0 || s >= p.c.n_slots) return false;
    const int n = p.c.lens[s];
    const int before = atomicExch(&p.claim[s], 1);
    if (before != 0 || n < 0 || n > p.c.max_pages * p.c.page_size) return false;
    *len = n;
    return true;
}

constexpr int kCluster = 8;

// Whether any CTA of the cluster has seen something bad; `round` counts the calls of a kernel.  Each
// CTA writes to the others' shared memory, so every CTA must have started (a barrier of the cluster
// comes before the first call); after the barrier here no CTA writes any more, and any may leave.
__device__ bool cluster_any(int bad, int round) {
    __shared__ int s_bad[2][kCluster];
    namespace cg = cooperative_groups;
    cg::cluster_group cl = cg::this_cluster();
    bad = __syncthreads_or(bad);
    if (threadIdx.x < kCluster) *cl.map_shared_rank(&s_bad[round][cl.block_rank()], threadIdx.x) = bad;
    cl.sync();
    int any = 0;
    for (int i = 0; i < kCluster; i++) any |= s_bad[round][i];
    return any != 0;
}

__device__ void refuse(const PlanParams& p, int bit) {
    if (threadIdx.x == 0) {
        atomicOr(&p.ctrl->status, bit);
        p.ctrl->valid = 0;
    }
}

// The first `want` free pages, lowest first, into free_list; false when there are fewer.  From page
// 0, 4096 pages a round, so a pool whose low pages are held costs the walk through them: append + free
// of three rows 12.5 us where the first page is free, 33 behind 90,000 held pages, 221 behind 900,000.
__device__ bool find_free(const PlanParams& p, int want, int* s_warp, int* s_total) {
    int found = 0;
    for (int p0 = 0; p0 < p.c.n_pages && found < want; p0 += 4 * kPlanThreads) {
        const int at = p0 + 4 * (int)threadIdx.x;
        int r[4], mine = 0;
#pragma unroll
        for (int e = 0; e < 4; e++) {
            r[e] = at + e < p.c.n_pages ? p.c.ref[at + e] : 1;
            mine += r[e] == 0;
        }
        int k = found + block_exclusive(mine, s_warp, s_total);
#pragma unroll
        for (int e = 0; e < 4; e++)
            if (r[e] == 0) {
                if (k < want) p.free_list[k] = at + e;
                k++;
            }
        found += *s_total;
        __syncthreads();
    }
    return found >= want;
}

// append (COMPACT = false) and compact: check, choose pages, write the tables.
template <bool COMPACT>
__global__ void __launch_bounds__(kPlanThreads) plan_rows_kernel(PlanParams p) {
    __shared__ int s_warp[32];
    __shared__ int s_total;
    allow_next_launch();
    const int tid = threadIdx.x, ps = p.c.page_size;
    for (int q = tid; q < p.n_req; q += kPlanThreads) clear_claim(p, p.slots[q]);
    __syncthreads();
    int bad = 0;
    if (tid == 0 && (p.off[0] != 0 || p.off[p.n_req] != p.T)) bad = 1;
    // pages each request needs, and its place in the list of free pages
    int carry = 0;
    for (int q0 = 0; q0 < p.n_req; q0 += kPlanThreads) {
        const int q = q0 + tid;
        int need = 0;
        if (q < p.n_req) {
            const int s = p.slots[q], cnt = p.off[q + 1] - p.off[q];
            int n, cow = -1;
            const bool ok = claim_slot(p, s, &n);
            const long long n_new = COMPACT ? cnt : (long long)n + cnt;
            if (!ok || cnt < 0 || cnt > p.T || n_new > (long long)p.c.max_pages * ps) {
                bad = 1;
            } else if (COMPACT) {
                need = pages_of(cnt, ps);
            } else {
                need = pages_of((int)n_new, ps) - pages_of(n, ps);
                if (cnt > 0 && n % ps != 0) {
                    const int last = p.c.page_table[(size_t)s * p.c.max_pages + n / ps];
                    if (last < 0 || last >= p.c.n_pages) bad = 1;
                    else if (p.c.ref[last] > 1) {
                        cow = last;
                        need++;
                    }
                }
            }
            p.old_len[q] = n;
            p.cow[q] = cow;
        }
        const int ex = block_exclusive(need, s_warp, &s_total);
        if (q < p.n_req) p.base[q] = carry + ex;
        carry += s_total;
        __syncthreads();
    }
    if (__syncthreads_or(bad)) return refuse(p, kStatusBounds);
    if (!find_free(p, carry, s_warp, &s_total)) return refuse(p, kStatusFull);
    // nothing was changed so far; a warp takes four requests at a time from here, so that their
    // lookups are in flight together
    const int warp = tid >> 5, lane = tid & 31;
    for (int q0 = 4 * warp; q0 < p.n_req; q0 += 4 * (kPlanThreads / 32)) {
        int s[4], n[4], cnt[4], base[4], cow[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int q = min(q0 + i, p.n_req - 1);
            s[i] = p.slots[q];
            n[i] = p.old_len[q];
            cnt[i] = q0 + i < p.n_req ? p.off[q + 1] - p.off[q] : 0;
            base[i] = p.base[q];
            cow[i] = p.cow[q];
        }
        if (COMPACT) {
            const int np = p.c.max_pages;
            for (int e = lane; e < np; e += 32) {
                int old[4], fresh[4];
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    old[i] = e < pages_of(n[i], ps) ? p.c.page_table[(size_t)s[i] * np + e] : -1;
                    fresh[i] = e < pages_of(cnt[i], ps) ? p.free_list[base[i] + e] : -1;
                }
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    if (q0 + i >= p.n_req || (e >= pages_of(n[i], ps) && fresh[i] < 0)) continue;
                    p.old_table[(size_t)(q0 + i) * np + e] = old[i];
                    if (old[i] >= 0 && old[i] < p.c.n_pages) atomicSub(&p.c.ref[old[i]], 1);
                    if (fresh[i] >= 0) p.c.ref[fresh[i]] = 1;
                    p.c.page_table[(size_t)s[i] * np + e] = fresh[i];
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const int first = pages_of(n[i], ps) - (cow[i] >= 0 ? 1 : 0), last = pages_of(n[i] + cnt[i], ps);
                if (q0 + i >= p.n_req) continue;
                for (int e = first + lane; e < last; e += 32) {
                    const int pg = p.free_list[base[i] + e - first];
                    p.c.page_table[(size_t)s[i] * p.c.max_pages + e] = pg;
                    p.c.ref[pg] = 1;
                }
                if (lane == 0 && cow[i] >= 0) atomicSub(&p.c.ref[cow[i]], 1);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; i++)
            if (lane == i && q0 + i < p.n_req) p.c.lens[s[i]] = COMPACT ? cnt[i] : n[i] + cnt[i];
    }
    if (tid == 0) p.ctrl->valid = 1;
}

// Threads of the cluster, and this one's number among them.
constexpr int kClusterThreads = kCluster * kPlanThreads;
__device__ __forceinline__ int cluster_thread() { return blockIdx.x * kPlanThreads + threadIdx.x; }

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kPlanThreads) fork_kernel(PlanParams p) {
    for (int q = cluster_thread(); q < p.n_req; q += kClusterThreads) {
        clear_claim(p, p.slots[q]);
        clear_claim(p, p.src_slots[q]);
    }
    cooperative_groups::this_cluster().sync();        // every CTA has started, and the claims are clear
    int bad = 0, n;
    for (int q = cluster_thread(); q < p.n_req; q += kClusterThreads)
        if (!claim_slot(p, p.slots[q], &n) || n != 0) bad = 1;
    bool any = cluster_any(bad, 0);                   // all slots are named
    bad = 0;
    for (int q = cluster_thread(); q < p.n_req; q += kClusterThreads) {
        const int a = p.src_slots[q];
        if (a < 0 || a >= p.c.n_slots || p.claim[a] != 0) {
            bad = 1;                                  // a source is no destination
        } else {
            n = p.c.lens[a];
            if (n < 0 || n > p.c.max_pages * p.c.page_size) bad = 1;
        }
    }
    any = cluster_any(bad, 1) || any;
    if (any) {
        if (blockIdx.x == 0) refuse(p, kStatusBounds);
        return;
    }
    // a warp takes four requests at a time, so that their lookups are in flight together
    const int warp = cluster_thread() >> 5, lane = threadIdx.x & 31, np = p.c.max_pages;
    for (int q0 = 4 * warp; q0 < p.n_req; q0 += 4 * (kClusterThreads / 32)) {
        int a[4], b[4], n[4], most = 0;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int q = min(q0 + i, p.n_req - 1);
            a[i] = p.src_slots[q];
            b[i] = p.slots[q];
        }
#pragma unroll
        for (int i = 0; i < 4; i++) {
            n[i] = q0 + i < p.n_req ? p.c.lens[a[i]] : 0;
            most = max(most, pages_of(n[i], p.c.page_size));
        }
        for (int e = lane; e < most; e += 32) {
            int pg[4];
#pragma unroll
            for (int i = 0; i < 4; i++) pg[i] = e < pages_of(n[i], p.c.page_size) ? p.c.page_table[(size_t)a[i] * np + e] : -1;
#pragma unroll
            for (int i = 0; i < 4; i++)
                if (e < pages_of(n[i], p.c.page_size)) {
                    if (pg[i] >= 0 && pg[i] < p.c.n_pages) atomicAdd(&p.c.ref[pg[i]], 1);
                    p.c.page_table[(size_t)b[i] * np + e] = pg[i];
                }
        }
#pragma unroll
        for (int i = 0; i < 4; i++)
            if (lane == i && q0 + i < p.n_req) p.c.lens[b[i]] = n[i];
    }
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kPlanThreads) free_kernel(PlanParams p) {
    for (int q = cluster_thread(); q < p.n_req; q += kClusterThreads) clear_claim(p, p.slots[q]);
    cooperative_groups::this_cluster().sync();        // every CTA has started, and the claims are clear
    int bad = 0, n;
    for (int q = cluster_thread(); q < p.n_req; q += kClusterThreads)
        if (!claim_slot(p, p.slots[q], &n)) bad = 1;
    const bool any = cluster_any(bad, 0);
    if (any) {
        if (blockIdx.x == 0) refuse(p, kStatusBounds);
        return;
    }
    const int warp = cluster_thread() >> 5, lane = threadIdx.x & 31, np = p.c.max_pages;
    for (int q0 = 4 * warp; q0 < p.n_req; q0 += 4 * (kClusterThreads / 32)) {
        int s[4], n[4], most = 0;
#pragma unroll
        for (int i = 0; i < 4; i++) s[i] = p.slots[min(q0 + i, p.n_req - 1)];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            n[i] = q0 + i < p.n_req ? pages_of(p.c.lens[s[i]], p.c.page_size) : 0;
            most = max(most, n[i]);
        }
        for (int e = lane; e < most; e += 32) {
            int pg[4];
#pragma unroll
            for (int i = 0; i < 4; i++) pg[i] = e < n[i] ? p.c.page_table[(size_t)s[i] * np + e] : -1;
#pragma unroll
            for (int i = 0; i < 4; i++)
                if (e < n[i]) {
                    if (pg[i] >= 0 && pg[i] < p.c.n_pages) atomicSub(&p.c.ref[pg[i]], 1);
                    p.c.page_table[(size_t)s[i] * np + e] = -1;
                }
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; i++)
            if (lane == i && q0 + i < p.n_req) p.c.lens[s[i]] = 0;
    }
}

// ------------------------------------------------------------------ copies
struct CopyParams {
    hstu_page_cache c;
    Control* ctrl;
    const int* old_len;
    const int* cow;
    const int* old_table;
    int n_req, T, nvec;
    const int32_t* slots;
    const int32_t* off;
    const int32_t* src_rows;   // append: source row of each new row (may be null); compact: keep_rows
    int n_src;                 // append: rows of k, v, ts
    const uint4* k;            // append: source rows
    const uint4* v;
    const int64_t* ts;
};

// Request of row r: off[q] <= r < off[q + 1].
__device__ __forceinline__ int request_of(const int32_t* off, int n_req, int r) {
    int lo = 0, hi = n_req - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (__ldg(off + mid) <= r) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Rows [0, T) are the new ones; append has n_req * page_size more places for the rows
// of the shared pages that are copied before they are written on.
template <bool COMPACT>
__global__ void __launch_bounds__(kCopyThreads) copy_rows_kernel(CopyParams p) {
    wait_for_prior_launch();
    if (p.ctrl->valid == 0) return;
    const int lane = threadIdx.x & 31, ps = p.c.page_size;
    const long long warp0 = ((long long)blockIdx.x * kCopyThreads + threadIdx.x) >> 5;
    const long long n_warps = ((long long)gridDim.x * kCopyThreads) >> 5;
    const long long total = (long long)p.T + (COMPACT ? 0 : (long long)p.n_req * ps);
    uint4* pk = static_cast<uint4*>(p.c.k);
    uint4* pv = static_cast<uint4*>(p.c.v);
    for (long long r0 = warp0 * kRowsPerWarp; r0 < total; r0 += n_warps * kRowsPerWarp) {
        // lane j < kRowsPerWarp resolves row r0 + j: source and destination rows, and whether
        // the source is the pool itself; src -2: nothing to do, -1: a row of zeros
        int src_mine = -2, dst_mine = 0, pool_mine = COMPACT;
        const long long r = r0 + lane;
        if (lane < kRowsPerWarp && r < p.T) {
            const int q = request_of(p.off, p.n_req, (int)r);
            const int at = (COMPACT ? 0 : p.old_len[q]) + (int)r - __ldg(p.off + q);
            const int s = p.slots[q];
            dst_mine = p.c.page_table[(size_t)s * p.c.max_pages + at / ps] * ps + at % ps;
            int f = p.src_rows ? __ldg(p.src_rows + r) : (int)r;
            if (COMPACT) {
                if (f >= 0 && f < p.old_len[q]) {
                    const int pg = p.old_table[(size_t)q * p.c.max_pages + f / ps];
                    src_mine = pg >= 0 && pg < p.c.n_pages ? pg * ps + f % ps : -1;
                } else {
                    src_mine = -1;
                }
            } else {
                src_mine = f >= 0 && f < p.n_src ? f : -1;
            }
            if (src_mine < 0) atomicOr(&p.ctrl->status, kStatusBounds);
        } else if (!COMPACT && lane < kRowsPerWarp && r < total) {
            const int q = (int)((r - p.T) / ps), row = (int)((r - p.T) % ps);
            const int pg = p.cow[q], n = p.old_len[q];
            // the whole page but the rows that are written on
            if (pg >= 0 && (row < n % ps || row - n % ps >= __ldg(p.off + q + 1) - __ldg(p.off + q))) {
                src_mine = pg * ps + row;
                dst_mine = p.c.page_table[(size_t)p.slots[q] * p.c.max_pages + n / ps] * ps + row;
                pool_mine = 1;
            }
        }
        if (src_mine >= -1) {
            const int64_t* ts = pool_mine ? p.c.ts : p.ts;
            p.c.ts[dst_mine] = src_mine >= 0 ? ts[src_mine] : 0;
        }
        if (__all_sync(kAll, src_mine == -2)) continue;
        int src[kRowsPerWarp], dst[kRowsPerWarp], pool[kRowsPerWarp];
#pragma unroll
        for (int j = 0; j < kRowsPerWarp; j++) {
            src[j] = __shfl_sync(kAll, src_mine, j);
            dst[j] = __shfl_sync(kAll, dst_mine, j);
            pool[j] = __shfl_sync(kAll, pool_mine, j);
        }
        for (int vb = 0; vb < p.nvec; vb += 64) {
            uint4 a[kRowsPerWarp][2], b[kRowsPerWarp][2];
#pragma unroll
            for (int j = 0; j < kRowsPerWarp; j++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    const int vi = vb + lane + 32 * e;
                    a[j][e] = b[j][e] = make_uint4(0, 0, 0, 0);
                    if (src[j] >= 0 && vi < p.nvec) {
                        const size_t o = (size_t)src[j] * p.nvec + vi;
                        a[j][e] = __ldcs((pool[j] ? pk : p.k) + o);
                        b[j][e] = __ldcs((pool[j] ? pv : p.v) + o);
                    }
                }
#pragma unroll
            for (int j = 0; j < kRowsPerWarp; j++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    const int vi = vb + lane + 32 * e;
                    if (src[j] >= -1 && vi < p.nvec) {
                        const size_t o = (size_t)dst[j] * p.nvec + vi;
                        __stcs(pk + o, a[j][e]);
                        __stcs(pv + o, b[j][e]);
                    }
                }
        }
    }
}

int launch_copy(bool compact, const CopyParams& p, cudaStream_t s) {
    const long long rows = (long long)p.T + (compact ? 0 : (long long)p.n_req * p.c.page_size);
    const long long warps = (rows + kRowsPerWarp - 1) / kRowsPerWarp;
    const long long blocks = std::min<long long>((warps * 32 + kCopyThreads - 1) / kCopyThreads, 148LL * 2);   // one resident wave
    if (blocks < 1) return HSTU_OK;
    return cuda_status(compact ? launch_early(copy_rows_kernel<true>, (int)blocks, kCopyThreads, 0, s, p)
                               : launch_early(copy_rows_kernel<false>, (int)blocks, kCopyThreads, 0, s, p));
}

// Checks common to the operators; *p gets the plan's parameters.
int plan_params(const hstu_page_cache* c, int32_t n_req, const int32_t* slots, void* workspace, size_t bytes,
                PlanParams* p) {
    const int st = check_cache(c);
    if (st != HSTU_OK) return st;
    if (n_req < 0) return HSTU_ERR_INVALID_ARG;
    const PageWs w = page_ws(*c);
    if (!aligned(workspace, 256) || bytes < w.total) return HSTU_ERR_WORKSPACE;
    if (n_req > 0 && !aligned(slots, 4)) return HSTU_ERR_INVALID_ARG;
    if (n_req > c->n_slots) return HSTU_ERR_INVALID_ARG;   // slots are named once
    char* base = static_cast<char*>(workspace);
    auto at = [&](size_t off) { return reinterpret_cast<int*>(base + off); };
    p->c = *c;
    p->ctrl = reinterpret_cast<Control*>(base);
    p->claim = at(w.claim);
    p->base = at(w.base);
    p->old_len = at(w.old_len);
    p->cow = at(w.cow);
    p->free_list = at(w.free_list);
    p->old_table = at(w.old_table);
    p->n_req = n_req;
    p->slots = slots;
    p->src_slots = nullptr;
    p->off = nullptr;
    p->T = 0;
    return HSTU_OK;
}

CopyParams copy_params(const PlanParams& p) {
    CopyParams q;
    q.c = p.c;
    q.ctrl = p.ctrl;
    q.old_len = p.old_len;
    q.cow = p.cow;
    q.old_table = p.old_table;
    q.n_req = p.n_req;
    q.T = p.T;
    q.nvec = (int)((long long)p.c.row_elems * (p.c.dtype == HSTU_F32 ? 4 : 2) / 16);
    q.slots = p.slots;
    q.off = p.off;
    q.src_rows = nullptr;
    q.n_src = 0;
    q.k = q.v = nullptr;
    q.ts = nullptr;
    return q;
}

}  // namespace
}  // namespace hstu

using namespace hstu;

size_t hstu_cache_workspace_bytes(const hstu_page_cache* cache) {
    return check_cache(cache) == HSTU_OK ? page_ws(*cache).total : 0;
}

int hstu_cache_append(const hstu_page_cache* cache, int32_t n_req, const int32_t* slots, const int32_t* row_offsets,
                      int32_t T, const int32_t* src_rows, int32_t n_src, const void* k, const void* v, const int64_t* ts,
                      void* workspace, size_t workspace_bytes, void* stream) {
    PlanParams p;
    const int st = plan_params(cache, n_req, slots, workspace, workspace_bytes, &p);
    if (st != HSTU_OK) return st;
    if (T < 0 || n_src < 0 || (!src_rows && n_src < T) || (T > 0 && n_req == 0)) return HSTU_ERR_INVALID_ARG;
    if (n_req == 0) return HSTU_OK;
    if (!aligned(row_offsets, 4) || (src_rows && !aligned(src_rows, 4))) return HSTU_ERR_INVALID_ARG;
    if (T > 0 && n_src > 0 && (!aligned(k, 16) || !aligned(v, 16) || !aligned(ts, 8))) return HSTU_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    p.off = row_offsets;
    p.T = T;
    plan_rows_kernel<false><<<1, kPlanThreads, 0, s>>>(p);
    const int e = cuda_status(cudaGetLastError());
    if (e != HSTU_OK || T == 0) return e;
    CopyParams q = copy_params(p);
    q.src_rows = src_rows;
    q.n_src = n_src;
    q.k = static_cast<const uint4*>(k);
    q.v = static_cast<const uint4*>(v);
    q.ts = ts;
    return launch_copy(false, q, s);
}

int hstu_cache_compact(const hstu_page_cache* cache, int32_t n_req, const int32_t* slots, const int32_t* keep_offsets,
                       int32_t K, const int32_t* keep_rows, void* workspace, size_t workspace_bytes, void* stream) {
    PlanParams p;
    const int st = plan_params(cache, n_req, slots, workspace, workspace_bytes, &p);
    if (st != HSTU_OK) return st;
    if (K < 0 || (K > 0 && n_req == 0)) return HSTU_ERR_INVALID_ARG;
    if (n_req == 0) return HSTU_OK;
    if (!aligned(keep_offsets, 4) || (K > 0 && !aligned(keep_rows, 4))) return HSTU_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    p.off = keep_offsets;
    p.T = K;
    plan_rows_kernel<true><<<1, kPlanThreads, 0, s>>>(p);
    const int e = cuda_status(cudaGetLastError());
    if (e != HSTU_OK || K == 0) return e;
    CopyParams q = copy_params(p);
    q.src_rows = keep_rows;
    return launch_copy(true, q, s);
}

int hstu_cache_fork(const hstu_page_cache* cache, int32_t n_req, const int32_t* src_slots, const int32_t* dst_slots,
                    void* workspace, size_t workspace_bytes, void* stream) {
    PlanParams p;
    const int st = plan_params(cache, n_req, dst_slots, workspace, workspace_bytes, &p);
    if (st != HSTU_OK) return st;
    if (n_req == 0) return HSTU_OK;
    if (!aligned(src_slots, 4)) return HSTU_ERR_INVALID_ARG;
    p.src_slots = src_slots;
    fork_kernel<<<kCluster, kPlanThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return cuda_status(cudaGetLastError());
}

int hstu_cache_free(const hstu_page_cache* cache, int32_t n_req, const int32_t* slots, void* workspace,
                    size_t workspace_bytes, void* stream) {
    PlanParams p;
    const int st = plan_params(cache, n_req, slots, workspace, workspace_bytes, &p);
    if (st != HSTU_OK) return st;
    if (n_req == 0) return HSTU_OK;
    free_kernel<<<kCluster, kPlanThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return cuda_status(cudaGetLastError());
}
