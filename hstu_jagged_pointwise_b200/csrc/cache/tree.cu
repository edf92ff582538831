// tree.cu -- trees of candidates scored over a paged history cache (tcgen05, sm_100a).
//
// For node c of tree b over a history of n rows, with depth(c) ancestors and position
// p_c = n + depth(c),
//   Y_c = (1/alpha) [ sum_j see(p_c, j) SiLU(q_c.k_j + rab_pos + rab_time) v_j
//                     + the same over c and its ancestors ],
// see(i, j) = i - j < W or j < S (HSTU blog, sections 3.1-3.2 for the sum and its biases,
// 4.2-4.3 for candidates over a cached history).  There is no softmax: parts of the sum
// over the history simply add, so a long history is split over CTAs with no statistics
// to join.  Three launches:
//   tree_prep    a CTA a tree: checks, depths by pointer doubling, the live part of the
//                history, and the work list (head, group of 64 nodes, split)
//   tree_attn    persistent; the sum over the history, 128 keys at a time
//   tree_finish  a CTA a node: adds the splits in order, the path's own terms, then
//                Y, LayerNorm and U in one pass over registers
//
// tree_attn works on transposed scores, so that few nodes still fill the tensor core's
// lanes: S^T = K Q^T (lanes = 128 keys, columns = 64 nodes), P^T = SiLU(.) in bf16 to
// shared memory, O^T += V^T P^T (lanes = head dims).  A thread owns one key: for keys far
// in the past both biases are the same for every node (the position is clamped, the time
// bucket is wide), so a warp mostly needs one constant a thread.  Only 16-node columns
// that hold nodes are computed.  With one node a tile costs its 64 KB of K and V and
// little else: the kernel is bound by HBM up to some 100 nodes a tree, and by the
// elementwise step and the tensor core above.
//
// One CTA = 10 warps, two CTAs per SM (110 KB of shared memory and 256 TMEM columns each,
// so that one loads while the other computes):
//   warps 0-7  elementwise (warp w: keys 32*(w%4).., 16-node chunks of parity w/4), epilogue
//   warp 8     producer: work fetch, page lookup, TMA of Q and of the K and V pages
//   warp 9     MMA issuer; S^T of the next tile is issued before this tile's P^T is waited for
// TMEM columns: S^T at [0, 64) and [64, 128), O^T at [128, 192).
// Every wait is bounded; on timeout the CTA sets a status bit, drains its copies and
// MMAs, frees TMEM and exits.
#include <math.h>

#include "../ew_bias.cuh"
#include "../ptx.cuh"
#include "cache_internal.h"

namespace hstu {
namespace {

using namespace ptx;

constexpr unsigned kAll = 0xffffffffu;
constexpr int kPrepThreads = 256;

// What tree_prep leaves for a tree: its nodes [off, off + m), history length n, live
// history rows [0, s) and [lo, n), live 128-row tiles [0, ts) and [w0, ceil(n / 128)),
// nv of them, cut into `splits` parts.
struct TreeInfo {
    int off, m, slot, n, s, lo, ts, w0, nv, splits, pad[2];
};

struct TreeParams {
    const int32_t* page_table;
    const int32_t* lens;
    const int64_t* ts_pages;
    int n_pages, n_slots, max_pages, ps;
    const int32_t* slots;
    const int32_t* node_off;
    const int32_t* parent;
    const int64_t* node_ts;
    const int32_t* n_sink;
    const int32_t* window;
    const float* rab_pos;
    const float* rab_time;
    Control* ctrl;             // valid: 0 at the start of a call, -1 after a bad tree or a timeout
    TreeInfo* info;            // [B]
    int* depth;                // [T]
    int4* items;               // {tree, head, group, split}
    float* part;               // [max_splits][T][H*d]: partial sums over the history
    long long max_items;
    int B, T, H, P, nb, ld, max_nodes, max_splits;
    float inv_alpha;
    DebugWait dbg;
    // tree_finish
    const __nv_bfloat16* q;
    const __nv_bfloat16* k;
    const __nv_bfloat16* v;
    const __nv_bfloat16* u;
    const float* gamma;
    const float* beta;
    float eps;
    __nv_bfloat16* y;
    __nv_bfloat16* o;
};

__device__ __forceinline__ int tile_of(const TreeInfo& t, int v) { return v < t.ts ? v : t.w0 + (v - t.ts); }
__device__ __forceinline__ bool live_row(const TreeInfo& t, int j) { return j < t.s || (j >= t.lo && j < t.n); }

// ------------------------------------------------------------------ prep
// The control block's item and work counters and its bad-tree flag are zeroed by the host
// before this launch.
__global__ void __launch_bounds__(kPrepThreads) tree_prep_kernel(TreeParams p) {
    extern __shared__ int s_tree[];                 // up[m], dist[m]
    __shared__ int s_base;
    const int b = blockIdx.x, tid = threadIdx.x;
    int bad = 0;
    const int off = p.node_off[b], m = p.node_off[b + 1] - off;
    if (b == 0 && p.node_off[0] != 0) bad = 1;
    if (b == p.B - 1 && p.node_off[p.B] != p.T) bad = 1;
    if (off < 0 || m < 0 || m > p.max_nodes || m > p.T - off) bad = 1;
    const int slot = p.slots[b];
    int n = 0, S = 0, W = 0x7fffffff;
    if (slot < 0 || slot >= p.n_slots) {
        bad = 1;
    } else {
        n = p.lens[slot];
        if (n < 0 || n > p.max_pages * p.ps) bad = 1;
    }
    if (p.window) {
        S = p.n_sink[b];
        W = p.window[b];
        if (S < 0 || W < 0) bad = 1;
    }
    if (__syncthreads_or(bad)) {
        if (tid == 0) {
            atomicOr(&p.ctrl->status, kStatusBounds);
            atomicExch(&p.ctrl->valid, -1);
        }
        return;
    }
    // ---- depths by pointer doubling: after step s, up = the 2^s-th ancestor, dist = how many were counted
    int* up = s_tree;
    int* dist = s_tree + p.max_nodes;
    for (int i = tid; i < m; i += kPrepThreads) {
        const int a = p.parent[off + i];
        if (a < -1 || a >= i) bad = 1;
        up[i] = a;
        dist[i] = a >= 0 ? 1 : 0;
    }
    bad = __syncthreads_or(bad);
    constexpr int kPer = kTreeMaxNodes / kPrepThreads;
    for (bool more = !bad; more;) {
        int nu[kPer], nd[kPer], any = 0;
#pragma unroll
        for (int e = 0; e < kPer; e++) {
            const int i = tid + e * kPrepThreads;
            nu[e] = -1;
            nd[e] = 0;
            if (i < m) {
                const int a = up[i];
                nd[e] = dist[i] + (a >= 0 ? dist[a] : 0);
                nu[e] = a >= 0 ? up[a] : -1;
                any |= nu[e] >= 0;
            }
        }
        more = __syncthreads_or(any);
#pragma unroll
        for (int e = 0; e < kPer; e++) {
            const int i = tid + e * kPrepThreads;
            if (i < m) {
                up[i] = nu[e];
                dist[i] = nd[e];
            }
        }
        __syncthreads();
    }
    for (int i = tid; i < m; i += kPrepThreads) p.depth[off + i] = dist[i];
    // ---- live part of the history: the sinks, and what the shallowest node's window reaches
    TreeInfo t;
    t.off = off;
    t.m = m;
    t.slot = slot;
    t.n = n;
    t.s = min(S, n);
    t.lo = W < 1 ? n : max(n - W + 1, 0);
    if (t.lo <= t.s) t.s = n, t.lo = n;              // one run
    const int nt = (n + kTileN - 1) / kTileN;
    t.ts = (t.s + kTileN - 1) / kTileN;
    t.w0 = t.lo < n ? max(t.lo / kTileN, t.ts) : nt;
    t.nv = m > 0 ? t.ts + max(nt - t.w0, 0) : 0;
    t.splits = min(t.nv, p.max_splits);
    t.pad[0] = t.pad[1] = 0;
    // every page with a live row must be in the pool
    if (m > 0)
        for (int e = tid; e < (n + p.ps - 1) / p.ps; e += kPrepThreads) {
            const int j0 = e * p.ps, j1 = min(j0 + p.ps, n) - 1;
            if (j0 < t.s || j1 >= t.lo) {
                const int pg = p.page_table[(size_t)slot * p.max_pages + e];
                if (pg < 0 || pg >= p.n_pages) bad = 1;
            }
        }
    bad = __syncthreads_or(bad);
    const int groups = (m + kTreeGroup - 1) / kTreeGroup;
    const int cnt = p.H * groups * t.splits;
    if (tid == 0) {
        p.info[b] = t;
        int base = bad ? 0 : atomicAdd(&p.ctrl->n_items, cnt);
        if (bad || (long long)base + cnt > p.max_items) {
            atomicOr(&p.ctrl->status, kStatusBounds);
            atomicExch(&p.ctrl->valid, -1);
            base = -1;
        }
        s_base = base;
    }
    __syncthreads();
    if (s_base < 0) return;
    // the groups of one (head, split) lie side by side: they read the same K and V
    for (int e = tid; e < cnt; e += kPrepThreads) {
        const int g = e % groups, r = e / groups;
        p.items[s_base + e] = make_int4(b, r / t.splits, g, r % t.splits);
    }
}

// ------------------------------------------------------------------ attention over the history
template <int D>
struct TreeSmem {
    static constexpr uint32_t kTileBytes = 128u * D * 2u;
    static constexpr uint32_t k = 0;
    static constexpr uint32_t v = k + kTileBytes;
    static constexpr uint32_t q = v + kTileBytes;                              // 64 nodes
    static constexpr uint32_t pt = q + (uint32_t)kTreeGroup * D * 2u;          // P^T: 128 keys x 64 nodes
    static constexpr uint32_t nts = pt + 128u * kTreeGroup * 2u;               // int64[8 warps][64] node times
    static constexpr uint32_t npos = nts + 8u * kTreeGroup * 8u;               // int32[8 warps][64] node positions
    static constexpr uint32_t rth = npos + 8u * kTreeGroup * 4u;               // float[64]: rab_time / 2
    static constexpr uint32_t item = rth + kMaxTBuckets * 4u;                  // int4[2]
    static constexpr uint32_t bars = item + 2u * 16u;                          // uint64[20]
    static constexpr uint32_t tmem = bars + 20u * 8u;
    static constexpr uint32_t abort_flag = tmem + 4u;
    static constexpr uint32_t rph = abort_flag + 12u;                          // float[2P-1]: rab_pos / 2
    static constexpr uint32_t alloc(int P) { return rph + 8u * (uint32_t)P + 1024u; }
};

enum {
    kQFull = 0, kQEmpty, kKFull, kKEmpty, kVFull, kVEmpty, kSFull0, kSFull1, kPFull, kPEmpty, kOFull, kOEmpty,
    kItFull0, kItFull1, kItEmpty0, kItEmpty1, kDrain, kNumBars
};

constexpr int kEwWarps = 8;
constexpr int kEwThreads = 32 * kEwWarps;
constexpr int kProducerWarp = kEwWarps;
constexpr int kMmaWarp = kEwWarps + 1;
constexpr int kThreads = 32 * (kEwWarps + 2);
constexpr uint32_t kTmemCols = 256;
constexpr uint32_t kSCol = 0;
constexpr uint32_t kOCol = 128;
constexpr uint32_t kPanel = 128u * 128u;                     // 128 rows x 128 B
constexpr uint32_t kHalfPanel = 64u * 128u;                  // 64 rows x 128 B

__device__ __forceinline__ void flag_timeout(const TreeParams& p, volatile int* abort_flag) {
    *abort_flag = 1;
    atomicOr(&p.ctrl->status, kStatusTimeout);
    atomicExch(&p.ctrl->valid, -1);
}

struct Item {
    int h, node0, cnt, v0, v1, split;
    TreeInfo t;
};

__device__ __forceinline__ Item load_item(const TreeParams& p, int4 it) {
    Item s;
    s.t = p.info[it.x];
    s.h = it.y;
    s.node0 = s.t.off + it.z * kTreeGroup;
    s.cnt = min(kTreeGroup, s.t.m - it.z * kTreeGroup);
    s.split = it.w;
    s.v0 = (int)((long long)s.t.nv * it.w / s.t.splits);
    s.v1 = (int)((long long)s.t.nv * (it.w + 1) / s.t.splits);
    return s;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 2)
tree_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const TreeParams p) {
    using L = TreeSmem<D>;
    constexpr int kPanels = D / 64;
    constexpr uint32_t kIdS = idesc_bf16_f32(128, kTreeGroup, 0, 0);   // S^T: K and Q K-major
    constexpr uint32_t kIdO = idesc_bf16_f32(D, kTreeGroup, 1, 1);     // O^T: V and P^T MN-major

    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    uint8_t* sm = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
    float* s_rph = reinterpret_cast<float*>(sm + L::rph);
    float* s_rth = reinterpret_cast<float*>(sm + L::rth);
    int4* s_item = reinterpret_cast<int4*>(sm + L::item);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::bars);
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(sm + L::tmem);
    volatile int* s_abort = reinterpret_cast<volatile int*>(sm + L::abort_flag);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    for (int i = tid; i < 2 * p.P - 1; i += kThreads) s_rph[i] = 0.5f * p.rab_pos[i];
    for (int i = tid; i < p.nb; i += kThreads) s_rth[i] = 0.5f * p.rab_time[i];
    if (tid == 0) {
        for (int i = 0; i < kNumBars; i++) {
            uint32_t c = 1;
            if (i == kPFull || i == kOEmpty) c = kEwThreads;
            if (i == kItEmpty0 || i == kItEmpty1) c = kEwThreads + 1;
            mbar_init(&bars[i], c);
        }
        *s_abort = 0;
        fence_mbar_init();
    }
    if (warp == kProducerWarp && lane == 0) {
        prefetch_tmap(&tm_q);
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
    }
    if (warp == kMmaWarp) {
        tmem_alloc(s_tmem, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;

    if (warp == kProducerWarp) {
        // ============================================================ producer
        // Lane e looks up and loads page box e of a tile (128 / ps boxes of ps rows).
        int it_use = 0, q_use = 0, k_use = 0, v_use = 0;
        bool ok = true;
        const int boxes = kTileN / p.ps;
        const int n_items = p.ctrl->valid == 0 ? p.ctrl->n_items : 0;
        while (true) {
            const int slot = it_use & 1;
            int4 it = make_int4(-1, 0, 0, 0);
            ok = mbar_wait(&bars[kItEmpty0 + slot], ((it_use >> 1) & 1) ^ 1, s_abort, p.dbg.limit);
            ok = __all_sync(kAll, ok);
            if (!ok) break;
            if (lane == 0) {
                const int idx = atomicAdd(&p.ctrl->counter, 1);
                if (idx < n_items) it = p.items[idx];
                s_item[slot] = it;
                mbar_arrive(&bars[kItFull0 + slot]);
            }
            it.x = __shfl_sync(kAll, it.x, 0);
            it.y = __shfl_sync(kAll, it.y, 0);
            it.z = __shfl_sync(kAll, it.z, 0);
            it.w = __shfl_sync(kAll, it.w, 0);
            it_use++;
            if (it.x < 0) break;
            const Item s = load_item(p, it);
            const int32_t* table = p.page_table + (size_t)s.t.slot * p.max_pages;
            // the page of this lane's box of tile v, -1 when it holds no live row
            auto page_of = [&](int v) {
                if (v >= s.v1 || lane >= boxes) return -1;
                const int j0 = tile_of(s.t, v) * kTileN + lane * p.ps, j1 = min(j0 + p.ps, s.t.n) - 1;
                return j0 < s.t.n && (j0 < s.t.s || j1 >= s.t.lo) ? table[j0 / p.ps] : -1;
            };
            auto load_boxes = [&](int pg, uint8_t* dst, const CUtensorMap* tm, uint64_t* bar) {
                const int live = __popc(__ballot_sync(kAll, pg >= 0));
                if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)live * p.ps * D * 2u);
                __syncwarp();
                if (pg >= 0)
                    for (int pn = 0; pn < kPanels; pn++)
                        tma_load_2d(dst + pn * kPanel + lane * p.ps * 128, tm, bar, s.h * D + pn * 64, pg * p.ps);
            };
            int pg = page_of(s.v0);
            ok = __all_sync(kAll, mbar_wait(&bars[kQEmpty], (q_use & 1) ^ 1, s_abort, p.dbg.limit));
            if (ok && p.dbg.withhold_first_load && q_use == 0) {
                // test hook: withhold this CTA's first Q tile, so the waits for it run out
                if (lane == 0) wait_for_abort(s_abort, 2 * p.dbg.limit);
                __syncwarp();
                ok = false;
            }
            if (!ok) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(&bars[kQFull], (uint32_t)kTreeGroup * D * 2u);
                for (int pn = 0; pn < kPanels; pn++)
                    tma_load_2d(sm + L::q + pn * kHalfPanel, &tm_q, &bars[kQFull], s.h * D + pn * 64, s.node0);
            }
            q_use++;
            for (int v = s.v0; v < s.v1; v++) {
                const int pg_next = page_of(v + 1);
                ok = __all_sync(kAll, mbar_wait(&bars[kKEmpty], (k_use & 1) ^ 1, s_abort, p.dbg.limit));
                if (!ok) break;
                load_boxes(pg, sm + L::k, &tm_k, &bars[kKFull]);
                k_use++;
                if (pg_next >= 0)
                    for (int pn = 0; pn < kPanels; pn++) {
                        tma_prefetch_2d(&tm_k, s.h * D + pn * 64, pg_next * p.ps);
                        tma_prefetch_2d(&tm_v, s.h * D + pn * 64, pg_next * p.ps);
                    }
                ok = __all_sync(kAll, mbar_wait(&bars[kVEmpty], (v_use & 1) ^ 1, s_abort, p.dbg.limit));
                if (!ok) break;
                load_boxes(pg, sm + L::v, &tm_v, &bars[kVFull]);
                v_use++;
                pg = pg_next;
            }
            if (!ok) break;
        }
        if (lane == 0) {
            if (!ok && !*s_abort) flag_timeout(p, s_abort);
            if (*s_abort) {
                // drain the copies this warp issued (at most the last one per buffer)
                volatile int dummy = 0;
                if (q_use) mbar_wait(&bars[kQFull], (q_use - 1) & 1, &dummy);
                if (k_use) mbar_wait(&bars[kKFull], (k_use - 1) & 1, &dummy);
                if (v_use) mbar_wait(&bars[kVFull], (v_use - 1) & 1, &dummy);
            }
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // ============================================================ MMA issuer
        int it_use = 0, q_use = 0, k_use = 0, v_use = 0, p_use = 0, o_use = 0, s_use = 0;
        bool ok = true;
        const uint32_t aK = smem_u32(sm + L::k), aV = smem_u32(sm + L::v), aQ = smem_u32(sm + L::q), aP = smem_u32(sm + L::pt);
        const uint64_t dK = sdesc_sw128(aK, 16, 1024), dQ = sdesc_sw128(aQ, 16, 1024);
        const uint64_t dV = sdesc_sw128(aV, kPanel, 1024), dP = sdesc_sw128(aP, 16, 1024);
        // S^T of the next tile into its TMEM buffer; K is free when it is done
        auto issue_s = [&]() -> bool {
            if (!mbar_wait(&bars[kKFull], k_use & 1, s_abort, p.dbg.limit)) return false;
            k_use++;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < D / 16; kk++) {
                const uint32_t off = (kk >> 2) * kPanel + (kk & 3) * 32, offq = (kk >> 2) * kHalfPanel + (kk & 3) * 32;
                mma_ss(tmem + kSCol + 64 * (s_use & 1), dK + (off >> 4), dQ + (offq >> 4), kIdS, kk > 0 ? 1u : 0u);
            }
            tc_commit(&bars[kSFull0 + (s_use & 1)]);
            tc_commit(&bars[kKEmpty]);
            s_use++;
            return true;
        };
        while (ok) {
            const int slot = it_use & 1;
            int4 it = make_int4(-1, 0, 0, 0);
            if (lane == 0) {
                ok = mbar_wait(&bars[kItFull0 + slot], (it_use >> 1) & 1, s_abort, p.dbg.limit);
                if (ok) it = s_item[slot];
            }
            ok = __shfl_sync(kAll, ok, 0);
            if (!ok) break;
            it.x = __shfl_sync(kAll, it.x, 0);
            it_use++;
            if (it.x < 0) break;
            if (lane == 0) {
                const Item s = load_item(p, it);
                ok = mbar_wait(&bars[kQFull], q_use & 1, s_abort, p.dbg.limit);
                q_use++;
                if (ok) ok = issue_s();
                for (int v = s.v0; ok && v < s.v1; v++) {
                    if (v + 1 < s.v1) ok = issue_s();
                    if (ok && v + 1 == s.v1) tc_commit(&bars[kQEmpty]);
                    if (ok) ok = mbar_wait(&bars[kPFull], p_use & 1, s_abort, p.dbg.limit);
                    if (ok) ok = mbar_wait(&bars[kVFull], v_use & 1, s_abort, p.dbg.limit);
                    if (ok && v == s.v0) ok = mbar_wait(&bars[kOEmpty], (o_use & 1) ^ 1, s_abort, p.dbg.limit);
                    if (!ok) break;
                    p_use++;
                    v_use++;
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < kTileN / 16; kk++)
                        mma_ss(tmem + kOCol, dV + (kk * 2048 >> 4), dP + (kk * 2048 >> 4), kIdO, (v > s.v0 || kk > 0) ? 1u : 0u);
                    tc_commit(&bars[kVEmpty]);
                    tc_commit(&bars[kPEmpty]);
                }
                if (ok) {
                    o_use++;
                    tc_commit(&bars[kOFull]);
                    mbar_arrive(&bars[kItEmpty0 + slot]);
                }
            }
            ok = __shfl_sync(kAll, ok, 0);
        }
        if (lane == 0) {
            if (!ok && !*s_abort) flag_timeout(p, s_abort);
            // every MMA this thread issued completes before TMEM is released
            volatile int dummy = 0;
            tc_commit(&bars[kDrain]);
            mbar_wait(&bars[kDrain], 0, &dummy);
        }
        __syncwarp();
    } else {
        // ============================================================ elementwise (warps 0-7)
        int it_use = 0, s_use = 0, p_use = 0, v_use = 0, o_use = 0;
        const int wq = warp & 3, g = warp >> 2;
        const int r = 32 * wq + lane;                        // TMEM lane = key of the tile
        const uint32_t lane_base = (uint32_t)(32 * wq) << 16;
        const uint32_t p_row = smem_u32(sm + L::pt) + r * 128;
        int64_t* w_nts = reinterpret_cast<int64_t*>(sm + L::nts) + warp * kTreeGroup;
        int32_t* w_npos = reinterpret_cast<int32_t*>(sm + L::npos) + warp * kTreeGroup;
        bool ok = true;
        while (ok) {
            const int slot = it_use & 1;
            ok = __all_sync(kAll, mbar_wait(&bars[kItFull0 + slot], (it_use >> 1) & 1, s_abort, p.dbg.limit));
            if (!ok) break;
            const int4 it = s_item[slot];
            it_use++;
            if (it.x < 0) break;
            const Item s = load_item(p, it);
            const int S = p.window ? p.n_sink[it.x] : 0, W = p.window ? p.window[it.x] : 0x7fffffff;
            const int32_t* table = p.page_table + (size_t)s.t.slot * p.max_pages;
            // the group's positions and times, and their ranges; places past the last node repeat it
            __syncwarp();
            int pmin = 0x7fffffff, pmax = 0;
            int64_t tmin = INT64_MAX, tmax = INT64_MIN;
#pragma unroll
            for (int e = 0; e < kTreeGroup / 32; e++) {
                const int c = s.node0 + min(lane + 32 * e, s.cnt - 1);
                const int pos = s.t.n + p.depth[c];
                const int64_t ts = p.node_ts[c];
                w_npos[lane + 32 * e] = pos;
                w_nts[lane + 32 * e] = ts;
                pmin = min(pmin, pos);
                pmax = max(pmax, pos);
                tmin = min(tmin, ts);
                tmax = max(tmax, ts);
            }
            pmin = __reduce_min_sync(kAll, pmin);
            pmax = __reduce_max_sync(kAll, pmax);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                tmin = min(tmin, (int64_t)__shfl_xor_sync(kAll, (long long)tmin, o));
                tmax = max(tmax, (int64_t)__shfl_xor_sync(kAll, (long long)tmax, o));
            }
            __syncwarp();
            const int n_chunks = (s.cnt + 15) / 16;
            // this thread's key of tile v: its index, or -1 when it is not live; its time a tile ahead
            auto key_of = [&](int v) {
                if (v >= s.v1) return -1;
                const int j = tile_of(s.t, v) * kTileN + r;
                return live_row(s.t, j) ? j : -1;
            };
            auto time_of = [&](int j) -> int64_t { return j >= 0 ? __ldg(p.ts_pages + (size_t)table[j / p.ps] * p.ps + j % p.ps) : 0; };
            int j = key_of(s.v0);
            int64_t tj = time_of(j);
            for (int v = s.v0; v < s.v1; v++) {
                const int j_next = key_of(v + 1);
                const int64_t tj_next = time_of(j_next);
                // ---- is the score's bias and visibility one value for all nodes?
                const bool dead = j < 0;
                float c0 = kMaskedHalfBias;
                bool same = true;
                if (!dead) {
                    const bool all = j < S || pmax - j < W, none = j >= S && pmin - j >= W;
                    uint64_t lo = 0, hi;
                    if (tj < tmin) lo = abs_diff_u64(tmin, tj);
                    else if (tj > tmax) lo = abs_diff_u64(tj, tmax);
                    hi = max(abs_diff_u64(tj, tmin), abs_diff_u64(tj, tmax));
                    const int tb_lo = time_bucket_of_delta(lo, p.nb), tb_hi = time_bucket_of_delta(hi, p.nb);
                    const bool pos1 = pmin == pmax || j - pmin <= -(p.P - 1);
                    same = none || (all && tb_lo == tb_hi && pos1);
                    if (same && !none) c0 = s_rph[pos_index(pmin, j, p.P)] + s_rth[tb_lo];
                }
                const bool fast = __all_sync(kAll, same);
                const bool ragged = __any_sync(kAll, dead);
                ok = mbar_wait(&bars[kSFull0 + (s_use & 1)], (s_use >> 1) & 1, s_abort, p.dbg.limit);
                // P^T of the tile before has been multiplied
                if (ok) ok = mbar_wait(&bars[kPEmpty], (p_use & 1) ^ 1, s_abort, p.dbg.limit);
                if (!__all_sync(kAll, ok)) { ok = false; break; }
                const uint32_t s_col = tmem + lane_base + kSCol + 64 * (s_use & 1);
                s_use++;
                p_use++;
                tc_fence_after();
#pragma unroll 1
                for (int c = g; c < n_chunks; c += 2) {
                    uint32_t sv[16], pk[8];
                    tmem_ld16(s_col + 16 * c, sv);
                    tmem_ld_wait(sv);
                    if (ragged) {
                        // rows that no node may see hold anything in shared memory
#pragma unroll
                        for (int e = 0; e < 16; e++) sv[e] = dead ? 0u : sv[e];
                    }
                    if (fast) {
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            const float2 h = fma2(make_float2(__uint_as_float(sv[e]), __uint_as_float(sv[e + 1])),
                                                  make_float2(0.5f, 0.5f), make_float2(c0, c0));
                            const float2 a = fma2(h, make_float2(tanh_approx(h.x), tanh_approx(h.y)), h);
                            pk[e >> 1] = pack_bf16x2(a.x, a.y);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            float a[2];
#pragma unroll
                            for (int f = 0; f < 2; f++) {
                                const int pos = w_npos[16 * c + e + f];
                                const int64_t ts = w_nts[16 * c + e + f];
                                const bool vis = !dead && (j < S || pos - j < W);
                                const float hb = vis ? s_rph[pos_index(pos, j, p.P)] + s_rth[time_bucket(ts, tj, p.nb)] : kMaskedHalfBias;
                                const float h = fmaf(__uint_as_float(sv[e + f]), 0.5f, hb);
                                a[f] = fmaf(h, tanh_approx(h), h);
                            }
                            pk[e >> 1] = pack_bf16x2(a[0], a[1]);
                        }
                    }
                    // row r of P^T, nodes 16c .. 16c + 15 (128-byte swizzle)
#pragma unroll
                    for (int e = 0; e < 2; e++)
                        st_shared_v4(p_row + (((uint32_t)(2 * c + e) ^ (r & 7)) * 16), pk[4 * e], pk[4 * e + 1], pk[4 * e + 2], pk[4 * e + 3]);
                }
                if (ragged) {
                    // V rows that are not live become zeros: P is zero there, but 0 * NaN is not
                    ok = mbar_wait(&bars[kVFull], v_use & 1, s_abort, p.dbg.limit);
                    if (!__all_sync(kAll, ok)) { ok = false; break; }
                    if (dead && g < kPanels) {
                        const uint32_t row = smem_u32(sm + L::v) + g * kPanel + r * 128;
#pragma unroll
                        for (int e = 0; e < 8; e++) st_shared_v4(row + 16 * e, 0u, 0u, 0u, 0u);
                    }
                }
                v_use++;
                fence_proxy_async_smem();
                tc_fence_before();
                mbar_arrive(&bars[kPFull]);
                j = j_next;
                tj = tj_next;
            }
            if (!ok) break;
            // ---------------- epilogue: O^T (lanes = head dims, columns = nodes) into the split's partial sums
            ok = __all_sync(kAll, mbar_wait(&bars[kOFull], o_use & 1, s_abort, p.dbg.limit));
            if (!ok) break;
            o_use++;
            tc_fence_after();
            // M = 128 puts head dim 32*wq + lane in this lane; M = 64 puts 16*wq + lane in lanes 0-15
            const int dim = D == 128 ? 32 * wq + lane : 16 * wq + lane;
            float* out = p.part + ((size_t)s.split * p.T + s.node0) * p.ld + (size_t)s.h * D + dim;
#pragma unroll 1
            for (int c = g; c < n_chunks; c += 2) {
                uint32_t ov[16];
                tmem_ld16(tmem + lane_base + kOCol + 16 * c, ov);
                tmem_ld_wait(ov);
                if (D == 128 || lane < 16) {
#pragma unroll
                    for (int e = 0; e < 16; e++)
                        if (16 * c + e < s.cnt) out[(size_t)(16 * c + e) * p.ld] = __uint_as_float(ov[e]);
                }
            }
            tc_fence_before();
            mbar_arrive(&bars[kOEmpty]);
            mbar_arrive(&bars[kItEmpty0 + slot]);
        }
        if (!ok && lane == 0 && !*s_abort) flag_timeout(p, s_abort);
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// ------------------------------------------------------------------ finish
__device__ __forceinline__ float block_sum(float x, float* s_red, int n_warps) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kAll, x, o);
    if (n_warps == 1) return x;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = x;
    __syncthreads();
    x = (threadIdx.x & 31) < n_warps ? s_red[threadIdx.x & 31] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kAll, x, o);
    return x;
}

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int e = 0; e < 4; e++) {
        x[2 * e] = __uint_as_float(w[e] << 16);
        x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
}

__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                              pack_bf16x2(x[6], x[7]));
}

// A CTA a node; thread t owns columns 8t .. 8t + 7.  Sums in fp32; Y and O_pre are each
// rounded once.  The block is rounded up to whole warps (idle threads hold zeros).
template <int D>
__global__ void tree_finish_kernel(TreeParams p) {
    __shared__ float s_red[32];
    if (p.ctrl->valid != 0) return;
    const int c = blockIdx.x, col = 8 * (int)threadIdx.x, n_warps = blockDim.x >> 5;
    const bool in = col < p.ld;
    // the tree of node c
    int lo = 0, hi = p.B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (__ldg(p.node_off + mid) <= c) lo = mid;
        else hi = mid - 1;
    }
    const TreeInfo t = p.info[lo];
    const int S = p.window ? p.n_sink[lo] : 0, W = p.window ? p.window[lo] : 0x7fffffff;
    const size_t row = (size_t)c * p.ld + col;
    float acc[8] = {};
    if (in)
        for (int sp = 0; sp < t.splits; sp++) {
            const float4* a = reinterpret_cast<const float4*>(p.part + (size_t)sp * p.T * p.ld + row);
            const float4 x = __ldcs(a), y = __ldcs(a + 1);
            acc[0] += x.x; acc[1] += x.y; acc[2] += x.z; acc[3] += x.w;
            acc[4] += y.x; acc[5] += y.y; acc[6] += y.z; acc[7] += y.w;
        }
    // the path: c itself, then its ancestors
    float q[8] = {};
    if (in) load8(p.q + row, q);
    const int pos_c = t.n + p.depth[c];
    const int64_t ts_c = p.node_ts[c];
    int d = 0;                                       // steps up from c
    for (int a = c; a >= 0; d++) {
        const int up = p.parent[a];
        const int pos_a = pos_c - d;
        if (d < W || pos_a < S) {
            float k[8] = {}, v[8] = {};
            if (in) {
                load8(p.k + (size_t)a * p.ld + col, k);
                load8(p.v + (size_t)a * p.ld + col, v);
            }
            float dot = 0.f;
#pragma unroll
            for (int e = 0; e < 8; e++) dot = fmaf(q[e], k[e], dot);
#pragma unroll
            for (int o = D / 16; o > 0; o >>= 1) dot += __shfl_xor_sync(kAll, dot, o);   // over the head's D / 8 threads
            const float z = dot + p.rab_pos[pos_index(pos_c, pos_a, p.P)] + p.rab_time[time_bucket(ts_c, p.node_ts[a], p.nb)];
            const float w = z * __fdividef(1.f, 1.f + __expf(-z));
#pragma unroll
            for (int e = 0; e < 8; e++) acc[e] = fmaf(w, v[e], acc[e]);
        }
        a = up >= 0 ? t.off + up : -1;
    }
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < 8; e++) {
        acc[e] = in ? acc[e] * p.inv_alpha : 0.f;
        sum += acc[e];
    }
    const float mu = block_sum(sum, s_red, n_warps) / (float)p.ld;
    float sq = 0.f;
    if (in) {
        store8(p.y + row, acc);
#pragma unroll
        for (int e = 0; e < 8; e++) sq = fmaf(acc[e] - mu, acc[e] - mu, sq);
    }
    const float rstd = rsqrtf(block_sum(sq, s_red, n_warps) / (float)p.ld + p.eps);
    if (in) {
        float u[8], o[8];
        load8(p.u + row, u);
#pragma unroll
        for (int e = 0; e < 8; e++) o[e] = fmaf((acc[e] - mu) * rstd, __ldg(p.gamma + col + e), __ldg(p.beta + col + e)) * u[e];
        store8(p.o + row, o);
    }
}

// ------------------------------------------------------------------ host
struct TreeWs {
    size_t info, depth, items, part, total;
    long long max_items;
    int max_splits;
};

// Parts a history may be cut into: enough work items for two resident CTAs an SM when the
// trees alone give fewer, one when they give more.  Four part sums a CTA slot: the last
// wave's tail against the partial sums' traffic (they are read once, in L2).
TreeWs tree_ws(const hstu_tree_dims& d, const hstu_page_cache& c) {
    TreeWs w;
    const long long groups = (long long)(d.T + kTreeGroup - 1) / kTreeGroup + d.B;   // at most
    const long long whole = (long long)d.H * ((long long)(d.T + kTreeGroup - 1) / kTreeGroup > d.B ? (d.T + kTreeGroup - 1) / kTreeGroup : d.B);
    const long long tiles = ((long long)c.max_pages * c.page_size + kTileN - 1) / kTileN;
    long long splits = whole > 0 ? (148 * 2 * 2 + whole - 1) / whole : 1;
    if (splits > tiles) splits = tiles;
    if (splits < 1) splits = 1;
    w.max_splits = (int)splits;
    w.max_items = (long long)d.H * groups * splits;
    size_t off = sizeof(Control);
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = align_up(off + bytes, 256);
        return at;
    };
    w.info = take((size_t)d.B * sizeof(TreeInfo));
    w.depth = take((size_t)d.T * 4);
    w.items = take((size_t)w.max_items * sizeof(int4));
    w.part = take((size_t)splits * d.T * d.H * d.d * 4);
    w.total = off;
    return w;
}

int check_tree(const hstu_tree_dims* d, const hstu_page_cache* c) {
    const int st = check_cache(c);
    if (st != HSTU_OK) return st;
    if (!d || d->B < 0 || d->T < 0 || d->H < 1 || d->max_nodes < 0 || (d->T > 0 && (d->B < 1 || d->max_nodes < 1)))
        return HSTU_ERR_INVALID_ARG;
    if (c->dtype != HSTU_BF16 || (d->d != 64 && d->d != 128)) return HSTU_ERR_UNSUPPORTED;
    if ((long long)d->H * d->d > 8192 || d->max_nodes > kTreeMaxNodes) return HSTU_ERR_UNSUPPORTED;
    if (d->H * d->d != c->row_elems) return HSTU_ERR_INVALID_ARG;
    if (d->n_pos < 1 || d->n_pos > kMaxPos || d->n_tbuckets < 1 || d->n_tbuckets > kMaxTBuckets) return HSTU_ERR_UNSUPPORTED;
    if (!(d->alpha > 0.f) || !isfinite(d->alpha) || !(d->ln_eps >= 0.f) || !isfinite(d->ln_eps)) return HSTU_ERR_INVALID_ARG;
    // item numbers are 32-bit
    if (tree_ws(*d, *c).max_items > 0x7fffffffLL) return HSTU_ERR_UNSUPPORTED;
    return HSTU_OK;
}

cudaError_t smem_limit(const void* fn, int bytes) {
    return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <int D>
cudaError_t launch_attn(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const TreeParams& p, int grid,
                        cudaStream_t s) {
    cudaError_t e = smem_limit((const void*)tree_attn_kernel<D>, TreeSmem<D>::alloc(kMaxPos));
    if (e != cudaSuccess) return e;
    tree_attn_kernel<D><<<grid, kThreads, TreeSmem<D>::alloc(p.P), s>>>(tq, tk, tv, p);
    return cudaGetLastError();
}

}  // namespace
}  // namespace hstu

using namespace hstu;

size_t hstu_tree_workspace_bytes(const hstu_tree_dims* dims, const hstu_page_cache* cache) {
    return check_tree(dims, cache) == HSTU_OK ? tree_ws(*dims, *cache).total : 0;
}

int hstu_tree_score(const hstu_tree_dims* dims, const hstu_page_cache* cache, const int32_t* slots,
                    const int32_t* node_offsets, const int32_t* parent, const int64_t* node_ts, const void* node_q,
                    const void* node_k, const void* node_v, const void* node_u, const int32_t* n_sink,
                    const int32_t* window, const float* rab_pos, const float* rab_time, const float* ln_gamma,
                    const float* ln_beta, void* y, void* o_pre, void* workspace, size_t workspace_bytes, void* stream) {
    const int st = check_tree(dims, cache);
    if (st != HSTU_OK) return st;
    const hstu_tree_dims& d = *dims;
    const hstu_page_cache& c = *cache;
    const TreeWs w = tree_ws(d, c);
    if (!aligned(workspace, 256) || workspace_bytes < w.total) return HSTU_ERR_WORKSPACE;
    if (d.T == 0) return HSTU_OK;
    if (!aligned(slots, 4) || !aligned(node_offsets, 4) || !aligned(parent, 4) || !aligned(node_ts, 8) ||
        !aligned(node_q, 16) || !aligned(node_k, 16) || !aligned(node_v, 16) || !aligned(node_u, 16) ||
        !aligned(rab_pos, 4) || !aligned(rab_time, 4) || !aligned(ln_gamma, 4) || !aligned(ln_beta, 4) ||
        !aligned(y, 16) || !aligned(o_pre, 16))
        return HSTU_ERR_INVALID_ARG;
    if ((n_sink != nullptr) != (window != nullptr) || (window && (!aligned(n_sink, 4) || !aligned(window, 4))))
        return HSTU_ERR_INVALID_ARG;
    if (c.n_slots < 1) return HSTU_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    char* base = static_cast<char*>(workspace);
    TreeParams p;
    p.page_table = c.page_table;
    p.lens = c.lens;
    p.ts_pages = c.ts;
    p.n_pages = c.n_pages;
    p.n_slots = c.n_slots;
    p.max_pages = c.max_pages;
    p.ps = c.page_size;
    p.slots = slots;
    p.node_off = node_offsets;
    p.parent = parent;
    p.node_ts = node_ts;
    p.n_sink = n_sink;
    p.window = window;
    p.rab_pos = rab_pos;
    p.rab_time = rab_time;
    p.ctrl = reinterpret_cast<Control*>(base);
    p.info = reinterpret_cast<TreeInfo*>(base + w.info);
    p.depth = reinterpret_cast<int*>(base + w.depth);
    p.items = reinterpret_cast<int4*>(base + w.items);
    p.part = reinterpret_cast<float*>(base + w.part);
    p.max_items = w.max_items;
    p.B = d.B;
    p.T = d.T;
    p.H = d.H;
    p.P = d.n_pos;
    p.nb = d.n_tbuckets;
    p.ld = d.H * d.d;
    p.max_nodes = d.max_nodes;
    p.max_splits = w.max_splits;
    p.inv_alpha = 1.0f / d.alpha;
    p.dbg = cache_debug_wait();
    p.q = static_cast<const __nv_bfloat16*>(node_q);
    p.k = static_cast<const __nv_bfloat16*>(node_k);
    p.v = static_cast<const __nv_bfloat16*>(node_v);
    p.u = static_cast<const __nv_bfloat16*>(node_u);
    p.gamma = ln_gamma;
    p.beta = ln_beta;
    p.eps = d.ln_eps;
    p.y = static_cast<__nv_bfloat16*>(y);
    p.o = static_cast<__nv_bfloat16*>(o_pre);

    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    // work counters and the bad-tree flag of this call; the status word stays
    if (e == cudaSuccess) e = cudaMemsetAsync(&p.ctrl->n_items, 0, 3 * sizeof(int), s);
    const int prep_smem = 2 * d.max_nodes * (int)sizeof(int);
    if (e == cudaSuccess) e = smem_limit((const void*)tree_prep_kernel, 2 * kTreeMaxNodes * (int)sizeof(int));
    if (e != cudaSuccess) return cuda_status(e);
    tree_prep_kernel<<<d.B, kPrepThreads, prep_smem, s>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_status(e);
    if (c.n_pages > 0) {
        CUtensorMap tq, tk, tv;
        const long long rows = (long long)c.n_pages * c.page_size;
        if (!make_tmap(&tq, node_q, d.T, p.ld, kTreeGroup) || !make_tmap(&tk, c.k, rows, p.ld, c.page_size) ||
            !make_tmap(&tv, c.v, rows, p.ld, c.page_size))
            return HSTU_ERR_CUDA;
        const int grid = (int)(w.max_items < 2LL * sms ? w.max_items : 2LL * sms);
        e = d.d == 128 ? launch_attn<128>(tq, tk, tv, p, grid, s) : launch_attn<64>(tq, tk, tv, p, grid, s);
        if (e != cudaSuccess) return cuda_status(e);
    }
    const int threads = (p.ld / 8 + 31) / 32 * 32;
    if (d.d == 128) tree_finish_kernel<128><<<d.T, threads, 0, s>>>(p);
    else tree_finish_kernel<64><<<d.T, threads, 0, s>>>(p);
    return cuda_status(cudaGetLastError());
}
