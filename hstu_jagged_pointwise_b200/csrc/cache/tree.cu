// tree.cu -- trees of candidates scored over a paged history cache (tcgen05, sm_100a).
//
// For node c of tree b over a history of n rows, with depth(c) ancestors and position
// p_c = n + depth(c),
//   Y_c = (1/alpha) [ sum_j see(p_c, j) SiLU(q_c.k_j + rab_pos + rab_time) v_j
//                     + the same over c and its ancestors ],
// see(i, j) = i - j < W or j < S (HSTU blog, sections 3.1-3.2 for the sum and its biases,
// 4.2-4.3 for candidates over a cached history).  There is no softmax: parts of the sum
// over the history simply add, so a long history is split over CTAs with no statistics
// to join.  Three launches: prep is an ordinary one, the other two start while the one before
// them ends (programmatic dependent launch) and wait for it before they read its results:
//   tree_prep    a CTA a tree: checks, depths by pointer doubling, the live part of the
//                history, and the work list (head, group of nodes, split)
//   tree_attn    persistent, a CTA an SM; the sum over the history, 128 keys at a time
//   tree_finish  one to eight warps a node: adds the splits in order, the path's own terms, then
//                Y, LayerNorm and U in one pass over registers.  A path is walked node by node, one
//                dependent load after another, so its depth is paid in latency and, for chains, its
//                square in L2 reads (one tree over 4096 events, H = 4, d = 128: chain of 64 nodes 50
//                us, 512 256, 2048 1.24 ms, 8192 12.1 ms; without depth 27, 40, 56, 117 us)
//
// tree_attn keeps a ring of 128-row K and V tiles in flight (160 KB at d = 128), filled by
// TMA page by page, and two score tiles in TMEM, so that the next tile's scores are
// multiplied while this tile's are turned into P.  It comes in two forms:
//   narrow  trees of up to 64 nodes: transposed, so that few nodes still fill the tensor
//           core's lanes.  S^T = K Q^T (lanes = keys, columns = 64 nodes), P^T in bf16 to
//           shared memory, O^T += V^T P^T (lanes = head dims).  Columns without nodes are
//           not computed: with one node a tile costs its 64 KB of K and V and little else,
//           and the kernel is bound by HBM.
//   wide    larger trees: S = Q K^T (lanes = 128 nodes), P in bf16 back into the score's
//           TMEM columns, O += P V.  Its products cost 1040 tensor cycles for 128 nodes
//           where the transposed ones take 1310 for 64.
// Bias: a history row far in the past has one position index (clamped) and one time bucket
// for all nodes of a warp, so most rows of scores need one constant a key.
//
// One CTA = 24 warps, each with little to wait for but its own input, since a wait that ends
// at once still costs some 200 cycles (at 128 keys x 128 nodes a tile takes about 1900):
//   0-15   elementwise and epilogue
//   16     producer: TMA of Q and of the K and V pages
//   17     issues the score products, up to two tiles ahead
//   18-21  key warps, a tile ahead: each lane looks up one key's time and decides how the
//          group's nodes see it, which keeps the elementwise path from scores to P short
//   22     issues the products with P
//   23     fetches work: the next item, its tree and its first pages, an item ahead
// Every wait is bounded; on timeout the CTA sets a status bit, drains its
// copies and MMAs, frees TMEM and exits.
#include <math.h>

#include <mutex>

#include "../ew_bias.cuh"
#include "../ptx.cuh"
#include "cache_internal.h"

namespace hstu {
namespace {

using namespace ptx;

constexpr unsigned kAll = 0xffffffffu;
constexpr int kPrepThreads = 256;
constexpr int kNarrow = 64, kWide = 128;   // nodes of a group in the two forms

// The scorer's words of the control block: items of tree_attn's work list and how many are taken,
// kBad = -1 after a bad tree or a timeout, CTAs of tree_attn that are done, kVerdict = kBad for
// tree_finish.  The last CTA of tree_attn sets kVerdict and clears the others for the next call.
// They lie in `pad`, which nothing else writes, so that a workspace may serve the page operators
// (which leave valid = 1) and the scorer in turn.
// The items are counted in 64 bits: where offsets are bad, trees may overlap, and a million of
// them claim more than 2^31 items (64 heads, 8192 nodes each) before the call is refused.
enum { kItems = 0, kTaken = 2, kBad = 3, kDone = 4, kVerdict = 5 };

__device__ __forceinline__ unsigned long long* items_claimed(Control* c) { return reinterpret_cast<unsigned long long*>(&c->pad[kItems]); }

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
    int n_pages, n_slots, max_pages, ps, ps_log;
    const int32_t* slots;
    const int32_t* node_off;
    const int32_t* parent;
    const int64_t* node_ts;
    const int32_t* n_sink;
    const int32_t* window;
    const float* rab_pos;
    const float* rab_time;
    Control* ctrl;
    TreeInfo* info;            // [B]
    int4* node;                // [T] {position, parent's row or -1, tree, splits}
    int4* items;               // {tree, head, group, split}
    float* part;               // [max_splits][T][H*d]: partial sums over the history
    long long max_items;
    int B, T, H, P, nb, ld, max_nodes, max_splits, min_tiles, group;
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
__global__ void __launch_bounds__(kPrepThreads) tree_prep_kernel(TreeParams p) {
    extern __shared__ int s_tree[];                 // up[m], dist[m]
    __shared__ int s_base;
    const int b = blockIdx.x, tid = threadIdx.x;
    allow_next_launch();
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
            atomicExch(&p.ctrl->pad[kBad], -1);
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
    t.splits = min((t.nv + p.min_tiles - 1) / p.min_tiles, p.max_splits);
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
    for (int i = tid; i < m; i += kPrepThreads) {
        const int a = p.parent[off + i];
        p.node[off + i] = make_int4(n + dist[i], a >= 0 ? off + a : -1, b, t.splits);
    }
    bad = __syncthreads_or(bad);
    const int groups = (m + p.group - 1) / p.group;
    const int cnt = p.H * groups * t.splits;
    if (tid == 0) {
        p.info[b] = t;
        long long base = bad ? 0 : (long long)atomicAdd(items_claimed(p.ctrl), (unsigned long long)cnt);
        if (bad || base + cnt > p.max_items) {
            atomicOr(&p.ctrl->status, kStatusBounds);
            atomicExch(&p.ctrl->pad[kBad], -1);
            base = -1;
        }
        s_base = (int)base;                          // max_items is below 2^31
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
constexpr int kPadLo = 160;

template <int D, bool WIDE>
struct TreeSmem {
    static constexpr int kSlots = D == 128 ? (WIDE ? 4 : 5) : 8;               // ring of K and V tiles
    static constexpr int kGroup = WIDE ? kWide : kNarrow;
    static constexpr uint32_t kTileBytes = 128u * D * 2u;
    static constexpr uint32_t kPBytes = WIDE ? 16u * 1024u : 128u * kNarrow * 2u;
    static constexpr uint32_t ring = 0;
    static constexpr uint32_t q = ring + kSlots * kTileBytes;
    static constexpr uint32_t pt = q + (uint32_t)kGroup * D * 2u;              // narrow: two P^T, 128 keys x 64 nodes;
                                                                               // wide: float[16 warps][32 x 16] staging
    // nodes of the item, two items: position, time, time relative to the group's earliest
    static constexpr uint32_t n64 = pt + 2u * kPBytes;                         // int64[2][128]
    static constexpr uint32_t n32 = n64 + 2u * 128u * 8u;                      // int32[2][128]
    static constexpr uint32_t npos = n32 + 2u * 128u * 4u;                     // int32[2][128]
    // keys of the tile, two tiles: half bias, time, relative time; mode and dead lanes of 32 keys
    static constexpr uint32_t k64 = npos + 2u * 128u * 4u;                     // int64[2][128]
    static constexpr uint32_t k32 = k64 + 2u * 128u * 8u;                      // int32[2][128]
    static constexpr uint32_t kc0 = k32 + 2u * 128u * 4u;                      // float[2][128]
    static constexpr uint32_t kmode = kc0 + 2u * 128u * 4u;                    // uint4[2][4]
    static constexpr uint32_t rth = kmode + 2u * 4u * 16u;                     // float[64]: rab_time / 2
    static constexpr uint32_t item = rth + kMaxTBuckets * 4u;                  // ItemSlot[2]
    static constexpr uint32_t bars = item + 2u * 160u;                         // uint64[40]
    static constexpr uint32_t tmem = bars + 40u * 8u;
    static constexpr uint32_t abort_flag = tmem + 4u;
    // rab_pos / 2, continued by its first entry for kPadLo entries below and by its last for 32 above
    static constexpr uint32_t rph = abort_flag + 12u;                          // float[kPadLo + 2P-1 + 32]
    static constexpr uint32_t alloc(int P) { return rph + 4u * (uint32_t)(kPadLo + 2 * P + 32) + 1024u; }
};
static_assert(TreeSmem<128, false>::alloc(kMaxPos) <= 227 * 1024 && TreeSmem<128, true>::alloc(kMaxPos) <= 227 * 1024, "shared memory");

constexpr int kMaxSlots = 8;
enum {
    kFull0 = 0, kEmpty0 = kFull0 + kMaxSlots, kQFull = kEmpty0 + kMaxSlots, kQEmpty, kSFull0, kSFull1, kPFull0, kPFull1, kKeys0, kKeys1,
    kOFull, kOEmpty, kItFull0, kItFull1, kItEmpty0, kItEmpty1, kPFree0, kPFree1, kDrainS, kDrainP, kNumBars
};
static_assert(kNumBars <= 40, "barrier space");

constexpr int kEwWarps = 16;
constexpr int kProducerWarp = kEwWarps;
constexpr int kScoreWarp = kEwWarps + 1;
constexpr int kKeyWarp = kEwWarps + 2;
constexpr int kKeyWarps = 4;
constexpr int kValueWarp = kKeyWarp + kKeyWarps;
constexpr int kFetchWarp = kValueWarp + 1;
constexpr int kThreads = 32 * (kFetchWarp + 1);
constexpr uint32_t kPanel = 128u * 128u;                     // 128 rows x 128 B

__device__ __forceinline__ void flag_timeout(const TreeParams& p, volatile int* abort_flag) {
    *abort_flag = 1;
    atomicOr(&p.ctrl->status, kStatusTimeout);
    atomicExch(&p.ctrl->pad[kBad], -1);
}

struct Item {
    int b, h, node0, cnt, v0, v1, split;   // b < 0: no more work
    TreeInfo t;
};

// An item in shared memory, with the pages of its first two tiles (-1 where a page box of a
// tile holds no live row).
struct ItemSlot {
    Item s;
    int pages[2][8];
    int pad[5];
};
static_assert(sizeof(ItemSlot) == 160, "item slot");

__device__ __forceinline__ Item load_item(const TreeParams& p, int4 it) {
    Item s;
    s.b = it.x;
    s.t = p.info[it.x];
    s.h = it.y;
    s.node0 = s.t.off + it.z * p.group;
    s.cnt = min(p.group, s.t.m - it.z * p.group);
    s.split = it.w;
    s.v0 = (int)((long long)s.t.nv * it.w / s.t.splits);
    s.v1 = (int)((long long)s.t.nv * (it.w + 1) / s.t.splits);
    return s;
}

// Ring of K and V tiles, filled in the order K0 K1 V0 K2 V1 ... V(m-1) of an item of m tiles.
__device__ __forceinline__ int ring_of_k(int v) { return v == 0 ? 0 : 2 * v - 1; }
__device__ __forceinline__ int ring_of_v(int v, int m) { return v + 1 < m ? 2 * v + 2 : 2 * v + 1; }

struct Ring {
    int slot = 0, phase = 0;
    __device__ __forceinline__ void next(int slots) {
        if (++slot == slots) {
            slot = 0;
            phase ^= 1;
        }
    }
    __device__ __forceinline__ void skip(int n, int slots) {
        slot += n;
        phase ^= (slot / slots) & 1;
        slot %= slots;
    }
};

// Positions and times of the nodes of a group.
struct NodeRange {
    int pmin, pmax, S, W;
    int64_t tmin, tmax;
    bool close;                // all times within 2^30
};

// How the nodes of a group see one key (this lane's), and how its quarter (32 keys, the
// warp's) is to be worked.  c0 is the part of half the bias that all nodes share: the time's,
// 0 where the bucket differs between nodes (a bit of `varied`), plus the position's unless
// kPos; a huge negative value where no node sees the key, which makes SiLU zero.
//   kPos   positions differ: add rab_pos[j - pos], read along a diagonal of the padded table
//   kWin   some node sees a key that another does not: mask each pair
//   kAny   times 2^30 or more apart under a varied bucket, or positions further apart than the
//          table's padding: each pair by the rules as they stand
enum { kPos = 1, kWin = 2, kAny = 4 };

struct KeyClass {
    float c0;
    int32_t tr;                // the key's time relative to the nodes' earliest
    uint32_t varied, mode;
};

__device__ __forceinline__ KeyClass classify_key(const NodeRange& n, int j, int j0, int64_t tj, const float* rph, const float* rth,
                                                 int P, int nb) {
    KeyClass k;
    const bool none = j < 0 || (j >= n.S && n.pmin - j >= n.W);
    const bool whole = j < n.S || n.pmax - j < n.W;
    uint64_t lo = 0;
    if (tj < n.tmin) lo = (uint64_t)n.tmin - (uint64_t)tj;
    else if (tj > n.tmax) lo = (uint64_t)tj - (uint64_t)n.tmax;
    const uint64_t hi = max(abs_diff_u64(tj, n.tmin), abs_diff_u64(tj, n.tmax));
    const int tb = time_bucket_of_delta(lo, nb);
    const bool varies = !none && tb != time_bucket_of_delta(hi, nb);
    const bool pos = __any_sync(kAll, !none && n.pmin != n.pmax && j - n.pmin > -(P - 1));
    k.c0 = varies ? 0.f : rth[tb];
    if (!pos) k.c0 += rph[pos_index(n.pmin, max(j, 0), P)];
    if (none) k.c0 = kMaskedHalfBias;
    k.tr = (int32_t)(uint32_t)((uint64_t)tj - (uint64_t)n.tmin);
    k.varied = __ballot_sync(kAll, varies);
    const bool any = __any_sync(kAll, varies && (!n.close || hi >= (1ull << 30))) || (pos && j0 - n.pmax + P - 1 < -kPadLo);
    k.mode = (pos ? kPos : 0) | (__any_sync(kAll, !none && !whole) ? kWin : 0) | (any ? kAny : 0);
    return k;
}

// bf16 pair of SiLU(s + 2 hb), from half the scores: h + h tanh(h).  One special-function call a
// score, where exp and a reciprocal take two: the hardware's tanh is off by up to 2^-11, so SiLU by up
// to |z| 2^-12.  P is rounded to bf16 (half a step, 2^-9 to 2^-8 of the value) because it is an operand
// of the bf16 product with V, whose other operand it has to match in type.
__device__ __forceinline__ uint32_t silu_pair(uint32_t s0, uint32_t s1, float hb0, float hb1) {
    const float2 h = fma2(make_float2(__uint_as_float(s0), __uint_as_float(s1)), make_float2(0.5f, 0.5f), make_float2(hb0, hb1));
    const float2 a = fma2(h, make_float2(tanh_approx(h.x), tanh_approx(h.y)), h);
    return pack_bf16x2(a.x, a.y);
}

// Half the time bias of a pair whose times are near.
__device__ __forceinline__ float near_time(int32_t tn, int32_t tk, const float* rth, int nbm1) {
    return rth[time_bucket_u32((uint32_t)abs(tn - tk), nbm1)];
}

// Any pair, by the rules as they stand.
__device__ __forceinline__ float any_bias(int pos, int64_t ts, int j, int64_t tj, const float* rph, const float* rth, int P, int nb) {
    return rph[pos_index(pos, j, P)] + rth[time_bucket(ts, tj, nb)];
}

template <int D, bool WIDE>
__global__ void __launch_bounds__(kThreads, 1)
tree_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const TreeParams p) {
    using L = TreeSmem<D, WIDE>;
    constexpr int kPanels = D / 64;
    constexpr int kSlots = L::kSlots;
    constexpr uint32_t kQPanel = (uint32_t)L::kGroup * 128u;           // one 64-column panel of Q
    constexpr uint32_t kSCols = WIDE ? 128u : 64u;                     // TMEM columns of a score tile
    constexpr uint32_t kOCol = 2u * kSCols;
    constexpr uint32_t kTmemCols = WIDE ? 512u : 256u;
    constexpr uint32_t kIdS = idesc_bf16_f32(128, L::kGroup, 0, 0);    // both operands K-major
    constexpr uint32_t kIdO = WIDE ? idesc_bf16_f32(128, D, 0, 1)      // O: P from TMEM, V MN-major
                                   : idesc_bf16_f32(D, kNarrow, 1, 1); // O^T: V and P^T MN-major

    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    uint8_t* sm = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
    float* s_rph = reinterpret_cast<float*>(sm + L::rph) + kPadLo;
    float* s_rth = reinterpret_cast<float*>(sm + L::rth);
    ItemSlot* s_item = reinterpret_cast<ItemSlot*>(sm + L::item);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::bars);
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(sm + L::tmem);
    volatile int* s_abort = reinterpret_cast<volatile int*>(sm + L::abort_flag);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    for (int i = tid - kPadLo; i < 2 * p.P - 1 + 32; i += kThreads) s_rph[i] = 0.5f * p.rab_pos[min(max(i, 0), 2 * p.P - 2)];
    for (int i = tid; i < p.nb; i += kThreads) s_rth[i] = 0.5f * p.rab_time[i];
    if (tid == 0) {
        for (int i = 0; i < kNumBars; i++) {
            uint32_t c = 1;
            if (i == kPFull0 || i == kPFull1) c = kEwWarps + kKeyWarps;
            if (i == kKeys0 || i == kKeys1) c = kKeyWarps;
            if (i == kOEmpty) c = kEwWarps;
            if (i == kItEmpty0 || i == kItEmpty1) c = kEwWarps + 2;
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
    if (warp == kScoreWarp) {
        tmem_alloc(s_tmem, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    allow_next_launch();
    wait_for_prior_launch();

    auto wait = [&](int bar, uint32_t parity) -> bool {
        return __all_sync(kAll, mbar_wait(&bars[bar], parity, s_abort, p.dbg.limit));
    };
    // this lane's page box of tile v of an item: its page, -1 when it holds no live row
    const int boxes = kTileN >> p.ps_log;
    auto box_page = [&](const Item& s, int v) {
        if (v >= s.v1 || lane >= boxes) return -1;
        const int j0 = tile_of(s.t, v) * kTileN + (lane << p.ps_log), j1 = min(j0 + p.ps, s.t.n) - 1;
        return j0 < s.t.n && (j0 < s.t.s || j1 >= s.t.lo) ? p.page_table[(size_t)s.t.slot * p.max_pages + (j0 >> p.ps_log)] : -1;
    };

    if (warp == kFetchWarp) {
        // ============================================================ work fetch
        const int n_items = p.ctrl->pad[kBad] == 0 ? (int)*items_claimed(p.ctrl) : 0;
        bool ok = true;
        for (int it_use = 0;; it_use++) {
            const int slot = it_use & 1;
            int idx = blockIdx.x;                           // the first item by position, the others by demand
            if (it_use > 0) {
                if (lane == 0) idx = atomicAdd(&p.ctrl->pad[kTaken], 1) + gridDim.x;
                idx = __shfl_sync(kAll, idx, 0);
            }
            Item s;
            s.b = -1;
            int pg0 = -1, pg1 = -1;
            if (idx < n_items) {
                s = load_item(p, p.items[idx]);
                pg0 = box_page(s, s.v0);
                pg1 = box_page(s, s.v0 + 1);
            }
            ok = wait(kItEmpty0 + slot, ((it_use >> 1) & 1) ^ 1);
            if (!ok) break;
            if (lane == 0) s_item[slot].s = s;
            if (lane < 8) {
                s_item[slot].pages[0][lane] = pg0;
                s_item[slot].pages[1][lane] = pg1;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[kItFull0 + slot]);
            if (s.b < 0) break;
        }
        if (lane == 0 && !ok && !*s_abort) flag_timeout(p, s_abort);
        __syncwarp();
    } else if (warp == kProducerWarp) {
        // ============================================================ producer
        // Lane e loads page box e of a tile (128 / ps boxes of ps rows).
        int used = 0;                                       // ring slots filled so far
        int q_use = 0;
        Ring ring;
        bool ok = true;
        for (int it_use = 0;; it_use++) {
            const int slot = it_use & 1;
            ok = wait(kItFull0 + slot, (it_use >> 1) & 1);
            if (!ok) break;
            const Item s = s_item[slot].s;
            if (s.b < 0) break;
            auto load_tile = [&](int pg, const CUtensorMap* tm) -> bool {
                if (!wait(kEmpty0 + ring.slot, ring.phase ^ 1)) return false;
                uint64_t* bar = &bars[kFull0 + ring.slot];
                const int live = __popc(__ballot_sync(kAll, pg >= 0));
                if (lane == 0) mbar_arrive_expect_tx(bar, ((uint32_t)live << p.ps_log) * D * 2u);
                __syncwarp();
                if (pg >= 0)
                    for (int pn = 0; pn < kPanels; pn++)
                        tma_load_2d(sm + L::ring + ring.slot * L::kTileBytes + pn * kPanel + (lane << p.ps_log) * 128, tm, bar,
                                    s.h * D + pn * 64, pg << p.ps_log);
                ring.next(kSlots);
                used++;
                return true;
            };
            int pg = lane < 8 ? s_item[slot].pages[0][lane] : -1, pg_next = lane < 8 ? s_item[slot].pages[1][lane] : -1;
            if (p.dbg.withhold_first_load && it_use == 0) {
                // test hook: withhold this CTA's first tiles, so the waits for them run out
                if (lane == 0) wait_for_abort(s_abort, 2 * p.dbg.limit);
                __syncwarp();
                ok = false;
                break;
            }
            // the first K tile goes ahead of Q, whose buffer is free only after the last item's last scores
            ok = load_tile(pg, &tm_k);
            if (ok) ok = wait(kQEmpty, (q_use & 1) ^ 1);
            if (!ok) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(&bars[kQFull], (uint32_t)L::kGroup * D * 2u);
                for (int pn = 0; pn < kPanels; pn++)
                    tma_load_2d(sm + L::q + pn * kQPanel, &tm_q, &bars[kQFull], s.h * D + pn * 64, s.node0);
            }
            q_use++;
            for (int v = s.v0; ok && v < s.v1; v++) {
                const int pg_after = box_page(s, v + 2);
                if (v + 1 < s.v1) ok = load_tile(pg_next, &tm_k);
                if (ok) ok = load_tile(pg, &tm_v);
                pg = pg_next;
                pg_next = pg_after;
            }
            if (!ok) break;
        }
        if (lane == 0) {
            if (!ok && !*s_abort) flag_timeout(p, s_abort);
            if (*s_abort) {
                // drain the copies this warp issued: the latest one of each buffer
                volatile int dummy = 0;
                if (q_use) mbar_wait(&bars[kQFull], (q_use - 1) & 1, &dummy);
                for (int i = 0; i < kSlots && i < used; i++) {
                    const int last = (used - 1 - i) / kSlots * kSlots + i;    // latest fill of slot i
                    mbar_wait(&bars[kFull0 + i], (last / kSlots) & 1, &dummy);
                }
            }
        }
        __syncwarp();
    } else if (warp == kScoreWarp || warp == kValueWarp) {
        // ============================================================ MMA issue
        // All lanes go through the same steps and one issues.
        const bool score = warp == kScoreWarp;
        int t_use = 0;
        Ring ring;                                          // first slot of the item
        bool ok = true;
        const uint32_t tm = __shfl_sync(kAll, tmem, 0);
        const uint32_t one = lane == 0;
        const uint32_t a_ring = smem_u32(sm + L::ring), a_pt = smem_u32(sm + L::pt);
        const uint64_t dQ = sdesc_sw128(smem_u32(sm + L::q), 16, 1024);
        for (int it_use = 0;; it_use++) {
            const int slot = it_use & 1;
            ok = wait(kItFull0 + slot, (it_use >> 1) & 1);
            if (!ok) break;
            const int b = s_item[slot].s.b, m = s_item[slot].s.v1 - s_item[slot].s.v0;
            if (b < 0) break;
            if (score) ok = wait(kQFull, it_use & 1);
            for (int v = 0; ok && v < m; v++, t_use++) {
                const uint32_t buf = t_use & 1, ph = (t_use >> 1) & 1;
                Ring at = ring;
                if (score) {
                    // scores of tile v into its TMEM buffer, once the tile two before has been multiplied
                    at.skip(ring_of_k(v), kSlots);
                    ok = wait(kPFree0 + buf, ph ^ 1);
                    if (ok) ok = wait(kFull0 + at.slot, at.phase);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t dK = sdesc_sw128(a_ring + at.slot * L::kTileBytes, 16, 1024);
#pragma unroll
                    for (int kk = 0; kk < D / 16; kk++) {
                        const uint32_t off = (kk >> 2) * kPanel + (kk & 3) * 32, offq = (kk >> 2) * kQPanel + (kk & 3) * 32;
                        const uint64_t k = dK + (off >> 4), q = dQ + (offq >> 4);
                        mma_ss_if(one, tm + kSCols * buf, WIDE ? q : k, WIDE ? k : q, kIdS, kk > 0 ? 1u : 0u);
                    }
                    tc_commit_if(one, &bars[kSFull0 + buf]);
                    tc_commit_if(one, &bars[kEmpty0 + at.slot]);
                    if (v + 1 == m) tc_commit_if(one, &bars[kQEmpty]);
                } else {
                    // O += P V
                    at.skip(ring_of_v(v, m), kSlots);
                    if (v == 0) ok = wait(kOEmpty, (it_use & 1) ^ 1);
                    if (ok) ok = wait(kFull0 + at.slot, at.phase);
                    if (ok) ok = wait(kPFull0 + buf, ph);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t dV = sdesc_sw128(a_ring + at.slot * L::kTileBytes, kPanel, 1024);
                    const uint64_t dP = sdesc_sw128(a_pt + buf * L::kPBytes, 16, 1024);
#pragma unroll
                    for (int kk = 0; kk < kTileN / 16; kk++) {
                        const uint32_t acc = (v > 0 || kk > 0) ? 1u : 0u;
                        // wide: P of keys 32c .. 32c+31 sits in the first 16 columns of score chunk c
                        if (WIDE) mma_ts_if(one, tm + kOCol, tm + kSCols * buf + 32 * (kk >> 1) + 8 * (kk & 1), dV + (kk * 2048 >> 4), kIdO, acc);
                        else mma_ss_if(one, tm + kOCol, dV + (kk * 2048 >> 4), dP + (kk * 2048 >> 4), kIdO, acc);
                    }
                    tc_commit_if(one, &bars[kEmpty0 + at.slot]);
                    tc_commit_if(one, &bars[kPFree0 + buf]);
                    if (v + 1 == m) tc_commit_if(one, &bars[kOFull]);
                }
            }
            if (!ok) break;
            ring.skip(2 * m, kSlots);
            if (lane == 0) mbar_arrive(&bars[kItEmpty0 + slot]);
        }
        if (lane == 0 && !ok && !*s_abort) flag_timeout(p, s_abort);
        __syncwarp();
        // every MMA issued completes before TMEM is released
        volatile int dummy = 0;
        const int drain = score ? kDrainS : kDrainP;
        tc_commit_if(one, &bars[drain]);
        mbar_wait(&bars[drain], 0, &dummy);
        __syncwarp();
    } else if (warp >= kKeyWarp && warp < kKeyWarp + kKeyWarps) {
        // ============================================================ key warps
        // Lane l of key warp w looks after key 32w + l of each tile.
        int it_use = 0, t_use = 0;
        Ring ring;                                           // first slot of the item
        const int kw = warp - kKeyWarp, r = 32 * kw + lane;
        bool ok = true;
        while (ok) {
            const int slot = it_use & 1;
            ok = wait(kItFull0 + slot, (it_use >> 1) & 1);
            if (!ok) break;
            const Item s = s_item[slot].s;
            it_use++;
            if (s.b < 0) break;
            const int32_t* table = p.page_table + (size_t)s.t.slot * p.max_pages;
            // the key of tile v (-1 when it is not live), its page two tiles ahead and its time one
            auto key_of = [&](int v) {
                if (v >= s.v1) return -1;
                const int j = tile_of(s.t, v) * kTileN + r;
                return live_row(s.t, j) ? j : -1;
            };
            auto page_of = [&](int j) { return j >= 0 ? __ldg(table + (j >> p.ps_log)) : 0; };
            auto time_of = [&](int j, int pg) -> int64_t {
                return j >= 0 ? __ldg(p.ts_pages + ((size_t)pg << p.ps_log) + (j & (p.ps - 1))) : 0;
            };
            int j = key_of(s.v0), j_next = key_of(s.v0 + 1);
            const int pg = page_of(j);
            int pg_next = page_of(j_next);
            // ranges over the group's nodes; places past the last one repeat it
            NodeRange nr;
            nr.S = p.window ? p.n_sink[s.b] : 0;
            nr.W = p.window ? p.window[s.b] : 0x7fffffff;
            int pos[L::kGroup / 32];
            int64_t ts[L::kGroup / 32];
            nr.pmin = 0x7fffffff;
            nr.pmax = 0;
            nr.tmin = INT64_MAX;
            nr.tmax = INT64_MIN;
#pragma unroll
            for (int e = 0; e < L::kGroup / 32; e++) {
                const int c = s.node0 + min(lane + 32 * e, s.cnt - 1);
                pos[e] = p.node[c].x;
                ts[e] = p.node_ts[c];
                nr.pmin = min(nr.pmin, pos[e]);
                nr.pmax = max(nr.pmax, pos[e]);
                nr.tmin = min(nr.tmin, ts[e]);
                nr.tmax = max(nr.tmax, ts[e]);
            }
            int64_t tj = time_of(j, pg);
            nr.pmin = __reduce_min_sync(kAll, nr.pmin);
            nr.pmax = __reduce_max_sync(kAll, nr.pmax);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                nr.tmin = min(nr.tmin, (int64_t)__shfl_xor_sync(kAll, (long long)nr.tmin, o));
                nr.tmax = max(nr.tmax, (int64_t)__shfl_xor_sync(kAll, (long long)nr.tmax, o));
            }
            nr.close = (uint64_t)nr.tmax - (uint64_t)nr.tmin < (1ull << 30);
            // the elementwise warps have left the item two before, whose place this is
#pragma unroll
            for (int e = 0; e < L::kGroup / 32; e++)
                if (e % kKeyWarps == kw) {
                    const int at = 128 * slot + lane + 32 * e;
                    reinterpret_cast<int32_t*>(sm + L::npos)[at] = pos[e];
                    reinterpret_cast<int64_t*>(sm + L::n64)[at] = ts[e];
                    reinterpret_cast<int32_t*>(sm + L::n32)[at] = (int32_t)(uint32_t)((uint64_t)ts[e] - (uint64_t)nr.tmin);
                }
            for (int v = s.v0; v < s.v1; v++, t_use++) {
                const int64_t tj_next = time_of(j_next, pg_next);
                const int j_after = key_of(v + 2);
                pg_next = page_of(j_after);
                const bool dead = j < 0;
                const uint32_t deads = __ballot_sync(kAll, dead), buf = t_use & 1;
                const KeyClass k = classify_key(nr, j, tile_of(s.t, v) * kTileN + 32 * kw, tj, s_rph, s_rth, p.P, p.nb);
                // the tile two before, whose place this is, has been turned into P
                ok = __all_sync(kAll, mbar_wait(&bars[kPFull0 + buf], ((t_use >> 1) & 1) ^ 1, s_abort, p.dbg.limit));
                if (!ok) break;
                const int at = 128 * buf + r;
                reinterpret_cast<float*>(sm + L::kc0)[at] = k.c0;
                reinterpret_cast<int32_t*>(sm + L::k32)[at] = k.tr;
                reinterpret_cast<int64_t*>(sm + L::k64)[at] = tj;
                if (lane == 0)
                    reinterpret_cast<uint4*>(sm + L::kmode)[4 * buf + kw] = make_uint4(k.mode, deads, k.varied, 0u);
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[kKeys0 + buf]);
                if (deads) {
                    // V rows that are not live become zeros: P is zero there, but 0 * NaN is not.
                    Ring at_v = ring;
                    at_v.skip(ring_of_v(v - s.v0, s.v1 - s.v0), kSlots);
                    // This warp runs ahead of the products, so the slot may still hold (or be about to
                    // receive) the tile before: first that one's release, then this one's arrival.  A
                    // phase alone cannot tell the tile before from this one.  (The release before that
                    // has come: P of the tile two before, which this warp has waited for, comes after
                    // the products of the tile four before; and this tile's own waits for this warp.)
                    ok = __all_sync(kAll, mbar_wait(&bars[kEmpty0 + at_v.slot], at_v.phase ^ 1, s_abort, p.dbg.limit) &&
                                              mbar_wait(&bars[kFull0 + at_v.slot], at_v.phase, s_abort, p.dbg.limit));
                    if (!ok) break;
                    if (dead) {
                        const uint32_t row = smem_u32(sm + L::ring) + at_v.slot * L::kTileBytes + r * 128;
#pragma unroll
                        for (int e = 0; e < 8 * kPanels; e++) st_shared_v4(row + (e >> 3) * kPanel + 16 * (e & 7), 0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                if (lane == 0) mbar_arrive(&bars[kPFull0 + buf]);
                j = j_next;
                j_next = j_after;
                tj = tj_next;
            }
            ring.skip(2 * (s.v1 - s.v0), kSlots);
        }
        if (!ok && lane == 0 && !*s_abort) flag_timeout(p, s_abort);
        __syncwarp();
    } else {
        // ============================================================ elementwise (warps 0-15)
        // narrow: warp w has keys 32*(w%4) .. +31 in its lanes and nodes 16*(w/4) .. +15 in columns;
        // wide: nodes 32*(w%4) .. +31 in its lanes and keys 32*(w/4) .. +31 in columns.
        int it_use = 0, t_use = 0, o_use = 0;
        const int wq = warp & 3, g = warp >> 2;
        const int kq = WIDE ? g : wq, nq = WIDE ? wq : g;    // key quarter, node quarter
        const int first = (WIDE ? 32 : 16) * nq;             // first node of the warp
        const uint32_t lane_base = (uint32_t)(32 * wq) << 16;
        const int np1 = p.P - 1, nbm1 = p.nb - 1;
        bool ok = true;
        while (ok) {
            const int slot = it_use & 1;
            ok = wait(kItFull0 + slot, (it_use >> 1) & 1);
            if (!ok) break;
            const Item s = s_item[slot].s;
            it_use++;
            if (s.b < 0) break;
            const int S = p.window ? p.n_sink[s.b] : 0, W = p.window ? p.window[s.b] : 0x7fffffff;
            const bool work = first < s.cnt;
            // this warp's nodes (written by the key warps before the item's first tile)
            const int32_t* npos = reinterpret_cast<const int32_t*>(sm + L::npos) + 128 * slot + first;
            const int32_t* n32 = reinterpret_cast<const int32_t*>(sm + L::n32) + 128 * slot + first;
            const int64_t* n64 = reinterpret_cast<const int64_t*>(sm + L::n64) + 128 * slot + first;
            for (int v = s.v0; v < s.v1; v++, t_use++) {
                const uint32_t buf = t_use & 1;
                ok = mbar_wait(&bars[kKeys0 + buf], (t_use >> 1) & 1, s_abort, p.dbg.limit);
                // the scores of this tile (and P of the tile two before has been multiplied)
                if (ok) ok = mbar_wait(&bars[kSFull0 + buf], (t_use >> 1) & 1, s_abort, p.dbg.limit);
                if (!__all_sync(kAll, ok)) { ok = false; break; }
                tc_fence_after();
                const uint4 md = reinterpret_cast<const uint4*>(sm + L::kmode)[4 * buf + kq];
                const uint32_t mode = md.x, deads = md.y, varied = md.z;
                const float* kc0 = reinterpret_cast<const float*>(sm + L::kc0) + 128 * buf + 32 * kq;
                const int32_t* k32 = reinterpret_cast<const int32_t*>(sm + L::k32) + 128 * buf + 32 * kq;
                const int64_t* k64 = reinterpret_cast<const int64_t*>(sm + L::k64) + 128 * buf + 32 * kq;
                const int j0 = tile_of(s.t, v) * kTileN + 32 * kq;            // first key of the quarter
                if (work && !WIDE) {
                    const uint32_t col = tmem + lane_base + kSCols * buf + 16 * g;
                    // row of P^T of this lane's key, nodes 16g .. 16g + 15 (128-byte swizzle)
                    const uint32_t p_row = smem_u32(sm + L::pt) + buf * L::kPBytes + (32 * kq + lane) * 128;
                    const bool dead = (deads >> lane) & 1;
                    const int j = j0 + lane;
                    if (mode & kAny) {
                        // rare: pair by pair, in little code
                        const int64_t tj = k64[lane];
#pragma unroll 1
                        for (int e = 0; e < 16; e += 2) {
                            uint32_t s0, s1;
                            tmem_ld2(col + e, s0, s1);
                            float hb[2];
#pragma unroll
                            for (int f = 0; f < 2; f++)
                                hb[f] = !dead && (j < S || npos[e + f] - j < W) ? any_bias(npos[e + f], n64[e + f], j, tj, s_rph, s_rth, p.P, p.nb)
                                                                                : kMaskedHalfBias;
                            // rows that no node may see hold anything in shared memory
                            const uint32_t x = silu_pair(dead ? 0u : s0, dead ? 0u : s1, hb[0], hb[1]);
                            asm volatile("st.shared.b32 [%0], %1;" ::"r"(p_row + (((uint32_t)(2 * g + (e >> 3)) ^ (lane & 7)) * 16) + (e & 7) * 2), "r"(x) : "memory");
                        }
                    } else {
                        uint32_t sv[16], pk[8];
                        tmem_ld16(col, sv);
                        const float c0 = kc0[lane];
                        tmem_ld_wait(sv);
                        if (deads) {
#pragma unroll
                            for (int e = 0; e < 16; e++) sv[e] = dead ? 0u : sv[e];
                        }
                        if ((mode | varied) == 0) {
#pragma unroll
                            for (int e = 0; e < 16; e += 2) pk[e >> 1] = silu_pair(sv[e], sv[e + 1], c0, c0);
                        } else if (mode == kPos && varied == 0) {
                            const float* rp = s_rph + np1 + j;
#pragma unroll
                            for (int e = 0; e < 16; e += 4) {
                                const int4 ps = *reinterpret_cast<const int4*>(npos + e);
                                pk[e >> 1] = silu_pair(sv[e], sv[e + 1], c0 + rp[-ps.x], c0 + rp[-ps.y]);
                                pk[(e >> 1) + 1] = silu_pair(sv[e + 2], sv[e + 3], c0 + rp[-ps.z], c0 + rp[-ps.w]);
                            }
                        } else {
                            const int cut = (mode & kWin) && j >= S ? W : 0x7fffffff;
                            const int32_t tr = k32[lane];
                            const bool mine = (varied >> lane) & 1;
                            const float* rp = s_rph + np1 + j;
#pragma unroll
                            for (int e = 0; e < 16; e += 4) {
                                const int4 ps = *reinterpret_cast<const int4*>(npos + e), ts = *reinterpret_cast<const int4*>(n32 + e);
                                const int pos[4] = {ps.x, ps.y, ps.z, ps.w}, tn[4] = {ts.x, ts.y, ts.z, ts.w};
                                float hb[4] = {c0, c0, c0, c0};
                                if (mode & kPos) {
#pragma unroll
                                    for (int f = 0; f < 4; f++) hb[f] += rp[-pos[f]];
                                }
                                if (varied) {
#pragma unroll
                                    for (int f = 0; f < 4; f++) {
                                        const float x = near_time(tn[f], tr, s_rth, nbm1);
                                        hb[f] += mine ? x : 0.f;
                                    }
                                }
                                if (mode & kWin) {
#pragma unroll
                                    for (int f = 0; f < 4; f++) hb[f] = pos[f] - j >= cut ? kMaskedHalfBias : hb[f];
                                }
                                pk[e >> 1] = silu_pair(sv[e], sv[e + 1], hb[0], hb[1]);
                                pk[(e >> 1) + 1] = silu_pair(sv[e + 2], sv[e + 3], hb[2], hb[3]);
                            }
                        }
#pragma unroll
                        for (int e = 0; e < 2; e++)
                            st_shared_v4(p_row + (((uint32_t)(2 * g + e) ^ (lane & 7)) * 16), pk[4 * e], pk[4 * e + 1], pk[4 * e + 2], pk[4 * e + 3]);
                    }
                    fence_proxy_async_smem();
                }
                if (work && WIDE) {
                    const uint32_t col = tmem + lane_base + kSCols * buf + 32 * g;
                    const int pos_c = npos[lane];
                    if (mode & kAny) {
                        // rare: pair by pair, in little code
#pragma unroll 1
                        for (int e = 0; e < 32; e += 2) {
                            uint32_t s0, s1;
                            tmem_ld2(col + e, s0, s1);
                            float hb[2];
#pragma unroll
                            for (int f = 0; f < 2; f++) {
                                const int j = j0 + e + f;
                                hb[f] = !((deads >> (e + f)) & 1) && (j < S || pos_c - j < W)
                                            ? any_bias(pos_c, n64[lane], j, k64[e + f], s_rph, s_rth, p.P, p.nb) : kMaskedHalfBias;
                            }
                            tmem_st1(col + (e >> 1), silu_pair((deads >> e) & 1 ? 0u : s0, (deads >> (e + 1)) & 1 ? 0u : s1, hb[0], hb[1]));
                        }
                    } else {
                        uint32_t sa[16], sb[16], pk[16];
                        tmem_ld16(col, sa);
                        tmem_ld16(col + 16, sb);
                        const int32_t tr_c = n32[lane];
                        const float* rp = s_rph + np1 + j0 - pos_c;      // of key 0 of the quarter (used where kPos)
                        const int cut = pos_c - W;                       // keys up to here are past the window
                        tmem_ld_wait(sa);
                        tmem_ld_wait(sb);
                        if (deads) {
#pragma unroll
                            for (int e = 0; e < 16; e++) {
                                sa[e] = (deads >> e) & 1 ? 0u : sa[e];
                                sb[e] = (deads >> (16 + e)) & 1 ? 0u : sb[e];
                            }
                        }
                        // Two straight paths (constants; constants and a diagonal of positions), and one
                        // with a branch for what four keys need: its branches keep the tanh of one
                        // group from overlapping the next's, which makes it half again as slow.
                        if ((mode | varied) == 0) {
#pragma unroll
                            for (int i = 0; i < 32; i += 4) {
                                uint32_t (&sv)[16] = i < 16 ? sa : sb;
                                const float4 c0 = *reinterpret_cast<const float4*>(kc0 + i);
                                pk[i >> 1] = silu_pair(sv[i & 15], sv[(i & 15) + 1], c0.x, c0.y);
                                pk[(i >> 1) + 1] = silu_pair(sv[(i & 15) + 2], sv[(i & 15) + 3], c0.z, c0.w);
                            }
                        } else if (mode == kPos && varied == 0) {
#pragma unroll
                            for (int i = 0; i < 32; i += 4) {
                                uint32_t (&sv)[16] = i < 16 ? sa : sb;
                                const float4 c0 = *reinterpret_cast<const float4*>(kc0 + i);
                                pk[i >> 1] = silu_pair(sv[i & 15], sv[(i & 15) + 1], c0.x + rp[i], c0.y + rp[i + 1]);
                                pk[(i >> 1) + 1] = silu_pair(sv[(i & 15) + 2], sv[(i & 15) + 3], c0.z + rp[i + 2], c0.w + rp[i + 3]);
                            }
                        } else {
#pragma unroll
                          for (int hf = 0; hf < 2; hf++) {
                            uint32_t (&sv)[16] = hf ? sb : sa;
#pragma unroll
                            for (int e = 0; e < 16; e += 4) {
                                const int i0 = 16 * hf + e;
                                const float4 c0 = *reinterpret_cast<const float4*>(kc0 + i0);
                                float hb[4] = {c0.x, c0.y, c0.z, c0.w};
                                if (mode & kPos) {
#pragma unroll
                                    for (int f = 0; f < 4; f++) hb[f] += rp[i0 + f];
                                }
                                if ((varied >> i0) & 15u) {
                                    const int4 tk = *reinterpret_cast<const int4*>(k32 + i0);
                                    const int tks[4] = {tk.x, tk.y, tk.z, tk.w};
#pragma unroll
                                    for (int f = 0; f < 4; f++) {
                                        const float x = near_time(tr_c, tks[f], s_rth, nbm1);
                                        hb[f] += (varied >> (i0 + f)) & 1 ? x : 0.f;
                                    }
                                }
                                if (mode & kWin) {
#pragma unroll
                                    for (int f = 0; f < 4; f++) hb[f] = j0 + i0 + f >= S && j0 + i0 + f <= cut ? kMaskedHalfBias : hb[f];
                                }
                                pk[8 * hf + (e >> 1)] = silu_pair(sv[e], sv[e + 1], hb[0], hb[1]);
                                pk[8 * hf + (e >> 1) + 1] = silu_pair(sv[e + 2], sv[e + 3], hb[2], hb[3]);
                            }
                          }
                        }
                        // P into the chunk's own, already read, columns
                        tmem_st16(col, pk);
                    }
                    tmem_st_wait();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[kPFull0 + buf]);
            }
            if (!ok) break;
            // ---------------- epilogue: the sums into the split's part
            ok = __all_sync(kAll, mbar_wait(&bars[kOFull], o_use & 1, s_abort, p.dbg.limit));
            if (!ok) break;
            o_use++;
            tc_fence_after();
            if (work && !WIDE) {
                // O^T: lanes = head dims, columns = nodes.  M = 128 puts head dim 32*wq + lane in this
                // lane; M = 64 puts 16*wq + lane in lanes 0-15
                const int dim = D == 128 ? 32 * wq + lane : 16 * wq + lane;
                float* out = p.part + ((size_t)s.split * p.T + s.node0 + first) * p.ld + (size_t)s.h * D + dim;
                uint32_t ov[16];
                tmem_ld16(tmem + lane_base + kOCol + 16 * g, ov);
                tmem_ld_wait(ov);
                if (D == 128 || lane < 16) {
#pragma unroll
                    for (int e = 0; e < 16; e++)
                        if (first + e < s.cnt) out[(size_t)e * p.ld] = __uint_as_float(ov[e]);
                }
            }
            if (work && WIDE) {
                // O: lanes = nodes, columns = head dims, a quarter of them for this warp.  16 columns at a
                // time go through shared memory (16-byte vectors, swizzled), so that four lanes store
                // 64 consecutive bytes of a node: from the lanes as they are each store instruction
                // touches 32 rows.
                float* stg = reinterpret_cast<float*>(sm + L::pt) + warp * 512;
#pragma unroll
                for (int hf = 0; hf < D / 64; hf++) {
                    uint32_t ov[16];
                    tmem_ld16(tmem + lane_base + kOCol + (D / 4) * g + 16 * hf, ov);
                    tmem_ld_wait(ov);
                    __syncwarp();
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        st_shared_v4(smem_u32(stg + 16 * lane + 4 * (e ^ ((lane >> 1) & 3))), ov[4 * e], ov[4 * e + 1], ov[4 * e + 2], ov[4 * e + 3]);
                    __syncwarp();
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const int nd = 8 * e + (lane >> 2);
                        const float4 x = *reinterpret_cast<const float4*>(stg + 16 * nd + 4 * ((lane & 3) ^ ((nd >> 1) & 3)));
                        if (first + nd < s.cnt)
                            *reinterpret_cast<float4*>(p.part + ((size_t)s.split * p.T + s.node0 + first + nd) * p.ld + (size_t)s.h * D +
                                                       (D / 4) * g + 16 * hf + 4 * (lane & 3)) = x;
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bars[kOEmpty]);
                mbar_arrive(&bars[kItEmpty0 + slot]);
            }
        }
        if (!ok && lane == 0 && !*s_abort) flag_timeout(p, s_abort);
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kScoreWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
    if (tid == 0) {
        __threadfence();
        if (atomicAdd(&p.ctrl->pad[kDone], 1) == (int)gridDim.x - 1) {
            __threadfence();
            p.ctrl->pad[kVerdict] = atomicAdd(&p.ctrl->pad[kBad], 0);
            *items_claimed(p.ctrl) = 0;
            p.ctrl->pad[kTaken] = p.ctrl->pad[kBad] = p.ctrl->pad[kDone] = 0;
        }
    }
}

// ------------------------------------------------------------------ finish
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kAll, x, o);
    return x;
}

__device__ __forceinline__ void open8(const uint4& a, float (&x)[8]) {
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

// WARPS warps a node; lane l of warp w owns columns 8 ((i WARPS + w) 32 + l) .. +7 of vectors
// i < NV, so that a head's d / 8 lanes are neighbours.  Sums in fp32; Y and O_pre are each
// rounded once, and O_pre comes from the unrounded Y.  Bound by HBM: the parts once, q, k,
// v, u once, two outputs; what it takes is latency (node, then parent and sums, then the two
// sums of the norm), so that all loads whose place is known are made at once, and the form for
// histories in one part (not SPLIT) keeps to 64 registers, four blocks an SM: 32 trees of 900 to
// 1024 nodes, whole scorer, 240 -> 227 us; held to them the form for several parts spills, and
// without, its four loads in flight take a single node over 16 parts from 19.8 to 18.8.
constexpr int kFinishThreads = 256;

template <int D, int NV, int WARPS, bool SPLIT>
__global__ void __launch_bounds__(kFinishThreads, NV == 1 && !SPLIT ? 4 : 1) tree_finish_kernel(TreeParams p) {
    __shared__ float s_red[2][kFinishThreads / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, w = warp % WARPS;
    const int c = blockIdx.x * (kFinishThreads / 32 / WARPS) + warp / WARPS;
    const bool live = c < p.T;                       // the same for all warps of a node
    const int cc = live ? c : p.T - 1;
    auto col = [&](int i) { return 8 * ((i * WARPS + w) * 32 + lane); };
    auto in = [&](int i) { return col(i) < p.ld; };
    const size_t row = (size_t)cc * p.ld;
    float acc[NV][8];
    uint4 q4[NV], k4[NV], v4[NV], u4[NV];            // kept packed while they are on their way
    auto load = [&](uint4 (&x)[NV], const __nv_bfloat16* base, size_t at) {
#pragma unroll
        for (int i = 0; i < NV; i++) x[i] = in(i) ? *reinterpret_cast<const uint4*>(base + at + col(i)) : make_uint4(0, 0, 0, 0);
    };
    load(q4, p.q, row);
    load(k4, p.k, row);
    load(v4, p.v, row);
    load(u4, p.u, row);
#pragma unroll
    for (int i = 0; i < NV; i++)
#pragma unroll
        for (int e = 0; e < 8; e++) acc[i][e] = 0.f;
    const int64_t ts_c = p.node_ts[cc];
    wait_for_prior_launch();
    if (p.ctrl->pad[kVerdict] != 0) return;
    const int4 nd = p.node[cc];                      // position, parent's row, tree, splits
    float4 part0[NV][2];                             // the first split's sums, on their way while the path is worked
#pragma unroll
    for (int i = 0; i < NV; i++)
        if (in(i)) {
            part0[i][0] = __ldcs(reinterpret_cast<const float4*>(p.part + row + col(i)));
            part0[i][1] = __ldcs(reinterpret_cast<const float4*>(p.part + row + col(i)) + 1);
        }
    const int S = p.window ? p.n_sink[nd.z] : 0, W = p.window ? p.window[nd.z] : 0x7fffffff;
    // the path: c itself, then its ancestors, each fetched while the one below it is worked
    int64_t ts_a = ts_c;
    for (int up = nd.y, d = 0;; d++) {               // d steps up from c
        uint4 nk4[NV], nv4[NV];
        int64_t ts_up = 0;
        int next = -1;
        if (up >= 0) {
            load(nk4, p.k, (size_t)up * p.ld);
            load(nv4, p.v, (size_t)up * p.ld);
            ts_up = p.node_ts[up];
            next = p.node[up].y;
        }
        const int pos_a = nd.x - d;
        if (d < W || pos_a < S) {
            const float bias = p.rab_pos[pos_index(nd.x, pos_a, p.P)] + p.rab_time[time_bucket(ts_c, ts_a, p.nb)];
#pragma unroll
            for (int i = 0; i < NV; i++) {
                float q[8], k[8], v[8], dot = 0.f;
                open8(q4[i], q);
                open8(k4[i], k);
                open8(v4[i], v);
#pragma unroll
                for (int e = 0; e < 8; e++) dot = fmaf(q[e], k[e], dot);
#pragma unroll
                for (int o = D / 16; o > 0; o >>= 1) dot += __shfl_xor_sync(kAll, dot, o);   // over the head's D / 8 lanes
                const float z = dot + bias;
                const float f = z * __fdividef(1.f, 1.f + __expf(-z));
#pragma unroll
                for (int e = 0; e < 8; e++) acc[i][e] = fmaf(f, v[e], acc[i][e]);
            }
        }
        if (up < 0) break;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            k4[i] = nk4[i];
            v4[i] = nv4[i];
        }
        ts_a = ts_up;
        up = next;
    }
    // the history, split by split, four on their way together
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; i++)
        if (in(i) && nd.w > 0) {
            acc[i][0] += part0[i][0].x; acc[i][1] += part0[i][0].y; acc[i][2] += part0[i][0].z; acc[i][3] += part0[i][0].w;
            acc[i][4] += part0[i][1].x; acc[i][5] += part0[i][1].y; acc[i][6] += part0[i][1].z; acc[i][7] += part0[i][1].w;
        }
    for (int sp = 1; SPLIT && sp < nd.w; sp += 4) {
#pragma unroll
        for (int i = 0; i < NV; i++)
            if (in(i)) {
                float4 x[4][2];
#pragma unroll
                for (int s = 0; s < 4; s++)
                    if (sp + s < nd.w) {
                        const float4* part = reinterpret_cast<const float4*>(p.part + (size_t)(sp + s) * p.T * p.ld + row + col(i));
                        x[s][0] = __ldcs(part);
                        x[s][1] = __ldcs(part + 1);
                    }
#pragma unroll
                for (int s = 0; s < 4; s++)
                    if (sp + s < nd.w) {
                        acc[i][0] += x[s][0].x; acc[i][1] += x[s][0].y; acc[i][2] += x[s][0].z; acc[i][3] += x[s][0].w;
                        acc[i][4] += x[s][1].x; acc[i][5] += x[s][1].y; acc[i][6] += x[s][1].z; acc[i][7] += x[s][1].w;
                    }
            }
    }
#pragma unroll
    for (int i = 0; i < NV; i++)
#pragma unroll
        for (int e = 0; e < 8; e++) {
            acc[i][e] *= p.inv_alpha;
            sum += acc[i][e];
        }
    // sum over the node's warps, in warp order
    auto node_sum = [&](float x, int which) {
        x = warp_sum(x);
        if (WARPS == 1) return x;
        if (lane == 0) s_red[which][warp] = x;
        __syncthreads();
        x = 0.f;
#pragma unroll
        for (int e = 0; e < WARPS; e++) x += s_red[which][warp - w + e];
        return x;
    };
    const float mu = node_sum(sum, 0) / (float)p.ld;
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < NV; i++)
        if (in(i)) {
            if (live) store8(p.y + row + col(i), acc[i]);
#pragma unroll
            for (int e = 0; e < 8; e++) sq = fmaf(acc[i][e] - mu, acc[i][e] - mu, sq);
        }
    const float rstd = rsqrtf(node_sum(sq, 1) / (float)p.ld + p.eps);
#pragma unroll
    for (int i = 0; i < NV; i++)
        if (live && in(i)) {
            float o[8], g[8], b[8], u[8];
            open8(u4[i], u);
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const float4 x = __ldg(reinterpret_cast<const float4*>(p.gamma + col(i)) + e), y = __ldg(reinterpret_cast<const float4*>(p.beta + col(i)) + e);
                g[4 * e] = x.x; g[4 * e + 1] = x.y; g[4 * e + 2] = x.z; g[4 * e + 3] = x.w;
                b[4 * e] = y.x; b[4 * e + 1] = y.y; b[4 * e + 2] = y.z; b[4 * e + 3] = y.w;
            }
#pragma unroll
            for (int e = 0; e < 8; e++)
                o[e] = fmaf((acc[i][e] - mu) * rstd, g[e], b[e]) * u[e];
            store8(p.o + row + col(i), o);
        }
}

// ------------------------------------------------------------------ host
struct TreeWs {
    size_t info, node, items, part, total;
    long long max_items;
    int max_splits, min_tiles, group;
};

// Groups: 64 nodes (narrow) where no tree has more, else 128 (wide).  Whole scorer, narrow / wide:
// 64 trees of one node over 4096 events 94 / 98 us, of 16 100 / 105, of 64 122 / 125; 32 trees of 65
// over 2048 70 / 61, of 128 70 / 63, of 512 178 / 145.
// Parts of a history: where the trees alone give at least four work items an SM, none (the sums
// go through HBM once); else so many that there are about sixteen an SM, of at least min_tiles
// tiles (an item's start costs about two tiles' time), which is eight where the work allows it
// and one for a single short history.  The parts' sums stay within 32 MB, which L2 holds.
// One part always / this rule: one node over 2048 events 25 / 19 us; 16 trees of 1 to 4 over 100 to
// 8192 76 / 64; 8 of 16 over 8192 69 / 39; 64 of one over 4096 to 8192 146 / 133; 48 of 5 to 60 over a
// window of 700 39 / 40.  At least 16 tiles in place of 8: 56 / 48 us for 48 of 5 to 61 over 0 to 2048.
TreeWs tree_ws(const hstu_tree_dims& d, const hstu_page_cache& c) {
    TreeWs w;
    w.group = d.max_nodes <= kNarrow ? kNarrow : kWide;
    const long long full = ((long long)d.T + w.group - 1) / w.group;
    const long long groups = full + d.B;                                    // at most
    const long long whole = d.H * (full > d.B ? full : (long long)d.B);     // at least, where no tree is empty
    const long long tiles = ((long long)c.max_pages * c.page_size + kTileN - 1) / kTileN;
    long long min_tiles = whole * tiles / (148 * 2);
    min_tiles = min_tiles < 1 ? 1 : (min_tiles > 8 ? 8 : min_tiles);
    long long splits = whole < 148 * 4 && whole > 0 ? (148 * 16 + whole - 1) / whole : 1;
    const long long by_size = (32LL << 20) / ((long long)d.T * d.H * d.d * 4 + 1);
    if (splits > by_size) splits = by_size;
    if (splits > (tiles + min_tiles - 1) / min_tiles) splits = (tiles + min_tiles - 1) / min_tiles;
    if (splits < 1) splits = 1;
    w.min_tiles = (int)min_tiles;
    w.max_splits = (int)splits;
    w.max_items = (long long)d.H * groups * splits;
    size_t off = sizeof(Control);
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = align_up(off + bytes, 256);
        return at;
    };
    w.info = take((size_t)d.B * sizeof(TreeInfo));
    w.node = take((size_t)d.T * sizeof(int4));
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

// Dynamic shared-memory limits and SM count, set and read once per device.
int prepare_device(int* sms) {
    static std::mutex mu;
    static int known[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_status(e);
    if (dev < 0 || dev >= 64) return HSTU_ERR_UNSUPPORTED;
    std::lock_guard<std::mutex> lk(mu);
    if (known[dev] == 0) {
        auto limit = [&](const void* fn, uint32_t bytes) {
            if (e == cudaSuccess) e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
        };
        limit((const void*)tree_prep_kernel, 2 * kTreeMaxNodes * sizeof(int));
        limit((const void*)tree_attn_kernel<64, false>, TreeSmem<64, false>::alloc(kMaxPos));
        limit((const void*)tree_attn_kernel<64, true>, TreeSmem<64, true>::alloc(kMaxPos));
        limit((const void*)tree_attn_kernel<128, false>, TreeSmem<128, false>::alloc(kMaxPos));
        limit((const void*)tree_attn_kernel<128, true>, TreeSmem<128, true>::alloc(kMaxPos));
        int n = 0;
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return cuda_status(e);
        known[dev] = n;
    }
    *sms = known[dev];
    return HSTU_OK;
}

template <int D, bool WIDE>
cudaError_t launch_attn(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const TreeParams& p, int grid,
                        cudaStream_t s) {
    return launch_early(tree_attn_kernel<D, WIDE>, grid, kThreads, TreeSmem<D, WIDE>::alloc(p.P), s, tq, tk, tv, p);
}

template <int D, bool SPLIT>
cudaError_t launch_finish(const TreeParams& p, cudaStream_t s) {
    // 256 columns a warp while that gives up to four warps a node, then eight warps
    const int warps = p.ld <= 256 ? 1 : p.ld <= 512 ? 2 : p.ld <= 1024 ? 4 : 8;
    const int per = kFinishThreads / 32 / warps, grid = (p.T + per - 1) / per;
    if (warps == 1) return launch_early(tree_finish_kernel<D, 1, 1, SPLIT>, grid, kFinishThreads, 0, s, p);
    if (warps == 2) return launch_early(tree_finish_kernel<D, 1, 2, SPLIT>, grid, kFinishThreads, 0, s, p);
    if (warps == 4) return launch_early(tree_finish_kernel<D, 1, 4, SPLIT>, grid, kFinishThreads, 0, s, p);
    if (p.ld <= 2048) return launch_early(tree_finish_kernel<D, 1, 8, SPLIT>, grid, kFinishThreads, 0, s, p);
    return launch_early(tree_finish_kernel<D, 4, 8, SPLIT>, grid, kFinishThreads, 0, s, p);
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
        !aligned(rab_pos, 4) || !aligned(rab_time, 4) || !aligned(ln_gamma, 16) || !aligned(ln_beta, 16) ||
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
    p.ps_log = c.page_size == 16 ? 4 : c.page_size == 32 ? 5 : c.page_size == 64 ? 6 : 7;
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
    p.node = reinterpret_cast<int4*>(base + w.node);
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
    p.min_tiles = w.min_tiles;
    p.group = w.group;
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

    int sms = 0;
    const int rc = prepare_device(&sms);
    if (rc != HSTU_OK) return rc;
    // with no page at all no tile is ever loaded; the queries then stand in as the pool
    CUtensorMap tq, tk, tv;
    const bool pool = c.n_pages > 0;
    const long long rows = pool ? (long long)c.n_pages * c.page_size : d.T;
    if (!make_tmap(&tq, node_q, d.T, p.ld, w.group) || !make_tmap(&tk, pool ? c.k : node_q, rows, p.ld, c.page_size) ||
        !make_tmap(&tv, pool ? c.v : node_q, rows, p.ld, c.page_size))
        return HSTU_ERR_CUDA;
    // An ordinary launch, and it has to stay one: the two after it read tables, queries and nodes before
    // their wait, which is right because prep starts only when all earlier work of the stream is done.
    tree_prep_kernel<<<d.B, kPrepThreads, 2 * d.max_nodes * (int)sizeof(int), s>>>(p);
    cudaError_t e = cudaGetLastError();
    const int grid = (int)(w.max_items < sms ? w.max_items : sms);
    const bool wide = w.group == kWide;
    if (e == cudaSuccess)
        e = d.d == 128 ? (wide ? launch_attn<128, true>(tq, tk, tv, p, grid, s) : launch_attn<128, false>(tq, tk, tv, p, grid, s))
                       : (wide ? launch_attn<64, true>(tq, tk, tv, p, grid, s) : launch_attn<64, false>(tq, tk, tv, p, grid, s));
    if (e == cudaSuccess && w.max_splits > 1) e = d.d == 128 ? launch_finish<128, true>(p, s) : launch_finish<64, true>(p, s);
    else if (e == cudaSuccess) e = d.d == 128 ? launch_finish<128, false>(p, s) : launch_finish<64, false>(p, s);
    return cuda_status(e);
}
