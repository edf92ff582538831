// schedule.cu -- device-side work list for the persistent attention kernels.
//
// One CTA validates the jagged offsets (and MTGR segment sizes), sorts the
// sequences by their number of key tiles (longest first, counting sort) and
// writes one work item per (sequence, head, query tile).  The items of one
// (sequence, head) are adjacent, so the CTAs that run them at the same time
// share that sequence's K/V tiles through L2; inside a group the heaviest
// query tile comes first.  Jagged, padding-free batches are the layout the
// MTGR pages describe (JaggedTensor + variable-length HSTU operator; the
// token-balanced batching of MTGR's training system motivates the sort).
#include "internal.h"

namespace hstu {

namespace {

constexpr int kThreads = 1024;

__device__ int n_q_tiles(const SchedParams& p, int Lq) {
    if (Lq <= 0) return 0;
    if (p.kind != HSTU_KIND_MFALCON) return (Lq + kTileM - 1) / kTileM;
    const int tpm = (p.b_m + kTileM - 1) / kTileM;     // tiles per full microbatch
    const int n_mb = (Lq + p.b_m - 1) / p.b_m;
    const int last = Lq - (n_mb - 1) * p.b_m;
    return (n_mb - 1) * tpm + (last + kTileM - 1) / kTileM;
}

// rows [row0, row_end) of query tile k (tile order inside a (sequence, head) group)
__device__ void tile_rows(const SchedParams& p, int Lq, int nt, int k, int* row0, int* row_end) {
    if (p.kind != HSTU_KIND_MFALCON) {
        const int t = p.ascending ? k : nt - 1 - k;      // heaviest tile first
        *row0 = t * kTileM;
        *row_end = min(*row0 + kTileM, Lq);
        return;
    }
    const int tpm = (p.b_m + kTileM - 1) / kTileM;
    const int mb = k / tpm, w = k % tpm;
    *row0 = mb * p.b_m + w * kTileM;
    *row_end = min(*row0 + kTileM, min((mb + 1) * p.b_m, Lq));
}

__device__ int block_exclusive_scan(int v, int* warp_sums, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int s = warp_sums[lane];
        int t = s;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            int y = __shfl_up_sync(0xffffffffu, t, o);
            if (lane >= o) t += y;
        }
        warp_sums[lane] = t - s;
        if (lane == 31) *total = t;
    }
    __syncthreads();
    int r = warp_sums[warp] + x - v;
    __syncthreads();
    return r;
}

// Blocks that clear p.zero, one an SM beside the schedule's: the schedule takes one SM for 4 us,
// in which the others write what two memsets took 2 x 1.5 us and more for (22000 tokens of 512,
// schedule and memsets 4.8 + 6.8 -> 7.6 us).
constexpr long long kZeroBlocks = 147;

// No loop is unrolled: each runs once or twice in a batch of a thousand sequences, and what a
// kernel this short takes is to a good part the fetch of its code (4.5 -> 4.0 us).
__global__ void __launch_bounds__(kThreads) schedule_kernel(SchedParams p) {
    __shared__ int hist[kSchedBins];
    __shared__ int warp_sums[32];
    __shared__ int s_total;
    __shared__ int s_carry;

    const int tid = threadIdx.x;
    allow_next_launch();
    if (blockIdx.x > 0) {
        const long long step = (long long)(gridDim.x - 1) * kThreads;
#pragma unroll 1
        for (long long i = (blockIdx.x - 1LL) * kThreads + tid; i < p.n_zero; i += step) p.zero[i] = make_uint4(0, 0, 0, 0);
        return;
    }
#pragma unroll 1
    for (int i = tid; i < kSchedBins; i += kThreads) hist[i] = 0;
    if (tid == 0) {
        p.ctrl->counter = 0;
        s_carry = 0;
    }

    // ---- 1. validate
    int bad = 0;
    if (tid == 0) {
        if (p.q_off[0] != 0 || p.q_off[p.B] != p.Tq) bad = 1;
        if (p.kv_off != p.q_off && (p.kv_off[0] != 0 || p.kv_off[p.B] != p.Tkv)) bad = 1;
    }
#pragma unroll 1
    for (int b = tid; b < p.B; b += kThreads) {
        const int Lq = p.q_off[b + 1] - p.q_off[b];
        if (Lq < 0 || Lq > p.max_q_len) bad = 1;
        if (p.kv_off != p.q_off) {
            const int Lk = p.kv_off[b + 1] - p.kv_off[b];
            if (Lk < 0 || Lk > p.max_kv_len) bad = 1;
        }
        if (p.kind == HSTU_KIND_MTGR || p.kind == HSTU_KIND_MFSEQ) {
            int S = 0, R = 0;
            segment_sizes(p.kind, p.n_static, p.n_rt, b, Lq, &S, &R);
            if (S < 0 || R < 0 || (long long)S + R > Lq) bad = 1;
        }
        if (p.kind == HSTU_KIND_WINDOW && (p.n_static[b] < 0 || p.n_rt[b] < 0)) bad = 1;
    }
    if (__syncthreads_or(bad)) {
        if (tid == 0) {
            atomicOr(&p.ctrl->status, kStatusBounds);
            p.ctrl->n_items = 0;
            p.ctrl->valid = 0;
        }
        return;
    }

    // ---- 2. counting sort of sequences by key-tile count, longest first
#pragma unroll 1
    for (int b = tid; b < p.B; b += kThreads) {
        const int Lk = p.kv_off[b + 1] - p.kv_off[b];
        const int key = min((Lk + kTileN - 1) / kTileN, kSchedBins - 1);
        atomicAdd(&hist[kSchedBins - 1 - key], 1);
    }
    __syncthreads();
    // exclusive scan over bins (4 bins per thread)
    {
        int v[4], s = 0;
#pragma unroll
        for (int e = 0; e < 4; e++) {
            v[e] = hist[tid * 4 + e];
            s += v[e];
        }
        int base = block_exclusive_scan(s, warp_sums, &s_total);
#pragma unroll
        for (int e = 0; e < 4; e++) {
            hist[tid * 4 + e] = base;
            base += v[e];
        }
    }
    __syncthreads();
#pragma unroll 1
    for (int b = tid; b < p.B; b += kThreads) {
        const int Lk = p.kv_off[b + 1] - p.kv_off[b];
        const int key = min((Lk + kTileN - 1) / kTileN, kSchedBins - 1);
        const int pos = atomicAdd(&hist[kSchedBins - 1 - key], 1);
        p.perm[pos] = b;
    }
    __syncthreads();

    // ---- 3. item base of every ranked sequence
#pragma unroll 1
    for (int r0 = 0; r0 < p.B; r0 += kThreads) {
        const int r = r0 + tid;
        int nt = 0;
        if (r < p.B) {
            const int b = p.perm[r];
            const int L = p.q_off[b + 1] - p.q_off[b];
            nt = n_q_tiles(p, L) + (p.cut ? sink_chunks(L, p.n_static[b]) - 1 : 0);
        }
        const int ex = block_exclusive_scan(nt, warp_sums, &s_total);
        if (r < p.B) p.seq_base[r] = s_carry + ex;
        __syncthreads();
        if (tid == 0) s_carry += s_total;
        __syncthreads();
    }
    const long long total_tiles = s_carry;
    if (total_tiles * p.H > p.max_items) {
        if (tid == 0) {
            atomicOr(&p.ctrl->status, kStatusBounds);
            p.ctrl->n_items = 0;
            p.ctrl->valid = 0;
        }
        return;
    }

    // ---- 4. items: (ranked sequence, head, tile)
    const int warp = tid >> 5, lane = tid & 31;
#pragma unroll 1
    for (int r = warp; r < p.B; r += kThreads / 32) {
        const int b = p.perm[r];
        const int Lq = p.q_off[b + 1] - p.q_off[b];
        const int nc = p.cut ? sink_chunks(Lq, p.n_static[b]) : 1;
        const int nt = n_q_tiles(p, Lq) + nc - 1;
        const long long base = (long long)p.seq_base[r] * p.H;
#pragma unroll 1
        for (int e = lane; e < nt * p.H; e += 32) {
            const int h = e / nt, k = e % nt;
            int row0, row_end;
            if (nc > 1) {
                // chunk k of the first key tile, then the other key tiles
                const int t = max(k - nc + 1, 0);
                p.items[base + e] = make_int4(b, t * kTileM, k < nc ? h | (k + 1) << 8 : h, min((t + 1) * kTileM, Lq));
                continue;
            }
            tile_rows(p, Lq, nt, k, &row0, &row_end);
            p.items[base + e] = make_int4(b, row0, h, row_end);
        }
    }
    if (tid == 0) {
        p.ctrl->n_items = (int)(total_tiles * p.H);
        p.ctrl->valid = 1;
    }
}

}  // namespace

cudaError_t launch_schedule(const SchedParams& p, cudaStream_t s) {
    // block 0 schedules; the others, one wave of them, clear p.zero
    const long long blocks = (p.n_zero + kThreads - 1) / kThreads;
    prof_begin(kProfSchedule, s);
    schedule_kernel<<<1 + (unsigned)(blocks < kZeroBlocks ? blocks : kZeroBlocks), kThreads, 0, s>>>(p);
    prof_end(kProfSchedule, s);
    return cudaGetLastError();
}

}  // namespace hstu
