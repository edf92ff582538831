// hstu_rules.cuh -- integer rules of jagged HSTU attention, as device functions.
//
// Every kernel (forward, backward, M-FALCON, the debug hook) takes its mask,
// relative-position index and time bucket from these functions, so the debug
// hook's output is exactly what the fused kernels use.
//
//   rab^{p,t} (Meta HSTU blog, section 3.2): a relative position bias plus a
//   time bias.  pidx = clamp(pos_j - pos_i, -(P-1), P-1) + (P-1);
//   bucket = min(nb-1, bit_length(|ts_i - ts_j|)).
//   MTGR dynamic mixed mask (MTGR deep-dive, section 2; MTGR arXiv report,
//   section 3.1): static tokens bidirectional, real-time causal, candidates
//   see themselves plus non-candidates with a strictly earlier timestamp.
//   Full-sequence M-FALCON (HSTU blog, section 4.2): [history ; candidates] in
//   one row, history causal, every candidate sees all history and itself (no
//   timestamp filter); it is the MTGR layout with no static part.
//   Window with sinks: token i sees token j <= i when i - j < R (the window) or
//   j < S (the first S tokens of the row, the sinks); positions are indices.
#pragma once
#include <stdint.h>

#define HSTU_KIND_CAUSAL 0
#define HSTU_KIND_MTGR 1
#define HSTU_KIND_MFALCON 2
#define HSTU_KIND_MFSEQ 3
#define HSTU_KIND_WINDOW 4

namespace hstu {

// Segment sizes of row b: S static tokens, R real-time / history tokens, the rest candidates.
// Window rows: S sinks and a window of R tokens (neither is bounded by the row's length).
__device__ __forceinline__ void segment_sizes(int kind, const int32_t* n_static, const int32_t* n_rt, int b,
                                              int L, int* S, int* R) {
    if (kind == HSTU_KIND_MTGR || kind == HSTU_KIND_WINDOW) {
        *S = n_static[b];
        *R = n_rt[b];
    } else if (kind == HSTU_KIND_MFSEQ) {
        *S = 0;
        *R = n_rt[b];
    } else {
        *S = L;
        *R = 0;
    }
}

// 0 static, 1 real-time, 2 candidate (MTGR rows); causal rows are all "static-causal".
__device__ __forceinline__ int token_class(int i, int S, int R) {
    return i < S ? 0 : (i < S + R ? 1 : 2);
}

// Position used by rab_pos.  MTGR candidates share the slot right after the history.
__device__ __forceinline__ int token_pos(int kind, int i, int S, int R) {
    return ((kind == HSTU_KIND_MTGR || kind == HSTU_KIND_MFSEQ) && i >= S + R) ? S + R : i;
}

__device__ __forceinline__ int pos_index(int pos_i, int pos_j, int P) {
    int dp = pos_j - pos_i;
    dp = max(dp, -(P - 1));
    dp = min(dp, P - 1);
    return dp + (P - 1);
}

// |a - b| of two int64 values without overflow.
__device__ __forceinline__ uint64_t abs_diff_u64(int64_t a, int64_t b) {
    return a >= b ? (uint64_t)a - (uint64_t)b : (uint64_t)b - (uint64_t)a;
}

// Bit length of |ts_i - ts_j| capped at nb-1 (bit_length(0) = 0).
__device__ __forceinline__ int time_bucket_of_delta(uint64_t d, int nb) {
    int bl = 64 - __clzll((long long)d);
    return min(bl, nb - 1);
}

__device__ __forceinline__ int time_bucket(int64_t ti, int64_t tj, int nb) {
    return time_bucket_of_delta(abs_diff_u64(ti, tj), nb);
}

// Mask of causal, window, MTGR and full-sequence M-FALCON rows (i, j local to the sequence).
__device__ __forceinline__ bool visible(int kind, int i, int j, int S, int R, int64_t ts_i,
                                        int64_t ts_j) {
    if (kind == HSTU_KIND_CAUSAL) return j <= i;
    if (kind == HSTU_KIND_WINDOW) return j <= i && (i - j < R || j < S);
    int ci = token_class(i, S, R), cj = token_class(j, S, R);
    if (ci == 0) return cj == 0;
    if (ci == 1) return cj == 0 || (cj == 1 && j <= i);
    return j == i || (cj != 2 && (kind == HSTU_KIND_MFSEQ || ts_j < ts_i));
}

// Tile-level classification of a (query tile, key tile) pair from segment
// sizes alone.  Rows [qa, qb] and columns [ka, kb] are clipped to [0, L).
// Returns 0 when no pair can be visible, 1 when some may be (evaluate the
// mask per element), 2 when every pair with j < L is visible.
// MTGR candidate rows against history are "partial": their timestamp filter is
// applied per element; full-sequence M-FALCON candidates see all history.
__device__ __forceinline__ int tile_class(int kind, int qa, int qb, int ka, int kb, int S, int R) {
    if (kind == HSTU_KIND_CAUSAL) {
        if (ka > qb) return 0;
        return (kb <= qa) ? 2 : 1;
    }
    if (kind == HSTU_KIND_MFALCON) return 2;
    if (kind == HSTU_KIND_WINDOW) {
        if (ka > qb) return 0;
        if (ka >= S && max(qa - kb, 0) >= R) return 0;          // past the sinks, before every row's window
        return kb <= qa && (kb < S || qb - ka < R) ? 2 : 1;
    }
    const int H = S + R;
    bool any = false;
    // static rows see static columns
    if (qa < S && ka < S) any = true;
    // real-time rows: static columns, or real-time columns up to the row
    int rlo = max(qa, S), rhi = min(qb, H - 1);
    if (rlo <= rhi) {
        if (ka < S) any = true;
        if (kb >= S && ka <= rhi && ka < H) any = true;
    }
    // candidate rows: themselves, and (timestamp-filtered) history
    int clo = max(qa, H), chi = qb;
    if (clo <= chi) {
        if (ka < H) any = true;
        if (max(clo, ka) <= min(chi, kb)) any = true;
    }
    if (!any) return 0;
    // full tiles: every column static and every row a non-candidate (static rows see
    // all static tokens, real-time rows too), or every row real-time and every column
    // at or before the first row (static or earlier real-time)
    if (kb < S && qb < H) return 2;
    if (qa >= S && qb < H && kb <= qa) return 2;
    if (kind == HSTU_KIND_MFSEQ && qa >= H && kb < H) return 2;   // candidates x history: no filter
    return 1;
}

// Backward of window rows: the sinks' key tile (keys 0 .. 127) is seen by every query of the
// sequence, however long, where other key tiles are seen by a window's worth.  Its queries
// are worked in chunks of kSinkChunk 128-query tiles, an item each, whose dK and dV meet in a
// sum of their own.  Sequences of one chunk and more than 128 sinks are not cut.  Whole layer
// backward, 4 sinks and a window of 64, uncut / 16 / 8 / 4 tiles: one sequence of 4096, one head
// of 128: 193 / 120 / 80 / 60 us; 8 of 2048, 4 heads: 195 / 195 / 174 / 160; 1 of 16384, 4 heads:
// 725 / 202 / 167 / 157.
constexpr int kSinkChunk = 4;

__device__ __forceinline__ int sink_chunks(int L, int S) {
    const int n = (L + 128 * kSinkChunk - 1) / (128 * kSinkChunk);
    return S >= 1 && S <= 128 && n > 1 ? n : 1;
}

// Whether any query of chunk k sees key r of the first key tile (past the window only the sinks
// are seen, and the chunk's sums of the other keys are neither written nor read).
__device__ __forceinline__ bool sink_chunk_sees(int k, int r, int S, int R) {
    return r < S || 128 * kSinkChunk * k - r < R;
}

// First place of a cut sequence's chunks in the partial sums: a sequence of more than 512
// tokens has at most L / 512 + 1 chunks, so two places for each 512 tokens before it keep
// the sequences apart.
__device__ __forceinline__ int sink_place(int off) { return 2 * (off / (128 * kSinkChunk)); }

}  // namespace hstu
