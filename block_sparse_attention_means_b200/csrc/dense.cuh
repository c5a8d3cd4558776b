// Operands and sequence bounds of the dense attention kernels.
#pragma once

#include "common.cuh"

namespace park {

struct Op4 {  // element (b, h, n, d) at p + (b sb + h sh + n sn + d) elements
    uint8_t* p;
    long long sb, sh, sn;
};

struct DenseArgs {
    int B, Hq, Hk, D, n_seq, causal;
    long long Nq, Nk;  // rows of a batch entry
    const int32_t *cu_q, *cu_k;
    float scale;
    Op4 q, k, v, o, d_o, dq, dk, dv;
    float* lse;  // [B, Hq, Nq], may be null in the forward pass
    int32_t* status;
};

// How the forward pass cuts its work: rows of a tile, row tiles of a key head, parts that the keys are split into (1:
// none) and the key tiles of a part; workspace for the parts.
struct DenseSplit {
    int rows;
    long long tiles;
    int n, chunk;
    size_t lse_off, bytes;
};
// How the kernel of dk and dv cuts its work: key tiles, parts that the steps (row tiles of all heads of a group) are split
// into (1: none), steps of a part; float32 workspace of the parts, dk after dv.
struct DkvSplit {
    long long tiles;
    int n, chunk;
    size_t dk_off, bytes;
};
constexpr int kDenseSMs = 148;  // SMs of a B200

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// The piece of work of one block: `tile`-th tile of a sequence.
struct SeqTile {
    int q0, nq, k0, nk, tile;  // first rows within the batch entry, rows, tile within the sequence
    int live;                  // 0: nothing to do
};

// Most tiles that the sequences can have: a packed batch holds at most
// N / tile + n_seq of them.
__host__ inline long long dense_tiles(long long n, int n_seq, int tile) {
    return n_seq > 0 ? n / tile + n_seq : (n + tile - 1) / tile;
}

// Tile x (of `rows` rows, counted along the queries, a query row counted `rep` times, or along the keys) -> sequence and
// tile.  Called by one whole warp; packed bounds are read 128 sequences at a time.  Bounds that are not 0 <= cu[s] <=
// cu[s+1] <= N make the sequence empty and set the status word.
__device__ inline SeqTile dense_resolve(const DenseArgs& a, int x, int rows, bool by_keys, int rep) {
    SeqTile t;
    if (a.n_seq == 0) {
        t.q0 = t.k0 = 0;
        t.nq = (int)a.Nq;
        t.nk = (int)a.Nk;
        t.tile = x;
        t.live = 1;
        return t;
    }
    constexpr int U = 4;  // sequences of a lane
    const int lane = threadIdx.x & 31;
    t.q0 = t.nq = t.k0 = t.nk = t.tile = t.live = 0;
    int before = 0;  // tiles of the sequences before this step's
    for (int s0 = 0; s0 < a.n_seq; s0 += 32 * U) {
        int q[U + 1], k[U + 1], nt[U], sum = 0;
        const int first = s0 + lane * U;
#pragma unroll
        for (int u = 0; u <= U; ++u) {
            q[u] = first + u <= a.n_seq ? a.cu_q[first + u] : 0;
            k[u] = first + u <= a.n_seq ? a.cu_k[first + u] : 0;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            nt[u] = 0;
            if (first + u < a.n_seq) {
                if (q[u] < 0 || q[u + 1] < q[u] || q[u + 1] > a.Nq || k[u] < 0 || k[u + 1] < k[u] || k[u + 1] > a.Nk) {
                    set_status(a.status, PARK_ERR_INDEX);
                } else {
                    const long long n = by_keys ? k[u + 1] - k[u] : (long long)(q[u + 1] - q[u]) * rep;
                    nt[u] = (int)((n + rows - 1) / rows);
                }
            }
            sum += nt[u];
        }
        int pre = sum;  // inclusive prefix over the lanes
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, pre, o);
            if (lane >= o) pre += v;
        }
        const int at = before + pre - sum;
        const unsigned hit = __ballot_sync(0xffffffffu, x >= at && x < at + sum);
        if (hit) {
            int e = x - at, q0 = 0, q1 = 0, k0 = 0, k1 = 0, tile = -1;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (tile < 0 && e < nt[u]) {
                    q0 = q[u];
                    q1 = q[u + 1];
                    k0 = k[u];
                    k1 = k[u + 1];
                    tile = e;
                }
                e -= nt[u];
            }
            const int src = __ffs(hit) - 1;
            t.q0 = __shfl_sync(0xffffffffu, q0, src);
            t.nq = __shfl_sync(0xffffffffu, q1, src) - t.q0;
            t.k0 = __shfl_sync(0xffffffffu, k0, src);
            t.nk = __shfl_sync(0xffffffffu, k1, src) - t.k0;
            t.tile = __shfl_sync(0xffffffffu, tile, src);
            t.live = 1;
            return t;
        }
        before += __shfl_sync(0xffffffffu, pre, 31);
    }
    return t;
}

// The x-th tile of a packed batch of at most 32 sequences in the order of falling work (key tiles of a row tile, row tiles of
// a key tile), so that the last CTAs to start are the shortest.  One lane for each sequence; a binary search finds the
// work C of tile x from how many tiles have more.
__device__ inline SeqTile dense_resolve_ranked(const DenseArgs& a, int x, int rows, bool by_keys, int rep) {
    constexpr int KT = 128;  // keys that count as one unit of a row tile's work
    const int lane = threadIdx.x & 31;
    int q0 = 0, nq = 0, k0 = 0, nk = 0;
    if (lane < a.n_seq) {
        const int qb = a.cu_q[lane + 1], kb = a.cu_k[lane + 1];
        q0 = a.cu_q[lane];
        k0 = a.cu_k[lane];
        nq = qb - q0;
        nk = kb - k0;
        if (q0 < 0 || qb < q0 || qb > a.Nq || k0 < 0 || kb < k0 || kb > a.Nk) {
            set_status(a.status, PARK_ERR_INDEX);
            q0 = k0 = nq = nk = 0;
        }
    }
    const int off = nk - nq, end = (nq + rows - 1) / rows;
    const int nt = by_keys ? (nk + rows - 1) / rows : (int)(((long long)nq * rep + rows - 1) / rows);
    // tiles of this lane's sequence with more work than C
    auto more = [&](int C) -> int {
        if (C < 0) return nt;
        if (by_keys) {
            if (C >= end) return 0;
            if (!a.causal) return nt;
            const long long v = (long long)(end - C) * rows + off;
            return v <= 0 ? 0 : (int)min((long long)nt, (v + rows - 1) / rows);
        }
        if (nk <= (long long)KT * C) return 0;
        if (!a.causal) return nt;
        const int z = KT * C - off;  // first row that sees more than C tiles of keys
        return z <= 0 ? nt : (z >= nq ? 0 : nt - (int)((long long)z * rep / rows));
    };
    int lo = 0, hi = __reduce_max_sync(0xffffffffu, by_keys ? end : (nk + KT - 1) / KT);
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (__reduce_add_sync(0xffffffffu, more(mid)) <= x)
            hi = mid;
        else
            lo = mid + 1;
    }
    const int above = more(lo), here = more(lo - 1) - above;  // tiles with more work, tiles with this work
    const int e = x - __reduce_add_sync(0xffffffffu, above);
    int pre = here;  // inclusive prefix over the lanes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, pre, o);
        if (lane >= o) pre += v;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, e >= pre - here && e < pre);
    SeqTile t;
    t.q0 = t.nq = t.k0 = t.nk = t.tile = t.live = 0;
    if (!hit) return t;
    const int src = __ffs(hit) - 1;
    t.q0 = __shfl_sync(0xffffffffu, q0, src);
    t.nq = __shfl_sync(0xffffffffu, nq, src);
    t.k0 = __shfl_sync(0xffffffffu, k0, src);
    t.nk = __shfl_sync(0xffffffffu, nk, src);
    t.tile = __shfl_sync(0xffffffffu, e - (pre - here) + (by_keys ? above : nt - above - here), src);
    t.live = 1;
    return t;
}

// Order of the blocks: `heads` (batch entries times heads) in groups of `group`; within a group the tiles by falling work,
// each for all heads of the group.  CTAs start in this order, so the last to start are short ones of the last group (head
// after head instead, the last head's long tiles start last).
struct DenseOrder {
    int tiles, heads, group;
};
// Where tiles differ in work, groups of alike size whose other side (keys for row tiles, rows for key tiles: `bytes` for each
// `share` heads) takes at most 128 MB together, about the L2; else head after head.  16,384 causal x 8 heads: 513 us head after
// head, 449 in one group.  Seven packed sequences, 41,331 rows: 2.62 ms in groups of 64 MB, 2.66 of 128, 2.71 of 256; the
// dk/dv kernel of a packed batch that needs 76 MB: 0.67 ms in groups of 64 MB, 0.51 of 128.
__host__ inline DenseOrder dense_order(const DenseArgs& a, long long tiles, int heads, long long bytes, int share) {
    DenseOrder o;
    o.tiles = (int)tiles;
    o.heads = heads;
    o.group = 1;
    if (a.causal || a.n_seq > 1) {
        const long long units = heads / share, fit = (128ll << 20) / (bytes > 0 ? bytes : 1);
        const long long groups = fit >= units ? 1 : (units + (fit > 1 ? fit : 1) - 1) / (fit > 1 ? fit : 1);
        o.group = (int)((units + groups - 1) / groups) * share;
    }
    return o;
}
// This block's head, and (one whole warp) its tile.
__device__ __forceinline__ int dense_block_head(const DenseOrder& o, int& x) {
    const int per = o.tiles * o.group, grp = blockIdx.x / per, r = blockIdx.x - grp * per;
    const int n = min(o.group, o.heads - grp * o.group);
    x = r / n;
    return grp * o.group + (r - x * n);
}
__device__ inline SeqTile dense_block_tile(const DenseArgs& a, const DenseOrder& o, int x, int rows, bool by_keys, int rep) {
    if (a.n_seq > 1 && a.n_seq <= 32) return dense_resolve_ranked(a, x, rows, by_keys, rep);
    // (causal: the last rows see the most keys, the first keys are seen by the most rows)
    return dense_resolve(a, by_keys ? x : o.tiles - 1 - x, rows, by_keys, rep);
}

// Row tiles (of `tile` rows) first .. end-1 of each head that see a key of the key tile starting at j0.
__device__ __forceinline__ void dense_row_tiles(const SeqTile& t, int j0, int causal, int tile, int& first, int& end) {
    first = causal ? max(0, j0 - (t.nk - t.nq)) / tile : 0;
    end = max(first, (t.nq + tile - 1) / tile);
}

// Keys that row i of a sequence sees: 0 .. dense_last_key (may be negative).
__device__ __forceinline__ int dense_last_key(int i, int nq, int nk, int causal) {
    return causal ? min(nk - 1, i + (nk - nq)) : nk - 1;
}

}  // namespace park
