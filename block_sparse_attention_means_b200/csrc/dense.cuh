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

// Tile x (of `rows` rows, counted along the queries or the keys, a query row
// counted `rep` times) -> sequence and tile.  Called by one whole warp; packed bounds are read 32
// sequences at a time.  Bounds that are not 0 <= cu[s] <= cu[s+1] <= N make
// the sequence empty and set the status word.
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
    const int lane = threadIdx.x & 31;
    t.q0 = t.nq = t.k0 = t.nk = t.tile = t.live = 0;
    int before = 0;  // tiles of the sequences before this step's
    for (int s0 = 0; s0 < a.n_seq; s0 += 32) {
        const int s = s0 + lane;
        int qa = 0, qb = 0, ka = 0, kb = 0;
        if (s < a.n_seq) {
            qa = a.cu_q[s];
            qb = a.cu_q[s + 1];
            ka = a.cu_k[s];
            kb = a.cu_k[s + 1];
            if (qa < 0 || qb < qa || qb > a.Nq || ka < 0 || kb < ka || kb > a.Nk) {
                set_status(a.status, PARK_ERR_INDEX);
                qb = qa = kb = ka = 0;
            }
        }
        const long long n = by_keys ? kb - ka : (long long)(qb - qa) * rep;
        const int nt = (int)((n + rows - 1) / rows);
        int pre = nt;  // inclusive prefix over the lanes
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, pre, o);
            if (lane >= o) pre += v;
        }
        const int first = before + pre - nt;
        const unsigned hit = __ballot_sync(0xffffffffu, x >= first && x < first + nt);
        if (hit) {
            const int src = __ffs(hit) - 1;
            t.q0 = __shfl_sync(0xffffffffu, qa, src);
            t.nq = __shfl_sync(0xffffffffu, qb, src) - t.q0;
            t.k0 = __shfl_sync(0xffffffffu, ka, src);
            t.nk = __shfl_sync(0xffffffffu, kb, src) - t.k0;
            t.tile = x - __shfl_sync(0xffffffffu, first, src);
            t.live = 1;
            return t;
        }
        before += __shfl_sync(0xffffffffu, pre, 31);
    }
    return t;
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
