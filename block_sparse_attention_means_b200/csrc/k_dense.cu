// Dense attention of float32 tensors, forward and backward, and the row sums
// delta_i = sum_d do_id o_id that the backward pass of either type starts with.
//
// Forward: one pass over the keys with the running maximum m and sum l of the
// Softmax,  o <- o 2^(m - m') + p v.  Backward in two kernels that form the
// scores again, one owning 64 query rows (dq) and one owning 64 key rows (dk, dv,
// summed over the query heads of the group): every sum has one owner and a fixed
// order, no atomics.
//   p = exp(s - lse),  ds = p (do v^T - delta),  dq = scale ds k,
//   dk = scale ds^T q,  dv = p^T do
//
// Bound by the FMA units and the shared-memory reads that feed them: tiles of 64 keys,
// R x 4 scores and R x D/16 outputs a thread (R = 8, 4 or 1 rows; 4 in the backward
// kernels), products in packed pairs; tiles stay in shared memory (row pitch D + 4
// floats: the 16 key rows that a half-warp reads with 16-byte loads hit all banks
// once) and the next ones are fetched beside the arithmetic.
// Tiles that a mask cuts take a variant whose products skip the hidden pairs, so
// that an infinity or NaN there stays out of the sums.
#include "dense.cuh"
#include "kernels.h"

namespace park {
namespace {

constexpr int TB = 64;          // query rows and key rows of a tile
constexpr int PP = TB + 4;      // row pitch of a probability tile

__device__ __forceinline__ float4 load4(const uint8_t* p, int i) {
    return *reinterpret_cast<const float4*>(p + 16 * (size_t)i);
}
// rows 0 .. n-1 of `src` (row stride in elements) into a [ROWS][D + 4] tile, zeros below
template <int D, int ROWS, int NT = 256>
__device__ __forceinline__ void load_tile(float* dst, const uint8_t* src, long long stride, int n) {
    constexpr int C = D / 4;
    for (int i = threadIdx.x; i < ROWS * C; i += NT) {
        const int r = i / C, c = i - r * C;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < n) v = load4(src + r * stride * 4, c);
        *reinterpret_cast<float4*>(dst + r * (D + 4) + 4 * c) = v;
    }
}

// The same, asynchronous: one group of copies, rows from n on as zeros.  Nothing is read for n <= 0.
template <int D, int NT = 256>
__device__ __forceinline__ void fetch_tile(float* dst, const uint8_t* src, long long stride, int n) {
    constexpr int C = D / 4;
    const uint32_t d0 = (uint32_t)__cvta_generic_to_shared(dst);
    for (int i = threadIdx.x; i < TB * C; i += NT) {
        const int r = i / C, c = i - r * C;
        const bool on = r < n;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d0 + (r * (D + 4) + 4 * c) * 4),
                     "l"(on ? src + r * stride * 4 + 16 * c : src), "r"(on ? 16 : 0)
                     : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
}
// The oldest group has landed: all but the newest N groups are waited for.
template <int N>
__device__ __forceinline__ void landed() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
    __syncthreads();
}

// s[i][j] = A[R ty + i] . B[tx + 16 j], even and odd elements in the halves of packed sums
template <int D, int R>
__device__ __forceinline__ void dot_tile(float (&s)[R][4], const float* A, const float* Bm, int ty, int tx) {
    float2 t[R][4];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) t[i][j] = make_float2(0.f, 0.f);
#pragma unroll(R > 4 ? 1 : 2)
    for (int d = 0; d < D; d += 4) {
        float4 b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4*>(Bm + (tx + 16 * j) * (D + 4) + d);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float4 a = *reinterpret_cast<const float4*>(A + (R * ty + i) * (D + 4) + d);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                t[i][j] = __ffma2_rn(make_float2(a.x, a.y), make_float2(b[j].x, b[j].y), t[i][j]);
                t[i][j] = __ffma2_rn(make_float2(a.z, a.w), make_float2(b[j].z, b[j].w), t[i][j]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = t[i][j].x + t[i][j].y;
}

// acc[i][c] += sum_k P[R ty + i][k] B[k][cols 2 tx + 32 c, + 1].  With MASK only pairs that see(row, k) allows enter.
template <int D, int R, bool MASK, typename F>
__device__ __forceinline__ void accumulate(float2 (&acc)[R][D / 32], const float* P, const float* Bm, int ty, int tx,
                                           F see, int k0 = 0, int k1 = TB) {
#pragma unroll 1
    for (int k = k0; k < k1; k += 4) {
        float4 p[R];
#pragma unroll
        for (int i = 0; i < R; ++i) p[i] = *reinterpret_cast<const float4*>(P + (R * ty + i) * PP + k);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            float2 b[D / 32];
#pragma unroll
            for (int c = 0; c < D / 32; ++c)
                b[c] = *reinterpret_cast<const float2*>(Bm + (k + kk) * (D + 4) + 2 * tx + 32 * c);
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const float pv = kk == 0 ? p[i].x : kk == 1 ? p[i].y : kk == 2 ? p[i].z : p[i].w;
                if (!MASK || see(R * ty + i, k + kk)) {
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) acc[i][c] = __ffma2_rn(make_float2(pv, pv), b[c], acc[i][c]);
                }
            }
        }
    }
}

__device__ __forceinline__ void store2(uint8_t* row, int col, float x, float y) {
    *reinterpret_cast<float2*>(row + 4 * col) = make_float2(x, y);
}

template <typename T>
__device__ __forceinline__ void store4(uint8_t* row, int i, float4 v) {
    if (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(row + 16 * i) = v;
    } else {
        const __nv_bfloat162 x = __floats2bfloat162_rn(v.x, v.y), y = __floats2bfloat162_rn(v.z, v.w);
        *reinterpret_cast<uint2*>(row + 8 * i) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
    }
}

template <typename T>
__device__ __forceinline__ uint8_t* row_ptr(const Op4& o, int b, int h, long long n) {
    return o.p + (b * o.sb + h * o.sh + n * o.sn) * (long long)sizeof(T);
}

__device__ __forceinline__ SeqTile resolve_block(const DenseArgs& a, const DenseOrder& o, int x, int rows, bool by_keys,
                                                 int rep) {
    __shared__ SeqTile sh;
    if (threadIdx.x < 32) {
        const SeqTile t = dense_block_tile(a, o, x, rows, by_keys, rep);
        if (threadIdx.x == 0) sh = t;
    }
    __syncthreads();
    return sh;
}

// Forward: 16 R rows of a sequence (counted token by token, the heads that share a key head side by side) and a part of
// its keys.  With several parts each writes its normalised o and its log2-sum, joined by k_dense_combine.
template <int D, int R>
__global__ void __launch_bounds__(256, D <= 64 || R == 1 ? 2 : 1)
    k_dense_fwd_simt(DenseArgs a, DenseOrder order, int n_split, int chunk, float* __restrict__ part_o, float* __restrict__ part_lse) {
    constexpr int BM = 16 * R;
    extern __shared__ __align__(16) float smem[];
    float* Qs = smem;
    float* Ks = Qs + BM * (D + 4);
    float* Vs = Ks + TB * (D + 4);
    float* Ps = Vs + TB * (D + 4);
    const int G = a.Hq / a.Hk;
    int x;
    const int bh = dense_block_head(order, x), b = bh / a.Hk, hk = bh - b * a.Hk, sp = blockIdx.z;
    const SeqTile t = resolve_block(a, order, x, BM, false, G);
    const int r0 = t.tile * BM;
    if (!t.live || r0 >= t.nq * G) return;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int rows = min(BM, t.nq * G - r0);
    {
        constexpr int C = D / 4;
        for (int i = tid; i < BM * C; i += 256) {
            const int r = i / C, c = i - r * C;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < rows) {
                const int tok = (r0 + r) / G, h = hk * G + (r0 + r - tok * G);
                v = load4(row_ptr<float>(a.q, b, h, t.q0 + tok), c);
            }
            *reinterpret_cast<float4*>(Qs + r * (D + 4) + 4 * c) = v;
        }
    }
    float2 acc[R][D / 32];
    float m[R], l[R];
    int last[R];  // last visible key of each row
#pragma unroll
    for (int i = 0; i < R; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
        last[i] = dense_last_key(min(r0 + R * ty + i, t.nq * G - 1) / G, t.nq, t.nk, a.causal);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) acc[i][c] = make_float2(0.f, 0.f);
    }
    const float sl2 = a.scale * kLog2e;
    const int least = dense_last_key(r0 / G, t.nq, t.nk, a.causal);  // of the first row
    int j_lo = 0, kend = dense_last_key((r0 + rows - 1) / G, t.nq, t.nk, a.causal) + 1;  // keys that any row sees
    if (n_split > 1) {
        j_lo = sp * chunk * TB;
        kend = min(kend, j_lo + chunk * TB);
    }
    auto key = [&](const Op4& o, int j) { return row_ptr<float>(o, b, hk, t.k0 + min(j, t.nk - 1)); };
    if (j_lo < kend) {
        fetch_tile<D>(Ks, key(a.k, j_lo), a.k.sn, t.nk - j_lo);
        fetch_tile<D>(Vs, key(a.v, j_lo), a.v.sn, t.nk - j_lo);
    }
    for (int j0 = j_lo; j0 < kend; j0 += TB) {
        // K of the next tile is fetched beside P V, V beside the next scores
        const int jn = j0 + TB, nn = jn < kend ? t.nk - jn : 0;
        landed<1>();
        const bool cut = j0 + TB - 1 > least;
        float s[R][4];
        dot_tile<D, R>(s, Qs, Ks, ty, tx);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            float mx = m[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] *= sl2;
                if (cut && j0 + tx + 16 * j > last[i]) s[i][j] = -INFINITY;
                mx = fmaxf(mx, s[i][j]);
            }
#pragma unroll
            for (int o = 8; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const float ref = mx == -INFINITY ? 0.f : mx;
            const float alpha = exp2f(m[i] - ref);
            m[i] = mx;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = exp2f(s[i][j] - ref);
                sum += p;
                Ps[(R * ty + i) * PP + tx + 16 * j] = p;
            }
            l[i] = l[i] * alpha + sum;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) acc[i][c] = __fmul2_rn(acc[i][c], make_float2(alpha, alpha));
        }
        __syncthreads();
        fetch_tile<D>(Ks, key(a.k, jn), a.k.sn, nn);
        landed<1>();
        if (cut)
            accumulate<D, R, true>(acc, Ps, Vs, ty, tx, [&](int r, int c) { return j0 + c <= last[r - R * ty]; });
        else
            accumulate<D, R, false>(acc, Ps, Vs, ty, tx, [](int, int) { return true; });
        __syncthreads();
        fetch_tile<D>(Vs, key(a.v, jn), a.v.sn, nn);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    const size_t rows_all = (size_t)a.B * a.Hq * a.Nq;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int r = r0 + R * ty + i;
        float sum = l[i];
#pragma unroll
        for (int o = 8; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (R * ty + i >= rows) continue;
        const int tok = r / G, h = hk * G + (r - tok * G);
        const bool none = m[i] == -INFINITY && sum == 0.f;
        const float inv = none ? 0.f : 1.f / sum, lse = none ? -INFINITY : m[i] + log2f(sum);
        const size_t id = ((size_t)b * a.Hq + h) * a.Nq + t.q0 + tok;
        uint8_t* row = n_split > 1 ? reinterpret_cast<uint8_t*>(part_o + (sp * rows_all + id) * D)
                                   : row_ptr<float>(a.o, b, h, t.q0 + tok);
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
            store2(row, 2 * tx + 32 * c, none ? 0.f : acc[i][c].x * inv, none ? 0.f : acc[i][c].y * inv);
        if (tx == 0) {
            if (n_split > 1)
                part_lse[sp * rows_all + id] = lse;
            else if (a.lse)
                a.lse[id] = lse * kLn2;
        }
    }
}

// Joins the parts of a split: o = sum_s w_s o_s, w_s = 2^(lse_s - M) / sum.  W warps share a row's parts (few rows have many
// parts, many rows few).
template <typename T, int W>
__global__ void __launch_bounds__(256)
    k_dense_combine(DenseArgs a, int n_split, const float* __restrict__ part_o, const float* __restrict__ part_lse) {
    __shared__ float4 sh_o[W][32];
    __shared__ float sh_sum[W];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, G = a.Hq / a.Hk, hk = blockIdx.y, b = blockIdx.z;
    const int x = W == 1 ? blockIdx.x * 8 + warp : blockIdx.x, w0 = W == 1 ? 0 : warp;
    if (x >= a.Nq * G) return;
    const SeqTile t = dense_resolve(a, x, 1, false, G);  // tiles of one row
    if (!t.live) return;                                 // (alike in all warps of a row)
    const size_t rows_all = (size_t)a.B * a.Hq * a.Nq;
    const int tok = t.tile / G, head = hk * G + (t.tile - tok * G);
    const size_t id = ((size_t)b * a.Hq + head) * a.Nq + t.q0 + tok;
    float M = -INFINITY;
    for (int s = lane; s < n_split; s += 32) M = fmaxf(M, part_lse[s * rows_all + id]);
    M = warp_max(M);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
#pragma unroll 4
    for (int s = w0; s < n_split; s += W) {
        const float ls = part_lse[s * rows_all + id];
        if (ls == -INFINITY) continue;  // (its part of o may not be written)
        const float w = exp2f(ls - M);  // (NaN where the row's scores are: M, which leaves NaN out, may be -inf then)
        sum += w;
        if (4 * lane < a.D) {
            const float4 o = *reinterpret_cast<const float4*>(part_o + (s * rows_all + id) * a.D + 4 * lane);
            acc.x = fmaf(w, o.x, acc.x);
            acc.y = fmaf(w, o.y, acc.y);
            acc.z = fmaf(w, o.z, acc.z);
            acc.w = fmaf(w, o.w, acc.w);
        }
    }
    if (W > 1) {
        sh_o[w0][lane] = acc;
        if (lane == 0) sh_sum[w0] = sum;
        __syncthreads();
        if (warp > 0) return;
        for (int i = 1; i < W; ++i) {
            const float4 o = sh_o[i][lane];
            acc = make_float4(acc.x + o.x, acc.y + o.y, acc.z + o.z, acc.w + o.w);
            sum += sh_sum[i];
        }
    }
    const bool none = M == -INFINITY && sum == 0.f;  // no visible key
    const float inv = none ? 0.f : 1.f / sum;
    if (4 * lane < a.D)
        store4<T>(row_ptr<T>(a.o, b, head, t.q0 + tok), lane, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
    if (a.lse && lane == 0) a.lse[id] = none ? M : (M + log2f(sum)) * kLn2;
}

// delta [B, Hq, Nq].  16 bytes a lane, 8 lanes a row up to 128 bytes and 16 or 32 above; four rows of a lane in flight.
template <typename T>
__global__ void __launch_bounds__(256) k_dense_delta(DenseArgs a, float* __restrict__ delta) {
    constexpr int E = 16 / sizeof(T);
    const int h = blockIdx.y, b = blockIdx.z, lane = threadIdx.x & 31;
    const int lpr = a.D <= 8 * E ? 8 : (a.D <= 16 * E ? 16 : 32), rpw = 32 / lpr, l = lane % lpr;
    const bool on = l * E < a.D;
    const long long n0 = ((long long)blockIdx.x * 8 + (threadIdx.x >> 5)) * rpw * 4 + lane / lpr;
    const uint8_t *po = row_ptr<T>(a.o, b, h, n0) + 16 * l, *pg = row_ptr<T>(a.d_o, b, h, n0) + 16 * l;
    uint4 o[4], g[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        o[u] = g[u] = make_uint4(0, 0, 0, 0);
        if (on && n0 + u * rpw < a.Nq) {
            o[u] = __ldg(reinterpret_cast<const uint4*>(po + u * rpw * a.o.sn * (long long)sizeof(T)));
            g[u] = __ldg(reinterpret_cast<const uint4*>(pg + u * rpw * a.d_o.sn * (long long)sizeof(T)));
        }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const uint32_t x[4] = {o[u].x, o[u].y, o[u].z, o[u].w}, y[4] = {g[u].x, g[u].y, g[u].z, g[u].w};
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (sizeof(T) == 4)
                s = fmaf(__uint_as_float(x[e]), __uint_as_float(y[e]), s);
            else
                s = fmaf(__uint_as_float(x[e] << 16), __uint_as_float(y[e] << 16),
                         fmaf(__uint_as_float(x[e] & 0xFFFF0000u), __uint_as_float(y[e] & 0xFFFF0000u), s));
        }
        for (int d = lpr / 2; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        if (l == 0 && n0 + u * rpw < a.Nq) delta[((size_t)b * a.Hq + h) * a.Nq + n0 + u * rpw] = s;
    }
}

// In the two backward kernels 256 threads form the scores and 256 others do v^T: one block fills the shared memory of an SM,
// and eight warps left the FMA units idle.  dq and dk/dv, 32 query heads on 8, 1,145 tokens: D = 128 865 and 1,258 us with
// 256 threads that did both, 887 and 1,182 with 512; D = 64 501 and 745, 476 and 674.  Halves of 128 threads with 8 x 4
// elements each, for fewer shared-memory reads: 957 and 1,229.
constexpr int kBwdThreads = 512;

template <int D>
__global__ void __launch_bounds__(kBwdThreads) k_dense_dq_simt(DenseArgs a, DenseOrder order, const float* __restrict__ delta) {
    extern __shared__ __align__(16) float smem[];
    float* Qs = smem;
    float* Gs = Qs + TB * (D + 4);
    float* Ks = Gs + TB * (D + 4);
    float* Vs = Ks + 2 * TB * (D + 4);  // (K twice)
    float* Ps = Vs + TB * (D + 4);
    int x;
    const int bh = dense_block_head(order, x), b = bh / a.Hq, h = bh - b * a.Hq, hk = h / (a.Hq / a.Hk);
    const SeqTile t = resolve_block(a, order, x, TB, false, 1);
    const int i0 = t.tile * TB;
    if (!t.live || i0 >= t.nq) return;
    const int tid = threadIdx.x, tx = tid & 15, ty = (tid >> 4) & 15;
    const bool second = tid >= 256;
    const int rows = min(TB, t.nq - i0);
    load_tile<D, TB, kBwdThreads>(Qs, row_ptr<float>(a.q, b, h, t.q0 + i0), a.q.sn, rows);
    load_tile<D, TB, kBwdThreads>(Gs, row_ptr<float>(a.d_o, b, h, t.q0 + i0), a.d_o.sn, rows);
    float2 acc[4][D / 32];
    float stat[4];  // of the rows 4 ty ..: lse in base 2, or delta in the second half
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i;
        const size_t at = ((size_t)b * a.Hq + h) * a.Nq + t.q0 + i0 + r;
        stat[i] = r < rows ? (second ? delta[at] : a.lse[at] * kLog2e) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < D / 32; ++c) acc[i][c] = make_float2(0.f, 0.f);
    const float sl2 = a.scale * kLog2e;
    const int kend = dense_last_key(i0 + rows - 1, t.nq, t.nk, a.causal) + 1;
    auto key = [&](const Op4& o, int j) { return row_ptr<float>(o, b, hk, t.k0 + min(j, t.nk - 1)); };
    if (kend > 0) {
        fetch_tile<D, kBwdThreads>(Ks, key(a.k, 0), a.k.sn, t.nk);
        fetch_tile<D, kBwdThreads>(Vs, key(a.v, 0), a.v.sn, t.nk);
    }
    float *Kj = Ks, *Kn = Ks + TB * (D + 4);
    for (int j0 = 0; j0 < kend; j0 += TB) {
        const int jn = j0 + TB, nn = jn < kend ? t.nk - jn : 0;
        landed<0>();
        fetch_tile<D, kBwdThreads>(Kn, key(a.k, jn), a.k.sn, nn);
        auto see = [&](int r, int c) { return j0 + c <= dense_last_key(i0 + r, t.nq, t.nk, a.causal); };
        const bool cut = j0 + TB - 1 > dense_last_key(i0, t.nq, t.nk, a.causal);
        float s[4][4];
        dot_tile<D, 4>(s, second ? Gs : Qs, second ? Vs : Kj, ty, tx);
        if (!second) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) Ps[(4 * ty + i) * PP + tx + 16 * j] = exp2f(s[i][j] * sl2 - stat[i]);
        }
        __syncthreads();
        fetch_tile<D, kBwdThreads>(Vs, key(a.v, jn), a.v.sn, nn);
        if (second) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float* at = Ps + (4 * ty + i) * PP + tx + 16 * j;
                    *at = cut && !see(4 * ty + i, tx + 16 * j) ? 0.f : *at * (s[i][j] - stat[i]);
                }
        }
        __syncthreads();
        // each half sums over half of the keys
        const int k0 = second ? TB / 2 : 0;
        if (cut)
            accumulate<D, 4, true>(acc, Ps, Kj, ty, tx, see, k0, k0 + TB / 2);
        else
            accumulate<D, 4, false>(acc, Ps, Kj, ty, tx, see, k0, k0 + TB / 2);
        float* swap = Kj;
        Kj = Kn;
        Kn = swap;
    }
    landed<0>();
    float* sum = Qs;  // the second half's sums
    if (second) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < D / 32; ++c) *reinterpret_cast<float2*>(sum + (4 * ty + i) * (D + 4) + 2 * tx + 32 * c) = acc[i][c];
    }
    __syncthreads();
    if (second) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i;
        if (r >= rows) continue;
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
            acc[i][c] = __fadd2_rn(acc[i][c], *reinterpret_cast<const float2*>(sum + r * (D + 4) + 2 * tx + 32 * c));
        uint8_t* row = row_ptr<float>(a.dq, b, h, t.q0 + i0 + r);
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
            store2(row, 2 * tx + 32 * c, acc[i][c].x * a.scale, acc[i][c].y * a.scale);
    }
}

// The first half of the threads goes on with dv, the second with dk.  The next step's rows travel through registers while
// these sums are formed (two more tiles do not fit in shared memory at D = 128).
template <int D>
__global__ void __launch_bounds__(kBwdThreads) k_dense_dkv_simt(DenseArgs a, DenseOrder order, const float* __restrict__ delta,
                                                                int n_split, int chunk, float* __restrict__ part_dv,
                                                                float* __restrict__ part_dk) {
    extern __shared__ __align__(16) float smem[];
    float* Ks = smem;
    float* Vs = Ks + TB * (D + 4);
    float* Qs = Vs + TB * (D + 4);
    float* Gs = Qs + TB * (D + 4);
    float* Ps = Gs + TB * (D + 4);
    float* Ds = Ps + TB * PP;
    int x;
    const int bh = dense_block_head(order, x), b = bh / a.Hk, hk = bh - b * a.Hk, sp = blockIdx.z;
    const SeqTile t = resolve_block(a, order, x, TB, true, 1);
    const int j0 = t.tile * TB;
    if (!t.live || j0 >= t.nk) return;
    const int G = a.Hq / a.Hk;
    const int tid = threadIdx.x, tx = tid & 15, ty = (tid >> 4) & 15;
    const bool second = tid >= 256;
    int first, end;
    dense_row_tiles(t, j0, a.causal, TB, first, end);
    const int per = end - first, s0 = n_split > 1 ? sp * chunk : 0;
    const int s1 = n_split > 1 ? min(per * G, s0 + chunk) : per * G;
    if (n_split > 1 && s0 >= s1) return;  // (no such part)
    const int keys = min(TB, t.nk - j0);
    load_tile<D, TB, kBwdThreads>(Ks, row_ptr<float>(a.k, b, hk, t.k0 + j0), a.k.sn, keys);
    load_tile<D, TB, kBwdThreads>(Vs, row_ptr<float>(a.v, b, hk, t.k0 + j0), a.v.sn, keys);
    float2 acc[4][D / 32];  // dv or dk
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < D / 32; ++c) acc[i][c] = make_float2(0.f, 0.f);
    const float sl2 = a.scale * kLog2e;
    constexpr int F = TB * D / 4 / kBwdThreads;  // 16-byte pieces of a tile for each thread
    float4 qn[F], gn[F];
    float stat[4];  // of the columns tx + 16 j: lse in base 2, or delta in the second half
    auto fetch = [&](int step) {  // the step's rows and statistics into registers
        const int h = hk * G + step / per, i0 = (first + step % per) * TB, rows = t.nq - i0;
        const uint8_t *qp = row_ptr<float>(a.q, b, h, t.q0 + i0), *gp = row_ptr<float>(a.d_o, b, h, t.q0 + i0);
#pragma unroll
        for (int f = 0; f < F; ++f) {
            const int i = tid + kBwdThreads * f, r = i / (D / 4), c = i - r * (D / 4);
            qn[f] = gn[f] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < rows) {
                qn[f] = load4(qp + r * a.q.sn * 4, c);
                gn[f] = load4(gp + r * a.d_o.sn * 4, c);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = tx + 16 * j;
            const size_t at = ((size_t)b * a.Hq + h) * a.Nq + t.q0 + i0 + c;
            stat[j] = c < rows ? (second ? delta[at] : a.lse[at] * kLog2e) : 0.f;
        }
    };
    auto keep = [&]() {
#pragma unroll
        for (int f = 0; f < F; ++f) {
            const int i = tid + kBwdThreads * f, r = i / (D / 4), c = i - r * (D / 4);
            *reinterpret_cast<float4*>(Qs + r * (D + 4) + 4 * c) = qn[f];
            *reinterpret_cast<float4*>(Gs + r * (D + 4) + 4 * c) = gn[f];
        }
        __syncthreads();
    };
    if (s0 < s1) {
        fetch(s0);
        keep();
    }
    for (int step = s0; step < s1; ++step) {
        const int i0 = (first + step % per) * TB, rows = min(TB, t.nq - i0);
        // r: key of the tile, c: query row of the tile
        auto see = [&](int r, int c) {
            return c < rows && r < keys && j0 + r <= dense_last_key(i0 + c, t.nq, t.nk, a.causal);
        };
        const bool cut = rows < TB || j0 + keys - 1 > dense_last_key(i0, t.nq, t.nk, a.causal);
        float s[4][4];
        dot_tile<D, 4>(s, second ? Vs : Ks, second ? Gs : Qs, ty, tx);
        if (!second) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int r = 4 * ty + i, c = tx + 16 * j;
                    const float p = exp2f(s[i][j] * sl2 - stat[j]);
                    Ps[r * PP + c] = cut && !see(r, c) ? 0.f : p;
                }
        }
        __syncthreads();
        if (second) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int r = 4 * ty + i, c = tx + 16 * j;
                    Ds[r * PP + c] = cut && !see(r, c) ? 0.f : Ps[r * PP + c] * (s[i][j] - stat[j]);
                }
            __syncwarp();  // (a row of ds comes from its own half-warp)
        }
        if (step + 1 < s1) fetch(step + 1);
        if (cut)
            accumulate<D, 4, true>(acc, second ? Ds : Ps, second ? Qs : Gs, ty, tx, see);
        else
            accumulate<D, 4, false>(acc, second ? Ds : Ps, second ? Qs : Gs, ty, tx, see);
        __syncthreads();
        if (step + 1 < s1) keep();
    }
    const Op4& out = second ? a.dk : a.dv;
    float* part = second ? part_dk : part_dv;
    const float f = second && n_split == 1 ? a.scale : 1.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i;
        if (r >= keys) continue;
        uint8_t* row = n_split > 1 ? reinterpret_cast<uint8_t*>(part + ((((size_t)sp * a.B + b) * a.Hk + hk) * a.Nk + t.k0 + j0 + r) * D)
                                   : row_ptr<float>(out, b, hk, t.k0 + j0 + r);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) store2(row, 2 * tx + 32 * c, acc[i][c].x * f, acc[i][c].y * f);
    }
}

// dk, dv = sums of the parts, in order; one warp a key row
template <typename T>
__global__ void __launch_bounds__(256)
    k_dense_dkv_reduce(DenseArgs a, int tile, int n_split, int chunk, const float* __restrict__ part_dv,
                       const float* __restrict__ part_dk) {
    const int lane = threadIdx.x & 31, hk = blockIdx.y, b = blockIdx.z;
    const int x = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (x >= a.Nk) return;
    const SeqTile t = dense_resolve(a, x, 1, true, 1);  // tiles of one key
    if (!t.live || 4 * lane >= a.D) return;
    int first, end;
    dense_row_tiles(t, t.tile / tile * tile, a.causal, tile, first, end);
    const int n = min(n_split, ((end - first) * (a.Hq / a.Hk) + chunk - 1) / chunk);  // parts that were written
    const size_t at = (((size_t)b * a.Hk + hk) * a.Nk + t.k0 + t.tile) * a.D + 4 * lane, step = (size_t)a.B * a.Hk * a.Nk * a.D;
    for (int w = 0; w < 2; ++w) {
        const float* src = (w ? part_dk : part_dv) + at;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int s = 0; s < n; ++s) {
            const float4 u = *reinterpret_cast<const float4*>(src + s * step);
            v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
        }
        const float f = w ? a.scale : 1.f;
        store4<T>(row_ptr<T>(w ? a.dk : a.dv, b, hk, t.k0 + t.tile), lane, make_float4(v.x * f, v.y * f, v.z * f, v.w * f));
    }
}

template <int D, int R>
int fwd_simt_r(const DenseArgs& a, const DenseSplit& sp, float* part_o, float* part_lse, cudaStream_t st) {
    const size_t sm = (size_t)((16 * R + 2 * TB) * (D + 4) + 16 * R * PP) * 4;
    {
        static std::atomic<uint64_t> done{0};
        allow_smem(k_dense_fwd_simt<D, R>, sm, done);
    }
    ::park::prof_begin(st);
    k_dense_fwd_simt<D, R><<<dim3((unsigned)(sp.tiles * a.B * a.Hk), 1, sp.n), 256, sm, st>>>(
        a, dense_order(a, sp.tiles, a.B * a.Hk, 8 * a.Nk * D, 1), sp.n, sp.chunk, part_o, part_lse);
    PARK_TRY_LAUNCH(R == 8 ? "k_dense_fwd_simt, 128 rows" : R == 4 ? "k_dense_fwd_simt, 64 rows" : "k_dense_fwd_simt, 16 rows", st);
    return PARK_OK;
}

template <int D>
int fwd_simt(const DenseArgs& a, void* ws, cudaStream_t st) {
    const DenseSplit sp = dense_split_simt(a.B, a.Hq, a.Hk, a.Nq, a.Nk, a.n_seq, a.D);
    if (sp.n > 65535) return PARK_ERR_UNSUPPORTED;
    float* part_o = static_cast<float*>(ws);
    float* part_lse = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + sp.lse_off);
    PARK_CHECK(sp.rows == 128 ? (fwd_simt_r<D, 8>(a, sp, part_o, part_lse, st))
               : sp.rows == 64 ? (fwd_simt_r<D, 4>(a, sp, part_o, part_lse, st))
                               : (fwd_simt_r<D, 1>(a, sp, part_o, part_lse, st)));
    return sp.n > 1 ? launch_dense_combine(a, PARK_F32, sp.n, part_o, part_lse, st) : PARK_OK;
}

template <int D>
int bwd_simt(const DenseArgs& a, const float* delta, float* parts, cudaStream_t st) {
    const size_t sq = (size_t)(5 * TB * (D + 4) + TB * PP) * 4, sk = (size_t)(4 * TB * (D + 4) + 2 * TB * PP) * 4;
    {
        static std::atomic<uint64_t> done{0};
        allow_smem(k_dense_dq_simt<D>, sq, done);
    }
    {
        static std::atomic<uint64_t> done{0};
        allow_smem(k_dense_dkv_simt<D>, sk, done);
    }
    if (a.Nq > 0) {
        ::park::prof_begin(st);
        const long long tiles = dense_tiles(a.Nq, a.n_seq, TB);
        k_dense_dq_simt<D><<<(unsigned)(tiles * a.B * a.Hq), kBwdThreads, sq, st>>>(
            a, dense_order(a, tiles, a.B * a.Hq, 8 * a.Nk * D, a.Hq / a.Hk), delta);
        PARK_TRY_LAUNCH("k_dense_dq_simt", st);
    }
    if (a.Nk == 0) return PARK_OK;
    const DkvSplit sp = dense_split_dkv(a.B, a.Hq, a.Hk, a.Nq, a.Nk, a.n_seq, D, TB);
    if (sp.n > 65535) return PARK_ERR_UNSUPPORTED;
    float* part_dk = parts + sp.dk_off / 4;
    ::park::prof_begin(st);
    k_dense_dkv_simt<D><<<dim3((unsigned)(sp.tiles * a.B * a.Hk), 1, sp.n), kBwdThreads, sk, st>>>(
        a, dense_order(a, sp.tiles, a.B * a.Hk, 8 * a.Nq * D * (a.Hq / a.Hk), 1), delta, sp.n, sp.chunk, parts, part_dk);
    PARK_TRY_LAUNCH("k_dense_dkv_simt", st);
    return sp.n > 1 ? launch_dense_dkv_reduce(a, PARK_F32, sp, TB, parts, part_dk, st) : PARK_OK;
}

}  // namespace

int launch_dense_combine(const DenseArgs& a, int dtype, int n_split, const float* part_o, const float* part_lse,
                         cudaStream_t st) {
    const long long rows = a.Nq * (a.Hq / a.Hk);
    const bool wide = n_split > 4 && rows * a.Hk * a.B <= 2048;
    const dim3 grid((unsigned)(wide ? rows : (rows + 7) / 8), a.Hk, a.B);
    ::park::prof_begin(st);
    if (dtype == PARK_BF16) {
        if (wide) k_dense_combine<bf16_t, 8><<<grid, 256, 0, st>>>(a, n_split, part_o, part_lse);
        else k_dense_combine<bf16_t, 1><<<grid, 256, 0, st>>>(a, n_split, part_o, part_lse);
    } else {
        if (wide) k_dense_combine<float, 8><<<grid, 256, 0, st>>>(a, n_split, part_o, part_lse);
        else k_dense_combine<float, 1><<<grid, 256, 0, st>>>(a, n_split, part_o, part_lse);
    }
    PARK_TRY_LAUNCH("k_dense_combine", st);
    return PARK_OK;
}

int launch_dense_dkv_reduce(const DenseArgs& a, int dtype, const DkvSplit& sp, int tile, const float* dv, const float* dk,
                            cudaStream_t st) {
    const dim3 grid((unsigned)((a.Nk + 7) / 8), a.Hk, a.B);
    ::park::prof_begin(st);
    if (dtype == PARK_BF16)
        k_dense_dkv_reduce<bf16_t><<<grid, 256, 0, st>>>(a, tile, sp.n, sp.chunk, dv, dk);
    else
        k_dense_dkv_reduce<float><<<grid, 256, 0, st>>>(a, tile, sp.n, sp.chunk, dv, dk);
    PARK_TRY_LAUNCH("k_dense_dkv_reduce", st);
    return PARK_OK;
}

// Parts are sized for the longest sequence that the bounds could hold, which the host does not know: a packed batch gets no
// more of them than fit in 256 MB (its parts of one length are then longer).  Without packing 80 MB are never exceeded.
static long long limit_chunk(long long chunk, long long steps, long long part_bytes) {
    long long most = (256ll << 20) / (part_bytes > 0 ? part_bytes : 1);
    if (most < 1) most = 1;
    const long long least = (steps + most - 1) / most;
    return chunk < least ? least : chunk;
}

// Few keys under many rows (text keys): the key tiles alone leave SMs idle, so the rows are split, about two CTAs for each
// SM, at least 8 steps each.
DkvSplit dense_split_dkv(int B, int Hq, int Hk, long long Nq, long long Nk, int n_seq, int D, int tile) {
    DkvSplit s;
    s.tiles = dense_tiles(Nk, n_seq, tile);
    s.n = 1;
    s.chunk = 0;
    const long long G = Hq / Hk, steps = (Nq + tile - 1) / tile * G, ctas = s.tiles * Hk * B;
    // (float32 steps are ten times as long, and up to four blocks for an SM are split too)
    const int waves = tile == 64 ? 4 : 2;
    if (ctas * 2 <= kDenseSMs * (tile == 64 ? 8 : 1)) {
        const long long work = n_seq > 0 ? (steps + n_seq * G) * ((s.tiles + n_seq - 1) / n_seq) * Hk : steps * ctas;
        long long chunk = (work + waves * kDenseSMs - 1) / (waves * kDenseSMs);
        if (chunk < 8) chunk = 8;
        chunk = limit_chunk(chunk, steps, 8ll * B * Hk * Nk * D);
        const long long n = (steps + chunk - 1) / chunk;  // (a sequence has at most all the steps)
        if (n > 1) {
            s.n = (int)n;
            s.chunk = (int)chunk;
        }
    }
    const size_t one = align_up((size_t)B * Hk * Nk * D * 4 * (size_t)s.n, 256);
    s.dk_off = s.n > 1 ? one : 0;
    s.bytes = s.n > 1 ? 2 * one : 0;
    return s;
}

// Splits the keys when the row tiles alone leave SMs idle: parts of equal length whatever the sequence (a packed batch
// holds at most kt key tiles in all, a batch entry has as many), of `chunk` key tiles, at least `least`; done when the row
// tiles are at most `wide` CTAs for two SMs.
static void split_keys(DenseSplit* s, int B, int Hq, int Hk, long long Nq, long long kt, int D, long long chunk, int wide,
                       int least) {
    s->n = 1;
    s->chunk = 0;
    if (chunk < least) chunk = least;
    const size_t rows = (size_t)B * Hq * Nq;
    chunk = limit_chunk(chunk, kt, 4ll * rows * (D + 1));
    const long long n = (kt + chunk - 1) / chunk;
    if (s->tiles * Hk * B * 2 <= kDenseSMs * wide && n > 1) {
        s->n = (int)n;
        s->chunk = (int)chunk;
    }
    s->lse_off = s->n > 1 ? align_up((size_t)s->n * rows * D * 4, 256) : 0;
    s->bytes = s->n > 1 ? s->lse_off + align_up((size_t)s->n * rows * 4, 256) : 0;
}

DenseSplit dense_split_tc(int B, int Hq, int Hk, long long Nq, long long Nk, int n_seq, int D) {
    // 256 rows and one CTA an SM, or, where those CTAs would fill no more than half of the SMs, 128 rows and two CTAs an SM
    // (8 heads x 2,048^2: 39 us against 60 with split keys; 300 x 20,000 keys 58 against 73; where both fill the GPU 256
    // rows are faster: 8 heads x 16,384^2 0.88 ms against 1.02, D = 64 0.78 against 0.89)
    DenseSplit s;
    const long long rows = Nq * (Hq / Hk);
    s.rows = dense_tiles(rows, n_seq, 256) * Hk * B * 2 <= kDenseSMs ? 128 : 256;
    s.tiles = dense_tiles(rows, n_seq, s.rows);
    // As many parts as run at once, two CTAs an SM: a few more start last and run alone.  In a packed batch (of single rows, one
    // row tile each) every sequence may have a part that is not full, so kt / chunk + n_seq parts fit, and not less than half as
    // many full ones.  24/8 heads, one row each, D = 128 and 64, captured, against parts that only come near that number: 119,056 +
    // 75,600 + 40,001 + 3,601 keys 178 and 143 us against 205 and 162, 119,056 + 40,001 129 and 94 against 135 and 102, 8 x 16,000
    // 115 and 90 against 125 and 94, 200,000 148 and 102 both, 4 x 60,000 176 and 131 against 176 and 125.  Parts of half the
    // length: 195 and 154, 141 and 109, 150 and 121, 156 and 111, 190 and 141.  8 heads x 1,100 rows x 20,000 keys 115 and 102
    // against 119 and 102, 300 x 119,056 199 and 178 against 193 and 174; 4 heads x 2,000 x 75,600 342 and 309 against 356 and
    // 317 (half the length 328 and 291).
    const long long kt = (Nk + 127) / 128 + n_seq, per = n_seq > 0 ? Hk : Hk * B * s.tiles;
    const long long fit = 2 * kDenseSMs / (per > 0 ? per : 1);  // (no rows: no tiles)
    long long parts = n_seq > 0 && fit - n_seq < fit / 2 ? fit / 2 : fit - n_seq;
    if (parts < 1) parts = 1;
    split_keys(&s, B, Hq, Hk, Nq, kt, D, (kt + parts - 1) / parts, 1, 3);
    return s;
}

DenseSplit dense_split_simt(int B, int Hq, int Hk, long long Nq, long long Nk, int n_seq, int D) {
    // 8 rows a thread (half the shared-memory reads of 4) where those tiles fill the SMs; one row a thread for single rows, and
    // for problems so small that a block for each pair of tiles is about one wave; 4 otherwise, with split keys where they do
    // not fill (1,500 causal rows x 2 heads, D = 64: 114 us with one row, 54 with 4)
    DenseSplit s;
    const long long rows = Nq * (Hq / Hk), mean = n_seq > 0 ? rows / n_seq : rows;
    const long long kt = (Nk + TB - 1) / TB / (n_seq > 0 ? n_seq : 1) + 1;
    if (mean >= 64 && dense_tiles(rows, n_seq, 128) * Hk * B >= kDenseSMs)
        s.rows = 128;
    else
        s.rows = mean < 32 || dense_tiles(rows, n_seq, 16) * kt * Hk * B <= 2 * kDenseSMs ? 16 : 64;
    s.tiles = dense_tiles(rows, n_seq, s.rows);
    // Parts of one key tile only while those fill no more than the SMs (captured: 256 x 2,048 keys, one head, D = 64, 14 us and
    // 19 with two; 1 x 500 x 8 heads, D = 128, 11 and 18; but 300 x 1,000 x 2 heads 33 and 28, 512^2 x 8, D = 64, 34 and 28)
    const long long keys = (Nk + TB - 1) / TB + n_seq;
    // About four blocks an SM (parts that fit as above: 8 heads, one row each, D = 128: 8 x 16,000 keys 666 us against 604, 4 x
    // 30,000 584 and 565, 100,000 481 and 479)
    const long long work = n_seq > 0 ? keys * Hk : keys * Hk * B * s.tiles;
    split_keys(&s, B, Hq, Hk, Nq, keys, D, (work + 4 * kDenseSMs - 1) / (4 * kDenseSMs), 2,
               s.tiles * Hk * B * keys > kDenseSMs ? 2 : 1);
    return s;
}

int launch_dense_delta(const DenseArgs& a, int dtype, float* delta, cudaStream_t st) {
    const int E = dtype == PARK_BF16 ? 8 : 4, lpr = a.D <= 8 * E ? 8 : (a.D <= 16 * E ? 16 : 32), rows = 32 / lpr * 4 * 8;
    const dim3 grid((unsigned)((a.Nq + rows - 1) / rows), a.Hq, a.B);
    ::park::prof_begin(st);
    if (dtype == PARK_BF16)
        k_dense_delta<bf16_t><<<grid, 256, 0, st>>>(a, delta);
    else
        k_dense_delta<float><<<grid, 256, 0, st>>>(a, delta);
    PARK_TRY_LAUNCH("k_dense_delta", st);
    return PARK_OK;
}

#define PARK_BY_D(F, ...)                                              \
    (a.D == 32 ? F<32>(__VA_ARGS__) : a.D == 64 ? F<64>(__VA_ARGS__) \
     : a.D == 96 ? F<96>(__VA_ARGS__) : F<128>(__VA_ARGS__))

int launch_dense_fwd_simt(const DenseArgs& a, void* ws, cudaStream_t st) { return PARK_BY_D(fwd_simt, a, ws, st); }

int launch_dense_bwd_simt(const DenseArgs& a, const float* delta, float* parts, cudaStream_t st) {
    return PARK_BY_D(bwd_simt, a, delta, parts, st);
}

}  // namespace park
