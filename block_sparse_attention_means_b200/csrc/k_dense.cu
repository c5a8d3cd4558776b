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
// Bound by the FMA units: 64 x 64 score tiles, 256 threads with 4 x 4 scores and
// 4 x D/16 outputs each; tiles stay in shared memory (row pitch D + 4 floats: the
// 16 key rows that a half-warp reads with 16-byte loads hit all banks once).
// Tiles that a mask cuts take a variant whose products skip the hidden pairs, so
// that an infinity or NaN there stays out of the sums.
#include "dense.cuh"
#include "kernels.h"

namespace park {
namespace {

constexpr int TB = 64;          // query rows and key rows of a tile
constexpr int PP = TB + 4;      // row pitch of a probability tile

template <typename T>
__device__ __forceinline__ float4 load4(const uint8_t* p, int i);
template <>
__device__ __forceinline__ float4 load4<float>(const uint8_t* p, int i) {
    return *reinterpret_cast<const float4*>(p + 16 * (size_t)i);
}
template <>
__device__ __forceinline__ float4 load4<bf16_t>(const uint8_t* p, int i) {
    const uint2 v = *reinterpret_cast<const uint2*>(p + 8 * (size_t)i);
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u), __uint_as_float(v.y << 16),
                       __uint_as_float(v.y & 0xFFFF0000u));
}

// rows 0 .. n-1 of `src` (row stride in elements) into a [64][D + 4] tile, zeros below
template <int D>
__device__ __forceinline__ void load_tile(float* dst, const uint8_t* src, long long stride, int n) {
    constexpr int C = D / 4;
    for (int i = threadIdx.x; i < TB * C; i += 256) {
        const int r = i / C, c = i - r * C;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < n) v = load4<float>(src + r * stride * 4, c);
        *reinterpret_cast<float4*>(dst + r * (D + 4) + 4 * c) = v;
    }
}

// s[i][j] = A[4 ty + i] . B[tx + 16 j]
template <int D>
__device__ __forceinline__ void dot_tile(float (&s)[4][4], const float* A, const float* Bm, int ty, int tx) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
        float4 a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(A + (4 * ty + i) * (D + 4) + d);
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4*>(Bm + (tx + 16 * j) * (D + 4) + d);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = fmaf(a[i].x, b[j].x, s[i][j]);
                s[i][j] = fmaf(a[i].y, b[j].y, s[i][j]);
                s[i][j] = fmaf(a[i].z, b[j].z, s[i][j]);
                s[i][j] = fmaf(a[i].w, b[j].w, s[i][j]);
            }
    }
}

// acc[i][c] += sum_k P[4 ty + i][k] B[k][col c], col c = 2 tx + 32 (c / 2) + c % 2.
// With MASK only pairs that see(row, k) allows enter the sum.
template <int D, bool MASK, typename F>
__device__ __forceinline__ void accumulate(float (&acc)[4][D / 16], const float* P, const float* Bm, int ty, int tx,
                                           F see) {
#pragma unroll 2
    for (int k = 0; k < TB; k += 4) {
        float4 p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const float4*>(P + (4 * ty + i) * PP + k);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                const float2 b = *reinterpret_cast<const float2*>(Bm + (k + kk) * (D + 4) + 2 * tx + 32 * c);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float pv = kk == 0 ? p[i].x : kk == 1 ? p[i].y : kk == 2 ? p[i].z : p[i].w;
                    if (!MASK || see(4 * ty + i, k + kk)) {
                        acc[i][2 * c] = fmaf(pv, b.x, acc[i][2 * c]);
                        acc[i][2 * c + 1] = fmaf(pv, b.y, acc[i][2 * c + 1]);
                    }
                }
            }
    }
}

__device__ __forceinline__ void store2(uint8_t* row, int col, float x, float y) {
    *reinterpret_cast<float2*>(row + 4 * col) = make_float2(x, y);
}

template <typename T>
__device__ __forceinline__ uint8_t* row_ptr(const Op4& o, int b, int h, long long n) {
    return o.p + (b * o.sb + h * o.sh + n * o.sn) * (long long)sizeof(T);
}

__device__ __forceinline__ SeqTile resolve_block(const DenseArgs& a, int x, bool by_keys) {
    __shared__ SeqTile sh;
    if (threadIdx.x < 32) {
        const SeqTile t = dense_resolve(a, x, TB, by_keys, 1);
        if (threadIdx.x == 0) sh = t;
    }
    __syncthreads();
    return sh;
}

template <int D>
__global__ void __launch_bounds__(256) k_dense_fwd_simt(DenseArgs a) {
    extern __shared__ __align__(16) float smem[];
    float* Qs = smem;
    float* Ks = Qs + TB * (D + 4);
    float* Vs = Ks + TB * (D + 4);
    float* Ps = Vs + TB * (D + 4);
    const SeqTile t = resolve_block(a, gridDim.x - 1 - blockIdx.x, false);  // causal: long rows first
    const int i0 = t.tile * TB;
    if (!t.live || i0 >= t.nq) return;
    const int h = blockIdx.y, b = blockIdx.z, hk = h / (a.Hq / a.Hk);
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int rows = min(TB, t.nq - i0);
    load_tile<D>(Qs, row_ptr<float>(a.q, b, h, t.q0 + i0), a.q.sn, rows);
    float acc[4][D / 16], m[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) acc[i][c] = 0.f;
    }
    const float sl2 = a.scale * kLog2e;
    const int kend = dense_last_key(i0 + rows - 1, t.nq, t.nk, a.causal) + 1;  // keys that any row sees
    for (int j0 = 0; j0 < kend; j0 += TB) {
        __syncthreads();
        load_tile<D>(Ks, row_ptr<float>(a.k, b, hk, t.k0 + j0), a.k.sn, min(TB, t.nk - j0));
        load_tile<D>(Vs, row_ptr<float>(a.v, b, hk, t.k0 + j0), a.v.sn, min(TB, t.nk - j0));
        __syncthreads();
        auto see = [&](int r, int c) { return j0 + c <= dense_last_key(i0 + r, t.nq, t.nk, a.causal); };
        const bool cut = j0 + TB - 1 > dense_last_key(i0, t.nq, t.nk, a.causal);
        float s[4][4];
        dot_tile<D>(s, Qs, Ks, ty, tx);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float mx = m[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] *= sl2;
                if (cut && !see(4 * ty + i, tx + 16 * j)) s[i][j] = -INFINITY;
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
                Ps[(4 * ty + i) * PP + tx + 16 * j] = p;
            }
            l[i] = l[i] * alpha + sum;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) acc[i][c] *= alpha;
        }
        __syncthreads();
        if (cut)
            accumulate<D, true>(acc, Ps, Vs, ty, tx, see);
        else
            accumulate<D, false>(acc, Ps, Vs, ty, tx, see);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i;
        float sum = l[i];
#pragma unroll
        for (int o = 8; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (r >= rows) continue;
        const float inv = m[i] == -INFINITY && !(sum != sum) ? 0.f : 1.f / sum;
        uint8_t* row = row_ptr<float>(a.o, b, h, t.q0 + i0 + r);
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
            store2(row, 2 * tx + 32 * c, inv == 0.f ? 0.f : acc[i][2 * c] * inv,
                      inv == 0.f ? 0.f : acc[i][2 * c + 1] * inv);
        if (a.lse && tx == 0)
            a.lse[((size_t)b * a.Hq + h) * a.Nq + t.q0 + i0 + r] = (m[i] + log2f(sum)) * kLn2;
    }
}

// delta [B, Hq, Nq]: one warp a row
template <typename T>
__global__ void __launch_bounds__(256) k_dense_delta(DenseArgs a, float* __restrict__ delta) {
    const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= (long long)a.B * a.Hq * a.Nq) return;
    const long long n = row % a.Nq, bh = row / a.Nq;
    const int h = (int)(bh % a.Hq), b = (int)(bh / a.Hq);
    float s = 0.f;
    if (4 * lane < a.D) {
        const float4 x = load4<T>(row_ptr<T>(a.o, b, h, n), lane), y = load4<T>(row_ptr<T>(a.d_o, b, h, n), lane);
        s = x.x * y.x + x.y * y.y + x.z * y.z + x.w * y.w;
    }
    s = warp_sum(s);
    if (lane == 0) delta[row] = s;
}

template <int D>
__global__ void __launch_bounds__(256) k_dense_dq_simt(DenseArgs a, const float* __restrict__ delta) {
    extern __shared__ __align__(16) float smem[];
    float* Qs = smem;
    float* Gs = Qs + TB * (D + 4);
    float* Ks = Gs + TB * (D + 4);
    float* Vs = Ks + TB * (D + 4);
    float* Ps = Vs + TB * (D + 4);
    const SeqTile t = resolve_block(a, gridDim.x - 1 - blockIdx.x, false);
    const int i0 = t.tile * TB;
    if (!t.live || i0 >= t.nq) return;
    const int h = blockIdx.y, b = blockIdx.z, hk = h / (a.Hq / a.Hk);
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int rows = min(TB, t.nq - i0);
    load_tile<D>(Qs, row_ptr<float>(a.q, b, h, t.q0 + i0), a.q.sn, rows);
    load_tile<D>(Gs, row_ptr<float>(a.d_o, b, h, t.q0 + i0), a.d_o.sn, rows);
    float acc[4][D / 16], lse2[4], del[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i;
        const size_t at = ((size_t)b * a.Hq + h) * a.Nq + t.q0 + i0 + r;
        lse2[i] = r < rows ? a.lse[at] * kLog2e : 0.f;
        del[i] = r < rows ? delta[at] : 0.f;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) acc[i][c] = 0.f;
    }
    const float sl2 = a.scale * kLog2e;
    const int kend = dense_last_key(i0 + rows - 1, t.nq, t.nk, a.causal) + 1;
    for (int j0 = 0; j0 < kend; j0 += TB) {
        __syncthreads();
        load_tile<D>(Ks, row_ptr<float>(a.k, b, hk, t.k0 + j0), a.k.sn, min(TB, t.nk - j0));
        load_tile<D>(Vs, row_ptr<float>(a.v, b, hk, t.k0 + j0), a.v.sn, min(TB, t.nk - j0));
        __syncthreads();
        auto see = [&](int r, int c) { return j0 + c <= dense_last_key(i0 + r, t.nq, t.nk, a.causal); };
        const bool cut = j0 + TB - 1 > dense_last_key(i0, t.nq, t.nk, a.causal);
        float s[4][4], dp[4][4];
        dot_tile<D>(s, Qs, Ks, ty, tx);
        dot_tile<D>(dp, Gs, Vs, ty, tx);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float ds = exp2f(s[i][j] * sl2 - lse2[i]) * (dp[i][j] - del[i]);
                if (cut && !see(4 * ty + i, tx + 16 * j)) ds = 0.f;
                Ps[(4 * ty + i) * PP + tx + 16 * j] = ds;
            }
        __syncthreads();
        if (cut)
            accumulate<D, true>(acc, Ps, Ks, ty, tx, see);
        else
            accumulate<D, false>(acc, Ps, Ks, ty, tx, see);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i;
        if (r >= rows) continue;
        uint8_t* row = row_ptr<float>(a.dq, b, h, t.q0 + i0 + r);
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
            store2(row, 2 * tx + 32 * c, acc[i][2 * c] * a.scale, acc[i][2 * c + 1] * a.scale);
    }
}

template <int D>
__global__ void __launch_bounds__(256) k_dense_dkv_simt(DenseArgs a, const float* __restrict__ delta) {
    extern __shared__ __align__(16) float smem[];
    float* Ks = smem;
    float* Vs = Ks + TB * (D + 4);
    float* Qs = Vs + TB * (D + 4);
    float* Gs = Qs + TB * (D + 4);
    float* Ps = Gs + TB * (D + 4);
    float* Ds = Ps + TB * PP;
    const SeqTile t = resolve_block(a, blockIdx.x, true);  // causal: the first keys have the most rows
    const int j0 = t.tile * TB;
    if (!t.live || j0 >= t.nk) return;
    const int hk = blockIdx.y, b = blockIdx.z, G = a.Hq / a.Hk;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int keys = min(TB, t.nk - j0);
    load_tile<D>(Ks, row_ptr<float>(a.k, b, hk, t.k0 + j0), a.k.sn, keys);
    load_tile<D>(Vs, row_ptr<float>(a.v, b, hk, t.k0 + j0), a.v.sn, keys);
    float dk[4][D / 16], dv[4][D / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < D / 16; ++c) dk[i][c] = dv[i][c] = 0.f;
    const float sl2 = a.scale * kLog2e;
    const int first = a.causal ? max(0, j0 - (t.nk - t.nq)) / TB * TB : 0;  // first row tile that sees a key here
    for (int g = 0; g < G; ++g) {
        const int h = hk * G + g;
        for (int i0 = first; i0 < t.nq; i0 += TB) {
            const int rows = min(TB, t.nq - i0);
            __syncthreads();
            load_tile<D>(Qs, row_ptr<float>(a.q, b, h, t.q0 + i0), a.q.sn, rows);
            load_tile<D>(Gs, row_ptr<float>(a.d_o, b, h, t.q0 + i0), a.d_o.sn, rows);
            __syncthreads();
            // r: key of the tile, c: query row of the tile
            auto see = [&](int r, int c) {
                return c < rows && r < keys && j0 + r <= dense_last_key(i0 + c, t.nq, t.nk, a.causal);
            };
            const bool cut = rows < TB || j0 + TB - 1 > dense_last_key(i0, t.nq, t.nk, a.causal);
            float s[4][4], dp[4][4];
            dot_tile<D>(s, Ks, Qs, ty, tx);
            dot_tile<D>(dp, Vs, Gs, ty, tx);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = tx + 16 * j;
                const size_t at = ((size_t)b * a.Hq + h) * a.Nq + t.q0 + i0 + c;
                const float lse2 = c < rows ? a.lse[at] * kLog2e : 0.f, del = c < rows ? delta[at] : 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float p = exp2f(s[i][j] * sl2 - lse2);
                    float ds = p * (dp[i][j] - del);
                    if (cut && !see(4 * ty + i, c)) p = ds = 0.f;
                    Ps[(4 * ty + i) * PP + c] = p;
                    Ds[(4 * ty + i) * PP + c] = ds;
                }
            }
            __syncthreads();
            if (cut) {
                accumulate<D, true>(dv, Ps, Gs, ty, tx, see);
                accumulate<D, true>(dk, Ds, Qs, ty, tx, see);
            } else {
                accumulate<D, false>(dv, Ps, Gs, ty, tx, see);
                accumulate<D, false>(dk, Ds, Qs, ty, tx, see);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i;
        if (r >= keys) continue;
        uint8_t* rk = row_ptr<float>(a.dk, b, hk, t.k0 + j0 + r);
        uint8_t* rv = row_ptr<float>(a.dv, b, hk, t.k0 + j0 + r);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            store2(rk, 2 * tx + 32 * c, dk[i][2 * c] * a.scale, dk[i][2 * c + 1] * a.scale);
            store2(rv, 2 * tx + 32 * c, dv[i][2 * c], dv[i][2 * c + 1]);
        }
    }
}

template <int D>
int fwd_simt(const DenseArgs& a, cudaStream_t st) {
    const size_t sm = (size_t)(3 * TB * (D + 4) + TB * PP) * 4;
    cudaFuncSetAttribute(k_dense_fwd_simt<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sm);
    const dim3 grid((unsigned)dense_tiles(a.Nq, a.n_seq, TB), a.Hq, a.B);
    ::park::prof_begin(st);
    k_dense_fwd_simt<D><<<grid, 256, sm, st>>>(a);
    PARK_TRY_LAUNCH("k_dense_fwd_simt", st);
    return PARK_OK;
}

template <int D>
int bwd_simt(const DenseArgs& a, const float* delta, cudaStream_t st) {
    const size_t sq = (size_t)(4 * TB * (D + 4) + TB * PP) * 4, sk = sq + (size_t)TB * PP * 4;
    cudaFuncSetAttribute(k_dense_dq_simt<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sq);
    cudaFuncSetAttribute(k_dense_dkv_simt<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sk);
    if (a.Nq > 0) {
        ::park::prof_begin(st);
        k_dense_dq_simt<D><<<dim3((unsigned)dense_tiles(a.Nq, a.n_seq, TB), a.Hq, a.B), 256, sq, st>>>(a, delta);
        PARK_TRY_LAUNCH("k_dense_dq_simt", st);
    }
    if (a.Nk == 0) return PARK_OK;
    ::park::prof_begin(st);
    k_dense_dkv_simt<D><<<dim3((unsigned)dense_tiles(a.Nk, a.n_seq, TB), a.Hk, a.B), 256, sk, st>>>(a, delta);
    PARK_TRY_LAUNCH("k_dense_dkv_simt", st);
    return PARK_OK;
}

}  // namespace

int launch_dense_delta(const DenseArgs& a, int dtype, float* delta, cudaStream_t st) {
    const long long rows = (long long)a.B * a.Hq * a.Nq;
    const unsigned blocks = (unsigned)((rows + 7) / 8);
    ::park::prof_begin(st);
    if (dtype == PARK_BF16)
        k_dense_delta<bf16_t><<<blocks, 256, 0, st>>>(a, delta);
    else
        k_dense_delta<float><<<blocks, 256, 0, st>>>(a, delta);
    PARK_TRY_LAUNCH("k_dense_delta", st);
    return PARK_OK;
}

#define PARK_BY_D(F, ...)                                              \
    (a.D == 32 ? F<32>(__VA_ARGS__) : a.D == 64 ? F<64>(__VA_ARGS__) \
     : a.D == 96 ? F<96>(__VA_ARGS__) : F<128>(__VA_ARGS__))

int launch_dense_fwd_simt(const DenseArgs& a, cudaStream_t st) { return PARK_BY_D(fwd_simt, a, st); }

int launch_dense_bwd_simt(const DenseArgs& a, const float* delta, cudaStream_t st) {
    return PARK_BY_D(bwd_simt, a, delta, st);
}

}  // namespace park
