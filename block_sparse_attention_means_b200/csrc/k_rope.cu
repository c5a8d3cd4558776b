// Rotary positions over (time, height, width) and the RMS norm of queries and
// keys for each head with the rotation in the same pass, forward and backward.
//
//   rotation   (a, b) -> (a cos - b sin, a sin + b cos) for each pair of a head,
//              angle = (scale pos) theta^(-j/n) of the axis that owns the pair
//   norm       y = R(w x r),  r = (mean x^2 + eps)^-1/2
//   backward   g = R^T dy, h = g w, xh = x r:
//              dx = r (h - xh mean(h xh)),  dw = sum over rows of g xh
//
// Bound by memory: every element is read once and written once (the backward
// pass reads x and dy and forms r again, which costs no traffic).  A warp owns one
// token and walks a side's heads, so the token's cos and sin are looked up once and
// stay in registers; the table (one entry for each position of an axis, not for
// each token) stays in L1/L2.  A head row lies on LPR = D/8 lanes (16 for D = 96, four
// of them idle) with 8 elements, four whole pairs, on each, in either pair order,
// so the rotation needs no exchange between lanes; the norm's sums are log2(LPR)
// shuffles.
#include "kernels.h"

namespace park {
namespace {

// Measured at 24 + 24 heads x 119,056 tokens and 40 + 40 x 75,600, D = 128, bf16.  Forward: 8 blocks of 4 warps 6.30 and
// 6.22 TB/s (6 blocks 5.30 and 5.38, 12 with two rows in flight 5.97 and 6.04).  Backward: 4 blocks 5.92 and 6.22 TB/s (3
// blocks 5.31 and 5.68, 6 blocks 5.39 and 5.69: more warps at once write to more places at once).
constexpr int kWarps = 4, kBlocks = 8;  // warps of a block, blocks of an SM
constexpr int kBwdWarps = 4, kBwdBlocks = 4, kBwdStages = 5;

// The four pairs of a lane, as packed float32 pairs (one instruction for two elements): a[i] = the first
// elements of pairs 2i and 2i + 1, b[i] their second ones.
struct Quad {
    float2 a[2], b[2];
};

struct RopeDev {
    const float2* table;
    const int32_t* pos;
    long long pos_sb;
    int e0, e1, e2, n0, n1, n2;
};

struct Heads {
    const uint8_t* x;
    const uint8_t* dy;  // backward only
    uint8_t* y;         // output; dx in the backward pass
    long long xb, xh, xn, db, dh, dn, yb, yh, yn;  // in bytes
    const void* w;
    int H;
};

template <typename T>
struct Raw;
template <>
struct alignas(16) Raw<bf16_t> {
    uint32_t v[4];
};
template <>
struct alignas(16) Raw<float> {
    uint32_t v[8];
};

// HALF = 0: elements 8l .. 8l+7 of the row; HALF = 1: 4l .. 4l+3 and D/2 + 4l ..
template <bool HALF>
__device__ __forceinline__ void load_raw(Raw<bf16_t>& r, const uint8_t* row, int l, int D) {
    if (HALF) {
        const uint2 a = __ldcs(reinterpret_cast<const uint2*>(row + 8 * l));
        const uint2 b = __ldcs(reinterpret_cast<const uint2*>(row + D + 8 * l));
        r.v[0] = a.x; r.v[1] = a.y; r.v[2] = b.x; r.v[3] = b.y;
    } else {
        const uint4 a = __ldcs(reinterpret_cast<const uint4*>(row + 16 * l));
        r.v[0] = a.x; r.v[1] = a.y; r.v[2] = a.z; r.v[3] = a.w;
    }
}
template <bool HALF>
__device__ __forceinline__ void load_raw(Raw<float>& r, const uint8_t* row, int l, int D) {
    const uint4 a = __ldcs(reinterpret_cast<const uint4*>(row + (HALF ? 16 * l : 32 * l)));
    const uint4 b = __ldcs(reinterpret_cast<const uint4*>(row + (HALF ? 2 * D + 16 * l : 32 * l + 16)));
    r.v[0] = a.x; r.v[1] = a.y; r.v[2] = a.z; r.v[3] = a.w;
    r.v[4] = b.x; r.v[5] = b.y; r.v[6] = b.z; r.v[7] = b.w;
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

template <bool HALF>
__device__ __forceinline__ Quad unpack(const Raw<bf16_t>& r) {
    Quad q;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (HALF) {
            q.a[i] = make_float2(lo_f(r.v[i]), hi_f(r.v[i]));
            q.b[i] = make_float2(lo_f(r.v[2 + i]), hi_f(r.v[2 + i]));
        } else {
            q.a[i] = make_float2(lo_f(r.v[2 * i]), lo_f(r.v[2 * i + 1]));
            q.b[i] = make_float2(hi_f(r.v[2 * i]), hi_f(r.v[2 * i + 1]));
        }
    }
    return q;
}
template <bool HALF>
__device__ __forceinline__ Quad unpack(const Raw<float>& r) {
    const float* v = reinterpret_cast<const float*>(r.v);
    Quad q;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        q.a[i] = HALF ? make_float2(v[2 * i], v[2 * i + 1]) : make_float2(v[4 * i], v[4 * i + 2]);
        q.b[i] = HALF ? make_float2(v[4 + 2 * i], v[5 + 2 * i]) : make_float2(v[4 * i + 1], v[4 * i + 3]);
    }
    return q;
}
template <bool HALF>
__device__ __forceinline__ void store_quad(const Quad& q, uint8_t* row, int l, int D, bf16_t) {
    if (HALF) {
        *reinterpret_cast<uint2*>(row + 8 * l) = make_uint2(pack2(q.a[0].x, q.a[0].y), pack2(q.a[1].x, q.a[1].y));
        *reinterpret_cast<uint2*>(row + D + 8 * l) = make_uint2(pack2(q.b[0].x, q.b[0].y), pack2(q.b[1].x, q.b[1].y));
    } else {
        *reinterpret_cast<uint4*>(row + 16 * l) = make_uint4(pack2(q.a[0].x, q.b[0].x), pack2(q.a[0].y, q.b[0].y),
                                                             pack2(q.a[1].x, q.b[1].x), pack2(q.a[1].y, q.b[1].y));
    }
}
template <bool HALF>
__device__ __forceinline__ void store_quad(const Quad& q, uint8_t* row, int l, int D, float) {
    if (HALF) {
        *reinterpret_cast<float4*>(row + 16 * l) = make_float4(q.a[0].x, q.a[0].y, q.a[1].x, q.a[1].y);
        *reinterpret_cast<float4*>(row + 2 * D + 16 * l) = make_float4(q.b[0].x, q.b[0].y, q.b[1].x, q.b[1].y);
    } else {
        *reinterpret_cast<float4*>(row + 32 * l) = make_float4(q.a[0].x, q.b[0].x, q.a[0].y, q.b[0].y);
        *reinterpret_cast<float4*>(row + 32 * l + 16) = make_float4(q.a[1].x, q.b[1].x, q.a[1].y, q.b[1].y);
    }
}

// The lane's four weights of each half of its pairs, 1 without weights.
template <bool HALF>
__device__ __forceinline__ Quad load_weights(const void* w, int wdtype, int l, int D, bool active) {
    float a[4], b[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int ia = HALF ? 4 * l + e : 8 * l + 2 * e, ib = HALF ? D / 2 + 4 * l + e : 8 * l + 2 * e + 1;
        if (!w || !active) {
            a[e] = b[e] = 1.f;
        } else if (wdtype == PARK_F32) {
            a[e] = static_cast<const float*>(w)[ia];
            b[e] = static_cast<const float*>(w)[ib];
        } else {
            a[e] = Elem<bf16_t>::to_float(static_cast<const bf16_t*>(w), ia);
            b[e] = Elem<bf16_t>::to_float(static_cast<const bf16_t*>(w), ib);
        }
    }
    Quad q;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        q.a[i] = make_float2(a[2 * i], a[2 * i + 1]);
        q.b[i] = make_float2(b[2 * i], b[2 * i + 1]);
    }
    return q;
}

// cos, sin and -sin of the lane's pairs
struct Turn {
    float2 c[2], s[2], n[2];
};

// cos and sin of the lane's four pairs (4l .. 4l+3) for token (b, n)
__device__ __forceinline__ void lookup_angles(const RopeDev& rp, int b, long long n, int l, bool active, float sign,
                                              float (&c)[4], float (&s)[4], int32_t* status) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        c[e] = 1.f;
        s[e] = 0.f;
    }
    if (!rp.table) return;
    int t, y, w;
    if (rp.pos) {
        const int32_t* p = rp.pos + b * rp.pos_sb + 3 * n;
        t = p[0];
        y = p[1];
        w = p[2];
        if (t < 0 || y < 0 || w < 0) return;
        if (t >= rp.e0 || y >= rp.e1 || w >= rp.e2) {
            set_status(status, PARK_ERR_INDEX);
            return;
        }
    } else {
        const long long plane = (long long)rp.e1 * rp.e2;
        const uint32_t n32 = (uint32_t)n, p32 = plane > n ? n32 + 1u : (uint32_t)plane;  // (n < 2^31)
        t = (int)(n32 / p32);
        if (t >= rp.e0) return;
        const uint32_t r = n32 - t * p32;
        y = (int)(r / (uint32_t)rp.e2);
        w = (int)(r - y * (uint32_t)rp.e2);
    }
    if (!active) return;
    const float2* t1 = rp.table + (size_t)rp.e0 * rp.n0;
    const float2* t2 = t1 + (size_t)rp.e1 * rp.n1;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        int j = 4 * l + e;
        const float2* at = nullptr;
        if (j < rp.n0) {
            at = rp.table + (size_t)t * rp.n0 + j;
        } else if ((j -= rp.n0) < rp.n1) {
            at = t1 + (size_t)y * rp.n1 + j;
        } else if ((j -= rp.n1) < rp.n2) {
            at = t2 + (size_t)w * rp.n2 + j;
        }
        if (at) {
            const float2 cs = __ldg(at);
            c[e] = cs.x;
            s[e] = sign * cs.y;
        }
    }
}

__device__ __forceinline__ Turn token_angles(const RopeDev& rp, int b, long long n, int l, bool active, float sign,
                                             int32_t* status) {
    float c[4], s[4];
    lookup_angles(rp, b, n, l, active, sign, c, s, status);
    Turn t;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        t.c[i] = make_float2(c[2 * i], c[2 * i + 1]);
        t.s[i] = make_float2(s[2 * i], s[2 * i + 1]);
        t.n[i] = make_float2(-s[2 * i], -s[2 * i + 1]);
    }
    return t;
}

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
template <int LPR>
__device__ __forceinline__ float2 row_sum(float2 v) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1)
        v = __fadd2_rn(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o)));
    return v;
}

__device__ __forceinline__ Quad rotate(const Quad& q, const Turn& t) {
    Quad r;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        r.a[i] = __ffma2_rn(q.b[i], t.n[i], __fmul2_rn(q.a[i], t.c[i]));
        r.b[i] = __ffma2_rn(q.a[i], t.s[i], __fmul2_rn(q.b[i], t.c[i]));
    }
    return r;
}
// sum of x y over the lane's elements
__device__ __forceinline__ float dot(const Quad& x, const Quad& y) {
    float2 v = __fmul2_rn(x.a[0], y.a[0]);
    v = __ffma2_rn(x.a[1], y.a[1], v);
    v = __ffma2_rn(x.b[0], y.b[0], v);
    v = __ffma2_rn(x.b[1], y.b[1], v);
    return v.x + v.y;
}
__device__ __forceinline__ Quad mul(const Quad& x, const Quad& y) {
    Quad r;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        r.a[i] = __fmul2_rn(x.a[i], y.a[i]);
        r.b[i] = __fmul2_rn(x.b[i], y.b[i]);
    }
    return r;
}
__device__ __forceinline__ Quad mul(const Quad& x, float f) {
    const float2 f2 = make_float2(f, f);
    return mul(x, Quad{{f2, f2}, {f2, f2}});
}
__device__ __forceinline__ Quad fma(const Quad& x, const Quad& y, const Quad& z) {
    Quad r;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        r.a[i] = __ffma2_rn(x.a[i], y.a[i], z.a[i]);
        r.b[i] = __ffma2_rn(x.b[i], y.b[i], z.b[i]);
    }
    return r;
}
__device__ __forceinline__ Quad fma(const Quad& x, float f, const Quad& z) {
    const float2 f2 = make_float2(f, f);
    return fma(x, Quad{{f2, f2}, {f2, f2}}, z);
}

// A warp owns a token and a chunk of the heads of Q or of K: blockIdx.y < cq counts the chunks of Q, the others those of K
// (one chunk each unless the tokens alone would not fill the SMs).
template <typename T, bool HALF, bool NORM, int LPR>
__global__ void __launch_bounds__(32 * kWarps, kBlocks)
    k_rope(Heads q, Heads k, RopeDev rp, int B, long long N, int D, float eps, int wdtype, float sign, int chunk, int cq,
           int32_t* status) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long tok = (long long)blockIdx.x * kWarps + warp;
    if (tok >= B * N) return;
    const int b = B == 1 ? 0 : (int)((uint32_t)tok / (uint32_t)N);  // (B N < 2^31)
    const long long n = tok - (long long)b * N;
    const bool isk = (int)blockIdx.y >= cq;
    const int h0 = ((int)blockIdx.y - (isk ? cq : 0)) * chunk, h1 = min(isk ? k.H : q.H, h0 + chunk);
    const long long xh = isk ? k.xh : q.xh, yh = isk ? k.yh : q.yh;
    const uint8_t* x = isk ? k.x + b * k.xb + n * k.xn : q.x + b * q.xb + n * q.xn;
    uint8_t* y = isk ? k.y + b * k.yb + n * k.yn : q.y + b * q.yb + n * q.yn;
    const int l = lane % LPR, grp = lane / LPR;
    const bool active = 8 * l < D;
    constexpr int RPW = 32 / LPR;  // rows of a warp step
    constexpr int kUnroll = 64 / sizeof(Raw<T>);  // rows in flight for each lane group: 64 bytes a lane fit the registers
    Raw<T> raw[kUnroll];
    auto load = [&](int u, int hh) {
        if (hh < h1 && active) {
            load_raw<HALF>(raw[u], x + hh * xh, l, D);
        } else {
#pragma unroll
            for (uint32_t& v : raw[u].v) v = 0u;
        }
    };
    // The first rows travel while the angles are looked up, the next ones while these are worked on (12 + 12 heads x 37,800
    // tokens, D = 128: the rotation of bf16 heads 5.0 -> 5.4 TB/s, norm and rotation in float32 5.6 -> 6.1, in bf16 4.8 -> 4.9).
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) load(u, h0 + grp + u * RPW);
    const Turn turn = token_angles(rp, b, n, l, active, sign, status);
    Quad w;
    if (NORM) w = load_weights<HALF>(isk ? k.w : q.w, wdtype, l, D, active);
    const float inv_d = 1.f / (float)D;
    for (int h = h0 + grp; h - grp < h1; h += RPW * kUnroll) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int hh = h + u * RPW;
            Quad v = unpack<HALF>(raw[u]);
            load(u, hh + RPW * kUnroll);
            if (NORM) {
                const float r = rsqrtf(row_sum<LPR>(dot(v, v)) * inv_d + eps);
                v = mul(v, mul(w, r));
            }
            if (hh < h1 && active) store_quad<HALF>(rotate(v, turn), y + hh * yh, l, D, T{});
        }
    }
}

// Asynchronous copy of the lane's part of a row into its own places of a stage in shared memory.  A float32 part is two
// 16-byte pieces: neighbours where they are neighbours in the row, else in a half of the stage each, so that the pieces of a
// 128-byte line lie as in memory (the other way round 3.6 instead of 5.3 TB/s, in both orders of pairs).
template <bool HALF>
__device__ __forceinline__ void copy_raw(Raw<bf16_t>* stage, const uint8_t* row, int lane, int l, int D) {
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(stage + lane);
    if (HALF) {
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(d), "l"(row + 8 * l) : "memory");
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(d + 8), "l"(row + D + 8 * l) : "memory");
    } else {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(row + 16 * l) : "memory");
    }
}
template <bool HALF>
__device__ __forceinline__ void copy_raw(Raw<float>* stage, const uint8_t* row, int lane, int l, int D) {
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(stage) + (HALF ? 16 : 32) * lane;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(row + (HALF ? 16 * l : 32 * l)) : "memory");
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d + (HALF ? 512 : 16)),
                 "l"(row + (HALF ? 2 * D + 16 * l : 32 * l + 16))
                 : "memory");
}
template <bool HALF>
__device__ __forceinline__ void read_raw(Raw<bf16_t>& r, const Raw<bf16_t>* stage, int lane) {
    r = stage[lane];
}
template <bool HALF>
__device__ __forceinline__ void read_raw(Raw<float>& r, const Raw<float>* stage, int lane) {
    const uint4* at = reinterpret_cast<const uint4*>(stage) + (HALF ? 1 : 2) * lane;
    const uint4 a = at[0], b = at[HALF ? 32 : 1];
    r.v[0] = a.x; r.v[1] = a.y; r.v[2] = a.z; r.v[3] = a.w;
    r.v[4] = b.x; r.v[5] = b.y; r.v[6] = b.z; r.v[7] = b.w;
}

// Backward of the norm and rotation.  Blocks below `bq` stride over the items (token, chunk of heads) of Q, the others over
// those of K; each warp keeps its part of dw in registers over all of its rows, the block adds the warps' parts in order
// and writes one partial row, and k_dw_reduce adds the blocks'.  A row needs three times the forward pass's
// arithmetic: with scalar arithmetic instruction issue was the bound (76 % busy), with packed pairs and loads into registers
// latency was; so the loads run kBwdStages steps ahead through the lane's own places in shared memory, across tokens.
template <typename T, bool HALF, int LPR>
__global__ void __launch_bounds__(32 * kBwdWarps, kBwdBlocks)
    k_norm_rope_bwd(Heads q, Heads k, RopeDev rp, int B, long long N, int D, float eps, int wdtype, int chunk, int bq,
                    float* __restrict__ part, int32_t* status) {
    __shared__ Raw<T> ring[kBwdWarps][kBwdStages][2][32];
    __shared__ float red[kBwdWarps][128];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int l = lane % LPR, grp = lane / LPR;
    const bool active = 8 * l < D;
    constexpr int RPW = 32 / LPR;
    const bool isk = (int)blockIdx.x >= bq;
    const int block = (int)blockIdx.x - (isk ? bq : 0), blocks = isk ? (int)gridDim.x - bq : bq;
    const int H = isk ? k.H : q.H;
    const long long xb = isk ? k.xb : q.xb, xh = isk ? k.xh : q.xh, xn = isk ? k.xn : q.xn;
    const long long gb = isk ? k.db : q.db, gh = isk ? k.dh : q.dh, gn = isk ? k.dn : q.dn;
    const long long yb = isk ? k.yb : q.yb, yh = isk ? k.yh : q.yh, yn = isk ? k.yn : q.yn;
    const uint8_t *px = isk ? k.x : q.x, *pg = isk ? k.dy : q.dy;
    uint8_t* py = isk ? k.y : q.y;
    const Quad w = load_weights<HALF>(isk ? k.w : q.w, wdtype, l, D, active);
    const float2 zero = make_float2(0.f, 0.f);
    Quad dw{{zero, zero}, {zero, zero}};
    const float inv_d = 1.f / (float)D;
    // (chunks are cut only for few tokens: the items' count fits 32 bits)
    const uint32_t n_chunks = (uint32_t)((H + chunk - 1) / chunk), items = (uint32_t)(B * N) * n_chunks;
    const uint32_t stride = (uint32_t)blocks * kBwdWarps, first = (uint32_t)block * kBwdWarps + warp;
    // walks: of the loads (x, dy) and of the arithmetic and stores (y)
    uint32_t it_in = first, it_at = first, n_at = 0;
    int left_in = 0, left_at = 0, b_at = 0;  // heads of the chunk that are left, from this lane group's
    const uint8_t *in_x = nullptr, *in_g = nullptr;
    uint8_t* at_y = nullptr;
    auto token = [&](uint32_t it, int& b, uint32_t& n, int& h0, int& left) {
        const uint32_t tok = n_chunks == 1 ? it : it / n_chunks, ch = it - tok * n_chunks;
        b = B == 1 ? 0 : (int)(tok / (uint32_t)N);
        n = tok - (uint32_t)b * (uint32_t)N;
        h0 = (int)ch * chunk;
        left = min(chunk, H - h0) - grp;
        h0 += grp;
    };
    auto enter_in = [&]() {
        if (it_in >= items) return;
        int b, h0;
        uint32_t n;
        token(it_in, b, n, h0, left_in);
        in_x = px + b * xb + n * xn + h0 * xh;
        in_g = pg + b * gb + n * gn + h0 * gh;
    };
    auto enter_at = [&]() {
        if (it_at >= items) return;
        int h0;
        token(it_at, b_at, n_at, h0, left_at);
        at_y = py + b_at * yb + n_at * yn + h0 * yh;
    };
    enter_in();
    enter_at();
    int slot_in = 0, slot = 0;
    auto fetch = [&]() {
        if (it_in < items) {
            if (left_in > 0 && active) {
                copy_raw<HALF>(ring[warp][slot_in][0], in_x, lane, l, D);
                copy_raw<HALF>(ring[warp][slot_in][1], in_g, lane, l, D);
            }
            left_in -= RPW;
            in_x += RPW * xh;
            in_g += RPW * gh;
            if (left_in + grp <= 0) {
                it_in = items - it_in > stride ? it_in + stride : items;
                enter_in();
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        slot_in = slot_in + 1 == kBwdStages ? 0 : slot_in + 1;
    };
#pragma unroll
    for (int i = 0; i < kBwdStages - 1; ++i) fetch();
    Turn turn;
    uint32_t angles_of = 0xffffffffu;
    while (it_at < items) {
        fetch();
        if (angles_of != it_at) {
            turn = token_angles(rp, b_at, n_at, l, active, -1.f, status);
            angles_of = it_at;
        }
        asm volatile("cp.async.wait_group %0;" ::"n"(kBwdStages - 1) : "memory");
        const bool on = left_at > 0 && active;
        Raw<T> rx, rd;
        if (on) {
            read_raw<HALF>(rx, ring[warp][slot][0], lane);
            read_raw<HALF>(rd, ring[warp][slot][1], lane);
        } else {
#pragma unroll
            for (uint32_t& v : rx.v) v = 0u;
#pragma unroll
            for (uint32_t& v : rd.v) v = 0u;
        }
        slot = slot + 1 == kBwdStages ? 0 : slot + 1;
        const Quad xx = unpack<HALF>(rx);
        const Quad g = rotate(unpack<HALF>(rd), turn);
        const Quad gx = mul(g, xx);
        const float2 sums = row_sum<LPR>(make_float2(dot(xx, xx), dot(gx, w)));  // sum x^2, sum h x
        const float r = rsqrtf(sums.x * inv_d + eps);
        dw = fma(gx, r, dw);  // (rows past the end hold zeros)
        // dx = r (g w - x r mean(h xh)), mean(h xh) = r sum(h x) / D; the mean first: r^3 alone leaves float32's range at rows
        // of 1e13
        const float mean = sums.y * r * inv_d;
        const Quad dx = fma(g, mul(w, r), mul(xx, -mean * r * r));
        if (on) store_quad<HALF>(dx, at_y, l, D, T{});
        left_at -= RPW;
        at_y += RPW * yh;
        if (left_at + grp <= 0) {
            it_at = items - it_at > stride ? it_at + stride : items;
            enter_at();
        }
    }
    // the lane groups of a warp, then the warps of the block, in a fixed order
    float da[4] = {dw.a[0].x, dw.a[0].y, dw.a[1].x, dw.a[1].y}, db[4] = {dw.b[0].x, dw.b[0].y, dw.b[1].x, dw.b[1].y};
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            da[e] += __shfl_xor_sync(0xffffffffu, da[e], o);
            db[e] += __shfl_xor_sync(0xffffffffu, db[e], o);
        }
    if (grp == 0 && active) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            red[warp][HALF ? 4 * l + e : 8 * l + 2 * e] = da[e];
            red[warp][HALF ? D / 2 + 4 * l + e : 8 * l + 2 * e + 1] = db[e];
        }
    }
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += 32 * kBwdWarps) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < kBwdWarps; ++i) v += red[i][d];
        part[(size_t)blockIdx.x * D + d] = v;
    }
}

// dw = sum over the partial rows of a side's blocks: 32 columns by 32 groups of rows, the groups added in order.
__global__ void __launch_bounds__(1024) k_dw_reduce(const float* __restrict__ part, int bq, int blocks, int D, float* dwq,
                                                    float* dwk) {
    __shared__ float red[32][33];
    const int lane = threadIdx.x & 31, g = threadIdx.x >> 5, d = blockIdx.x * 32 + lane;
    const int i0 = blockIdx.y ? bq : 0, i1 = blockIdx.y ? blocks : bq;
    float v = 0.f;
#pragma unroll 8
    for (int i = i0 + g; i < i1; i += 32) v += part[(size_t)i * D + d];
    red[g][lane] = v;
    __syncthreads();
    const float t = warp_sum(red[lane][g]);  // warp g: column g
    float* out = blockIdx.y ? dwk : dwq;
    if (out && lane == 0) out[blockIdx.x * 32 + g] = t;
}

__global__ void k_rope_table(float2* table, int extent, int n, double theta, double scale) {
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= extent * n) return;
    const int pos = i / n, j = i - pos * n;
    double s, c;
    sincos(scale * pos * pow(theta, -(double)j / (double)n), &s, &c);
    table[i] = make_float2((float)c, (float)s);
}

RopeDev rope_dev(const park_rope_axes* r, const int32_t* pos, long long pos_sb) {
    RopeDev d{};
    if (r) {
        d.table = reinterpret_cast<const float2*>(r->table);
        d.pos = pos;
        d.pos_sb = pos_sb;
        d.e0 = r->extent[0];
        d.e1 = r->extent[1];
        d.e2 = r->extent[2];
        d.n0 = r->pairs[0];
        d.n1 = r->pairs[1];
        d.n2 = r->pairs[2];
    }
    return d;
}

Heads heads(const park_operand* x, const park_operand* y, const park_operand* dy, const void* w, int elt) {
    Heads h{};
    if (!x) return h;
    h.x = static_cast<const uint8_t*>(x->ptr);
    h.xb = x->sb * elt;
    h.xh = x->sh * elt;
    h.xn = x->sn * elt;
    h.y = static_cast<uint8_t*>(y->ptr);
    h.yb = y->sb * elt;
    h.yh = y->sh * elt;
    h.yn = y->sn * elt;
    if (dy) {
        h.dy = static_cast<const uint8_t*>(dy->ptr);
        h.db = dy->sb * elt;
        h.dh = dy->sh * elt;
        h.dn = dy->sn * elt;
    }
    h.w = w;
    h.H = x->H;
    return h;
}

// Heads of a chunk: all of a side when the tokens of both sides alone give every SM its 64 warps, else as few as
// fill them, at least one step of a warp.
int head_chunk(long long tokens, int H, int rpw, int num_sms) {
    const long long want = (32ll * num_sms + tokens - 1) / tokens;
    long long chunk = (H + want - 1) / want;
    chunk = (chunk + rpw - 1) / rpw * rpw;
    return (int)(chunk < rpw ? rpw : chunk);
}

}  // namespace

int launch_rope_table(const park_rope_axes* r, double theta, const double* scale, cudaStream_t st) {
    float2* t = reinterpret_cast<float2*>(r->table);
    for (int a = 0; a < 3; ++a) {
        const int n = r->extent[a] * r->pairs[a];
        if (n == 0) continue;
        ::park::prof_begin(st);
        k_rope_table<<<(n + 255) / 256, 256, 0, st>>>(t, r->extent[a], r->pairs[a], theta, scale[a]);
        PARK_TRY_LAUNCH("k_rope_table", st);
        t += n;
    }
    return PARK_OK;
}

int launch_rope(const park_operand* q, const park_operand* k, const park_operand* yq, const park_operand* yk,
                const void* wq, const void* wk, int wdtype, float eps, bool norm, const park_rope_axes* rope,
                const int32_t* pos, long long pos_sb, bool inverse, int B, long long N, int D, int dtype,
                int32_t* status, int num_sms, cudaStream_t st) {
    const int elt = dtype == PARK_BF16 ? 2 : 4;
    const Heads hq = heads(q, yq, nullptr, wq, elt), hk = heads(k, yk, nullptr, wk, elt);
    const RopeDev rp = rope_dev(rope, pos, pos_sb);
    const int lpr = D == 32 ? 4 : (D == 64 ? 8 : 16);
    const int chunk = head_chunk(B * N, hq.H > hk.H ? hq.H : hk.H, 32 / lpr, num_sms);
    const int cq = (hq.H + chunk - 1) / chunk, ck = (hk.H + chunk - 1) / chunk;
    const dim3 grid((unsigned)((B * N + kWarps - 1) / kWarps), (unsigned)(cq + ck));
    const float sign = inverse ? -1.f : 1.f;
    if (grid.y > 65535u) return PARK_ERR_UNSUPPORTED;
    const bool half = rope && rope->half;
    ::park::prof_begin(st);
#define GO(T, HALF, NORM, LPR) \
    k_rope<T, HALF, NORM, LPR><<<grid, 32 * kWarps, 0, st>>>(hq, hk, rp, B, N, D, eps, wdtype, sign, chunk, cq, status)
#define GO_L(T, HALF, NORM)                     \
    do {                                        \
        if (lpr == 4) GO(T, HALF, NORM, 4);     \
        else if (lpr == 8) GO(T, HALF, NORM, 8); \
        else GO(T, HALF, NORM, 16);             \
    } while (0)
#define GO_H(T, NORM)                 \
    do {                              \
        if (half) GO_L(T, true, NORM); \
        else GO_L(T, false, NORM);    \
    } while (0)
    if (dtype == PARK_BF16) {
        if (norm) GO_H(bf16_t, true);
        else GO_H(bf16_t, false);
    } else {
        if (norm) GO_H(float, true);
        else GO_H(float, false);
    }
#undef GO_H
#undef GO_L
#undef GO
    PARK_TRY_LAUNCH(norm ? "k_qk_norm_rope" : "k_rope", st);
    return PARK_OK;
}

int norm_rope_bwd_blocks(long long tokens) {
    // two sides at least; small calls cut a token's heads into chunks, so they may take more blocks than tokens / warps
    const long long b = 2 + (tokens * 8 + kBwdWarps - 1) / kBwdWarps, most = (long long)kBwdBlocks * 148;
    return (int)(b < most ? b : most);
}

int launch_norm_rope_bwd(const park_operand* dyq, const park_operand* dyk, const park_operand* q,
                         const park_operand* k, const park_operand* dq, const park_operand* dk, const void* wq,
                         const void* wk, int wdtype, float eps, const park_rope_axes* rope, const int32_t* pos,
                         long long pos_sb, float* dwq, float* dwk, int B, long long N, int D, int dtype, float* part,
                         int32_t* status, int num_sms, cudaStream_t st) {
    const int elt = dtype == PARK_BF16 ? 2 : 4;
    const Heads hq = heads(q, dq, dyq, wq, elt), hk = heads(k, dk, dyk, wk, elt);
    const RopeDev rp = rope_dev(rope, pos, pos_sb);
    const int lpr = D == 32 ? 4 : (D == 64 ? 8 : 16);
    const int Hm = hq.H > hk.H ? hq.H : hk.H, chunk = N ? head_chunk(B * N, Hm, 32 / lpr, num_sms) : Hm;
    const int blocks = norm_rope_bwd_blocks(B * N);
    int bq = (int)((long long)blocks * hq.H / (hq.H + hk.H));  // shares of the blocks as the sides' rows
    bq = bq < 1 ? 1 : (bq > blocks - 1 ? blocks - 1 : bq);
    const bool half = rope && rope->half;
    ::park::prof_begin(st);
#define GO(T, HALF, LPR)                                                                                             \
    k_norm_rope_bwd<T, HALF, LPR><<<blocks, 32 * kBwdWarps, 0, st>>>(hq, hk, rp, B, N, D, eps, wdtype, chunk, bq, \
                                                                     part, status)
#define GO_L(T, HALF)                    \
    do {                                 \
        if (lpr == 4) GO(T, HALF, 4);    \
        else if (lpr == 8) GO(T, HALF, 8); \
        else GO(T, HALF, 16);            \
    } while (0)
    if (dtype == PARK_BF16) {
        if (half) GO_L(bf16_t, true);
        else GO_L(bf16_t, false);
    } else {
        if (half) GO_L(float, true);
        else GO_L(float, false);
    }
#undef GO_L
#undef GO
    PARK_TRY_LAUNCH("k_norm_rope_bwd", st);
    if (!dwq && !dwk) return PARK_OK;
    ::park::prof_begin(st);
    k_dw_reduce<<<dim3(D / 32, 2), 1024, 0, st>>>(part, bq, blocks, D, dwq, dwk);
    PARK_TRY_LAUNCH("k_dw_reduce", st);
    return PARK_OK;
}

}  // namespace park
