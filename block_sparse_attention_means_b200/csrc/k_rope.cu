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
// token and walks its heads, so the token's cos and sin are looked up once and stay
// in registers for all heads of Q and K; the table (one entry for each position of
// an axis, not for each token) stays in L1/L2.  A head row lies on LPR = D/8 lanes
// (16 for D = 96, four of them idle) with 8 elements, four whole pairs, on each, in
// either pair order, so the rotation needs no exchange between lanes; the norm's
// sums are log2(LPR) shuffles.  Four rows are in flight for each lane group before
// the first is used.
#include "kernels.h"

namespace park {
namespace {

constexpr int kWarps = 8;    // warps of a block
constexpr int kUnroll = 4;   // head rows in flight for each lane group

struct Quad {  // the four pairs of a lane
    float a[4], b[4];
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
struct Raw<bf16_t> {
    uint32_t v[4];
};
template <>
struct Raw<float> {
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
    if (HALF) {
        q.a[0] = lo_f(r.v[0]); q.a[1] = hi_f(r.v[0]); q.a[2] = lo_f(r.v[1]); q.a[3] = hi_f(r.v[1]);
        q.b[0] = lo_f(r.v[2]); q.b[1] = hi_f(r.v[2]); q.b[2] = lo_f(r.v[3]); q.b[3] = hi_f(r.v[3]);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            q.a[e] = lo_f(r.v[e]);
            q.b[e] = hi_f(r.v[e]);
        }
    }
    return q;
}
template <bool HALF>
__device__ __forceinline__ Quad unpack(const Raw<float>& r) {
    Quad q;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        q.a[e] = __uint_as_float(r.v[HALF ? e : 2 * e]);
        q.b[e] = __uint_as_float(r.v[HALF ? 4 + e : 2 * e + 1]);
    }
    return q;
}
template <bool HALF>
__device__ __forceinline__ void store_quad(const Quad& q, uint8_t* row, int l, int D, bf16_t) {
    if (HALF) {
        *reinterpret_cast<uint2*>(row + 8 * l) = make_uint2(pack2(q.a[0], q.a[1]), pack2(q.a[2], q.a[3]));
        *reinterpret_cast<uint2*>(row + D + 8 * l) = make_uint2(pack2(q.b[0], q.b[1]), pack2(q.b[2], q.b[3]));
    } else {
        *reinterpret_cast<uint4*>(row + 16 * l) = make_uint4(pack2(q.a[0], q.b[0]), pack2(q.a[1], q.b[1]),
                                                             pack2(q.a[2], q.b[2]), pack2(q.a[3], q.b[3]));
    }
}
template <bool HALF>
__device__ __forceinline__ void store_quad(const Quad& q, uint8_t* row, int l, int D, float) {
    if (HALF) {
        *reinterpret_cast<float4*>(row + 16 * l) = make_float4(q.a[0], q.a[1], q.a[2], q.a[3]);
        *reinterpret_cast<float4*>(row + 2 * D + 16 * l) = make_float4(q.b[0], q.b[1], q.b[2], q.b[3]);
    } else {
        *reinterpret_cast<float4*>(row + 32 * l) = make_float4(q.a[0], q.b[0], q.a[1], q.b[1]);
        *reinterpret_cast<float4*>(row + 32 * l + 16) = make_float4(q.a[2], q.b[2], q.a[3], q.b[3]);
    }
}

// The lane's four weights of each half of its pairs, 1 without weights.
template <bool HALF>
__device__ __forceinline__ Quad load_weights(const void* w, int wdtype, int l, int D, bool active) {
    Quad q;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int ia = HALF ? 4 * l + e : 8 * l + 2 * e, ib = HALF ? D / 2 + 4 * l + e : 8 * l + 2 * e + 1;
        if (!w || !active) {
            q.a[e] = q.b[e] = 1.f;
        } else if (wdtype == PARK_F32) {
            q.a[e] = static_cast<const float*>(w)[ia];
            q.b[e] = static_cast<const float*>(w)[ib];
        } else {
            q.a[e] = Elem<bf16_t>::to_float(static_cast<const bf16_t*>(w), ia);
            q.b[e] = Elem<bf16_t>::to_float(static_cast<const bf16_t*>(w), ib);
        }
    }
    return q;
}

// cos and sin of the lane's four pairs (4l .. 4l+3) for token (b, n)
__device__ __forceinline__ void token_angles(const RopeDev& rp, int b, long long n, int l, bool active, float sign,
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
        if (n >= plane * rp.e0) return;
        t = (int)(n / plane);
        const int r = (int)(n - t * plane);
        y = r / rp.e2;
        w = r - y * rp.e2;
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

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ Quad rotate(const Quad& q, const float (&c)[4], const float (&s)[4]) {
    Quad r;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        r.a[e] = q.a[e] * c[e] - q.b[e] * s[e];
        r.b[e] = q.a[e] * s[e] + q.b[e] * c[e];
    }
    return r;
}

// Work items are (token, chunk of the concatenated heads of Q and K); the launch
// cuts the heads into chunks only when the tokens alone would not fill the SMs.
template <typename T, bool HALF, bool NORM, int LPR>
__global__ void __launch_bounds__(32 * kWarps)
    k_rope(Heads q, Heads k, RopeDev rp, int B, long long N, int D, float eps, int wdtype, float sign, int chunk,
           int32_t* status) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long tok = (long long)blockIdx.x * kWarps + warp;
    if (tok >= B * N) return;
    const int b = (int)(tok / N);
    const long long n = tok - (long long)b * N;
    const int l = lane % LPR, grp = lane / LPR;
    const bool active = 8 * l < D;
    constexpr int RPW = 32 / LPR;  // rows of a warp step
    float c[4], s[4];
    token_angles(rp, b, n, l, active, sign, c, s, status);
    Quad wq, wk;
    if (NORM) {
        wq = load_weights<HALF>(q.w, wdtype, l, D, active);
        wk = load_weights<HALF>(k.w, wdtype, l, D, active);
    }
    const int Ht = q.H + k.H;
    const int h0 = blockIdx.y * chunk, h1 = min(Ht, h0 + chunk);
    const float inv_d = 1.f / (float)D;
    for (int h = h0 + grp; h - grp < h1; h += RPW * kUnroll) {
        Raw<T> raw[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int hh = h + u * RPW;
            const bool isk = hh >= q.H;
            const uint8_t* row = isk ? k.x + b * k.xb + (hh - q.H) * k.xh + n * k.xn : q.x + b * q.xb + hh * q.xh + n * q.xn;
            if (hh < h1 && active) {
                load_raw<HALF>(raw[u], row, l, D);
            } else {
#pragma unroll
                for (uint32_t& v : raw[u].v) v = 0u;
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int hh = h + u * RPW;
            const bool isk = hh >= q.H;
            Quad v = unpack<HALF>(raw[u]);
            if (NORM) {
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) ss += v.a[e] * v.a[e] + v.b[e] * v.b[e];
                const float r = rsqrtf(row_sum<LPR>(ss) * inv_d + eps);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v.a[e] *= r * (isk ? wk.a[e] : wq.a[e]);
                    v.b[e] *= r * (isk ? wk.b[e] : wq.b[e]);
                }
            }
            if (hh < h1 && active) {
                uint8_t* row = isk ? k.y + b * k.yb + (hh - q.H) * k.yh + n * k.yn
                                   : q.y + b * q.yb + hh * q.yh + n * q.yn;
                store_quad<HALF>(rotate(v, c, s), row, l, D, T{});
            }
        }
    }
}

// Backward of the norm and rotation.  Blocks stride over the items; each warp keeps
// its part of dw (both sides) in registers over all of its rows, the block adds the
// warps' parts in order and writes one partial row, and k_dw_reduce adds the blocks'.
template <typename T, bool HALF, int LPR>
__global__ void __launch_bounds__(32 * kWarps)
    k_norm_rope_bwd(Heads q, Heads k, RopeDev rp, int B, long long N, int D, float eps, int wdtype, int chunk,
                    int n_chunks, float* __restrict__ part, int32_t* status) {
    __shared__ float red[kWarps][2][128];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int l = lane % LPR, grp = lane / LPR;
    const bool active = 8 * l < D;
    constexpr int RPW = 32 / LPR;
    constexpr int U = 2;  // rows in flight (x and dy each)
    const Quad wq = load_weights<HALF>(q.w, wdtype, l, D, active), wk = load_weights<HALF>(k.w, wdtype, l, D, active);
    Quad dwq, dwk;
#pragma unroll
    for (int e = 0; e < 4; ++e) dwq.a[e] = dwq.b[e] = dwk.a[e] = dwk.b[e] = 0.f;
    const int Ht = q.H + k.H;
    const float inv_d = 1.f / (float)D;
    const long long items = (long long)B * N * n_chunks;
    for (long long it = (long long)blockIdx.x * kWarps + warp; it < items; it += (long long)gridDim.x * kWarps) {
        const long long tok = it / n_chunks;
        const int ch = (int)(it - tok * n_chunks);
        const int b = (int)(tok / N);
        const long long n = tok - (long long)b * N;
        float c[4], s[4];
        token_angles(rp, b, n, l, active, -1.f, c, s, status);
        const int h0 = ch * chunk, h1 = min(Ht, h0 + chunk);
        for (int h = h0 + grp; h - grp < h1; h += RPW * U) {
            Raw<T> rx[U], rd[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int hh = h + u * RPW;
                const bool isk = hh >= q.H;
                if (hh < h1 && active) {
                    load_raw<HALF>(rx[u], isk ? k.x + b * k.xb + (hh - q.H) * k.xh + n * k.xn
                                              : q.x + b * q.xb + hh * q.xh + n * q.xn, l, D);
                    load_raw<HALF>(rd[u], isk ? k.dy + b * k.db + (hh - q.H) * k.dh + n * k.dn
                                              : q.dy + b * q.db + hh * q.dh + n * q.dn, l, D);
                } else {
#pragma unroll
                    for (uint32_t& v : rx[u].v) v = 0u;
#pragma unroll
                    for (uint32_t& v : rd[u].v) v = 0u;
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int hh = h + u * RPW;
                const bool isk = hh >= q.H;
                Quad x = unpack<HALF>(rx[u]);
                const Quad g = rotate(unpack<HALF>(rd[u]), c, s);
                float ss = 0.f, hx = 0.f;
                Quad hg;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    hg.a[e] = g.a[e] * (isk ? wk.a[e] : wq.a[e]);
                    hg.b[e] = g.b[e] * (isk ? wk.b[e] : wq.b[e]);
                    ss += x.a[e] * x.a[e] + x.b[e] * x.b[e];
                    hx += hg.a[e] * x.a[e] + hg.b[e] * x.b[e];
                }
                const float r = rsqrtf(row_sum<LPR>(ss) * inv_d + eps);
                const float m = row_sum<LPR>(hx) * r * inv_d;  // mean(h xh)
                Quad dx;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float xa = x.a[e] * r, xb = x.b[e] * r;
                    dx.a[e] = r * (hg.a[e] - xa * m);
                    dx.b[e] = r * (hg.b[e] - xb * m);
                    // rows past the end hold zeros and add nothing
                    if (isk) {
                        dwk.a[e] += g.a[e] * xa;
                        dwk.b[e] += g.b[e] * xb;
                    } else {
                        dwq.a[e] += g.a[e] * xa;
                        dwq.b[e] += g.b[e] * xb;
                    }
                }
                if (hh < h1 && active)
                    store_quad<HALF>(dx, isk ? k.y + b * k.yb + (hh - q.H) * k.yh + n * k.yn
                                             : q.y + b * q.yb + hh * q.yh + n * q.yn, l, D, T{});
            }
        }
    }
    // the lane groups of a warp, then the warps of the block, in a fixed order
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            dwq.a[e] += __shfl_xor_sync(0xffffffffu, dwq.a[e], o);
            dwq.b[e] += __shfl_xor_sync(0xffffffffu, dwq.b[e], o);
            dwk.a[e] += __shfl_xor_sync(0xffffffffu, dwk.a[e], o);
            dwk.b[e] += __shfl_xor_sync(0xffffffffu, dwk.b[e], o);
        }
    if (grp == 0 && active) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int ia = HALF ? 4 * l + e : 8 * l + 2 * e, ib = HALF ? D / 2 + 4 * l + e : 8 * l + 2 * e + 1;
            red[warp][0][ia] = dwq.a[e];
            red[warp][0][ib] = dwq.b[e];
            red[warp][1][ia] = dwk.a[e];
            red[warp][1][ib] = dwk.b[e];
        }
    }
    __syncthreads();
    const int side = threadIdx.x >> 7, d = threadIdx.x & 127;
    if (d < D) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += red[w][side][d];
        part[((size_t)blockIdx.x * 2 + side) * D + d] = v;
    }
}

// dw[side][d] = sum over the blocks' partial rows; one warp for each 32 columns of a
// row group, eight row groups added in order.
__global__ void __launch_bounds__(256) k_dw_reduce(const float* __restrict__ part, int blocks, int D, float* dwq,
                                                   float* dwk) {
    __shared__ float red[8][32];
    const int side = blockIdx.y, d = blockIdx.x * 32 + (threadIdx.x & 31), g = threadIdx.x >> 5;
    float v = 0.f;
    for (int i = g; i < blocks; i += 8) v += part[((size_t)i * 2 + side) * D + d];
    red[g][threadIdx.x & 31] = v;
    __syncthreads();
    if (g == 0) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) t += red[i][threadIdx.x];
        float* out = side ? dwk : dwq;
        if (out) out[d] = t;
    }
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

// Head chunks of an item: whole tokens when those give every SM its 64 warps, else
// as many chunks as fill them, at least one step of a warp each.
int head_chunk(long long tokens, int Ht, int rpw, int num_sms) {
    const long long want = (64ll * num_sms + tokens - 1) / tokens;
    long long chunk = (Ht + want - 1) / want;
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
    const int Ht = hq.H + hk.H, lpr = D == 32 ? 4 : (D == 64 ? 8 : 16);
    const int chunk = head_chunk(B * N, Ht, 32 / lpr, num_sms);
    const dim3 grid((unsigned)((B * N + kWarps - 1) / kWarps), (unsigned)((Ht + chunk - 1) / chunk));
    const float sign = inverse ? -1.f : 1.f;
    if (grid.y > 65535u) return PARK_ERR_UNSUPPORTED;
    const bool half = rope && rope->half;
    ::park::prof_begin(st);
#define GO(T, HALF, NORM, LPR) \
    k_rope<T, HALF, NORM, LPR><<<grid, 32 * kWarps, 0, st>>>(hq, hk, rp, B, N, D, eps, wdtype, sign, chunk, status)
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
    if (tokens == 0) return 1;  // (writes dw = 0)
    const long long b = (tokens * 4 + kWarps - 1) / kWarps;  // (small calls: several chunks of heads for each token)
    return (int)(b < 592 ? b : 592);                          // four blocks for each of 148 SMs
}

int launch_norm_rope_bwd(const park_operand* dyq, const park_operand* dyk, const park_operand* q,
                         const park_operand* k, const park_operand* dq, const park_operand* dk, const void* wq,
                         const void* wk, int wdtype, float eps, const park_rope_axes* rope, const int32_t* pos,
                         long long pos_sb, float* dwq, float* dwk, int B, long long N, int D, int dtype, float* part,
                         int32_t* status, int num_sms, cudaStream_t st) {
    const int elt = dtype == PARK_BF16 ? 2 : 4;
    const Heads hq = heads(q, dq, dyq, wq, elt), hk = heads(k, dk, dyk, wk, elt);
    const RopeDev rp = rope_dev(rope, pos, pos_sb);
    const int Ht = hq.H + hk.H, lpr = D == 32 ? 4 : (D == 64 ? 8 : 16);
    const int chunk = N ? head_chunk(B * N, Ht, 32 / lpr, num_sms) : Ht, nch = (Ht + chunk - 1) / chunk;
    const int blocks = norm_rope_bwd_blocks(B * N);
    const bool half = rope && rope->half;
    ::park::prof_begin(st);
#define GO(T, HALF, LPR)                                                                                             \
    k_norm_rope_bwd<T, HALF, LPR><<<blocks, 32 * kWarps, 0, st>>>(hq, hk, rp, B, N, D, eps, wdtype, chunk, nch, part, \
                                                                  status)
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
    k_dw_reduce<<<dim3(D / 32, 2), 256, 0, st>>>(part, blocks, D, dwq, dwk);
    PARK_TRY_LAUNCH("k_dw_reduce", st);
    return PARK_OK;
}

}  // namespace park
