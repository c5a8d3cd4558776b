// Dense attention, backward, bf16 on the 5th-generation tensor cores.
//
//   p = 2^(scale log2(e) s - lse log2(e)),  ds = p (do v^T - delta)
//   dq = scale ds k,  dk = scale ds^T q,  dv = p^T do
//
// Two kernels, each the only writer of its sums, so no atomics and the same bits
// every time; the price is that the scores and do v^T are formed twice.
//
// k_dense_dq_tc owns 128 query rows and walks the keys; k_dense_dkv_tc owns 128 keys and
// walks the query rows of all heads of the group, with the products transposed (keys are
// the rows).  Both run four products of 128 x 128 x D a step in full tensor memory:
//   dq:  S = Q K^T | dP = dO V^T | dQ += dS K | B += P K
//   dkv: S^T = K Q^T | dP^T = V dO^T | dV += P^T dO | dK += dS^T Q
// with P over S's columns and dS over dP's.  Order of the MMAs: the product with P of
// step j, S(j+1), the product with dS of step j, dP(j+1): the exponentials of a step run
// beside the product with the last step's dS and dP(j), its dS beside the product with P and S(j+1).
//
// What B = sum_j p_j k_j is for: sum_j ds_j is 0, so dq = scale sum_j ds_j (k_j - c) for
// any c.  The roundings of ds (bf16 operand) and of o (which delta is computed from) break
// the zero sum, and the keys that a row attends to have much in common: its error would be
// that common part times the sum's.  With r = the sum of the rounded ds, dq - r B takes c = B
// out.  The same walk gives sum_j p_j (dp_j - delta), which is what delta is off by: it is
// added to delta for the second kernel.  On rows whose keys share a direction (scores of +-6)
// the errors of dq and dk were 7.5e-3 and 6e-3 of their norms without this.
//
// In both, 256 threads work on a 128 x 128 tile, two on a row with 64 columns each; the
// half h of a bf16 operand lies on the first 32 of its own 64 columns (a second part on the
// others), so a thread only overwrites what it has read itself.  p and ds are rounded to bf16 as operands.
//
// Tiles that a mask cuts are cleaned by the same threads before the product that sums
// over the hidden rows: infinities and NaN become 0 (0 x NaN is NaN); what visible rows
// hold of them reaches dq and dk through ds, and dv in its epilogue.
//
// Every wait is time-bounded (PARK_ERR_TIMEOUT); on a failed wait the roles leave their
// loops, copies and MMAs in flight are waited for and TMEM is freed.
#include <type_traits>

#include "dense_tc.cuh"

namespace park {
namespace {

template <int NP>
struct BwdCfg {
    static constexpr int ST = NP == 2 ? 5 : 8;  // ring stages beside two resident tiles
    static constexpr uint32_t tile = NP * kPanel;
};

struct DqSmem {
    uint64_t own_full, kv_full[8], kv_empty[8], s_full, p_full[2], dp_full, ds_full, final_bar;
    uint32_t tmem_base;
    int abort;
    SeqTile seq;
    float sum[2][2][kTile];  // [column half][exact, of the rounded ds][row]
};
struct DkvSmem {
    uint64_t own_full, in_full[8], in_empty[8], s_full, p_full[2], dp_full, ds_full, stat_full[2], stat_empty[2], final_bar;
    uint32_t tmem_base;
    int abort, poison;
    int fine;  // from this step on p and ds have a second part
    SeqTile seq;
    alignas(16) float lse2[2][kTile], delta[2][kTile];  // both negated
};
template <int NP, typename S>
constexpr size_t bwd_smem() { return (size_t)(2 + BwdCfg<NP>::ST) * BwdCfg<NP>::tile + sizeof(S); }

// Pair e of exponentials.  At 128 columns the four products take longer than the exponentials and all of them go to
// the special-function unit (moving two of eight pairs to the FMA pipe: dq 1.43 -> 1.51 ms at 16,384 x 8 heads); at
// 64 columns the products are half as long and two of eight pairs go to the FMA pipe (dk/dv 0.56 -> 0.51 ms at
// 8,192 causal, 16/4 heads).
template <int NP>
__device__ __forceinline__ float2 ex2_pair(int e, float2 x) {
    return NP == 1 && e % 4 == 0 ? ex2_poly2(x) : make_float2(ex2(x.x), ex2(x.y));
}
// K = 16 steps of a product over 128 rows of which the threads deliver their first 32 columns, then the others
__device__ constexpr int part_step(int part, int x) { return 2 * part + (x & 1) + 4 * (x >> 1); }

// Pairs of columns c0 + 2e, c0 + 2e + 1: 0 outside lo .. hi.  (A hidden row's lse and delta may be NaN, so p and ds
// are hidden once they are formed.)
template <int N>
__device__ __forceinline__ void hide(uint32_t (&pk)[N], int c0, int lo, int hi) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const int c = c0 + 2 * e;
        pk[e] &= (c >= lo && c <= hi ? 0x0000FFFFu : 0u) | (c + 1 >= lo && c + 1 <= hi ? 0xFFFF0000u : 0u);
    }
}

// A key that draws kDominant times its share of the rows' attention gives a row of dv (and of dk) so much larger than the others
// that the roundings of p and ds to bf16 in it stand out in the tensor as a whole.  Two steps after one is seen, its
// tile's p and ds get a second bf16 part and a second product.  75,600 rows of which many attend to the same few
// keys, one of them with half of dv's norm: dv and dk were 2.3e-3 and 2.5e-3 of their norms off, now 1.7e-3, which is the rounding of the result.
// Steps that a mask cuts are not looked at, and nothing changes before the third step: in sequences of a few tiles a row of
// dv cannot outweigh the others by so much.  dq needs nothing like it, its rows are averages.
// Where no key is dominant, the looking costs the dk/dv kernel alone 1.5 % (D = 128: 3.07 -> 3.12 ms at 32,768 x 4 heads) to 6 %
// (D = 64: 338 -> 358 us at 8,192 causal, 16/4 heads).
constexpr float kDominant = 64.f;
constexpr int kSample = 8;  // steps of which one is looked at

// What bf16 left of pairs of p or ds, as bf16: with it an operand has 16 bits.
template <int N>
__device__ __forceinline__ void rest(uint32_t (&lo)[N], const uint32_t* pk, const uint32_t (&x)[2 * N]) {
#pragma unroll
    for (int e = 0; e < N; ++e)
        lo[e] = bf2(f_of(x[2 * e]) - f_of(pk[e] << 16), f_of(x[2 * e + 1]) - f_of(pk[e] & 0xFFFF0000u));
}

// 64 columns at `col` of this thread's lane
__device__ __forceinline__ void ld64(uint32_t col, uint32_t (&x)[2][32]) {
    tmem_ld32(col, x[0]);
    tmem_ld32(col + 32, x[1]);
}

template <int NP>
__global__ void __launch_bounds__(384, 1)
    k_dense_dq_tc(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmG,
                  const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, DenseArgs a,
                  DenseOrder order, float* __restrict__ delta, uint64_t wait_ns) {
    using C = BwdCfg<NP>;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* Qs = smem;
    uint8_t* Gs = smem + C::tile;
    uint8_t* ring = smem + 2 * C::tile;
    DqSmem& sh = *reinterpret_cast<DqSmem*>(ring + C::ST * C::tile);
    if (smem_u32(smem) & 1023u) {  // the swizzle is by address
        set_status(a.status, PARK_ERR_CUDA);
        return;
    }
    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    volatile int* abort = &sh.abort;
    int x_tile;
    const int bh = dense_block_head(order, x_tile), b = a.B == 1 ? 0 : bh / a.Hq, h = bh - b * a.Hq, hk = h / (a.Hq / a.Hk);
    if (warp == 0) {
        const SeqTile t = dense_block_tile(a, order, x_tile, kTile, false, 1);
        if (lane == 0) {
            sh.seq = t;
            mbar_init(&sh.own_full, 1);
            for (int s = 0; s < C::ST; ++s) {
                mbar_init(&sh.kv_full[s], 1);
                mbar_init(&sh.kv_empty[s], 1);
            }
            mbar_init(&sh.s_full, 1);
            mbar_init(&sh.p_full[0], 256);
            mbar_init(&sh.p_full[1], 256);
            mbar_init(&sh.dp_full, 1);
            mbar_init(&sh.ds_full, 256);
            mbar_init(&sh.final_bar, 1);
            sh.abort = 0;
            mbar_fence_init();
        }
    } else if (warp == 9) {
        tmem_alloc(&sh.tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem_base;
    const SeqTile t = sh.seq;
    const int i0 = t.tile * kTile, rows = t.live ? min(kTile, t.nq - i0) : 0;
    const int kend = rows > 0 ? dense_last_key(i0 + rows - 1, t.nq, t.nk, a.causal) + 1 : 0;
    const int nt = kend > 0 ? (kend + kTile - 1) / kTile : 0;
    const int cut = (dense_last_key(i0, t.nq, t.nk, a.causal) + 1) / kTile;  // first tile that a row sees in part

    if (warp >= 8) {
        reg_dec<56>();
        if (warp == 8 && lane == 0 && nt > 0) {
            tma_prefetch_desc(&tmK);
            tma_prefetch_desc(&tmV);
            mbar_arrive_expect_tx(&sh.own_full, 2 * C::tile);
            for (int p = 0; p < NP; ++p) {
                tma_load_4d(Qs + p * kPanel, &tmQ, &sh.own_full, 64 * p, t.q0 + i0, h, b);
                tma_load_4d(Gs + p * kPanel, &tmG, &sh.own_full, 64 * p, t.q0 + i0, h, b);
            }
            int issued = 0;
            for (int i = 0; i < 2 * nt; ++i) {  // K_0 V_0 K_1 V_1 ...
                const int st = i % C::ST, round = i / C::ST;
                if (round > 0 && !wait_bar(&sh.kv_empty[st], (round - 1) & 1, abort, wait_ns)) break;
                mbar_arrive_expect_tx(&sh.kv_full[st], C::tile);
                for (int p = 0; p < NP; ++p)
                    tma_load_4d(ring + st * C::tile + p * kPanel, i & 1 ? &tmV : &tmK, &sh.kv_full[st], 64 * p,
                                t.k0 + (i >> 1) * kTile, hk, b);
                ++issued;
            }
            int dummy = 0;  // copies in flight land before the CTA may exit
            wait_bar(&sh.own_full, 0, &dummy, 100000000ull);
            for (int i = max(0, issued - C::ST); i < issued; ++i)
                wait_bar(&sh.kv_full[i % C::ST], (i / C::ST) & 1, &dummy, 100000000ull);
        } else if (warp == 9) {
            const uint32_t idS = idesc_bf16(128, 128, 0, 0), idQ = idesc_bf16(128, 64 * NP, 0, 1);
            const bool lead = elect_one();
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            const uint64_t dA[2] = {sdesc_sw128(smem_u32(Qs), 16, 1024), sdesc_sw128(smem_u32(Gs), 16, 1024)};
            const uint64_t dB = sdesc_sw128(smem_u32(ring), 16, 1024), dBt = sdesc_sw128(smem_u32(ring), kPanel, 1024);
            // w = 0: S of tile j = Q K^T; w = 1: dP = dO V^T
            auto issue_s = [&](int j, int w) -> bool {
                const int i = 2 * j + w, st = i % C::ST;
                if (!wait_warp(&sh.kv_full[st], (i / C::ST) & 1, abort, wait_ns)) return false;
                tc_fence_after();
                const uint64_t ba = dB + ((st * C::tile) >> 4);
                if (lead) {
#pragma unroll
                    for (int kk = 0; kk < 4 * NP; ++kk) {
                        const uint32_t off = ((kk >> 2) * kPanel + (kk & 3) * 32) >> 4;
                        umma_bf16(tm + 128 * w, dA[w] + off, ba + off, idS, kk > 0);
                    }
                    if (w) umma_commit(&sh.kv_empty[st]);  // V_j is read once
                    umma_commit(w ? &sh.dp_full : &sh.s_full);
                }
                __syncwarp();
                return true;
            };
            // w = 0: B += P K; w = 1: dQ += dS K
            auto issue_g = [&](int j, int w) -> bool {
                const int st = (2 * j) % C::ST;
                const uint64_t ka = dBt + ((st * C::tile) >> 4);
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    if ((w == 0 || part == 0) &&
                        !wait_warp(w ? &sh.ds_full : &sh.p_full[part], j & 1, abort, wait_ns))
                        return false;
                    tc_fence_after();
                    if (lead) {
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const int kk = part_step(part, x);
                            umma_bf16_ts(tm + 256 + 128 * w, tm + 128 * w + 64 * (kk >> 2) + 8 * (kk & 3),
                                         ka + ((kk * 2048) >> 4), idQ, j > 0 || part > 0 || x > 0);
                        }
                        if (part == 1 && w) umma_commit(&sh.kv_empty[st]);
                    }
                    __syncwarp();
                }
                return true;
            };
            bool ok = nt > 0 && wait_warp(&sh.own_full, 0, abort, wait_ns) && issue_s(0, 0) && issue_s(0, 1);
            for (int j = 0; j < nt && ok; ++j)
                ok = issue_g(j, 0) && (j + 1 >= nt || issue_s(j + 1, 0)) && issue_g(j, 1) &&
                     (j + 1 >= nt || issue_s(j + 1, 1));
            if (lead) umma_commit(&sh.final_bar);
            __syncwarp();
            int dummy = 0;
            wait_bar(&sh.final_bar, 0, &dummy, 100000000ull);
        }
        __syncwarp();
    } else {
        reg_inc<216>();
        const int quad = warp & 3, hc = warp >> 2, row = 32 * quad + lane;
        const uint32_t trow = tmem + ((uint32_t)(32 * quad) << 16);
        const bool live = row < rows;
        const size_t at = ((size_t)b * a.Hq + h) * a.Nq + t.q0 + i0 + row;
        const float INF = __int_as_float(0x7f800000);
        // a row without keys (lse = -inf) and the rows past the end: p = 2^-inf = 0
        float lse2 = live ? a.lse[at] * kLog2e : INF;
        if (lse2 == -INF) lse2 = INF;
        const float del = live ? delta[at] : 0.f;
        const int seen = live ? dense_last_key(i0 + row, t.nq, t.nk, a.causal) : -1;
        const float2 sl22 = make_float2(a.scale * kLog2e, a.scale * kLog2e), nl = make_float2(-lse2, -lse2);
        const float2 nd = make_float2(-del, -del);
        float2 r2 = make_float2(0.f, 0.f), rb2 = make_float2(0.f, 0.f);  // sums of ds: exact, rounded
        bool ok = true;
        for (int j = 0; j < nt; ++j) {
            if (!__all_sync(0xffffffffu, wait_bar(&sh.s_full, j & 1, abort, wait_ns))) {
                ok = false;
                break;
            }
            tc_fence_after();
            uint32_t s[2][32];
            ld64(trow + 64 * hc, s);
            tmem_ld_wait();
            tmem_ld_dep(s[0]);
            tmem_ld_dep(s[1]);
            const int lim = seen - j * kTile - 64 * hc;  // columns 0 .. lim of this half are visible
            if (j >= cut) {
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (32 * c + e > lim) s[c][e] = 0xff800000u;  // p = 0
                // K_j, which S has been formed from, is cleaned for the sums over its rows
                const int st = (2 * j) % C::ST;
                if (!__all_sync(0xffffffffu, wait_bar(&sh.kv_full[st], ((2 * j) / C::ST) & 1, abort, wait_ns))) {
                    ok = false;
                    break;
                }
                uint4* k4 = reinterpret_cast<uint4*>(ring + st * C::tile);
                for (int e = threadIdx.x; e < (int)(C::tile / 16); e += 256) clean16(k4 + e);
                fence_proxy_async_smem();
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t pk[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float2 p = ex2_pair<NP>(e, __ffma2_rn(make_float2(f_of(s[c][2 * e]), f_of(s[c][2 * e + 1])), sl22, nl));
                    s[c][2 * e] = __float_as_uint(p.x);
                    s[c][2 * e + 1] = __float_as_uint(p.y);
                    pk[e] = bf2(p.x, p.y);
                }
                tmem_st16(trow + 64 * hc + 16 * c, pk);
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&sh.p_full[c]);
            }
            if (!__all_sync(0xffffffffu, wait_bar(&sh.dp_full, j & 1, abort, wait_ns))) {
                ok = false;
                break;
            }
            tc_fence_after();
            uint32_t pk[32];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t g[32];
                tmem_ld32(trow + 128 + 64 * hc + 32 * c, g);
                tmem_ld_wait();
                tmem_ld_dep(g);
                if (j >= cut) {  // what a hidden value makes of dP does not meet p = 0
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (32 * c + e > lim) g[e] = 0u;
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float2 x = __fmul2_rn(__fadd2_rn(make_float2(f_of(g[2 * e]), f_of(g[2 * e + 1])), nd),
                                                make_float2(f_of(s[c][2 * e]), f_of(s[c][2 * e + 1])));
                    const uint32_t w = bf2(x.x, x.y);
                    r2 = __fadd2_rn(r2, x);
                    rb2 = __fadd2_rn(rb2, make_float2(f_of(w << 16), f_of(w & 0xFFFF0000u)));
                    pk[16 * c + e] = w;
                }
            }
            tmem_st32(trow + 128 + 64 * hc, pk);
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&sh.ds_full);
        }
        sh.sum[hc][0][row] = r2.x + r2.y;
        sh.sum[hc][1][row] = rb2.x + rb2.y;
        named_bar_sync(1, 256);
        if (nt > 0 && ok) ok = __all_sync(0xffffffffu, wait_bar(&sh.final_bar, 0, abort, wait_ns)) && !__any_sync(0xffffffffu, *abort != 0);
        if (ok) {
            tc_fence_after();
            const float r = sh.sum[0][1][row] + sh.sum[1][1][row];
            if (live && hc == 0) delta[at] = del + (sh.sum[0][0][row] + sh.sum[1][0][row]);
            uint8_t* out = a.dq.p + (b * a.dq.sb + h * a.dq.sh + (t.q0 + i0 + (long long)row) * a.dq.sn) * 2;
#pragma unroll
            for (int c = 0; c < NP; ++c) {
                const int d0 = 32 * (2 * c + hc);  // the halves take alternate groups of 32 columns
                if (d0 >= a.D) break;
                uint32_t o[32], bk[32];
                __syncwarp();
                if (nt > 0) {
                    tmem_ld32(trow + 384 + d0, o);
                    tmem_ld32(trow + 256 + d0, bk);
                    tmem_ld_wait();
                    tmem_ld_dep(o);
                    tmem_ld_dep(bk);
                }
                if (live) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        uint32_t w[4];
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const int y = e + 2 * x;
                            w[x] = nt > 0 ? bf2(fmaf(-r, f_of(bk[y]), f_of(o[y])) * a.scale,
                                                fmaf(-r, f_of(bk[y + 1]), f_of(o[y + 1])) * a.scale)
                                          : 0u;
                        }
                        *reinterpret_cast<uint4*>(out + 2 * (d0 + e)) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (threadIdx.x == 0 && sh.abort) set_status(a.status, PARK_ERR_TIMEOUT);
}

template <int NP>
__global__ void __launch_bounds__(384, 1)
    k_dense_dkv_tc(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmG,
                   const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, DenseArgs a,
                   DenseOrder order, const float* __restrict__ delta, int n_split, int chunk, float* __restrict__ part_dv,
                   float* __restrict__ part_dk, uint64_t wait_ns) {
    using C = BwdCfg<NP>;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* Ks = smem;
    uint8_t* Vs = smem + C::tile;
    uint8_t* ring = smem + 2 * C::tile;
    DkvSmem& sh = *reinterpret_cast<DkvSmem*>(ring + C::ST * C::tile);
    if (smem_u32(smem) & 1023u) {  // the swizzle is by address
        set_status(a.status, PARK_ERR_CUDA);
        return;
    }
    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    volatile int *abort = &sh.abort, *fine_from = &sh.fine;
    int x_tile;
    const int bh = dense_block_head(order, x_tile), b = a.B == 1 ? 0 : bh / a.Hk, hk = bh - b * a.Hk, sp = blockIdx.z;
    if (warp == 0) {
        const SeqTile t = dense_block_tile(a, order, x_tile, kTile, true, 1);
        if (lane == 0) {
            sh.seq = t;
            mbar_init(&sh.own_full, 1);
            for (int s = 0; s < C::ST; ++s) {
                mbar_init(&sh.in_full[s], 1);
                mbar_init(&sh.in_empty[s], 1);
            }
            mbar_init(&sh.s_full, 1);
            mbar_init(&sh.p_full[0], 256);
            mbar_init(&sh.p_full[1], 256);
            mbar_init(&sh.dp_full, 1);
            mbar_init(&sh.ds_full, 256);
            for (int s = 0; s < 2; ++s) {
                mbar_init(&sh.stat_full[s], 32);
                mbar_init(&sh.stat_empty[s], 256);
            }
            mbar_init(&sh.final_bar, 1);
            sh.abort = 0;
            sh.poison = 0;
            sh.fine = 0x7fffffff;
            mbar_fence_init();
        }
    } else if (warp == 9) {
        tmem_alloc(&sh.tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem_base;
    const SeqTile t = sh.seq;
    const int G = a.Hq / a.Hk;
    const int j0 = t.tile * kTile, keys = t.live ? min(kTile, t.nk - j0) : 0;
    // row tiles first .. end-1 of each head of the group see a key of this tile; this part has steps s0 .. s0 + steps - 1
    int first, end;
    dense_row_tiles(t, j0, a.causal, kTile, first, end);
    const int per = keys > 0 ? end - first : 0, s0 = n_split > 1 ? sp * chunk : 0;
    const int steps = max(0, n_split > 1 ? min(chunk, per * G - s0) : per * G);
    const int head0 = hk * G + (per > 0 ? s0 / per : 0), it0 = first + (per > 0 ? s0 % per : 0);

    if (warp >= 8) {
        reg_dec<56>();
        if (warp == 8 && lane == 0 && steps > 0) {
            tma_prefetch_desc(&tmQ);
            tma_prefetch_desc(&tmG);
            mbar_arrive_expect_tx(&sh.own_full, 2 * C::tile);
            for (int p = 0; p < NP; ++p) {
                tma_load_4d(Ks + p * kPanel, &tmK, &sh.own_full, 64 * p, t.k0 + j0, hk, b);
                tma_load_4d(Vs + p * kPanel, &tmV, &sh.own_full, 64 * p, t.k0 + j0, hk, b);
            }
            int issued = 0, head = head0, it = it0;
            for (int i = 0; i < 2 * steps; ++i) {  // Q_0 dO_0 Q_1 dO_1 ...
                const int st = i % C::ST, round = i / C::ST;
                if (round > 0 && !wait_bar(&sh.in_empty[st], (round - 1) & 1, abort, wait_ns)) break;
                mbar_arrive_expect_tx(&sh.in_full[st], C::tile);
                for (int p = 0; p < NP; ++p)
                    tma_load_4d(ring + st * C::tile + p * kPanel, i & 1 ? &tmG : &tmQ, &sh.in_full[st], 64 * p,
                                t.q0 + it * kTile, head, b);
                ++issued;
                if ((i & 1) && ++it == end) {
                    it = first;
                    ++head;
                }
            }
            int dummy = 0;
            wait_bar(&sh.own_full, 0, &dummy, 100000000ull);
            for (int i = max(0, issued - C::ST); i < issued; ++i)
                wait_bar(&sh.in_full[i % C::ST], (i / C::ST) & 1, &dummy, 100000000ull);
        } else if (warp == 9) {
            const uint32_t idS = idesc_bf16(128, 128, 0, 0), idG = idesc_bf16(128, 64 * NP, 0, 1);
            const bool lead = elect_one();
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            const uint64_t dA[2] = {sdesc_sw128(smem_u32(Ks), 16, 1024), sdesc_sw128(smem_u32(Vs), 16, 1024)};
            const uint64_t dB = sdesc_sw128(smem_u32(ring), 16, 1024), dBt = sdesc_sw128(smem_u32(ring), kPanel, 1024);
            // w = 0: S^T of step j = K Q^T; w = 1: dP^T = V dO^T
            auto issue_s = [&](int j, int w) -> bool {
                const int i = 2 * j + w, st = i % C::ST;
                if (!wait_warp(&sh.in_full[st], (i / C::ST) & 1, abort, wait_ns)) return false;
                tc_fence_after();
                const uint64_t ba = dB + ((st * C::tile) >> 4);
                if (lead) {
#pragma unroll
                    for (int kk = 0; kk < 4 * NP; ++kk) {
                        const uint32_t off = ((kk >> 2) * kPanel + (kk & 3) * 32) >> 4;
                        umma_bf16(tm + 128 * w, dA[w] + off, ba + off, idS, kk > 0);
                    }
                    umma_commit(w ? &sh.dp_full : &sh.s_full);
                }
                __syncwarp();
                return true;
            };
            // w = 0: dV += P^T dO; w = 1: dK += dS^T Q
            auto issue_g = [&](int j, int w, bool fine) -> bool {
                const int st = (2 * j + 1 - w) % C::ST;
                const uint64_t ba = dBt + ((st * C::tile) >> 4);
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    if ((w == 0 || part == 0) &&
                        !wait_warp(w ? &sh.ds_full : &sh.p_full[part], j & 1, abort, wait_ns))
                        return false;
                    tc_fence_after();
                    if (lead) {
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const int kk = part_step(part, x);
                            umma_bf16_ts(tm + 256 + 128 * w, tm + 128 * w + 64 * (kk >> 2) + 8 * (kk & 3),
                                         ba + ((kk * 2048) >> 4), idG, j > 0 || part > 0 || x > 0);
                        }
                        if (part == 1 && fine) {  // (rolled up: unrolled, the ordinary steps took a tenth longer)
#pragma unroll 1
                            for (int kk = 0; kk < 8; ++kk)
                                umma_bf16_ts(tm + 256 + 128 * w, tm + 128 * w + 64 * (kk >> 2) + 32 + 8 * (kk & 3),
                                             ba + ((kk * 2048) >> 4), idG, 1);
                        }
                        if (part == 1) umma_commit(&sh.in_empty[st]);
                    }
                    __syncwarp();
                }
                return true;
            };
            bool ok = steps > 0 && wait_warp(&sh.own_full, 0, abort, wait_ns) && issue_s(0, 0) && issue_s(0, 1);
            for (int j = 0; j < steps && ok; ++j) {
                const bool fine = __any_sync(0xffffffffu, *fine_from <= j);  // (set two steps ago or earlier, or not meant for this one)
                ok = issue_g(j, 0, fine) && (j + 1 >= steps || issue_s(j + 1, 0)) && issue_g(j, 1, fine) &&
                     (j + 1 >= steps || issue_s(j + 1, 1));
            }
            if (lead) umma_commit(&sh.final_bar);
            __syncwarp();
            int dummy = 0;
            wait_bar(&sh.final_bar, 0, &dummy, 100000000ull);
        } else if (warp == 10) {
            // lse and delta of each step's 128 rows
            const float INF = __int_as_float(0x7f800000);
            int head = head0, it = it0;
            for (int j = 0; j < steps; ++j) {
                const int st = j & 1, round = j >> 1;
                if (round > 0 && !__all_sync(0xffffffffu, wait_bar(&sh.stat_empty[st], (round - 1) & 1, abort, wait_ns))) break;
                const size_t at = ((size_t)b * a.Hq + head) * a.Nq + t.q0;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int c = lane + 32 * e, i = it * kTile + c;
                    float l = i < t.nq ? a.lse[at + i] * -kLog2e : -INF;
                    if (l == INF) l = -INF;  // a row without keys
                    sh.lse2[st][c] = l;
                    sh.delta[st][c] = i < t.nq ? -delta[at + i] : 0.f;
                }
                mbar_arrive(&sh.stat_full[st]);
                if (++it == end) {
                    it = first;
                    ++head;
                }
            }
        }
        __syncwarp();
    } else {
        reg_inc<216>();
        const int quad = warp & 3, hc = warp >> 2, row = 32 * quad + lane;
        const uint32_t trow = tmem + ((uint32_t)(32 * quad) << 16);
        const float2 sl22 = make_float2(a.scale * kLog2e, a.scale * kLog2e);
        const int off = t.nk - t.nq;
        // of a step's rows, for this thread's half of them (lanes past the last key never find one)
        const float share = row < keys ? kDominant / 2 / kSample * kTile / t.nk : __int_as_float(0x7f800000);
        float2 mass2 = make_float2(0.f, 0.f);
        bool ok = true, fine = false;
        int it = it0;
        // one step; the rows' columns are lo .. hi of the thread's, FINE: p and ds in two parts
        auto step = [&](auto fine_c, int j, int i0, bool cut, int lo, int hi) -> bool {
            constexpr bool FINE = decltype(fine_c)::value;
            const int st = j & 1;
            uint32_t s[2][32];
            ld64(trow + 64 * hc, s);
            tmem_ld_wait();
            tmem_ld_dep(s[0]);
            tmem_ld_dep(s[1]);
            if (cut) {
                // S and dP have been formed from Q and dO: now they are cleaned for the sums over their rows
                const int sq = (2 * j) % C::ST, sg = (2 * j + 1) % C::ST;
                if (!__all_sync(0xffffffffu, wait_bar(&sh.dp_full, j & 1, abort, wait_ns) &&
                                                 wait_bar(&sh.in_full[sq], ((2 * j) / C::ST) & 1, abort, wait_ns) &&
                                                 wait_bar(&sh.in_full[sg], ((2 * j + 1) / C::ST) & 1, abort, wait_ns))) return false;
                uint4* q4 = reinterpret_cast<uint4*>(ring + sq * C::tile);
                uint4* g4 = reinterpret_cast<uint4*>(ring + sg * C::tile);
                for (int e = threadIdx.x; e < (int)(C::tile / 16); e += 256) {
                    clean16(q4 + e);
                    if (clean16(g4 + e) && i0 + (e >> 3) % kTile < t.nq) sh.poison = 1;
                }
                fence_proxy_async_smem();
            }
            const float4* lp = reinterpret_cast<const float4*>(&sh.lse2[st][64 * hc]);  // negated
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t pk[16];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float4 l = lp[8 * c + e];
                    const float2 x = ex2_pair<NP>(2 * e, __ffma2_rn(make_float2(f_of(s[c][4 * e]), f_of(s[c][4 * e + 1])), sl22,
                                                                make_float2(l.x, l.y)));
                    const float2 y = ex2_pair<NP>(2 * e + 1, __ffma2_rn(make_float2(f_of(s[c][4 * e + 2]), f_of(s[c][4 * e + 3])),
                                                                    sl22, make_float2(l.z, l.w)));
                    s[c][4 * e] = __float_as_uint(x.x);
                    s[c][4 * e + 1] = __float_as_uint(x.y);
                    s[c][4 * e + 2] = __float_as_uint(y.x);
                    s[c][4 * e + 3] = __float_as_uint(y.y);
                    pk[2 * e] = bf2(x.x, x.y);
                    pk[2 * e + 1] = bf2(y.x, y.y);
                }
                if (cut) hide(pk, 32 * c, lo, hi);
                tmem_st16(trow + 64 * hc + 16 * c, pk);
                if (FINE) {
                    uint32_t low[16];
                    rest(low, pk, s[c]);
                    if (cut) hide(low, 32 * c, lo, hi);
                    tmem_st16(trow + 64 * hc + 32 + 16 * c, low);
                } else if (j % kSample == 0 && !cut) {
#pragma unroll
                    for (int e = 0; e < 32; e += 2) mass2 = __fadd2_rn(mass2, make_float2(f_of(s[c][e]), f_of(s[c][e + 1])));
                    if (c == 1 && __any_sync(0xffffffffu, mass2.x + mass2.y > share * max(j + 1, t.nk >> 10)) && *fine_from > j + 2)
                        *fine_from = j + 2;
                }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&sh.p_full[c]);
            }
            // what all steps before this one set is there: S of this step was issued after their p
            fine = __any_sync(0xffffffffu, *fine_from <= j + 1);
            if (!__all_sync(0xffffffffu, wait_bar(&sh.dp_full, j & 1, abort, wait_ns))) return false;
            tc_fence_after();
            const float4* dp4 = reinterpret_cast<const float4*>(&sh.delta[st][64 * hc]);  // negated
            uint32_t pk[32];
#pragma unroll
            for (int c = 1; c >= 0; --c) {  // (in this order the second parts only cover what has been read)
                uint32_t g[32];
                tmem_ld32(trow + 128 + 64 * hc + 32 * c, g);
                tmem_ld_wait();
                tmem_ld_dep(g);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float4 d = dp4[8 * c + e];
                    const float2 x = __fmul2_rn(
                        __fadd2_rn(make_float2(f_of(g[4 * e]), f_of(g[4 * e + 1])), make_float2(d.x, d.y)),
                        make_float2(f_of(s[c][4 * e]), f_of(s[c][4 * e + 1])));
                    const float2 y = __fmul2_rn(
                        __fadd2_rn(make_float2(f_of(g[4 * e + 2]), f_of(g[4 * e + 3])), make_float2(d.z, d.w)),
                        make_float2(f_of(s[c][4 * e + 2]), f_of(s[c][4 * e + 3])));
                    pk[16 * c + 2 * e] = bf2(x.x, x.y);
                    pk[16 * c + 2 * e + 1] = bf2(y.x, y.y);
                    g[4 * e] = __float_as_uint(x.x);
                    g[4 * e + 1] = __float_as_uint(x.y);
                    g[4 * e + 2] = __float_as_uint(y.x);
                    g[4 * e + 3] = __float_as_uint(y.y);
                }
                if (FINE) {
                    uint32_t low[16];
                    rest(low, pk + 16 * c, g);
                    if (cut) hide(low, 32 * c, lo, hi);
                    tmem_st16(trow + 128 + 64 * hc + 32 + 16 * c, low);
                }
            }
            mbar_arrive(&sh.stat_empty[st]);
            if (cut) hide(pk, 0, lo, hi);
            tmem_st32(trow + 128 + 64 * hc, pk);
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&sh.ds_full);
            return true;
        };
        for (int j = 0; j < steps; ++j) {
            const int st = j & 1, i0 = it * kTile;
            if (++it == end) it = first;
            if (!__all_sync(0xffffffffu, wait_bar(&sh.stat_full[st], (j >> 1) & 1, abort, wait_ns) &&
                                             wait_bar(&sh.s_full, j & 1, abort, wait_ns))) {
                ok = false;
                break;
            }
            tc_fence_after();
            // columns lo .. hi of this half are visible to this thread's key
            // (keys past the end are lanes of their own, which nothing sums over and nothing writes)
            const bool cut = i0 + kTile > t.nq || j0 + keys - 1 > dense_last_key(i0, t.nq, t.nk, a.causal);
            const int lo = (a.causal ? j0 + row - off - i0 : 0) - 64 * hc, hi = t.nq - 1 - i0 - 64 * hc;
            ok = fine ? step(std::true_type{}, j, i0, cut, lo, hi) : step(std::false_type{}, j, i0, cut, lo, hi);
            if (!ok) break;
        }
        if (steps > 0 && ok) ok = __all_sync(0xffffffffu, wait_bar(&sh.final_bar, 0, abort, wait_ns)) && !__any_sync(0xffffffffu, *abort != 0);
        if (ok && !(n_split > 1 && steps == 0)) {  // (a part without steps is not written)
            tc_fence_after();
            const bool live = row < keys, split = n_split > 1;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const Op4& out_op = w ? a.dk : a.dv;
                uint8_t* out = out_op.p + (b * out_op.sb + hk * out_op.sh + (t.k0 + j0 + (long long)row) * out_op.sn) * 2;
                float* part = (w ? part_dk : part_dv) +
                              ((((size_t)sp * a.B + b) * a.Hk + hk) * a.Nk + t.k0 + j0 + row) * a.D;
                const float f = w ? a.scale : 1.f;
#pragma unroll
                for (int c = 0; c < NP; ++c) {
                    const int d0 = 32 * (2 * c + hc);
                    if (d0 >= a.D) break;
                    uint32_t o[32];
                    __syncwarp();
                    if (steps > 0) {
                        tmem_ld32(trow + 256 + 128 * w + d0, o);
                        tmem_ld_wait();
                        tmem_ld_dep(o);
                    }
                    if (w == 0 && sh.poison && live) {
                        // infinities and NaN of dO rows that do see this key, in the tiles that were cleaned
                        for (int g = 0; g < G; ++g)
                            for (int i = first * kTile; i < t.nq; ++i) {
                                const int ib = i / kTile * kTile;
                                if (!(ib + kTile > t.nq || j0 + keys - 1 > dense_last_key(ib, t.nq, t.nk, a.causal))) {
                                    i = ib + kTile - 1;  // (not cut)
                                    continue;
                                }
                                if (j0 + row > dense_last_key(i, t.nq, t.nk, a.causal)) continue;
                                const uint16_t* gr = reinterpret_cast<const uint16_t*>(
                                                         a.d_o.p + (b * a.d_o.sb + (hk * G + g) * a.d_o.sh +
                                                                    (t.q0 + (long long)i) * a.d_o.sn) * 2) + d0;
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    if ((gr[e] & 0x7F80u) == 0x7F80u)
                                        o[e] = __float_as_uint(f_of(o[e]) + f_of((uint32_t)gr[e] << 16));
                            }
                    }
                    if (live && split) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<uint4*>(part + d0 + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                    } else if (live) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            uint32_t x4[4];
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                x4[x] = steps > 0 ? bf2(f_of(o[e + 2 * x]) * f, f_of(o[e + 2 * x + 1]) * f) : 0u;
                            *reinterpret_cast<uint4*>(out + 2 * (d0 + e)) = make_uint4(x4[0], x4[1], x4[2], x4[3]);
                        }
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (threadIdx.x == 0 && sh.abort) set_status(a.status, PARK_ERR_TIMEOUT);
}

template <int NP>
int bwd_tc(const DenseArgs& a, const CUtensorMap* m, float* delta, float* parts, cudaStream_t st) {
    constexpr size_t sq = bwd_smem<NP, DqSmem>(), sk = bwd_smem<NP, DkvSmem>();
    {
        static std::atomic<uint64_t> done{0};
        allow_smem(k_dense_dq_tc<NP>, sq, done);
    }
    {
        static std::atomic<uint64_t> done{0};
        allow_smem(k_dense_dkv_tc<NP>, sk, done);
    }
    if (a.Nq > 0) {
        const long long tiles = dense_tiles(a.Nq, a.n_seq, kTile);
        const DenseOrder order = dense_order(a, tiles, a.B * a.Hq, 4 * a.Nk * a.D, a.Hq / a.Hk);
        ::park::prof_begin(st);
        k_dense_dq_tc<NP><<<(unsigned)(tiles * a.B * a.Hq), 384, sq, st>>>(m[0], m[1], m[2], m[3], a, order, delta,
                                                                           wait_limit_ns());
        PARK_TRY_LAUNCH("k_dense_dq_tc", st);
    }
    if (a.Nk > 0) {
        const DkvSplit sp = dense_split_dkv(a.B, a.Hq, a.Hk, a.Nq, a.Nk, a.n_seq, a.D, kTile);
        if (sp.n > 65535) return PARK_ERR_UNSUPPORTED;
        float* part_dk = parts + sp.dk_off / 4;
        const DenseOrder order = dense_order(a, sp.tiles, a.B * a.Hk, 4 * a.Nq * a.D * (a.Hq / a.Hk), 1);
        ::park::prof_begin(st);
        k_dense_dkv_tc<NP><<<dim3((unsigned)(sp.tiles * a.B * a.Hk), 1, sp.n), 384, sk, st>>>(
            m[0], m[1], m[2], m[3], a, order, delta, sp.n, sp.chunk, parts, part_dk, wait_limit_ns());
        PARK_TRY_LAUNCH("k_dense_dkv_tc", st);
        if (sp.n > 1) return launch_dense_dkv_reduce(a, PARK_BF16, sp, kTile, parts, part_dk, st);
    }
    return PARK_OK;
}

}  // namespace

int launch_dense_bwd_tc(const DenseArgs& a, float* delta, float* parts, cudaStream_t st) {
    if (a.Nq == 0 && a.Nk == 0) return PARK_OK;
    CUtensorMap m[4];
    const Op4* ops[4] = {&a.q, &a.d_o, &a.k, &a.v};
    for (int i = 0; i < 4; ++i) {
        const bool qs = i < 2, empty = qs ? a.Nq == 0 : a.Nk == 0;
        // an empty side is never loaded; its map still has to be valid
        const Op4& op = empty ? (qs ? a.k : a.q) : *ops[i];
        PARK_CHECK(map_4d(&m[i], op, empty ? 1 : a.B, empty ? 1 : qs ? a.Hq : a.Hk, empty ? 1 : qs ? a.Nq : a.Nk, a.D,
                          kTile));
    }
    return a.D <= 64 ? bwd_tc<1>(a, m, delta, parts, st) : bwd_tc<2>(a, m, delta, parts, st);
}

}  // namespace park
