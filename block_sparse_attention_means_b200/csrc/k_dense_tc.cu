// Dense attention, forward, bf16 on the 5th-generation tensor cores.
//
//   o_i = sum_j p_ij v_j / l_i,  p_ij = 2^(s_ij log2(e) scale - m_i),  one pass over the keys
//
// A CTA owns 256 query rows as two tiles of 128 ("stages") over one key head.  With
// grouped heads the rows of a sequence are counted token by token, the group's heads
// side by side (row r = token r / G, head r % G), so a single token fills G rows and
// its keys are read once for the whole group.  K and V arrive by TMA in tiles of 128
// keys, each in its own ring (a wait for a phase is sound only for a role that has seen the
// stage's phase before, and warp 10 sees V alone); the head dimension is padded to 64 or 128 by the copy's
// zero fill.  Tensor memory: S_0 | S_1 (128 columns each) | O_0 | O_1.  Per key tile
// and stage: S = Q K^T; the stage's four warps, one thread a row, turn S into P (bf16,
// over S's own columns, the A operand of the next product); O += P V.  The two stages
// alternate, so the tensor cores work on one while the other is in its Softmax:
//   S0(j+1) follows PV0(j), S1(j+1) follows PV1(j), MMAs of one thread run in issue order,
// which also means that s_full(j+1) implies that PV(j) is done: a stage may then rescale
// its O.  It does so only when its running maximum grows by more than 2^8 (P stays
// below 2^8, exact in the end since O and l carry the same reference).
//
// P is rounded to bf16, the only operand type beside V's; l sums the unrounded values.  Each rounding is off by 1.7e-3 at root
// mean square, so o, a weighted sum of many, is 1.2e-3 to 1.7e-3 of its norm off before its own rounding of 1.65e-3: 2.0e-3 to
// 2.3e-3 measured.  A second bf16 part of P would double the products with V, half of this kernel's.
//
// Warps 0-7: Softmax (stage = warp / 4) and epilogue; 8: TMA; 9: MMA; 10: forwards the V
// tiles to the MMA warp and, in tiles that a mask cuts, replaces infinities and NaN by 0:
// 0 x NaN is NaN, so a hidden row would reach all rows of its tile.  What the rows do see
// of them is added in the epilogue.
//
// When the row tiles do not fill the GPU, the keys are split over CTAs; each writes its
// part's normalised O in float32 and its log-sum-exp, and k_dense_combine joins them.
//
// Every wait is time-bounded (PARK_ERR_TIMEOUT); on a failed wait the roles leave their
// loops, copies and MMAs in flight are waited for and TMEM is freed.
#include "dense_tc.cuh"

namespace park {

using namespace sm100;

namespace {

constexpr float kRescale = 8.f;        // log2 units

// NP: 64-column panels of the padded head dimension.  NS: 128-row stages of a CTA.  Two stages share each K and V tile and
// one CTA fills an SM; one stage leaves room for a second CTA, whose work covers this one's start and end.
template <int NP, int NS>
struct FwdCfg {
    static constexpr int KS = NS == 2 ? (NP == 2 ? 3 : 4) : (NP == 2 ? 1 : 2);  // ring stages of K
    static constexpr int VS = NS == 2 ? (NP == 2 ? 2 : 4) : (NP == 2 ? 1 : 2);  // and of V
    static constexpr uint32_t tile = NP * kPanel;
    static constexpr size_t smem = (size_t)(NS + KS + VS) * tile + 1024;
    static constexpr int threads = 128 * NS + 128, ctas = NS == 2 ? 1 : 2;
    static constexpr int tmem_cols = NS == 2 ? 512 : 256, O = 128 * NS;  // S_0 (S_1) O_0 (O_1)
    // registers of a Softmax thread and of the others: 256 x 216 + 128 x 56 of the 384 x 168 that a launch of two stages
    // holds, 128 x 200 + 128 x 56 = 256 x 128 of one
    static constexpr int soft_regs = NS == 2 ? 216 : 200, misc_regs = 56;
};

struct FwdSmem {
    uint64_t q_full[2], k_full[4], k_empty[4], v_full[4], v_clean[4], v_empty[4], s_full[2], p_full[2][2], o_full[2], final_bar;
    uint32_t tmem_base;
    int abort, poison;
    SeqTile seq;
};

// Pairs of exponentials that go to the FMA pipe (see ex2_poly2): two of eight.  All on the special-function unit, an
// iteration's exponentials take as long as its products: 1233 / 810 TFLOP/s at 16,384 x 8 heads, D = 128 / 64; with one
// pair in four moved 1248 / 814, with three in eight 1203 / 830.
__device__ constexpr bool poly_pair(int e) { return e % 4 == 0; }

// Row of a group's rows -> token (a division only where heads share keys).
__device__ __forceinline__ int token_of(int r, int G) { return G == 1 ? r : r / G; }

// Walks rows r, r + RS, r + 2 RS .. of a tensor whose rows are counted token by token, heads side by side: offset of the
// row from the first head's first token, in bytes.
template <int RS>
struct RowWalk {
    int g, G, dg;
    long long at, step, carry;
    __device__ __forceinline__ RowWalk(int r, int G_, long long sh, long long sn) : G(G_) {
        const int tk = token_of(r, G), q = G == 1 ? RS : RS / G;
        g = r - tk * G;
        dg = RS - q * G;
        at = (tk * sn + g * sh) * 2;
        step = (q * sn + dg * sh) * 2;
        carry = (sn - G * sh) * 2;
    }
    __device__ __forceinline__ void next() {
        at += step;
        g += dg;
        if (g >= G) {
            g -= G;
            at += carry;
        }
    }
};

// The CTA's piece: rows r0 .. of the sequence's nq G rows, key tiles j_lo .. j_lo + nt[t] - 1 of stage t.
template <int NS>
struct Piece {
    int r0, rows, nt[NS], j_lo, jmax;
};
template <int NS>
__device__ __forceinline__ Piece<NS> fwd_piece(const SeqTile& t, int G, int causal, int n_split, int sp, int chunk) {
    Piece<NS> p;
    p.r0 = t.tile * NS * kTile;
    p.rows = t.live ? min(NS * kTile, t.nq * G - p.r0) : 0;
    p.jmax = 0;
    p.j_lo = n_split > 1 ? sp * chunk : 0;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
        const int last = min(p.rows, (s + 1) * kTile) - 1;  // last row of the stage
        int n = 0;
        if (last >= s * kTile) {
            const int kend = dense_last_key(token_of(p.r0 + last, G), t.nq, t.nk, causal) + 1;
            n = kend > 0 ? (kend + kTile - 1) / kTile : 0;
            n = max(0, (n_split > 1 ? min(n, p.j_lo + chunk) : n) - p.j_lo);
        }
        p.nt[s] = n;
        p.jmax = max(p.jmax, n);
    }
    return p;
}

template <int NP, int NS>
__global__ void __launch_bounds__(FwdCfg<NP, NS>::threads, FwdCfg<NP, NS>::ctas)
    k_dense_fwd_tc(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, DenseArgs a,
                   DenseOrder order, int n_split, int chunk, float* __restrict__ part_o, float* __restrict__ part_lse, uint64_t wait_ns) {
    using C = FwdCfg<NP, NS>;
    extern __shared__ __align__(1024) uint8_t dsmem[];
    __shared__ FwdSmem sh;
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dsmem) + 1023) & ~uintptr_t(1023));
    uint8_t* Qs = base;                 // NS tiles
    uint8_t* Ks = base + NS * C::tile;  // rings
    uint8_t* Vs = Ks + C::KS * C::tile;
    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    volatile int* abort = &sh.abort;
    int x_tile;
    const int bh = dense_block_head(order, x_tile), b = a.B == 1 ? 0 : bh / a.Hk, hk = bh - b * a.Hk, sp = blockIdx.z;
    if (warp == 0) {
        const SeqTile t = dense_block_tile(a, order, x_tile, NS * kTile, false, a.Hq / a.Hk);
        if (lane == 0) {
            sh.seq = t;
            for (int s = 0; s < NS; ++s) {
                mbar_init(&sh.q_full[s], 128);
                mbar_init(&sh.s_full[s], 1);
                mbar_init(&sh.p_full[s][0], 128);
                mbar_init(&sh.p_full[s][1], 128);
                mbar_init(&sh.o_full[s], 1);
            }
            for (int s = 0; s < C::KS; ++s) {
                mbar_init(&sh.k_full[s], 1);
                mbar_init(&sh.k_empty[s], 1);
            }
            for (int s = 0; s < C::VS; ++s) {
                mbar_init(&sh.v_full[s], 1);
                mbar_init(&sh.v_clean[s], 1);
                mbar_init(&sh.v_empty[s], 1);
            }
            mbar_init(&sh.final_bar, 1);
            sh.abort = 0;
            sh.poison = 0;
            mbar_fence_init();
        }
    } else if (warp == 4 * NS + 1) {
        tmem_alloc(&sh.tmem_base, C::tmem_cols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem_base;
    const SeqTile t = sh.seq;
    const int G = a.Hq / a.Hk;
    const Piece<NS> pc = fwd_piece<NS>(t, G, a.causal, n_split, sp, chunk);
    // first key tile (counted within the piece) that some row does not see whole
    const int cut = (dense_last_key(token_of(pc.r0, G), t.nq, t.nk, a.causal) + 1) / kTile - pc.j_lo;

    if (warp >= 4 * NS) {
        reg_dec<C::misc_regs>();
        if (warp == 4 * NS && lane == 0) {
            // ---------------------------------------------------------------- TMA
            tma_prefetch_desc(&tmK);
            tma_prefetch_desc(&tmV);
            int nk = 0, nv = 0;  // tiles issued
            for (int j = 0; j < pc.jmax; ++j) {
                const int n = t.k0 + (pc.j_lo + j) * kTile;
                const int ks = j % C::KS, vs = j % C::VS;
                if (j >= C::KS && !wait_bar(&sh.k_empty[ks], (j / C::KS - 1) & 1, abort, wait_ns)) break;
                mbar_arrive_expect_tx(&sh.k_full[ks], C::tile);
                for (int p = 0; p < NP; ++p)
                    tma_load_4d(Ks + ks * C::tile + p * kPanel, &tmK, &sh.k_full[ks], 64 * p, n, hk, b);
                ++nk;
                if (j >= C::VS && !wait_bar(&sh.v_empty[vs], (j / C::VS - 1) & 1, abort, wait_ns)) break;
                mbar_arrive_expect_tx(&sh.v_full[vs], C::tile);
                for (int p = 0; p < NP; ++p)
                    tma_load_4d(Vs + vs * C::tile + p * kPanel, &tmV, &sh.v_full[vs], 64 * p, n, hk, b);
                ++nv;
            }
            int dummy = 0;  // copies in flight land before the CTA may exit
            for (int j = max(0, nk - C::KS); j < nk; ++j)
                wait_bar(&sh.k_full[j % C::KS], (j / C::KS) & 1, &dummy, 100000000ull);
            for (int j = max(0, nv - C::VS); j < nv; ++j)
                wait_bar(&sh.v_full[j % C::VS], (j / C::VS) & 1, &dummy, 100000000ull);
        } else if (warp == 4 * NS + 1) {
            // ---------------------------------------------------------------- MMA
            const uint32_t idS = idesc_bf16(128, 128, 0, 0), idO = idesc_bf16(128, 64 * NP, 0, 1);
            const bool lead = elect_one();
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            const uint64_t dQ = sdesc_sw128(smem_u32(Qs), 16, 1024), dK = sdesc_sw128(smem_u32(Ks), 16, 1024);
            const uint64_t dV = sdesc_sw128(smem_u32(Vs), kPanel, 1024);
            auto issue_S = [&](int s, int j) -> bool {
                const int st = j % C::KS;
                if (!wait_warp(&sh.k_full[st], (j / C::KS) & 1, abort, wait_ns)) return false;
                tc_fence_after();
                const uint64_t qa = dQ + ((s * C::tile) >> 4), ka = dK + ((st * C::tile) >> 4);
                if (lead) {
#pragma unroll
                    for (int kk = 0; kk < 4 * NP; ++kk) {
                        const uint32_t off = ((kk >> 2) * kPanel + (kk & 3) * 32) >> 4;
                        umma_bf16(tm + 128 * s, qa + off, ka + off, idS, kk > 0);
                    }
                    umma_commit(&sh.s_full[s]);
                    // the last stage that uses K_j frees it
                    if (s == NS - 1 || pc.nt[NS - 1] <= j) umma_commit(&sh.k_empty[st]);
                }
                __syncwarp();
                return true;
            };
            bool ok = true;
            for (int s = 0; s < NS && ok; ++s)
                if (pc.nt[s] > 0) {
                    ok = wait_warp(&sh.q_full[s], 0, abort, wait_ns);
                    if (ok) ok = issue_S(s, 0);
                }
            for (int j = 0; j < pc.jmax && ok; ++j) {
                const int st = j % C::VS;
                const uint64_t va = dV + ((st * C::tile) >> 4);
                if (!wait_warp(&sh.v_clean[st], (j / C::VS) & 1, abort, wait_ns)) break;
                for (int s = 0; s < NS && ok; ++s) {
                    if (j >= pc.nt[s]) continue;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (!wait_warp(&sh.p_full[s][h], j & 1, abort, wait_ns)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        if (lead) {
#pragma unroll
                            for (int kk = 4 * h; kk < 4 * h + 4; ++kk)
                                umma_bf16_ts(tm + C::O + 64 * NP * s, tm + 128 * s + 8 * kk, va + ((kk * 2048) >> 4), idO,
                                             j > 0 || kk > 0);
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                    if (lead) {
                        if (j + 1 == pc.nt[s]) umma_commit(&sh.o_full[s]);
                        if (s == NS - 1 || pc.nt[NS - 1] <= j) umma_commit(&sh.v_empty[st]);
                    }
                    __syncwarp();
                    if (j + 1 < pc.nt[s]) ok = issue_S(s, j + 1);
                }
            }
            if (lead) umma_commit(&sh.final_bar);  // every MMA is done before TMEM is released
            __syncwarp();
            int dummy = 0;
            wait_bar(&sh.final_bar, 0, &dummy, 100000000ull);
        } else if (warp == 4 * NS + 2) {
            // ---------------------------------------------------------------- V tiles: forward, clean where cut
            for (int j = 0; j < pc.jmax; ++j) {
                const int st = j % C::VS;
                if (!__all_sync(0xffffffffu, wait_bar(&sh.v_full[st], (j / C::VS) & 1, abort, wait_ns))) break;
                if (j >= cut) {
                    const int n0 = (pc.j_lo + j) * kTile;
                    uint4* v = reinterpret_cast<uint4*>(Vs + st * C::tile);
                    for (int e = lane; e < (int)(C::tile / 16); e += 32) {
                        // (128 rows of 8 pieces to a panel; rows behind the last key poison nothing)
                        if (clean16(v + e) && n0 + (e >> 3) % kTile < t.nk) sh.poison = 1;
                    }
                    fence_proxy_async_smem();
                    __threadfence_block();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.v_clean[st]);
            }
        }
        __syncwarp();
    } else {
        // -------------------------------------------------------------------- Softmax
        reg_inc<C::soft_regs>();
        const int s = warp >> 2, quad = warp & 3, row = 32 * quad + lane;
        const uint32_t trow = tmem + ((uint32_t)(32 * quad) << 16);
        const uint32_t scol = trow + 128 * s, ocol = trow + C::O + 64 * NP * s;
        const int nt = pc.nt[s];
        const bool live = kTile * s + row < pc.rows;
        // The warp's 32 rows move 16 bytes a lane: piece `pc16` of row (lane / PR) and of every (32 / PR)-th row after it.
        constexpr int PR = 8 * NP, RS = 32 / PR;  // pieces of a row, rows of a step
        uint8_t* qt = Qs + s * C::tile;
        const int pc16 = lane % PR, row0 = kTile * s + 32 * quad + lane / PR;
        const bool piece = pc16 < a.D / 8;
        if (nt > 0) {
            RowWalk<RS> w(pc.r0 + row0, G, a.q.sh, a.q.sn);
            const uint8_t* qb = a.q.p + (b * a.q.sb + hk * (long long)G * a.q.sh + t.q0 * a.q.sn) * 2 + 16 * pc16;
            const uint32_t dst = smem_u32(qt) + (pc16 >> 3) * kPanel;
#pragma unroll 4
            for (int i = 0; i < PR; ++i) {
                const int rr = 32 * quad + lane / PR + i * RS;
                const bool on = piece && row0 + i * RS < pc.rows;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + rr * 128 + (((pc16 & 7) ^ (rr & 7)) << 4)),
                             "l"(qb + (on ? w.at : 0)), "r"(on ? 16 : 0)
                             : "memory");  // (0 bytes read: zeros)
                w.next();
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_proxy_async_smem();
            mbar_arrive(&sh.q_full[s]);
        }
        const float sl2 = a.scale * kLog2e, NI = __int_as_float(0xff800000);
        const float2 sl22 = make_float2(sl2, sl2);
        const int seen = live ? dense_last_key(token_of(pc.r0 + kTile * s + row, G), t.nq, t.nk, a.causal) : -1;  // last visible key
        float m = NI;
        float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        bool ok = true;
        for (int j = 0; j < nt; ++j) {
            if (!__all_sync(0xffffffffu, wait_bar(&sh.s_full[s], j & 1, abort, wait_ns))) {
                ok = false;
                break;
            }
            tc_fence_after();
            uint32_t x[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(scol + 32 * c, x[c]);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld_dep(x[c]);
            if (j >= cut) {
                const int lim = seen - (pc.j_lo + j) * kTile;  // columns 0 .. lim are visible
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (32 * c + e > lim) x[c][e] = 0xff800000u;
            }
            float tm[4] = {NI, NI, NI, NI};
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int e = 0; e < 32; e += 2) tm[(e >> 1) & 3] = max3(tm[(e >> 1) & 3], f_of(x[c][e]), f_of(x[c][e + 1]));
            const float tmax = fmaxf(fmaxf(tm[0], tm[1]), fmaxf(tm[2], tm[3])) * sl2;
            if (j == 0) {
                m = tmax;
            } else if (__any_sync(0xffffffffu, tmax > m + kRescale)) {
                // decided per warp; rows that keep their reference get a factor of 1
                const float mn = tmax > m + kRescale ? tmax : m;
                const float f = mn == m ? 1.f : ex2(m - mn);
#pragma unroll
                for (int c = 0; c < 2 * NP; ++c) {
                    uint32_t o[32];
                    tmem_ld32(ocol + 32 * c, o);
                    tmem_ld_wait();
                    tmem_ld_dep(o);
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(f_of(o[e]) * f);
                    tmem_st32(ocol + 32 * c, o);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) l2[e] = __fmul2_rn(l2[e], make_float2(f, f));
                m = mn;
            }
            const float mr = m == NI ? 0.f : m;  // a row that has seen no key yet: P = 0
            const float2 nm = make_float2(-mr, -mr);
#pragma unroll
            for (int h = 0; h < 2; ++h) {  // the MMA warp starts on the first 64 keys while the others follow
                uint32_t pk[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const int c = 2 * h + (e >> 4), y = 2 * (e & 15);
                    const float2 d = __ffma2_rn(make_float2(f_of(x[c][y]), f_of(x[c][y + 1])), sl22, nm);
                    const float2 pe = poly_pair(e) ? ex2_poly2(d) : make_float2(ex2(d.x), ex2(d.y));
                    l2[e & 1] = __fadd2_rn(l2[e & 1], pe);
                    pk[e] = bf2(pe.x, pe.y);
                }
                tmem_st32(scol + 32 * h, pk);
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&sh.p_full[s][h]);
            }
        }
        // ---------------------------------------------------------------- epilogue
        const float l = (l2[0].x + l2[0].y) + (l2[1].x + l2[1].y);
        if (nt > 0 && ok) ok = __all_sync(0xffffffffu, wait_bar(&sh.o_full[s], 0, abort, wait_ns));
        if (ok) {
            tc_fence_after();
            int r = pc.r0 + kTile * s + row;  // (formed again: nothing of it has to live through the loop)
            asm volatile("" : "+r"(r));
            const int tok = token_of(r, G), head = hk * G + (r - tok * G);
            const bool poison = sh.poison != 0;
            const bool none = m == NI && l == 0.f;  // no visible key (or every score -inf)
            const float inv = none ? 0.f : 1.f / l;
            const size_t row_id = ((size_t)b * a.Hq + head) * a.Nq + t.q0 + tok;
            const size_t rows_all = (size_t)a.B * a.Hq * a.Nq;
            const bool split = n_split > 1;
            if (live) {
                const float lse = none ? NI : (m + log2f(l));
                if (split)
                    part_lse[sp * rows_all + row_id] = lse;
                else if (a.lse)
                    a.lse[row_id] = lse * kLn2;
            }
            float* prow = part_o + (sp * rows_all + row_id) * a.D;
            if (!(split && nt == 0)) {  // (a part without keys is only its lse)
#pragma unroll 1
                for (int c = 0; 32 * c < a.D; ++c) {
                    uint32_t o[32];
                    __syncwarp();
                    if (nt > 0) {
                        tmem_ld32(ocol + 32 * c, o);
                        tmem_ld_wait();
                        tmem_ld_dep(o);
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {  // (rows without a key: O = 0, inv = 0)
                            const float2 x = __fmul2_rn(make_float2(f_of(o[e]), f_of(o[e + 1])), make_float2(inv, inv));
                            o[e] = __float_as_uint(x.x);
                            o[e + 1] = __float_as_uint(x.y);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = 0u;
                    }
                    if (poison && live) {  // infinities and NaN that the row does see in the cut tiles
                        const int k1 = min(seen + 1, (pc.j_lo + nt) * kTile);
                        for (int key = max(0, pc.j_lo + cut) * kTile; key < k1; ++key) {
                            const uint16_t* vr = reinterpret_cast<const uint16_t*>(
                                                     a.v.p + (b * a.v.sb + hk * a.v.sh + (t.k0 + (long long)key) * a.v.sn) * 2) + 32 * c;
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if ((vr[e] & 0x7F80u) == 0x7F80u)
                                    o[e] = __float_as_uint(f_of(o[e]) + f_of((uint32_t)vr[e] << 16));
                        }
                    }
                    if (live && split) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<uint4*>(prow + 32 * c + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                    } else if (!split) {  // through the stage's own Q tile, which no MMA reads any more
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
                            *reinterpret_cast<uint4*>(qt + (c >> 1) * kPanel + row * 128 +
                                                      ((((4 * c + (e >> 3)) & 7) ^ (row & 7)) << 4)) =
                                make_uint4(bf2(f_of(o[e]), f_of(o[e + 1])), bf2(f_of(o[e + 2]), f_of(o[e + 3])),
                                           bf2(f_of(o[e + 4]), f_of(o[e + 5])), bf2(f_of(o[e + 6]), f_of(o[e + 7])));
                    }
                }
            }
            if (!split) {  // whole rows
                __syncwarp();
                RowWalk<RS> w(pc.r0 + row0, G, a.o.sh, a.o.sn);
                uint8_t* ob = a.o.p + (b * a.o.sb + hk * (long long)G * a.o.sh + t.q0 * a.o.sn) * 2 + 16 * pc16;
#pragma unroll 4
                for (int i = 0; i < PR; ++i) {
                    const int rr = 32 * quad + lane / PR + i * RS;
                    const uint4 v = *reinterpret_cast<const uint4*>(qt + (pc16 >> 3) * kPanel + rr * 128 + (((pc16 & 7) ^ (rr & 7)) << 4));
                    if (piece && row0 + i * RS < pc.rows) *reinterpret_cast<uint4*>(ob + w.at) = v;
                    w.next();
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 4 * NS + 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::tmem_cols);
    }
    if (threadIdx.x == 0 && sh.abort) set_status(a.status, PARK_ERR_TIMEOUT);
}

template <int NP, int NS>
int fwd_tc(const DenseArgs& a, const CUtensorMap& mK, const CUtensorMap& mV, const DenseSplit& sp, float* part_o,
           float* part_lse, cudaStream_t st) {
    using C = FwdCfg<NP, NS>;
    {
        static std::atomic<uint64_t> done{0};
        allow_smem(k_dense_fwd_tc<NP, NS>, C::smem, done);
    }
    const DenseOrder order = dense_order(a, sp.tiles, a.B * a.Hk, 4 * a.Nk * a.D, 1);
    const dim3 grid((unsigned)(sp.tiles * a.B * a.Hk), 1, sp.n);
    ::park::prof_begin(st);
    k_dense_fwd_tc<NP, NS><<<grid, C::threads, C::smem, st>>>(mK, mV, a, order, sp.n, sp.chunk, part_o, part_lse, wait_limit_ns());
    PARK_TRY_LAUNCH(NS == 2 ? "k_dense_fwd_tc, 256 rows" : "k_dense_fwd_tc, 128 rows", st);
    return PARK_OK;
}

}  // namespace

int launch_dense_fwd_tc(const DenseArgs& a, void* ws, cudaStream_t st) {
    const DenseSplit sp = dense_split_tc(a.B, a.Hq, a.Hk, a.Nq, a.Nk, a.n_seq, a.D);
    if (sp.n > 65535) return PARK_ERR_UNSUPPORTED;
    CUtensorMap mK, mV;
    // without keys nothing is loaded; the maps still have to be valid
    PARK_CHECK(map_4d(&mK, a.Nk ? a.k : a.q, a.Nk ? a.B : 1, a.Nk ? a.Hk : 1, a.Nk ? a.Nk : 1, a.D, kTile));
    PARK_CHECK(map_4d(&mV, a.Nk ? a.v : a.q, a.Nk ? a.B : 1, a.Nk ? a.Hk : 1, a.Nk ? a.Nk : 1, a.D, kTile));
    float* part_o = static_cast<float*>(ws);
    float* part_lse = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + sp.lse_off);
    PARK_CHECK(sp.rows == 256 ? (a.D <= 64 ? fwd_tc<1, 2>(a, mK, mV, sp, part_o, part_lse, st)
                                           : fwd_tc<2, 2>(a, mK, mV, sp, part_o, part_lse, st))
                              : (a.D <= 64 ? fwd_tc<1, 1>(a, mK, mV, sp, part_o, part_lse, st)
                                           : fwd_tc<2, 1>(a, mK, mV, sp, part_o, part_lse, st)));
    return sp.n > 1 ? launch_dense_combine(a, PARK_BF16, sp.n, part_o, part_lse, st) : PARK_OK;
}

}  // namespace park
