// Parts that the dense attention kernels on tcgen05 share.
#pragma once

#include "dense.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace park {

using namespace sm100;

constexpr int kTile = 128;         // rows of a tile
constexpr uint32_t kPanel = 16384;  // 128 rows of 64 bf16

__device__ __forceinline__ float f_of(uint32_t u) { return __uint_as_float(u); }
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t bf2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <int N>
__device__ __forceinline__ void reg_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int n, int h, int b) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];"
        ::"r"(smem_u32(dst)), "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(n), "r"(h), "r"(b)
        : "memory");
}
// Time-bounded wait for the phase of the given parity, as mbar_wait but counting SM cycles
// (at most 2 for each ns of the limit): reading the global timer costs more than most of these waits.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (true) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort) return false;
        if ((uint64_t)(clock64() - t0) > 2 * limit_ns) {
            *abort = 1;
            return false;
        }
    }
}
// Warp index as a value that the compiler knows to be the same in all lanes.
__device__ __forceinline__ int uniform_warp() { return __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0); }
// True in one lane of a converged warp, always the same one.  The MMA warp runs its loop with all lanes and
// issues under this predicate: its operands then live in uniform registers.  Issued from an
// `if (lane == 0)` branch, each tcgen05.mma waited for their transfer and took about 95 cycles instead of
// the 64 that a 128 x 128 x 16 product needs.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
// wait_bar by a whole warp
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
    return __all_sync(0xffffffffu, wait_bar(bar, parity, abort, limit_ns));
}
// 2^x of a pair on the FMA pipe: x = n + r with n the nearest integer (from the low bits of x + 1.5 2^23)
// and |r| <= 1/2, 2^r by its minimax polynomial of degree 4 in relative error (Remez exchange, 2^-18.5;
// P is rounded to 2^-8 next), times 2^n.  x <= 128 here; below -127 the factor 2^n is 0.  NaN stays NaN.
__device__ __forceinline__ float2 ex2_poly2(float2 x) {
    const float2 magic = make_float2(12582912.f, 12582912.f);
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(x.x) : "f"(-127.f));
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(x.y) : "f"(-127.f));
    const float2 t = __fadd2_rn(x, magic);
    const float2 n = __fadd2_rn(t, make_float2(-12582912.f, -12582912.f));
    const float2 r = __fadd2_rn(x, make_float2(-n.x, -n.y));
    float2 p = __ffma2_rn(r, make_float2(0.009570102207f, 0.009570102207f), make_float2(0.05591785908f, 0.05591785908f));
    p = __ffma2_rn(p, r, make_float2(0.2402474433f, 0.2402474433f));
    p = __ffma2_rn(p, r, make_float2(0.6931217909f, 0.6931217909f));
    p = __ffma2_rn(p, r, make_float2(0.9999992847f, 0.9999992847f));
    const float2 e = make_float2(__uint_as_float((__float_as_uint(t.x) << 23) + 0x3F800000u),
                                 __uint_as_float((__float_as_uint(t.y) << 23) + 0x3F800000u));
    return __fmul2_rn(p, e);
}
// a 16-byte piece with an infinity or NaN among its bf16
__device__ __forceinline__ uint32_t nonfinite2(uint32_t w) { return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u; }

// Replaces the infinities and NaN of a 16-byte piece by 0; true if there were any.
__device__ __forceinline__ bool clean16(uint4* at) {
    uint4 w = *at;
    if (!(nonfinite2(w.x) | nonfinite2(w.y) | nonfinite2(w.z) | nonfinite2(w.w))) return false;
    uint32_t* u = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
    for (int x = 0; x < 4; ++x) u[x] &= ~(((nonfinite2(u[x]) >> 15) & 0x00010001u) * 0xFFFFu);
    *at = w;
    return true;
}

// 4-D map [B][H][N][D], boxes of 64 x box_rows, 128-byte swizzle; what lies past D or N reads as 0.
inline int map_4d(CUtensorMap* m, const Op4& op, int B, int H, long long N, int D, int box_rows) {
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)N, (cuuint64_t)H, (cuuint64_t)B};
    // strides of axes of length 1 are never used: any valid value does
    const cuuint64_t st[3] = {(cuuint64_t)(N > 1 ? op.sn * 2 : 256), (cuuint64_t)(H > 1 ? op.sh * 2 : 256),
                              (cuuint64_t)(B > 1 ? op.sb * 2 : 256)};
    const cuuint32_t box[4] = {64, (cuuint32_t)box_rows, 1, 1};
    return make_tma_map_4d(m, op.p, dims, st, box);
}

}  // namespace park
