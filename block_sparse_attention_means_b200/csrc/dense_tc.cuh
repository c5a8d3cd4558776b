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
