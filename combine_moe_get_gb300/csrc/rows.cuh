// rows.cuh -- eight bf16 at a time and blocks of 128 channels in E4M3, for the
// kernels that pass once over rows (swiglu.cu, norm.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "moe_common.cuh"

namespace moe {

// 16 bytes that this kernel reads once (coherent: the same thread may write its result there)
__device__ __forceinline__ uint4 load_once(const void *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

__device__ __forceinline__ void widen(const uint4 &v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 narrow(const float (&x)[8]) {
    uint4 v;
    __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    return v;
}

// E4M3 codes of 128 channels held by 16 neighbouring lanes, eight each, and their
// scale amax / 448 (its rounded product with 1 / 448, corrected by what that leaves:
// off by 2^-24 of it). Codes are those of x * r with r the fast reciprocal, off x / scale by
// at most 2^-22 of it: where a quotient is that near the middle between two codes,
// either may come out. Scales whose reciprocal could overflow, or that are not normal, take the division. NaN has no part
// in amax and keeps its code; with an infinity the scale is infinite, its code NaN and all others 0.
__device__ __forceinline__ float quantise(const float (&x)[8], uint2 &codes) {
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    constexpr float k = 1.0f / 448.0f;
    const float q0 = amax * k;
    float scale = fmaf(fmaf(-q0, 448.0f, amax), k, q0);
    uint32_t q[4];
    if (amax > 5.7e-28f && amax < 3.0e38f) {   // far inside what has a normal scale and reciprocal
        float r;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(scale));
#pragma unroll
        for (int i = 0; i < 4; ++i)
            q[i] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(x[2 * i] * r, x[2 * i + 1] * r), __NV_SATFINITE, __NV_E4M3);
    } else {
        scale = amax / 448.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = x[2 * i], b = x[2 * i + 1];
            q[i] = (uint32_t)__nv_cvt_float2_to_fp8x2(
                make_float2(scale > 0 || isnan(a) ? a / scale : 0.0f, scale > 0 || isnan(b) ? b / scale : 0.0f), __NV_SATFINITE,
                __NV_E4M3);
        }
    }
    codes = make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
    return scale;
}

}  // namespace moe
