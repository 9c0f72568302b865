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
// scale amax / 448. Codes are those of x * RN(1 / scale), off x / scale by at most
// 3 * 2^-24 of it: where a quotient is that near the middle between two codes, either may come out.
// Scales whose reciprocal could overflow take the division. NaN has no part in amax
// and keeps its code; with an infinity the scale is infinite, its code NaN and all others 0.
__device__ __forceinline__ float quantise(const float (&x)[8], uint2 &codes) {
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float scale = amax / 448.0f;
    const bool tiny = scale < 7.8886090522e-31f;   // 2^-100
    const float r = tiny ? 0.0f : 1.0f / scale;
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a = x[2 * i] * r, b = x[2 * i + 1] * r;
        if (tiny) {
            a = scale > 0 ? x[2 * i] / scale : isnan(x[2 * i]) ? x[2 * i] : 0.0f;
            b = scale > 0 ? x[2 * i + 1] / scale : isnan(x[2 * i + 1]) ? x[2 * i + 1] : 0.0f;
        }
        q[i] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    }
    codes = make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
    return scale;
}

}  // namespace moe
