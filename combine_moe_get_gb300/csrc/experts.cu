// experts.cu -- the experts' products of a few tokens (moe_experts).
//
//   h[t, j]  = silu(G x_t) * (U x_t),  [G; U] = w13[e], e = topk_idx[t, j]
//   out[t]   = sum_j topk_weights[t, j] * (w2[e] h[t, j])
//
// One warp per element of h, then one warp per element of out; every sum is
// fp32, in a fixed order, and out is rounded once to bf16.
#include <algorithm>
#include <cuda_bf16.h>

#include "moe_common.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kFull = 0xffffffffu;

struct ExpertArgs {
    ExpertsLaunch p;
    float *h;   // [T * k, I]
    TraceArgs trace;
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

__device__ __forceinline__ float e4m3_value(uint8_t c) {
    const int e = c >> 3 & 15, m = c & 7;
    if ((c & 0x7f) == 0x7f) return __int_as_float(0x7fc00000);
    const float v = e == 0 ? (float)m * 0x1p-9f : (float)(8 + m) * exp2f((float)(e - 10));
    return c & 0x80 ? -v : v;
}

// element i of weight row `row` (of length K)
__device__ __forceinline__ float weight(const void *w, const float *scales, size_t row, int K, int i) {
    if (scales == nullptr) return __bfloat162float(static_cast<const __nv_bfloat16 *>(w)[row * K + i]);
    return e4m3_value(static_cast<const uint8_t *>(w)[row * K + i]) * scales[row * (K / 128) + i / 128];
}

__global__ void __launch_bounds__(kThreads) experts_up_kernel(const ExpertArgs a) {
    WarpTrace wt(a.trace, MOE_TRACE_EXPERTS);
    grid_dependency_wait();
    const ExpertsLaunch &p = a.p;
    const int lane = threadIdx.x & 31, entry = blockIdx.y;
    const int64_t e = p.topk_idx[entry];
    if (e < 0 || e >= p.num_experts) {
        if (e != -1 && threadIdx.x == 0) report(p.status, MOE_ERR_BAD_TOPK);
        return;
    }
    const __nv_bfloat16 *x = static_cast<const __nv_bfloat16 *>(p.x) + (size_t)(entry / p.num_topk) * p.hidden;
    const int H = p.hidden, I = p.intermediate;
    for (int i = blockIdx.x * (kThreads / 32) + threadIdx.x / 32; i < I; i += gridDim.x * (kThreads / 32)) {
        const size_t g = (size_t)e * 2 * I + i, u = g + I;
        float sg = 0.0f, su = 0.0f;
        for (int c = lane; c < H; c += 32) {
            const float v = __bfloat162float(x[c]);
            sg += v * weight(p.w13, p.w13_scales, g, H, c);
            su += v * weight(p.w13, p.w13_scales, u, H, c);
        }
        sg = warp_sum(sg);
        su = warp_sum(su);
        if (lane == 0) a.h[(size_t)entry * I + i] = sg / (1.0f + expf(-sg)) * su;
    }
}

__global__ void __launch_bounds__(kThreads) experts_down_kernel(const ExpertArgs a) {
    WarpTrace wt(a.trace, MOE_TRACE_EXPERTS);
    grid_dependency_wait();
    const ExpertsLaunch &p = a.p;
    const int lane = threadIdx.x & 31, t = blockIdx.y;
    const int H = p.hidden, I = p.intermediate;
    for (int o = blockIdx.x * (kThreads / 32) + threadIdx.x / 32; o < H; o += gridDim.x * (kThreads / 32)) {
        float acc = 0.0f;
        for (int j = 0; j < p.num_topk; ++j) {
            const int entry = t * p.num_topk + j;
            const int64_t e = p.topk_idx[entry];
            if (e < 0 || e >= p.num_experts) continue;
            float s = 0.0f;
            for (int c = lane; c < I; c += 32)
                s += a.h[(size_t)entry * I + c] * weight(p.w2, p.w2_scales, (size_t)e * H + o, I, c);
            acc += p.topk_weights[entry] * warp_sum(s);
        }
        if (lane == 0) static_cast<__nv_bfloat16 *>(p.out)[(size_t)t * H + o] = __float2bfloat16_rn(acc);
    }
}

}  // namespace

size_t experts_workspace_bytes(int T, int H, int I, int k, int E) {
    return (size_t)T * k * I * sizeof(float);
}

int launch_experts(const ExpertsLaunch &L) {
    if (L.num_tokens == 0) return MOE_OK;
    const ExpertArgs a{L, static_cast<float *>(L.workspace), trace_args()};
    const cudaStream_t s = static_cast<cudaStream_t>(L.stream);
    const bool overlap = tuning().overlap != 0;
    const int warps = kThreads / 32;
    cudaError_t e = launch_kernel(experts_up_kernel, dim3((L.intermediate + warps - 1) / warps,
                                  L.num_tokens * L.num_topk), dim3(kThreads), 0, s, overlap, a);
    if (e == cudaSuccess)
        e = launch_kernel(experts_down_kernel, dim3((L.hidden + warps - 1) / warps, L.num_tokens), dim3(kThreads), 0,
                          s, overlap, a);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe
