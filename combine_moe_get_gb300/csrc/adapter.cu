// adapter.cu -- a shared projection with the low-rank adapter of each row
// (moe_adapter_linear).
//
//   v[t]   = scales[a] * (A_a x_t),  a = adapter_idx[t]
//   out[t] = W x_t + B_a v[t]        (W x_t alone where a = -1)
//
// One warp per element of v, then one warp per element of out; sums and v are
// fp32, out is rounded once to bf16.
#include <algorithm>
#include <cuda_bf16.h>

#include "moe_common.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kFull = 0xffffffffu;

struct AdapterArgs {
    AdapterLaunch p;
    float *v;   // [T, r]
    TraceArgs trace;
};

__device__ __forceinline__ float warp_dot(const __nv_bfloat16 *x, const __nv_bfloat16 *y, int n, int lane) {
    float s = 0.0f;
    for (int c = lane; c < n; c += 32) s += __bfloat162float(x[c]) * __bfloat162float(y[c]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
    return s;
}

__global__ void __launch_bounds__(kThreads) adapter_shrink_kernel(const AdapterArgs a) {
    WarpTrace wt(a.trace, MOE_TRACE_ADAPTER_SHRINK);
    grid_dependency_wait();
    const AdapterLaunch &p = a.p;
    const int lane = threadIdx.x & 31;
    for (int t = blockIdx.x; t < p.num_tokens; t += gridDim.x) {
        const int id = p.adapter_idx[t];
        if (id < 0 || id >= p.num_adapters) {
            if (id != -1 && threadIdx.x == 0) report(p.status, MOE_ERR_BAD_ADAPTER);
            continue;
        }
        const __nv_bfloat16 *x = static_cast<const __nv_bfloat16 *>(p.x) + (size_t)t * p.in_features;
        for (int i = threadIdx.x / 32; i < p.rank; i += kThreads / 32) {
            const __nv_bfloat16 *w = static_cast<const __nv_bfloat16 *>(p.a) + ((size_t)id * p.rank + i) * p.in_features;
            const float s = warp_dot(x, w, p.in_features, lane);
            if (lane == 0) a.v[(size_t)t * p.rank + i] = p.scales[id] * s;
        }
    }
}

__global__ void __launch_bounds__(kThreads) adapter_project_kernel(const AdapterArgs a) {
    WarpTrace wt(a.trace, MOE_TRACE_ADAPTER_PROJECT);
    grid_dependency_wait();
    const AdapterLaunch &p = a.p;
    const int lane = threadIdx.x & 31;
    for (int t = blockIdx.x; t < p.num_tokens; t += gridDim.x) {
        const int id = p.adapter_idx[t];
        const __nv_bfloat16 *x = static_cast<const __nv_bfloat16 *>(p.x) + (size_t)t * p.in_features;
        for (int o = blockIdx.y * (kThreads / 32) + threadIdx.x / 32; o < p.out_features;
             o += gridDim.y * (kThreads / 32)) {
            float s = warp_dot(x, static_cast<const __nv_bfloat16 *>(p.w) + (size_t)o * p.in_features, p.in_features, lane);
            if (id >= 0 && id < p.num_adapters) {
                const __nv_bfloat16 *b = static_cast<const __nv_bfloat16 *>(p.b) + ((size_t)id * p.out_features + o) * p.rank;
                for (int i = 0; i < p.rank; ++i) s += a.v[(size_t)t * p.rank + i] * __bfloat162float(b[i]);
            }
            if (lane == 0) static_cast<__nv_bfloat16 *>(p.out)[(size_t)t * p.out_features + o] = __float2bfloat16_rn(s);
        }
    }
}

}  // namespace

size_t adapter_workspace_bytes(int T, int K, int N, int L, int r) { return (size_t)T * r * sizeof(float); }

int launch_adapter_linear(const AdapterLaunch &L) {
    if (L.num_tokens == 0) return MOE_OK;
    const AdapterArgs a{L, static_cast<float *>(L.workspace), trace_args()};
    const cudaStream_t s = static_cast<cudaStream_t>(L.stream);
    const bool overlap = tuning().overlap != 0;
    cudaError_t e = launch_kernel(adapter_shrink_kernel, dim3(L.num_tokens), dim3(kThreads), 0, s, overlap, a);
    if (e == cudaSuccess)
        e = launch_kernel(adapter_project_kernel, dim3(L.num_tokens, std::min((L.out_features + 7) / 8, 1024)),
                          dim3(kThreads), 0, s, overlap, a);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe
