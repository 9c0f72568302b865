// norm.cu -- root-mean-square norm of rows behind the residual's addition:
//
//   h = x + residual,  y = h * rsqrt(mean(h^2) + eps) * weight
//   with n = h * r, r = rsqrt(mean(h^2) + eps), d = dy * weight:
//   dh = r (d - n mean(d n)) + dresidual,  dweight = sum over rows of dy n
//
// One pass over the rows, bound by HBM: a row stays in the registers of its threads
// (kVec times 8 channels each) between the sum of squares and the output. The sums
// are fp32; h enters them unrounded, and is rounded to bf16 only where it is stored.
#include "rows.cuh"

namespace moe {
namespace {

constexpr int kMaxWarps = 32;

struct NormArgs {
    const __nv_bfloat16 *x, *residual;   // backward: h, and the gradient that reaches the residual (or null)
    const __nv_bfloat16 *grad;
    const void *weight;
    bool wide_weight;                    // fp32
    float eps;
    __nv_bfloat16 *out, *residual_out;   // backward: grad_x
    uint8_t *codes;
    float *scales;
    float *parts, *grad_weight;          // backward: [parts][H] sums of a CTA's rows each
    int T, H, num_parts;
    int row_warps;                       // warps of a row
    TraceArgs trace;
};

__device__ __forceinline__ void load_weight(const NormArgs &a, int col, float (&w)[8]) {
    if (a.wide_weight) {
        const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(a.weight) + col);
        const float4 lo = __ldg(p), hi = __ldg(p + 1);
        w[0] = lo.x, w[1] = lo.y, w[2] = lo.z, w[3] = lo.w, w[4] = hi.x, w[5] = hi.y, w[6] = hi.z, w[7] = hi.w;
    } else {
        widen(__ldg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.weight) + col)), w);
    }
}

// Sums of N values over the warps of this thread's row, in a fixed order. `place` alternates from call to call, so
// that one barrier is enough. Every thread of the CTA calls it.
template <int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*space)[kMaxWarps], int row_warps) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if (row_warps == 1) return;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, first = warp / row_warps * row_warps;
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (lane == 0) space[i][warp] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = lane < row_warps ? space[i][first + lane] : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    }
}

template <int kVec, bool kCodes>
__global__ __launch_bounds__(kVec < 8 ? 512 : 1024) void norm_kernel(const __grid_constant__ NormArgs a) {
    const WarpTrace trace(a.trace, MOE_TRACE_NORM);
    __shared__ float space[1][kMaxWarps];
    grid_dependency_wait();
    grid_launch_dependents();
    const int threads = a.row_warps * 32, sub = threadIdx.x / threads, tid = threadIdx.x - sub * threads;
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x / threads) + sub;
    const bool live = row < a.T;
    const size_t base = (size_t)row * a.H;
    uint4 x[kVec], res[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        const int col = (j * threads + tid) * 8;
        x[j] = res[j] = make_uint4(0, 0, 0, 0);
        if (live && col < a.H) {
            x[j] = load_once(a.x + base + col);
            if (a.residual) res[j] = load_once(a.residual + base + col);
        }
    }
    float h[kVec][8], sum[1] = {};
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        widen(x[j], h[j]);
        if (a.residual) {
            float r[8];
            widen(res[j], r);
#pragma unroll
            for (int i = 0; i < 8; ++i) h[j][i] += r[i];
            const int col = (j * threads + tid) * 8;
            if (a.residual_out && live && col < a.H) *reinterpret_cast<uint4 *>(a.residual_out + base + col) = narrow(h[j]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[0] = fmaf(h[j][i], h[j][i], sum[0]);
    }
    row_sums(sum, space, a.row_warps);
    const float r = rsqrtf(sum[0] / a.H + a.eps);
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        const int col = (j * threads + tid) * 8;
        const bool in = live && col < a.H;
        float w[8] = {};
        if (in) load_weight(a, col, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[j][i] = h[j][i] * r * w[i];
        if (a.out && in) *reinterpret_cast<uint4 *>(a.out + base + col) = narrow(h[j]);
        if constexpr (kCodes) {   // H is a multiple of 128: 16 lanes are in the row or not
            uint2 codes;
            const float scale = quantise(h[j], codes);
            if (in) {
                *reinterpret_cast<uint2 *>(a.codes + base + col) = codes;
                if ((threadIdx.x & 15) == 0) a.scales[(base + col) / 128] = scale;
            }
        }
    }
}

// A CTA takes every num_parts-th row and keeps the weight's gradient of its columns in registers.
template <int kVec>
__global__ __launch_bounds__(kVec < 8 ? 512 : 1024) void norm_backward_kernel(const __grid_constant__ NormArgs a) {
    const WarpTrace trace(a.trace, MOE_TRACE_NORM_BACKWARD);
    __shared__ float space[2][2][kMaxWarps];
    grid_dependency_wait();
    grid_launch_dependents();
    const int threads = blockDim.x, tid = threadIdx.x;
    float dw[kVec][8] = {};
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x, turn ^= 1) {
        const size_t base = (size_t)row * a.H;
        uint4 h4[kVec], g4[kVec], res[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            const int col = (j * threads + tid) * 8;
            h4[j] = g4[j] = res[j] = make_uint4(0, 0, 0, 0);
            if (col < a.H) {
                h4[j] = load_once(a.x + base + col);
                g4[j] = load_once(a.grad + base + col);
                if (a.residual) res[j] = load_once(a.residual + base + col);
            }
        }
        float sum[2] = {};   // of h^2 and of d h
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            const int col = (j * threads + tid) * 8;
            float h[8], g[8], w[8] = {};
            widen(h4[j], h);
            widen(g4[j], g);
            if (col < a.H) load_weight(a, col, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                sum[0] = fmaf(h[i], h[i], sum[0]);
                sum[1] = fmaf(g[i] * w[i], h[i], sum[1]);
            }
        }
        row_sums(sum, space[turn], a.row_warps);
        const float r = rsqrtf(sum[0] / a.H + a.eps), m = r * r * (sum[1] / a.H);   // m h = n mean(d n)
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            const int col = (j * threads + tid) * 8;
            if (col >= a.H) continue;
            float h[8], g[8], w[8], add[8];
            widen(h4[j], h);
            widen(g4[j], g);
            widen(res[j], add);
            load_weight(a, col, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                dw[j][i] = fmaf(g[i], h[i] * r, dw[j][i]);
                add[i] += r * (g[i] * w[i] - h[i] * m);
            }
            *reinterpret_cast<uint4 *>(a.out + base + col) = narrow(add);
        }
    }
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        const int col = (j * threads + tid) * 8;
        if (col >= a.H) continue;
        float4 *p = reinterpret_cast<float4 *>(a.parts + (size_t)blockIdx.x * a.H + col);
        p[0] = make_float4(dw[j][0], dw[j][1], dw[j][2], dw[j][3]);
        p[1] = make_float4(dw[j][4], dw[j][5], dw[j][6], dw[j][7]);
    }
}

// The weight's gradient: the CTAs' sums, in order. 32 columns a CTA, its 8 warps every eighth part each.
__global__ __launch_bounds__(256) void norm_weight_kernel(const __grid_constant__ NormArgs a) {
    const WarpTrace trace(a.trace, MOE_TRACE_NORM_WEIGHT);
    __shared__ float space[8][32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, col = blockIdx.x * 32 + lane;
    float sum = 0.0f;
    if (col < a.H)
#pragma unroll 8
        for (int p = warp; p < a.num_parts; p += 8) sum += __ldcg(a.parts + (size_t)p * a.H + col);
    space[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && col < a.H) {
#pragma unroll
        for (int i = 1; i < 8; ++i) sum += space[i][lane];
        a.grad_weight[col] = sum;
    }
}

// Vectors of 8 channels that a thread holds, for rows of H: `most` warps a row at best, else as many as fit.
int vectors(int H, int most_warps) {
    int v = 1;
    while (v < 8 && (H + v * 256 - 1) / (v * 256) > most_warps) v *= 2;
    return v;
}

// CTAs of the backward kernel, each with a part of the weight's gradient.
int backward_parts(int T) {
    const int most = 2 * device_sm_count();
    return T < most ? T : most;
}

template <int kVec>
cudaError_t launch_forward(NormArgs &a, cudaStream_t s) {
    a.row_warps = (a.H + kVec * 256 - 1) / (kVec * 256);
    const int rows = a.row_warps >= 8 ? 1 : 8 / a.row_warps;
    const dim3 grid((unsigned)(((int64_t)a.T + rows - 1) / rows)), block(rows * a.row_warps * 32);
    return a.codes ? launch_kernel(norm_kernel<kVec, true>, grid, block, 0, s, tuning().overlap != 0, a)
                   : launch_kernel(norm_kernel<kVec, false>, grid, block, 0, s, tuning().overlap != 0, a);
}

template <int kVec>
cudaError_t launch_backward(NormArgs &a, cudaStream_t s) {
    a.row_warps = (a.H + kVec * 256 - 1) / (kVec * 256);
    return launch_kernel(norm_backward_kernel<kVec>, dim3(a.num_parts), dim3(a.row_warps * 32), 0, s, tuning().overlap != 0, a);
}

}  // namespace

size_t norm_backward_workspace_bytes(int T, int H) { return (size_t)(T < 512 ? T : 512) * H * sizeof(float); }

int launch_norm(const NormLaunch &L) {
    if (L.num_tokens == 0) return MOE_OK;
    NormArgs a{};
    a.x = static_cast<const __nv_bfloat16 *>(L.x), a.residual = static_cast<const __nv_bfloat16 *>(L.residual);
    a.weight = L.weight, a.wide_weight = L.weight_type == MOE_NORM_WEIGHT_F32;
    a.eps = L.eps;
    a.out = static_cast<__nv_bfloat16 *>(L.out), a.residual_out = static_cast<__nv_bfloat16 *>(L.residual_out);
    a.codes = static_cast<uint8_t *>(L.codes), a.scales = L.scales;
    a.T = L.num_tokens, a.H = L.hidden;
    a.trace = trace_args();
    const cudaStream_t s = static_cast<cudaStream_t>(L.stream);
    cudaError_t e;
    switch (vectors(a.H, 16)) {
        case 1: e = launch_forward<1>(a, s); break;
        case 2: e = launch_forward<2>(a, s); break;
        case 4: e = launch_forward<4>(a, s); break;
        default: e = launch_forward<8>(a, s); break;
    }
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int launch_norm_backward(const NormLaunch &L) {
    const cudaStream_t s = static_cast<cudaStream_t>(L.stream);
    if (L.num_tokens == 0)
        return cudaMemsetAsync(L.grad_weight, 0, (size_t)L.hidden * sizeof(float), s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
    NormArgs a{};
    a.x = static_cast<const __nv_bfloat16 *>(L.x), a.residual = static_cast<const __nv_bfloat16 *>(L.residual);
    a.grad = static_cast<const __nv_bfloat16 *>(L.grad);
    a.weight = L.weight, a.wide_weight = L.weight_type == MOE_NORM_WEIGHT_F32;
    a.eps = L.eps;
    a.out = static_cast<__nv_bfloat16 *>(L.out);
    a.parts = static_cast<float *>(L.workspace), a.grad_weight = L.grad_weight;
    a.T = L.num_tokens, a.H = L.hidden;
    a.num_parts = backward_parts(a.T) < 512 ? backward_parts(a.T) : 512;
    a.trace = trace_args();
    cudaError_t e;
    switch (vectors(a.H, 16)) {
        case 1: e = launch_backward<1>(a, s); break;
        case 2: e = launch_backward<2>(a, s); break;
        case 4: e = launch_backward<4>(a, s); break;
        default: e = launch_backward<8>(a, s); break;
    }
    if (e == cudaSuccess)
        e = launch_kernel(norm_weight_kernel, dim3((a.H + 31) / 32), dim3(256), 0, s, tuning().overlap != 0, a);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe
