// swiglu.cu -- the gated activation between the experts' two products, row by row:
//
//   h[r, i]  = weight[r] * silu(g[r, i]) * u[r, i],   [g; u] = gate_up[r], silu(z) = z / (1 + exp(-z))
//   dg = dh * weight * u * s (1 + g (1 - s)),  du = dh * weight * g s,  dweight[r] = sum_i dh g s u,  s = 1 / (1 + exp(-g))
//
// One pass over the rows, bound by HBM. A warp takes 256 channels of a row: 16 bytes
// of gate and of up a lane, so that 16 lanes hold a block of 128 and its largest
// magnitude takes four shuffles.
#include "rows.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;         // pieces that a warp loads before it works on the first
constexpr int kPiece = 256;        // channels of a warp's piece

struct SwigluArgs {
    const __nv_bfloat16 *gate_up, *grad;
    const float *row_weights;
    const int32_t *num_rows;
    void *out;             // h; backward: grad_gate_up
    float *scales;         // E4M3
    float *grad_weights;   // backward
    int32_t *status;
    int M, I;
    TraceArgs trace;
};

__device__ __forceinline__ int rows_in_use(const SwigluArgs &a) {
    if (a.num_rows == nullptr) return a.M;
    const int n = __ldg(a.num_rows), cut = min(max(n, 0), a.M);
    if (cut != n && blockIdx.x == 0 && threadIdx.x == 0) report(a.status, MOE_ERR_CAPACITY);
    return cut;
}

// exp and the quotient are the fast ones, off by some 2^-21 of the sigmoid: an eighth of an E4M3 or bf16 rounding's 2^-9 at most
__device__ __forceinline__ float sigmoid(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }

template <bool kE4m3>
__global__ __launch_bounds__(kThreads) void swiglu_kernel(const __grid_constant__ SwigluArgs a) {
    const WarpTrace trace(a.trace, MOE_TRACE_SWIGLU);
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int pieces = (a.I + kPiece - 1) / kPiece;
    const int64_t total = (int64_t)rows_in_use(a) * pieces;
    const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
    for (int64_t u0 = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32; u0 < total; u0 += warps * kUnroll) {
        uint4 g[kUnroll], u[kUnroll];
        int64_t row[kUnroll];
        int col[kUnroll];
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) {
            const int64_t piece = u0 + j * warps;
            row[j] = div_count(piece, pieces);
            col[j] = (int)(piece - row[j] * pieces) * kPiece + lane * 8;
            g[j] = u[j] = make_uint4(0, 0, 0, 0);
            if (piece < total && col[j] < a.I) {
                const __nv_bfloat16 *p = a.gate_up + (size_t)row[j] * 2 * a.I + col[j];
                g[j] = load_once(p);
                u[j] = load_once(p + a.I);
            }
        }
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) {
            if (u0 + j * warps >= total) break;
            const float w = a.row_weights == nullptr ? 1.0f : __ldg(a.row_weights + row[j]);
            float z[8], v[8];
            widen(g[j], z);
            widen(u[j], v);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = z[i] * sigmoid(z[i]) * v[i] * w;
            const size_t at = (size_t)row[j] * a.I + col[j];
            if constexpr (kE4m3) {   // I is a multiple of 128: 16 lanes are in it or not
                uint2 codes;
                const float scale = quantise(v, codes);
                if (col[j] < a.I) {
                    *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.out) + at) = codes;
                    if ((lane & 15) == 0) a.scales[at / 128] = scale;
                }
            } else if (col[j] < a.I) {
                *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + at) = narrow(v);
            }
        }
    }
}

// A warp takes whole rows where their weights want a gradient (a row's sum stays in
// the warp, in a fixed order), else pieces.
template <bool kWeights>
__global__ __launch_bounds__(kThreads) void swiglu_backward_kernel(const __grid_constant__ SwigluArgs a) {
    const WarpTrace trace(a.trace, MOE_TRACE_SWIGLU_BACKWARD);
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int pieces = (a.I + kPiece - 1) / kPiece;
    const int rows = rows_in_use(a);
    const int64_t total = kWeights ? rows : (int64_t)rows * pieces;
    const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
    for (int64_t u = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32; u < total; u += warps) {
        const int64_t row = kWeights ? u : div_count(u, pieces);
        const int first = kWeights ? 0 : (int)(u - row * pieces) * kPiece, last = kWeights ? a.I : min(a.I, first + kPiece);
        const float w = a.row_weights == nullptr ? 1.0f : __ldg(a.row_weights + row);
        float sum = 0.0f;
        for (int col = first + lane * 8; col < last; col += kPiece) {
            const __nv_bfloat16 *p = a.gate_up + (size_t)row * 2 * a.I + col;
            float z[8], v[8], d[8];
            const uint4 g4 = load_once(p), u4 = load_once(p + a.I), d4 = load_once(a.grad + (size_t)row * a.I + col);
            widen(g4, z);
            widen(u4, v);
            widen(d4, d);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float s = sigmoid(z[i]), silu = z[i] * s, up = v[i], dh = d[i] * w;
                if constexpr (kWeights) sum = fmaf(d[i], silu * up, sum);
                v[i] = dh * silu;
                z[i] = dh * up * s * fmaf(z[i], 1.0f - s, 1.0f);
            }
            __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + (size_t)row * 2 * a.I + col;
            *reinterpret_cast<uint4 *>(out) = narrow(z);
            *reinterpret_cast<uint4 *>(out + a.I) = narrow(v);
        }
        if constexpr (kWeights) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane == 0) a.grad_weights[row] = sum;
        }
    }
}

int blocks_for(int64_t warps, int per_sm) {
    const int64_t blocks = (warps + kThreads / 32 - 1) / (kThreads / 32), most = (int64_t)device_sm_count() * per_sm;
    return (int)(blocks < most ? blocks : most);
}

}  // namespace

int launch_swiglu(const SwigluLaunch &L) {
    if (L.num_rows_most == 0) return MOE_OK;
    const SwigluArgs a{static_cast<const __nv_bfloat16 *>(L.gate_up), nullptr, L.row_weights, L.num_rows, L.out, L.out_scales,
                       nullptr, L.status, L.num_rows_most, L.intermediate, trace_args()};
    const int64_t pieces = (int64_t)a.M * ((a.I + kPiece - 1) / kPiece);
    const dim3 grid(blocks_for(pieces, 8));
    const cudaStream_t s = static_cast<cudaStream_t>(L.stream);
    const cudaError_t e = L.out_scales ? launch_kernel(swiglu_kernel<true>, grid, dim3(kThreads), 0, s, tuning().overlap != 0, a)
                                       : launch_kernel(swiglu_kernel<false>, grid, dim3(kThreads), 0, s, tuning().overlap != 0, a);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int launch_swiglu_backward(const SwigluLaunch &L) {
    if (L.num_rows_most == 0) return MOE_OK;
    const SwigluArgs a{static_cast<const __nv_bfloat16 *>(L.gate_up), static_cast<const __nv_bfloat16 *>(L.grad), L.row_weights,
                       L.num_rows, L.out, nullptr, L.grad_row_weights, L.status, L.num_rows_most, L.intermediate,
                       trace_args()};
    const int64_t pieces = L.grad_row_weights ? a.M : (int64_t)a.M * ((a.I + kPiece - 1) / kPiece);
    const dim3 grid(blocks_for(pieces, 8));
    const cudaStream_t s = static_cast<cudaStream_t>(L.stream);
    const cudaError_t e =
        L.grad_row_weights
            ? launch_kernel(swiglu_backward_kernel<true>, grid, dim3(kThreads), 0, s, tuning().overlap != 0, a)
            : launch_kernel(swiglu_backward_kernel<false>, grid, dim3(kThreads), 0, s, tuning().overlap != 0, a);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe
