// swiglu.cu -- the gated activation between the experts' two products, row by row:
//
//   h[r, i]  = weight[r] * silu(g[r, i]) * u[r, i],   [g; u] = gate_up[r], silu(z) = z / (1 + exp(-z))
//   dg = dh * weight * u * s (1 + g (1 - s)),  du = dh * weight * g s,  dweight[r] = sum_i dh g s u,  s = 1 / (1 + exp(-g))
//
// One pass over the rows, bound by HBM. A warp takes 256 channels of a row: 16 bytes
// of gate and of up a lane, so that 16 lanes hold a block of 128 and its largest
// magnitude takes four shuffles. 32768 x 2048: 62 us to bf16 (6.5 TB/s), 54 to E4M3
// (6.3 TB/s; 60 with one element to an instruction and as many registers as the
// compiler takes, 40, which leaves out a quarter of the warps); the gradient 107
// (6.3 TB/s). Four pieces to a warp, loaded at once, were no faster than one, and
// slower in small calls; the next piece's loads ahead of this one's sums were slower.
#include "rows.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 3;         // backward: vectors that a thread loads before it works on the first
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
    int row_warps;         // backward
    TraceArgs trace;
};

__device__ __forceinline__ int rows_in_use(const SwigluArgs &a) {
    if (a.num_rows == nullptr) return a.M;
    const int n = __ldg(a.num_rows), cut = min(max(n, 0), a.M);
    if (cut != n && blockIdx.x == 0 && threadIdx.x == 0) report(a.status, MOE_ERR_CAPACITY);
    return cut;
}

// Two fp32 to an instruction.
struct Two {
    uint64_t v;
    __device__ Two(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
    __device__ explicit Two(float a) : Two(a, a) {}
    __device__ void parts(float &a, float &b) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
};
__device__ __forceinline__ Two operator*(Two a, Two b) {
    asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(a.v) : "l"(b.v));
    return a;
}
__device__ __forceinline__ Two operator+(Two a, Two b) {
    asm("add.rn.f32x2 %0, %0, %1;" : "+l"(a.v) : "l"(b.v));
    return a;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
    asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(a.v) : "l"(b.v), "l"(c.v));
    return a;
}
// exp and the reciprocal are the fast ones, the exponent rounded before: off by 2^-22 + |z| 2^-23 of the sigmoid (2^-16 at most,
// where bf16's rounding has 2^-9) down to z = -87.3; below, where the reciprocal is no normal number, the sigmoid is 0
__device__ __forceinline__ Two sigmoid(Two z) {
    float a, b;
    (z * Two(-1.4426950408889634f)).parts(a, b);   // log2(e)
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(a));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(b));
    (Two(a, b) + Two(1.0f)).parts(a, b);
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(a));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(b));
    return Two(a, b);
}

// Pieces of 256 channels in order, a warp's own `step` apart, without a division for each.
struct Pieces {
    int64_t row;
    int piece, pieces, step_piece;
    int64_t step_row;
    __device__ Pieces(int64_t first, int64_t step, int n) : pieces(n) {
        row = div_count(first, n), piece = (int)(first - row * n);
        step_row = div_count(step, n), step_piece = (int)(step - step_row * n);
    }
    __device__ void next() {
        row += step_row, piece += step_piece;
        if (piece >= pieces) piece -= pieces, ++row;
    }
};

template <bool kE4m3>
__global__ __launch_bounds__(kThreads, 8) void swiglu_kernel(const __grid_constant__ SwigluArgs a) {
    const WarpTrace trace(a.trace, MOE_TRACE_SWIGLU);
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t rows = rows_in_use(a);
    Pieces p((int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32, (int64_t)gridDim.x * (kThreads / 32),
             (a.I + kPiece - 1) / kPiece);
    for (; p.row < rows; p.next()) {
        const int col = p.piece * kPiece + lane * 8;
        const bool in = col < a.I;
        const size_t at = (size_t)p.row * a.I + col;
        uint4 g = make_uint4(0, 0, 0, 0), u = g;
        if (in) {
            const __nv_bfloat16 *from = a.gate_up + at + (size_t)p.row * a.I;
            g = load_once(from);
            u = load_once(from + a.I);
        }
        const float w = a.row_weights == nullptr ? 1.0f : __ldg(a.row_weights + p.row);
        float z[8], v[8];
        widen(g, z);
        widen(u, v);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const Two gate(z[i], z[i + 1]);
            (gate * sigmoid(gate) * Two(w) * Two(v[i], v[i + 1])).parts(v[i], v[i + 1]);
        }
        if constexpr (kE4m3) {   // I is a multiple of 128: 16 lanes are in it or not
            uint2 codes;
            const float scale = quantise(v, codes);
            if (in) {
                *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.out) + at) = codes;
                if ((lane & 15) == 0) a.scales[at / 128] = scale;
            }
        } else if (in) {
            *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + at) = narrow(v);
        }
    }
}

struct Gradients {
    uint4 gate, up;
};
// Of eight channels; returns their part of the row weight's gradient.
__device__ __forceinline__ float gradients(const uint4 &g4, const uint4 &u4, const uint4 &d4, float w, Gradients &out) {
    float z[8], v[8], d[8];
    widen(g4, z);
    widen(u4, v);
    widen(d4, d);
    Two sum(0.0f);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const Two gate(z[i], z[i + 1]), up(v[i], v[i + 1]), dh(d[i], d[i + 1]), s = sigmoid(gate), silu = gate * s, wdh = dh * Two(w);
        sum = fma2(dh, silu * up, sum);
        (wdh * silu).parts(v[i], v[i + 1]);
        (wdh * up * s * fma2(gate, fma2(s, Two(-1.0f), Two(1.0f)), Two(1.0f))).parts(z[i], z[i + 1]);
    }
    out.gate = narrow(z);
    out.up = narrow(v);
    float even, odd;
    sum.parts(even, odd);
    return even + odd;
}

// `row_warps` warps to a row, up to kUnroll times 8 channels a thread at once; a row's sum of the weight's gradient is
// added up in a fixed order.
__global__ __launch_bounds__(kThreads, 3) void swiglu_backward_kernel(const __grid_constant__ SwigluArgs a) {
    const WarpTrace trace(a.trace, MOE_TRACE_SWIGLU_BACKWARD);
    __shared__ float space[2][kThreads / 32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int sub = warp / a.row_warps, threads = a.row_warps * 32, tid = threadIdx.x - sub * threads;
    const int per = kThreads / threads, rows = rows_in_use(a);
    int turn = 0;
    for (int64_t first = (int64_t)blockIdx.x * per; first < rows; first += (int64_t)gridDim.x * per, turn ^= 1) {
        const int64_t row = first + sub;
        const bool live = row < rows;
        const float w = live && a.row_weights != nullptr ? __ldg(a.row_weights + row) : 1.0f;
        const __nv_bfloat16 *from = a.gate_up + (size_t)row * 2 * a.I, *grad = a.grad + (size_t)row * a.I;
        __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + (size_t)row * 2 * a.I;
        float sum = 0.0f;
        if (live)
            for (int col0 = tid * 8; col0 < a.I; col0 += kUnroll * threads * 8) {
                uint4 g4[kUnroll], u4[kUnroll], d4[kUnroll];
#pragma unroll
                for (int j = 0; j < kUnroll; ++j) {
                    const int col = col0 + j * threads * 8;
                    if (col < a.I) {
                        g4[j] = load_once(from + col);
                        u4[j] = load_once(from + a.I + col);
                        d4[j] = load_once(grad + col);
                    }
                }
#pragma unroll
                for (int j = 0; j < kUnroll; ++j) {
                    const int col = col0 + j * threads * 8;
                    if (col < a.I) {
                        Gradients r;
                        sum += gradients(g4[j], u4[j], d4[j], w, r);
                        *reinterpret_cast<uint4 *>(out + col) = r.gate;
                        *reinterpret_cast<uint4 *>(out + a.I + col) = r.up;
                    }
                }
            }
        if (a.grad_weights == nullptr) continue;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (a.row_warps > 1) {
            if (lane == 0) space[turn][warp] = sum;
            __syncthreads();   // one is enough: the next row's sums go to the other half
            sum = 0.0f;
            for (int i = 0; i < a.row_warps; ++i) sum += space[turn][sub * a.row_warps + i];
        }
        if (live && tid == 0) a.grad_weights[row] = sum;
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
                       nullptr, L.status, L.num_rows_most, L.intermediate, 0, trace_args()};
    const int64_t pieces = (int64_t)a.M * ((a.I + kPiece - 1) / kPiece);
    const dim3 grid(blocks_for(pieces, 16));
    const cudaStream_t s = static_cast<cudaStream_t>(L.stream);
    const cudaError_t e = L.out_scales ? launch_kernel(swiglu_kernel<true>, grid, dim3(kThreads), 0, s, tuning().overlap != 0, a)
                                       : launch_kernel(swiglu_kernel<false>, grid, dim3(kThreads), 0, s, tuning().overlap != 0, a);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int launch_swiglu_backward(const SwigluLaunch &L) {
    if (L.num_rows_most == 0) return MOE_OK;
    SwigluArgs a{static_cast<const __nv_bfloat16 *>(L.gate_up), static_cast<const __nv_bfloat16 *>(L.grad), L.row_weights,
                 L.num_rows, L.out, nullptr, L.grad_row_weights, L.status, L.num_rows_most, L.intermediate, 1, trace_args()};
    while (a.row_warps < kThreads / 32 && a.I > a.row_warps * 256 * kUnroll) a.row_warps *= 2;
    const dim3 grid(blocks_for((int64_t)a.M * a.row_warps, 3));
    const cudaStream_t s = static_cast<cudaStream_t>(L.stream);
    return launch_kernel(swiglu_backward_kernel, grid, dim3(kThreads), 0, s, tuning().overlap != 0, a) == cudaSuccess
               ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe
