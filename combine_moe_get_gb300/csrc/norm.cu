// norm.cu -- root-mean-square norm of rows behind the residual's addition:
//
//   h = x + residual,  y = h * rsqrt(mean(h^2) + eps) * weight
//   with n = h * r, r = rsqrt(mean(h^2) + eps), d = dy * weight:
//   dh = r (d - n mean(d n)) + dresidual,  dweight = sum over rows of dy n
//
// One pass over the rows, bound by HBM: a row stays in the registers of its threads
// (kVec times 8 channels each) between the sum of squares and the output. The sums
// are fp32; h enters them unrounded, and is rounded to bf16 only where it is stored.
// 4096 x 7168 with a residual, to bf16: 36 us (6.5 TB/s); 16384 x 7168 to E4M3: 127
// (6.5 TB/s); the gradient of 4096 x 7168 45 (5.2 TB/s).
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
    int32_t *status;
    WaitLimits limits;
    int stages;
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

// Sum over a row of what its threads have, v[j] for its vectors j * row_warps * 32 + thread: over the lanes of each 32
// vectors, then over those, so that equal rows have equal bits whichever way they are laid out over warps. `first` is the
// row's place in `space`. Every thread of the CTA calls it.
template <int kVec>
__device__ __forceinline__ float row_sum(const float (&v)[kVec], float *space, int first, int row_warps) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32 % row_warps;
    float sum;
    int o = 16;
    if constexpr (kVec == 4) {   // halves of a warp take two of the four on, quarters one
        const bool upper = lane & 16, odd = lane & 8;
        const float a = (upper ? v[2] : v[0]) + __shfl_xor_sync(0xffffffffu, upper ? v[0] : v[2], 16);
        const float b = (upper ? v[3] : v[1]) + __shfl_xor_sync(0xffffffffu, upper ? v[1] : v[3], 16);
        sum = (odd ? b : a) + __shfl_xor_sync(0xffffffffu, odd ? a : b, 8);
        o = 4;
    } else if constexpr (kVec == 2) {
        const bool upper = lane & 16;
        sum = (upper ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, upper ? v[0] : v[1], 16);
        o = 8;
    } else {
        sum = v[0];
    }
#pragma unroll
    for (; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const int n = row_warps * kVec;
    if (n == 1) return sum;
    constexpr int kShare = 32 / kVec;
    if (lane % kShare == 0) space[first + lane / kShare * row_warps + warp] = sum;
    __syncthreads();
    sum = lane < n ? space[first + lane] : 0.0f;
    if (kVec == 4 && lane + 32 < n) sum += space[first + lane + 32];
#pragma unroll
    for (o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return sum;
}

// Registers, for as many rows at once: 40 for two vectors (with 42 a third row of 14 warps does not fit beside two: 4096 x 7168 to
// both types takes 55 us, not 47), 64 for four (86: 16384 x 7168 to E4M3 194 us, not 134).
template <int kVec, bool kCodes>
__global__ __launch_bounds__(512, kVec == 4 ? 2 : 3) void norm_kernel(const __grid_constant__ NormArgs a) {
    const WarpTrace trace(a.trace, MOE_TRACE_NORM);
    __shared__ float space[64];   // a value for 256 channels of each row
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
    float h[kVec][8], sums[kVec] = {};
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
        for (int i = 0; i < 8; ++i) sums[j] = fmaf(h[j][i], h[j][i], sums[j]);
    }
    const float r = rsqrtf(row_sum(sums, space, sub * a.row_warps * kVec, a.row_warps) / a.H + a.eps);
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

// Barrier `id` for `threads` of the CTA; whether all of them say `yes`.
__device__ __forceinline__ bool barrier_all(int id, int threads, bool yes) {
    uint32_t all;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %3, 0;\n\tbarrier.cta.red.and.pred p, %1, %2, p;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(all) : "r"(id), "r"(threads), "r"((uint32_t)yes) : "memory");
    return all != 0;
}

// What is waited for is mostly there: the rest stays out of line (3000 x 14336 took 66.4 us with it in place, not 65.2).
static __device__ __noinline__ bool wait_longer(uint64_t *bar, uint32_t parity, uint64_t ns) {
    return mbar_wait_bounded(bar, parity, ns);
}

// Two vectors a thread and 28 warps, in groups where rows are short: fewer shuffles a row than with one vector, and two
// rows at once where 28 warps in step would all wait for each row's sums. Rows beyond 14336 take four and 16 warps.
__host__ __device__ constexpr int backward_warps(int vec) { return vec == 2 ? 28 : 16; }

// Rows on their way to a group of warps: h, the gradient and the residual's gradient of a row to a stage.
constexpr int kMostStages = 8;
struct RowRing {
    char *at;
    uint64_t *full;
    int stages, arrays, row_bytes;
    __device__ int stage_bytes() const { return arrays * row_bytes; }
    // By one thread; nothing for rows past the last.
    __device__ void fetch(const NormArgs &a, int64_t row, int slot, uint64_t policy) const {
        if (row >= a.T) return;
        mbar_arrive_expect_tx(full + slot, stage_bytes());
        const size_t from = (size_t)row * a.H;
        char *to = at + (size_t)slot * stage_bytes();
        bulk_load(to, a.x + from, row_bytes, full + slot, policy);
        bulk_load(to + row_bytes, a.grad + from, row_bytes, full + slot, policy);
        if (arrays == 3) bulk_load(to + 2 * row_bytes, a.residual + from, row_bytes, full + slot, policy);
    }
    __device__ uint4 read(int slot, int array, int col) const {
        return *reinterpret_cast<const uint4 *>(at + (size_t)slot * stage_bytes() + array * row_bytes + col * 2);
    }
};

// The CTA's groups of `row_warps` warps take rows in turn, and keep the weight's gradient of their columns in registers;
// at the end the groups' sums are added up in shared memory, in order. Rows come through rings in shared memory, as
// many ahead as it holds. 4096 x 7168: 45 us, the weight's sums included (5.2 TB/s); with loads into registers, one row
// ahead, 81; one vector a thread 54.
template <int kVec>
__global__ __launch_bounds__(backward_warps(kVec) * 32) void norm_backward_kernel(const __grid_constant__ NormArgs a) {
    const WarpTrace trace(a.trace, MOE_TRACE_NORM_BACKWARD);
    __shared__ float space[2][2][kMaxWarps];
    __shared__ uint64_t full[kMaxWarps][kMostStages];
    extern __shared__ __align__(128) char rings[];
    const int threads = a.row_warps * 32, groups = blockDim.x / threads, group = threadIdx.x / threads;
    const int tid = threadIdx.x - group * threads, lane = threadIdx.x & 31, warp = threadIdx.x / 32, first = group * a.row_warps;
    RowRing ring{nullptr, full[group], a.stages, a.residual ? 3 : 2, a.H * 2};
    ring.at = rings + (size_t)group * a.stages * ring.stage_bytes();
    if (tid == 0) {
        for (int i = 0; i < a.stages; ++i) mbar_init(ring.full + i, 1);
        fence_barrier_init();
    }
    __syncthreads();
    grid_dependency_wait();
    grid_launch_dependents();
    float dw[kVec][8] = {};
    const int64_t step = (int64_t)gridDim.x * groups;
    int64_t row = (int64_t)blockIdx.x * groups + group;
    const uint64_t policy = policy_evict_first();
    if (tid == 0)
        for (int i = (int)blockIdx.x == a.limits.withheld_cta; i < a.stages; ++i) ring.fetch(a, row + i * step, i, policy);
    int slot = 0, turn = 0;
    uint32_t round = 0;
    bool ok = true;
    for (; row < a.T; row += step, turn ^= 1) {
        ok = mbar_try_wait(ring.full + slot, round) || wait_longer(ring.full + slot, round, a.limits.wait_ns);
        uint4 now[kVec][3];
        float sum[2] = {};   // of h^2 and of d h
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            const int col = (j * threads + tid) * 8;
            now[j][0] = now[j][1] = now[j][2] = make_uint4(0, 0, 0, 0);
            if (col >= a.H) continue;
            now[j][0] = ring.read(slot, 0, col);
            now[j][1] = ring.read(slot, 1, col);
            if (a.residual) now[j][2] = ring.read(slot, 2, col);
            float h[8], g[8], w[8];
            widen(now[j][0], h);
            widen(now[j][1], g);
            load_weight(a, col, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                sum[0] = fmaf(h[i], h[i], sum[0]);
                sum[1] = fmaf(g[i] * w[i], h[i], sum[1]);
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
        if (a.row_warps > 1) {   // the two halves of `space` in turn, so that one barrier a row is enough
            if (lane == 0) space[turn][0][warp] = sum[0], space[turn][1][warp] = sum[1];
            ok = barrier_all(1 + group, threads, ok);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                sum[i] = lane < a.row_warps ? space[turn][i][first + lane] : 0.0f;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
            }
        } else {
            ok = __all_sync(0xffffffffu, ok);
        }
        if (!ok) break;   // the group as one
        if (tid == 0) ring.fetch(a, row + a.stages * step, slot, policy);   // every thread has read the stage
        if (++slot == a.stages) slot = 0, round ^= 1;
        const float r = rsqrtf(sum[0] / a.H + a.eps), m = r * r * (sum[1] / a.H);   // m h = n mean(d n)
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            const int col = (j * threads + tid) * 8;
            if (col >= a.H) continue;
            float h[8], g[8], w[8], add[8];
            widen(now[j][0], h);
            widen(now[j][1], g);
            widen(now[j][2], add);
            load_weight(a, col, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                dw[j][i] = fmaf(g[i], h[i] * r, dw[j][i]);
                add[i] += r * (g[i] * w[i] - h[i] * m);
            }
            *reinterpret_cast<uint4 *>(a.out + (size_t)row * a.H + col) = narrow(add);
        }
    }
    if (!ok && tid == 0) {
        report(a.status, MOE_ERR_TIMEOUT);
        for (int i = 0; i < a.stages && row + i * step < a.T; ++i) {   // rows on their way all the same
            mbar_wait_bounded(ring.full + slot, round, a.limits.wait_ns);
            if (++slot == a.stages) slot = 0, round ^= 1;
        }
    }
    __syncthreads();   // no copy is under way: every stage that was fetched has been waited for
    float *sums = reinterpret_cast<float *>(rings);   // [groups][H]: half of the smallest ring
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        const int col = (j * threads + tid) * 8;
        if (col >= a.H) continue;
        float4 *to = reinterpret_cast<float4 *>(groups > 1 ? sums + group * a.H + col : a.parts + (size_t)blockIdx.x * a.H + col);
        to[0] = make_float4(dw[j][0], dw[j][1], dw[j][2], dw[j][3]);
        to[1] = make_float4(dw[j][4], dw[j][5], dw[j][6], dw[j][7]);
    }
    if (groups == 1) return;
    __syncthreads();
    for (int col = threadIdx.x * 4; col < a.H; col += blockDim.x * 4) {
        float4 sum = *reinterpret_cast<const float4 *>(sums + col);
        for (int g = 1; g < groups; ++g) {
            const float4 v = *reinterpret_cast<const float4 *>(sums + g * a.H + col);
            sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
        }
        *reinterpret_cast<float4 *>(a.parts + (size_t)blockIdx.x * a.H + col) = sum;
    }
}

// The weight's gradient: the CTAs' sums, in order. 32 columns a CTA, its 16 warps every 16th part each.
constexpr int kWeightWarps = 16;
__global__ __launch_bounds__(kWeightWarps * 32) void norm_weight_kernel(const __grid_constant__ NormArgs a) {
    const WarpTrace trace(a.trace, MOE_TRACE_NORM_WEIGHT);
    __shared__ float space[kWeightWarps][32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, col = blockIdx.x * 32 + lane;
    float sum = 0.0f;
    if (col < a.H)
#pragma unroll 8
        for (int p = warp; p < a.num_parts; p += kWeightWarps) sum += __ldcg(a.parts + (size_t)p * a.H + col);
    space[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && col < a.H) {
#pragma unroll
        for (int i = 1; i < kWeightWarps; ++i) sum += space[i][lane];
        a.grad_weight[col] = sum;
    }
}

// Vectors of 8 channels that a thread holds so that a row of H takes at most `most_warps` warps.
int vectors(int H, int most_warps) {
    int v = 1;
    while ((H + v * 256 - 1) / (v * 256) > most_warps) v *= 2;
    return v;
}

constexpr int kRingBytes = 200 << 10;   // of a CTA's rings
constexpr int kMaxParts = 160;   // CTAs of the backward kernel, each with a part of the weight's gradient

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
    // as many rows at once as a CTA has warps for (15: a barrier each), one CTA an SM
    int groups = backward_warps(kVec) / a.row_warps;
    if (groups > 15) groups = 15;
    const int ctas = device_sm_count() < kMaxParts ? device_sm_count() : kMaxParts;
    if (groups > (a.T + ctas - 1) / ctas) groups = (a.T + ctas - 1) / ctas;
    const int64_t need = ((int64_t)a.T + groups - 1) / groups;
    a.num_parts = need < ctas ? (int)need : ctas;
    const int stage = groups * (a.residual ? 3 : 2) * a.H * 2;   // at most 96 KB
    a.stages = kRingBytes / stage < kMostStages ? kRingBytes / stage : kMostStages;
    const size_t smem = (size_t)a.stages * stage;   // two stages at least, of 4 H bytes a group: room for the groups' sums
    const int rc = ensure_dynamic_smem((const void *)norm_backward_kernel<kVec>, kRingBytes);
    if (rc != MOE_OK) return cudaErrorUnknown;
    return launch_kernel(norm_backward_kernel<kVec>, dim3(a.num_parts), dim3(groups * a.row_warps * 32), smem, s,
                         tuning().overlap != 0, a);
}

}  // namespace

size_t norm_backward_workspace_bytes(int T, int H) { return (size_t)(T < kMaxParts ? T : kMaxParts) * H * sizeof(float); }

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
    // Fewer warps with more of a row each, where that keeps enough of them at work. us (7 of them the launch's), at most 8
    // warps / 16: 4096 channels, 16384 rows to E4M3 85 / 95, to bf16 85 / 91, 128 rows 9.4 / 9.4; 7168 channels to E4M3 alone
    // 134 / 143, 4096 rows 42 / 44; but with bf16 rows 4096 rows 50 / 48, 128 rows 11.4 / 9.4. In a graph, without the 7:
    // 16384 rows to E4M3 alone 5120 channels 92 / 99, 6144 109 / 112, 8192 143 / 150, to bf16 99 / 98, 119 / 118, 157 / 156, to
    // both 113 / 114, 134 / 134, 177 / 177; 4096 rows to both 32.4 / 32.1, 37.9 / 37.1, 48.7 / 48.2; 128 rows to E4M3 alone
    // the other way, 4.3 to 4.7 / 3.4 to 3.9.
    switch (vectors(a.H, a.H <= 4096 || (a.H <= 8192 && !a.out) ? 8 : 16)) {
        case 1: e = launch_forward<1>(a, s); break;
        case 2: e = launch_forward<2>(a, s); break;
        default: e = launch_forward<4>(a, s); break;
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
    a.status = L.status;
    a.limits = wait_limits();
    a.trace = trace_args();
    cudaError_t e;
    e = a.H <= 14336 ? launch_backward<2>(a, s) : launch_backward<4>(a, s);
    if (e == cudaSuccess)
        e = launch_kernel(norm_weight_kernel, dim3((a.H + 31) / 32), dim3(kWeightWarps * 32), 0, s, tuning().overlap != 0, a);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe
