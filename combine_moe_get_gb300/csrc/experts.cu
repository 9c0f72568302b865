// experts.cu -- the experts' products of a few tokens (moe_experts).
//
//   h[t, j]  = silu(G x_t) * (U x_t),  [G; U] = w13[e], e = topk_idx[t, j]
//   out[t]   = sum_j topk_weights[t, j] * (w2[e] h[t, j])
//
// Two kernels. The plan kernel (one CTA) sorts the valid entries by expert and
// cuts each expert's into groups of at most `cols` entries. The experts kernel
// (one CTA per SM, launched cooperatively) runs skinny.cuh's body over two
// lines of work: phase 0 makes h (a tile is 128 gate and the same 128 up rows,
// so that one thread holds both sums of an element), phase 1 multiplies h by w2
// (a tile is 256 rows) into y, one fp32 row per entry. A group's phase 1 waits
// until all its h tiles are done; the loads of w2 do not wait, so the stream of
// weights goes on across the border. When all of y is there, all CTAs add each
// token's rows in entry order with their weights and round once to bf16.
//
// h is rounded to bf16: it is the operand of a bf16 product, and the rounding's
// effect on an output is of the size of that output's own rounding.
#include <algorithm>
#include <cuda_bf16.h>

#include "skinny.cuh"

namespace moe {
namespace {

using skinny::kRows;

// Device workspace: byte offsets.
struct Space {
    size_t words, groups, order, h, y, partial, total;
};
constexpr int kReady = skinny::kWords;   // then a word per group: its finished h tiles

int columns(int T, bool e4m3) { return std::min((T + 15) / 16 * 16, e4m3 ? 64 : 128); }

Space space(int T, int H, int I, int k, int cols) {
    Space s{};
    skinny::Cut cut;
    const size_t n = (size_t)T * k;   // groups are at most as many as entries
    s.words = cut.take((kReady + n) * 4);
    s.groups = cut.take(n * sizeof(int4));
    s.order = cut.take(n * 4);
    s.h = cut.take(n * I * 2);
    s.y = cut.take(n * H * 4);
    s.partial = cut.take(skinny::partial_floats(cols) * 4);
    s.total = cut.at;
    return s;
}

// ------------------------------------------------------------------ experts

struct ExpertsArgs {
    CUtensorMap w13, w2, x, h_map;
    const int64_t *topk_idx;
    const float *topk_weights;
    const float *s13, *s2;
    uint32_t *words;
    const int4 *groups;
    const int *order;
    __nv_bfloat16 *h;
    float *y, *partials;
    __nv_bfloat16 *out;
    int32_t *status;
    int T, H, I, k, E;
    skinny::Shape shape;
    uint32_t tmem_cols;
    TraceArgs trace;
};

template <bool kE4m3>
struct ExpertsProblem {
    const ExpertsArgs &a;
    int G;
    int32_t *status;
    int tiles[2], kbs[2];   // tiles per group and K blocks per tile of the two phases

    __device__ explicit ExpertsProblem(const ExpertsArgs &args) : a(args), G((int)args.words[skinny::kGroupsWord]), status(args.status) {
        constexpr int block = kE4m3 ? 128 : 64;
        tiles[0] = (a.I + kRows - 1) / kRows;
        tiles[1] = (a.H + 2 * kRows - 1) / (2 * kRows);
        kbs[0] = (a.H + block - 1) / block;
        kbs[1] = (a.I + block - 1) / block;
    }

    template <class F>
    __device__ bool segments(F f) const {
        for (int phase = 0; phase < 2; ++phase) {
            const skinny::Line line((int64_t)G * tiles[phase], kbs[phase], gridDim.x);
            const bool ok = line.each(blockIdx.x, [&](int64_t tile, skinny::Segment &s) {
                s.phase = phase;
                s.group = (int)(tile / tiles[phase]);
                s.f = (int)(tile - (int64_t)s.group * tiles[phase]);
                const int4 g = a.groups[s.group];
                s.first = g.y;
                s.n = g.z;
                s.a_bytes = skinny::kHalf;
                s.two = true;
                if (phase == 0) {
                    s.a_map = &a.w13;
                    s.row0 = g.x * 2 * a.I + s.f * kRows;
                    s.row1 = s.row0 + a.I;
                    s.row_end = a.E * 2 * a.I;
                } else {
                    s.a_map = &a.w2;
                    s.row0 = g.x * a.H + s.f * 2 * kRows;
                    s.row1 = s.row0 + kRows;
                    s.row_end = a.E * a.H;
                }
                return f(s);
            });
            if (!ok) return false;
        }
        return true;
    }

    // ---- loads of B: x rows of the group's entries, or their rows of h
    struct Rows {
        int r[4];
    };
    __device__ bool b_ready(const skinny::Segment &s) const {
        if (s.phase == 0) return true;
        if (!skinny::wait_count(a.words + kReady + s.group, tiles[0])) return false;
        fence_proxy_async();
        return true;
    }
    __device__ Rows b_rows(const skinny::Segment &s, int lane) const {
        Rows rows{};
        if (s.phase == 0)
#pragma unroll
            for (int i = 0; i < 4; ++i) rows.r[i] = a.order[s.first + min(4 * lane + i, s.n - 1)] / a.k;
        return rows;
    }
    __device__ uint32_t b_bytes(const skinny::Segment &s) const {
        return s.phase == 0 ? (s.n + 3) / 4 * 512 : (s.n + 7) / 8 * 1024;
    }
    __device__ void b_load(const skinny::Segment &s, const Rows &rows, int col, uint32_t dst, uint64_t *bar,
                           int lane) const {
        const uint64_t policy = policy_evict_last();
        if (s.phase == 0) {
            if (4 * lane < s.n)
                tma_gather4(dst + lane * 512, &a.x, col, rows.r[0], rows.r[1], rows.r[2], rows.r[3], bar, policy);
        } else if (8 * lane < s.n) {
            tma_load(dst + lane * 1024, &a.h_map, col, s.first + 8 * lane, bar, policy);
        }
    }

    // ---- sums
    __device__ const float *scales(int phase) const { return phase == 0 ? a.s13 : a.s2; }
    __device__ float *partial(int phase, int cta, int slot) const {
        return a.partials + ((size_t)(phase * skinny::kMaxCtas + cta) * 2 + slot) * 2 * a.shape.cols * kRows;
    }
    __device__ uint32_t *arrivals(int phase, int cta) const {
        return a.words + skinny::kArrivals + phase * skinny::kMaxCtas + cta;
    }
    __device__ bool emit_ready(const skinny::Segment &) const { return true; }
    struct Emit {
        const ExpertsArgs &a;
        const skinny::Segment &s;
        int row;
        __device__ Emit(const ExpertsProblem &p, const skinny::Segment &seg, int r) : a(p.a), s(seg), row(r) {}
        __device__ void operator()(int col, const float *v0, const float *v1) const {
            if (s.phase == 0) {
                const int i = s.f * kRows + row;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (col + j >= s.n || i >= a.I) continue;
                    const float g = v0[j];
                    a.h[(size_t)(s.first + col + j) * a.I + i] = __float2bfloat16_rn(g / (1.0f + expf(-g)) * v1[j]);
                }
            } else {
                const int o = s.f * 2 * kRows + row;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (col + j >= s.n) continue;
                    float *y = a.y + (size_t)a.order[s.first + col + j] * a.H + o;
                    if (o < a.H) y[0] = v0[j];
                    if (o + kRows < a.H) y[kRows] = v1[j];
                }
            }
        }
    };
    __device__ void tile_done(const skinny::Segment &s) const {
        fence_proxy_async();   // h is read by TMA
        __threadfence();
        skinny::readers_sync();
        if (threadIdx.x == skinny::kThreads - skinny::kReaders)
            skinny::add_acq_rel(s.phase == 0 ? a.words + kReady + s.group : a.words + skinny::kDoneWord, 1);
    }

    // out[t] = sum_j w[t, j] y[t, j], eight columns to a thread
    __device__ bool finish() const {
        const int thread = threadIdx.x - (skinny::kThreads - skinny::kReaders);
        bool ok = true;
        if (thread == 0) ok = skinny::wait_count(a.words + skinny::kDoneWord, (uint32_t)G * tiles[1]);
        if (!skinny::readers_agree(ok)) return false;
        const int pieces = a.H / 8;
        const int64_t all = (int64_t)a.T * pieces;
        for (int64_t i = (int64_t)blockIdx.x * skinny::kReaders + thread; i < all;
             i += (int64_t)gridDim.x * skinny::kReaders) {
            const int t = (int)(i / pieces), o = (int)(i - (int64_t)t * pieces) * 8;
            float acc[8] = {};
#pragma unroll 4
            for (int j = 0; j < a.k; ++j) {
                const int64_t e = a.topk_idx[(size_t)t * a.k + j];
                if (e < 0 || e >= a.E) continue;
                const float w = a.topk_weights[(size_t)t * a.k + j];
                const float4 *y = reinterpret_cast<const float4 *>(a.y + ((size_t)t * a.k + j) * a.H + o);
                const float4 lo = __ldcg(y), hi = __ldcg(y + 1);
                acc[0] = fmaf(w, lo.x, acc[0]), acc[1] = fmaf(w, lo.y, acc[1]);
                acc[2] = fmaf(w, lo.z, acc[2]), acc[3] = fmaf(w, lo.w, acc[3]);
                acc[4] = fmaf(w, hi.x, acc[4]), acc[5] = fmaf(w, hi.y, acc[5]);
                acc[6] = fmaf(w, hi.z, acc[6]), acc[7] = fmaf(w, hi.w, acc[7]);
            }
            __nv_bfloat162 b[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) b[j] = __floats2bfloat162_rn(acc[2 * j], acc[2 * j + 1]);
            *reinterpret_cast<uint4 *>(a.out + (size_t)t * a.H + o) = *reinterpret_cast<const uint4 *>(b);
        }
        return true;
    }
};

template <bool kE4m3>
__global__ void __launch_bounds__(skinny::kThreads, 1) experts_kernel(const __grid_constant__ ExpertsArgs a) {
    WarpTrace wt(a.trace, MOE_TRACE_EXPERTS);
    grid_dependency_wait();
    const ExpertsProblem<kE4m3> p(a);
    skinny::run<kE4m3>(p, a.shape, a.tmem_cols);
}

}  // namespace

size_t experts_workspace_bytes(int T, int H, int I, int k, int E) {
    return space(T, H, I, k, columns(T, false)).total;   // bf16 weights: the larger of the two
}

int launch_experts(const ExpertsLaunch &L) {
    const int T = L.num_tokens, H = L.hidden, I = L.intermediate, k = L.num_topk, E = L.num_experts;
    if (T == 0) return MOE_OK;
    const bool e4m3 = L.w13_scales != nullptr;
    const int cols = columns(T, e4m3);
    const Space sp = space(T, H, I, k, cols);
    char *ws = static_cast<char *>(L.workspace);
    const cudaStream_t s = static_cast<cudaStream_t>(L.stream);

    const skinny::PlanArgs<int64_t> plan{L.topk_idx, T * k, E, cols, reinterpret_cast<uint32_t *>(ws + sp.words),
                                         kReady + T * k, reinterpret_cast<int4 *>(ws + sp.groups),
                                         reinterpret_cast<int *>(ws + sp.order), MOE_ERR_BAD_TOPK, L.status,
                                         trace_args()};
    ExpertsArgs a{};
    if (!make_tensor_map(&a.w13, L.w13, e4m3, (uint64_t)E * 2 * I, H, kRows) ||
        !make_tensor_map(&a.w2, L.w2, e4m3, (uint64_t)E * H, I, kRows) ||
        !make_tensor_map(&a.x, L.x, false, T, H, 1) ||
        !make_tensor_map(&a.h_map, ws + sp.h, false, (uint64_t)T * k, I, 8))
        return MOE_ERR_CUDA;
    a.topk_idx = L.topk_idx;
    a.topk_weights = L.topk_weights;
    a.s13 = L.w13_scales;
    a.s2 = L.w2_scales;
    a.words = plan.words;
    a.groups = plan.groups;
    a.order = plan.order;
    a.h = reinterpret_cast<__nv_bfloat16 *>(ws + sp.h);
    a.y = reinterpret_cast<float *>(ws + sp.y);
    a.partials = reinterpret_cast<float *>(ws + sp.partial);
    a.out = static_cast<__nv_bfloat16 *>(L.out);
    a.status = L.status;
    a.T = T, a.H = H, a.I = I, a.k = k, a.E = E;
    a.shape = skinny::Shape{cols, skinny::Shape::stages_for(cols, e4m3)};
    a.tmem_cols = skinny::Shape::tmem_cols(cols, e4m3);
    a.trace = trace_args();

    const int rc = skinny::launch_plan(plan, s);
    if (rc != MOE_OK) return rc;
    return skinny::launch_resident(e4m3 ? experts_kernel<true> : experts_kernel<false>, a,
                                   skinny::Shape::smem(cols, e4m3), s);
}

}  // namespace moe
