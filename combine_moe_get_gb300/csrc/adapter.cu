// adapter.cu -- a shared projection with the low-rank adapter of each row
// (moe_adapter_linear).
//
//   v[t]   = scales[a] * (A_a x_t),  a = adapter_idx[t]
//   out[t] = W x_t + B_a v[t]        (W x_t alone where a = -1)
//
// Two kernels. The plan kernel sorts the rows by adapter into groups. The
// adapter kernel (one CTA per SM, launched cooperatively) runs skinny.cuh's body
// over two lines of work: phase 0 multiplies each group's x rows by its A (up to
// 128 rows of A are one product) into v, phase 1 multiplies all rows of x, in
// their own order, by W. Phase 1's products do not need v; only the readers of
// its sums do: they add B_a v[t] in fp32 before the one rounding to bf16, each
// thread for its own row of W and B, so an adapter's values meet no other
// row's sums, not even as a product with zero.
#include <algorithm>
#include <cuda_bf16.h>

#include "skinny.cuh"

namespace moe {
namespace {

using skinny::kRows;

struct Space {
    size_t words, groups, order, v, partial, total;   // byte offsets
};

int columns(int T) { return std::min((T + 15) / 16 * 16, 128); }

Space space(int T, int r, int cols) {
    Space s{};
    skinny::Cut cut;
    s.words = cut.take((size_t)skinny::kWords * 4);
    s.groups = cut.take((size_t)T * sizeof(int4));   // groups are at most as many as rows
    s.order = cut.take((size_t)T * 4);
    s.v = cut.take((size_t)T * r * 4);
    s.partial = cut.take(skinny::partial_floats(cols) * 4);
    s.total = cut.at;
    return s;
}

struct AdapterArgs {
    CUtensorMap w, a_map, x, x_rows;   // x: one row a box (gather), x_rows: `cols` rows
    const int32_t *idx;
    const __nv_bfloat16 *b;
    const float *scales;
    uint32_t *words;
    const int4 *groups;
    const int *order;
    float *v, *partials;
    __nv_bfloat16 *out;
    int32_t *status;
    int T, K, N, L, r;
    skinny::Shape shape;
    uint32_t tmem_cols;
    TraceArgs trace;
};

__device__ __forceinline__ float bf16_low(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_high(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

struct AdapterProblem {
    const AdapterArgs &a;
    int G;
    int32_t *status;
    int chunks, tiles, kbs;   // row chunks, feature tiles of W, K blocks

    __device__ explicit AdapterProblem(const AdapterArgs &args)
        : a(args), G((int)args.words[skinny::kGroupsWord]), status(args.status) {
        chunks = (a.T + a.shape.cols - 1) / a.shape.cols;
        tiles = (a.N + 2 * kRows - 1) / (2 * kRows);
        kbs = (a.K + 63) / 64;
    }

    template <class F>
    __device__ bool segments(F f) const {
        for (int phase = 0; phase < 2; ++phase) {
            const skinny::Line line(phase == 0 ? G : (int64_t)chunks * tiles, kbs, gridDim.x);
            const bool ok = line.each(blockIdx.x, [&](int64_t tile, skinny::Segment &s) {
                s.phase = phase;
                if (phase == 0) {
                    const int4 g = a.groups[tile];
                    s.group = g.x;
                    s.f = 0;
                    s.first = g.y;
                    s.n = g.z;
                    s.a_map = &a.a_map;
                    s.row0 = g.x * a.r;
                    s.a_bytes = a.r * 128;
                    s.two = false;
                } else {
                    const int chunk = (int)(tile / tiles);
                    s.group = 0;
                    s.f = (int)(tile - (int64_t)chunk * tiles);
                    s.first = chunk * a.shape.cols;
                    s.n = min(a.shape.cols, a.T - s.first);
                    s.a_map = &a.w;
                    s.row0 = s.f * 2 * kRows;
                    s.row1 = s.row0 + kRows;
                    s.a_bytes = skinny::kHalf;
                    s.two = true;
                }
                return f(s);
            });
            if (!ok) return false;
        }
        return true;
    }

    // ---- loads of B
    struct Rows {
        int r[4];
    };
    __device__ bool b_ready(const skinny::Segment &) const { return true; }
    __device__ Rows b_rows(const skinny::Segment &s, int lane) const {
        Rows rows{};
        if (s.phase == 0)
#pragma unroll
            for (int i = 0; i < 4; ++i) rows.r[i] = a.order[s.first + min(4 * lane + i, s.n - 1)];
        return rows;
    }
    __device__ uint32_t b_bytes(const skinny::Segment &s) const {
        return s.phase == 0 ? (s.n + 3) / 4 * 512 : a.shape.cols * 128;
    }
    __device__ void b_load(const skinny::Segment &s, const Rows &rows, int col, uint32_t dst, uint64_t *bar,
                           int lane) const {
        const uint64_t policy = policy_evict_last();
        if (s.phase == 0) {
            if (4 * lane < s.n)
                tma_gather4(dst + lane * 512, &a.x, col, rows.r[0], rows.r[1], rows.r[2], rows.r[3], bar, policy);
        } else if (lane == 0) {
            tma_load(dst, &a.x_rows, col, s.first, bar, policy);   // rows past T read as 0
        }
    }

    // ---- sums
    __device__ float *partial(int phase, int cta, int slot) const {
        return a.partials + ((size_t)(phase * skinny::kMaxCtas + cta) * 2 + slot) * 2 * a.shape.cols * kRows;
    }
    __device__ uint32_t *arrivals(int phase, int cta) const {
        return a.words + skinny::kArrivals + phase * skinny::kMaxCtas + cta;
    }
    // phase 1 adds what phase 0 made
    __device__ bool emit_ready(const skinny::Segment &s) const {
        if (s.phase == 0) return true;
        bool ok = true;
        if (threadIdx.x == skinny::kThreads - skinny::kReaders)
            ok = skinny::wait_count(a.words + skinny::kDoneWord, (uint32_t)G);
        return skinny::readers_agree(ok);
    }
    struct Emit {
        const AdapterArgs &a;
        const skinny::Segment &s;
        int row;
        __device__ Emit(const AdapterProblem &p, const skinny::Segment &seg, int r) : a(p.a), s(seg), row(r) {}
        __device__ void operator()(int col, const float *v0, const float *v1) const {
            if (s.phase == 0) {
                if (row >= a.r) return;
                const float scale = a.scales[s.group];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (col + j < s.n) a.v[(size_t)a.order[s.first + col + j] * a.r + row] = scale * v0[j];
                return;
            }
            const int o0 = s.f * 2 * kRows + row, o1 = o0 + kRows;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (col + j >= s.n) continue;
                const int t = s.first + col + j, id = a.idx[t];
                float x0 = v0[j], x1 = v1[j];
                if (id >= 0 && id < a.L) {
                    const float4 *v = reinterpret_cast<const float4 *>(a.v + (size_t)t * a.r);
                    const uint4 *b0 = reinterpret_cast<const uint4 *>(a.b + ((size_t)id * a.N + min(o0, a.N - 1)) * a.r);
                    const uint4 *b1 = reinterpret_cast<const uint4 *>(a.b + ((size_t)id * a.N + min(o1, a.N - 1)) * a.r);
                    for (int i = 0; i < a.r / 8; ++i) {
                        const float4 lo = __ldcg(v + 2 * i), hi = __ldcg(v + 2 * i + 1);
                        const uint4 p = __ldg(b0 + i), q = __ldg(b1 + i);
                        x0 = fmaf(bf16_low(p.x), lo.x, x0), x0 = fmaf(bf16_high(p.x), lo.y, x0);
                        x0 = fmaf(bf16_low(p.y), lo.z, x0), x0 = fmaf(bf16_high(p.y), lo.w, x0);
                        x0 = fmaf(bf16_low(p.z), hi.x, x0), x0 = fmaf(bf16_high(p.z), hi.y, x0);
                        x0 = fmaf(bf16_low(p.w), hi.z, x0), x0 = fmaf(bf16_high(p.w), hi.w, x0);
                        x1 = fmaf(bf16_low(q.x), lo.x, x1), x1 = fmaf(bf16_high(q.x), lo.y, x1);
                        x1 = fmaf(bf16_low(q.y), lo.z, x1), x1 = fmaf(bf16_high(q.y), lo.w, x1);
                        x1 = fmaf(bf16_low(q.z), hi.x, x1), x1 = fmaf(bf16_high(q.z), hi.y, x1);
                        x1 = fmaf(bf16_low(q.w), hi.z, x1), x1 = fmaf(bf16_high(q.w), hi.w, x1);
                    }
                }
                if (o0 < a.N) a.out[(size_t)t * a.N + o0] = __float2bfloat16_rn(x0);
                if (o1 < a.N) a.out[(size_t)t * a.N + o1] = __float2bfloat16_rn(x1);
            }
        }
    };
    __device__ void tile_done(const skinny::Segment &s) const {
        if (s.phase == 1) return;
        __threadfence();
        skinny::readers_sync();
        if (threadIdx.x == skinny::kThreads - skinny::kReaders) skinny::add_acq_rel(a.words + skinny::kDoneWord, 1);
    }
    __device__ bool finish() const { return true; }
};

__global__ void __launch_bounds__(skinny::kThreads, 1) adapter_kernel(const __grid_constant__ AdapterArgs a) {
    WarpTrace wt(a.trace, MOE_TRACE_ADAPTER);
    grid_dependency_wait();
    const AdapterProblem p(a);
    skinny::run<false>(p, a.shape, a.tmem_cols);
}

}  // namespace

size_t adapter_workspace_bytes(int T, int K, int N, int L, int r) { return space(T, r, columns(T)).total; }

int launch_adapter_linear(const AdapterLaunch &L) {
    const int T = L.num_tokens, K = L.in_features, N = L.out_features, r = L.rank;
    if (T == 0) return MOE_OK;
    const int cols = columns(T);
    const Space sp = space(T, r, cols);
    char *ws = static_cast<char *>(L.workspace);
    const cudaStream_t s = static_cast<cudaStream_t>(L.stream);

    const skinny::PlanArgs<int32_t> plan{L.adapter_idx, T, L.num_adapters, cols,
                                         reinterpret_cast<uint32_t *>(ws + sp.words), skinny::kWords,
                                         reinterpret_cast<int4 *>(ws + sp.groups),
                                         reinterpret_cast<int *>(ws + sp.order), MOE_ERR_BAD_ADAPTER, L.status,
                                         trace_args()};
    AdapterArgs a{};
    if (!make_tensor_map(&a.w, L.w, false, N, K, kRows) ||
        !make_tensor_map(&a.a_map, L.a, false, (uint64_t)L.num_adapters * r, K, r) ||
        !make_tensor_map(&a.x, L.x, false, T, K, 1) || !make_tensor_map(&a.x_rows, L.x, false, T, K, cols))
        return MOE_ERR_CUDA;
    a.idx = L.adapter_idx;
    a.b = static_cast<const __nv_bfloat16 *>(L.b);
    a.scales = L.scales;
    a.words = plan.words;
    a.groups = plan.groups;
    a.order = plan.order;
    a.v = reinterpret_cast<float *>(ws + sp.v);
    a.partials = reinterpret_cast<float *>(ws + sp.partial);
    a.out = static_cast<__nv_bfloat16 *>(L.out);
    a.status = L.status;
    a.T = T, a.K = K, a.N = N, a.L = L.num_adapters, a.r = r;
    a.shape = skinny::Shape{cols, skinny::Shape::stages_for(cols, false)};
    a.tmem_cols = skinny::Shape::tmem_cols(cols, false);
    a.trace = trace_args();
    const int rc = skinny::launch_plan(plan, s);
    if (rc != MOE_OK) return rc;
    return skinny::launch_resident(adapter_kernel, a, skinny::Shape::smem(cols, false), s);
}

}  // namespace moe
