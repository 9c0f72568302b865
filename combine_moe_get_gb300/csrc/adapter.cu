// adapter.cu -- a shared projection with the low-rank adapter of each row
// (moe_adapter_linear).
//
//   v[t]   = scales[i] * (A_i x_t),  i = adapter_idx[t]
//   out[t] = W x_t + B_i v[t]        (W x_t alone where i = -1)
//
// An adapter's values meet the sums of its own rows only, not even as a product
// with zero in another row's. Two ways to do that, in two or three kernels:
//
// Grouped (many rows to an adapter): the plan kernel sorts the rows by adapter,
// rows without one last, and cuts groups of one adapter; the sort kernel copies
// x in that order. The projection runs
// skinny.cuh's body over two lines: phase 0 multiplies a group's x rows by its A
// into v, phase 1 multiplies them by W and then, as more K blocks of the same
// sums, v by B. v is held as the sum of two bf16 (16 bits of it), the operands
// of two products.
//
// Row by row (few rows to an adapter): the shrink kernel makes v in fp32, four
// warps to a row of A, and the projection multiplies all rows, in their own
// order, by W; the readers of its sums add B_i v[t] in fp32, each thread for its
// own row of B. The projection's loads do not depend on the shrink kernel, so it
// is launched to overlap it.
#include <algorithm>
#include <climits>
#include <cuda_bf16.h>

#include "skinny.cuh"

namespace moe {
namespace {

using skinny::kRows;

// Grouped costs another pass over W for every group that is not full, about
// (L + 1) / 2 of them; row by row costs a pass over A for every row, from caches
// that are about half as fast for it.
bool grouped(int T, int N, int L, int r) { return (int64_t)4 * T * r > (int64_t)std::min(L + 1, T) * N; }

int columns(int T) { return std::min((T + 15) / 16 * 16, 128); }

struct Space {
    size_t words, groups, order, v, x, partial, total;   // byte offsets
};
constexpr int kReady = skinny::kWords;   // then a word per group: its v is done

Space space(int T, int K, int N, int L, int r, int cols) {
    Space s{};
    skinny::Cut cut;
    s.words = cut.take(((size_t)kReady + T) * 4);
    s.groups = cut.take((size_t)T * sizeof(int4));   // groups are at most as many as rows
    s.order = cut.take((size_t)T * 4);
    s.v = cut.take((size_t)(T + 8) * r * 4);         // fp32, or two bf16
    s.x = cut.take(grouped(T, N, L, r) ? (size_t)T * K * 2 : 0);   // rows of x, sorted
    s.partial = cut.take(skinny::partial_floats(2, cols) * 4);
    s.total = cut.at;
    return s;
}

struct AdapterArgs {
    CUtensorMap w, a_map, b_map, x, v_map;   // x: `cols` rows a box, of x or of its sorted copy
    const int32_t *idx;
    const __nv_bfloat16 *b;
    const float *scales;
    uint32_t *words;
    const int4 *groups;
    const int *order;
    void *v;
    float *partials;
    __nv_bfloat16 *out;
    int32_t *status;
    int T, K, N, L, r;
    skinny::Shape shape;
    uint32_t tmem_cols;
    TraceArgs trace;
};

__device__ __forceinline__ float bf16_low(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_high(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// What both ways share.
struct AdapterBase {
    static constexpr bool kHalves = true, kConvert = false;
    const AdapterArgs &a;
    int32_t *status;
    int tiles, kbs;   // feature tiles of W, K blocks of x
    __device__ explicit AdapterBase(const AdapterArgs &args) : a(args), status(args.status) {
        tiles = (a.N + 2 * kRows - 1) / (2 * kRows);
        kbs = (a.K + 63) / 64;
    }
    __device__ float *partial(int line, int cta, int slot) const {
        return a.partials + ((size_t)(line * skinny::kMaxCtas + cta) * 2 + slot) * 2 * a.shape.cols * kRows;
    }
    __device__ uint32_t *arrivals(int line, int cta) const {
        return a.words + skinny::kArrivals + line * skinny::kMaxCtas + cta;
    }
    template <class Team>
    __device__ bool emit_ready(const skinny::Segment &) const { return true; }
    __device__ bool finish() const { return true; }
};

// ------------------------------------------------------------------ grouped

struct SortArgs {
    const uint4 *x;
    uint4 *sorted;
    const int *order;
    int T, pieces;   // rows, 16-byte pieces of a row
    TraceArgs trace;
};

// sorted[p] = x[order[p]], one CTA per row. (Gathering the rows by TMA in the
// products' loads instead, four rows a copy, took 22 cycles a row: 2.5 times the
// whole projection's time at 128 rows to a tile.)
__global__ void __launch_bounds__(256) adapter_sort_kernel(const SortArgs s) {
    WarpTrace wt(s.trace, MOE_TRACE_ADAPTER_SORT);
    grid_dependency_wait();
    grid_launch_dependents();
    const uint4 *from = s.x + (size_t)s.order[blockIdx.x] * s.pieces;
    uint4 *to = s.sorted + (size_t)blockIdx.x * s.pieces;
    for (int i = threadIdx.x; i < s.pieces; i += 256) to[i] = __ldg(from + i);
}

struct GroupedAdapter : AdapterBase {
    static constexpr bool kAdders = true;
    static constexpr int kReaders = 512;
    using Ahead = skinny::NothingAhead;
    int G, with_adapter;   // groups; those before it have an adapter
    int more;              // K blocks of v's first part

    __device__ explicit GroupedAdapter(const AdapterArgs &args) : AdapterBase(args) {
        G = (int)a.words[skinny::kGroupsWord];
        with_adapter = (int)a.words[skinny::kNamedWord];
        more = (a.r + 63) / 64;
    }

    template <class F, class End = skinny::Nothing>
    __device__ bool segments(F f, End end_line = End()) const {
        for (int phase = 0; phase < 2; ++phase) {
            const skinny::Line line(phase == 0 ? with_adapter : (int64_t)G * tiles, phase == 0 ? kbs : kbs + 2 * more,
                                    gridDim.x, skinny::kSlackWork);
            const bool ok = line.each(blockIdx.x, [&](int64_t tile, skinny::Segment &s) {
                s.line = s.phase = phase;
                s.group = phase == 0 ? (int)tile : (int)skinny::quotient(tile, tiles);
                s.f = phase == 0 ? 0 : (int)(tile - (int64_t)s.group * tiles);
                const int4 g = a.groups[s.group];
                s.first = g.y;
                s.n = g.z;
                s.set = g.x;
                s.two = phase == 1;
                s.row0 = phase == 0 ? g.x * a.r : s.f * 2 * kRows;
                s.row1 = s.row0 + kRows;
                s.b_from = phase == 1 && g.x < a.L ? kbs : INT_MAX;
                return f(s);
            });
            if (!ok || !end_line()) return false;
        }
        return true;
    }

    __device__ void a_load(const skinny::Segment &s, int kb, uint32_t dst, uint64_t *bar, uint64_t policy) const {
        if (s.phase == 0) {
            mbar_arrive_expect_tx(bar, a.r * 128);
            tma_load(dst, &a.a_map, kb * 64, s.row0, bar, policy);
            return;
        }
        // rows behind the last adapter's B read as 0: groups without an adapter
        const bool is_w = kb < kbs;
        const CUtensorMap *map = is_w ? &a.w : &a.b_map;
        const int col = is_w ? kb * 64 : (kb - kbs) % more * 64, row = is_w ? s.row0 : s.set * a.N + s.row0;
        mbar_arrive_expect_tx(bar, 2 * skinny::kHalf);
        tma_load(dst, map, col, row, bar, policy);
        tma_load(dst + skinny::kHalf, map, col, row + kRows, bar, policy);
    }
    struct Rows {};
    __device__ Rows b_rows(const skinny::Segment &, int) const { return Rows{}; }
    __device__ bool b_ready(const skinny::Segment &s) const {
        if (!skinny::wait_count(a.words + kReady + s.group, skinny::kTileWeight)) return false;
        fence_proxy_async();
        return true;
    }
    __device__ uint32_t b_bytes(const skinny::Segment &s, int kb) const {
        return kb < kbs ? a.shape.cols * 128 : (s.n + 7) / 8 * 1024;
    }
    __device__ void b_load(const skinny::Segment &s, const Rows &, int kb, uint32_t dst, uint64_t *bar, uint64_t policy,
                           int lane) const {
        if (kb < kbs) {
            if (lane == 0) tma_load(dst, &a.x, kb * 64, s.first, bar, policy);   // the next groups' rows fill the box
        } else if (8 * lane < s.n) {
            // v's first parts [T, r], then the second ones; behind both, zeros for groups without an adapter
            const int part = (kb - kbs) / more, row = s.set < a.L ? part * a.T + s.first + 8 * lane : 2 * a.T;
            tma_load(dst + lane * 1024, &a.v_map, (kb - kbs) % more * 64, row, bar, policy);
        }
    }

    struct Emit {
        const AdapterArgs &a;
        const skinny::Segment &s;
        int row, half;
        __device__ Emit(const GroupedAdapter &p, const skinny::Segment &seg, const skinny::Share<true> &me)
            : a(p.a), s(seg), row(me.row), half(me.side & 1) {}
        __device__ void operator()(int col, const float *sums) const {
            if (s.phase == 0) {
                if (half != 0 || row >= a.r) return;
                const float scale = a.scales[s.set];
                __nv_bfloat16 *v = static_cast<__nv_bfloat16 *>(a.v);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (col + j >= s.n) continue;
                    const float x = scale * sums[j];
                    const __nv_bfloat16 hi = __float2bfloat16_rn(x);
                    const float rest = x - __bfloat162float(hi);
                    const size_t at = (size_t)(s.first + col + j) * a.r + row;
                    v[at] = hi;
                    v[(size_t)a.T * a.r + at] = __float2bfloat16_rn(isfinite(rest) ? rest : 0.0f);
                }
                return;
            }
            const int o = s.row0 + half * kRows + row;
            if (o >= a.N) return;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (col + j < s.n) a.out[(size_t)a.order[s.first + col + j] * a.N + o] = __float2bfloat16_rn(sums[j]);
        }
    };
    __device__ void before_signal(const skinny::Segment &s) const {
        if (s.phase == 0) fence_proxy_async();   // v is read by TMA
    }
    __device__ void tile_done(const skinny::Segment &s, uint32_t weight) const {
        if (s.phase == 0) skinny::count_up(a.words + kReady + s.group, weight);
    }
};

__global__ void __launch_bounds__(skinny::threads_of<GroupedAdapter>(), 1)
    adapter_grouped_kernel(const __grid_constant__ AdapterArgs a) {
    WarpTrace wt(a.trace, MOE_TRACE_ADAPTER);
    if (threadIdx.x == 0)
        for (const CUtensorMap *m : {&a.w, &a.x, &a.a_map, &a.b_map, &a.v_map}) tma_prefetch_map(m);
    skinny::run<false, GroupedAdapter>([&] {
        grid_dependency_wait();
        return GroupedAdapter(a);
    }, a.shape, a.tmem_cols);
}

// ------------------------------------------------------------------ row by row

struct ShrinkArgs {
    const __nv_bfloat16 *x, *a;
    const int32_t *idx;
    const float *scales;
    float *v;            // [T, r]
    uint32_t *words;
    int T, K, L, r;
    int32_t *status;
    TraceArgs trace;
};

constexpr int kShrinkRows = 8;   // rows of A to a CTA: two groups of four warps, a quarter of K to a warp, four rows to a warp

__global__ void __launch_bounds__(256) adapter_shrink_kernel(const ShrinkArgs s) {
    WarpTrace wt(s.trace, MOE_TRACE_ADAPTER_SHRINK);
    grid_dependency_wait();
    grid_launch_dependents();   // the projection's loads, of inputs that are complete by now
    __shared__ float sums[8][4];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = (s.r + kShrinkRows - 1) / kShrinkRows;
    const int t = blockIdx.x / per, row0 = (blockIdx.x - t * per) * kShrinkRows;
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < skinny::kWords; i += 256) s.words[i] = 0;
    const int id = s.idx[t];
    if (id < 0 || id >= s.L) {
        if (id != -1 && row0 == 0 && threadIdx.x == 0) report(s.status, MOE_ERR_BAD_ADAPTER);
        return;
    }
    const int first = row0 + (warp >> 2) * 4, last = s.r - 1;
    const __nv_bfloat16 *x = s.x + (size_t)t * s.K;
    const __nv_bfloat16 *rows[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) rows[i] = s.a + ((size_t)id * s.r + min(first + i, last)) * s.K;
    float acc[4] = {};
#pragma unroll 4
    for (int c = ((warp & 3) * 32 + lane) * 8; c < s.K; c += 1024) {
        const uint4 p = __ldg(reinterpret_cast<const uint4 *>(x + c));
        const uint32_t pw[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 q = __ldg(reinterpret_cast<const uint4 *>(rows[i] + c));
            const uint32_t qw[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc[i] = fmaf(bf16_low(pw[j]), bf16_low(qw[j]), acc[i]);
                acc[i] = fmaf(bf16_high(pw[j]), bf16_high(qw[j]), acc[i]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
        if (lane == 0) sums[warp][i] = acc[i];
    }
    __syncthreads();
    const int i = threadIdx.x;
    if (i < kShrinkRows && row0 + i < s.r) {
        const int g = i / 4 * 4;
        s.v[(size_t)t * s.r + row0 + i] =
            s.scales[id] * (((sums[g][i & 3] + sums[g + 1][i & 3]) + sums[g + 2][i & 3]) + sums[g + 3][i & 3]);
    }
}

struct RowAdapter : AdapterBase {
    static constexpr bool kAdders = false;
    static constexpr int kReaders = 256;
    int chunks;
    __device__ explicit RowAdapter(const AdapterArgs &args) : AdapterBase(args) {
        chunks = (a.T + a.shape.cols - 1) / a.shape.cols;
    }

    template <class F, class End = skinny::Nothing>
    __device__ bool segments(F f, End end_line = End()) const {
        const skinny::Line line((int64_t)chunks * tiles, kbs, gridDim.x,
                                a.shape.cols > 32 ? skinny::kSlackWork : skinny::kSlackBytes);
        const bool ok = line.each(blockIdx.x, [&](int64_t tile, skinny::Segment &s) {
            s.line = s.phase = 0;
            s.group = (int)skinny::quotient(tile, tiles);
            s.f = (int)(tile - (int64_t)s.group * tiles);
            s.first = s.group * a.shape.cols;
            s.n = min(a.shape.cols, a.T - s.first);
            s.two = true;
            s.row0 = s.f * 2 * kRows;
            s.row1 = s.row0 + kRows;
            s.b_from = INT_MAX;
            return f(s);
        });
        return ok && end_line();
    }

    __device__ void a_load(const skinny::Segment &s, int kb, uint32_t dst, uint64_t *bar, uint64_t policy) const {
        mbar_arrive_expect_tx(bar, 2 * skinny::kHalf);
        tma_load(dst, &a.w, kb * 64, s.row0, bar, policy);
        tma_load(dst + skinny::kHalf, &a.w, kb * 64, s.row1, bar, policy);
    }
    struct Rows {};
    __device__ bool b_ready(const skinny::Segment &) const { return true; }
    __device__ Rows b_rows(const skinny::Segment &, int) const { return Rows{}; }
    __device__ uint32_t b_bytes(const skinny::Segment &, int) const { return a.shape.cols * 128; }
    __device__ void b_load(const skinny::Segment &s, const Rows &, int kb, uint32_t dst, uint64_t *bar, uint64_t policy,
                           int lane) const {
        if (lane == 0) tma_load(dst, &a.x, kb * 64, s.first, bar, policy);   // rows past T read as 0
    }

    // B v of eight columns for one row of W and B
    struct Part {
        const AdapterArgs &a;
        const skinny::Segment &s;
        int o;                    // the row
        const __nv_bfloat16 *b;   // ... in the first adapter
        __device__ Part(const RowAdapter &p, const skinny::Segment &seg, const skinny::Share<true> &me)
            : a(p.a), s(seg), o(seg.row0 + (me.side & 1) * kRows + me.row) {
            b = a.b + (size_t)min(o, a.N - 1) * a.r;
        }
        __device__ static float dot(const uint4 &w, const float *v, float x) {
            const float4 lo = *reinterpret_cast<const float4 *>(v), hi = *reinterpret_cast<const float4 *>(v + 4);
            x = fmaf(bf16_low(w.x), lo.x, x), x = fmaf(bf16_high(w.x), lo.y, x);
            x = fmaf(bf16_low(w.y), lo.z, x), x = fmaf(bf16_high(w.y), lo.w, x);
            x = fmaf(bf16_low(w.z), hi.x, x), x = fmaf(bf16_high(w.z), hi.y, x);
            return fmaf(bf16_high(w.w), hi.w, fmaf(bf16_low(w.w), hi.z, x));
        }
        __device__ void add(int col, float *x) const {
            int id[8];
            bool same = true;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                id[j] = a.idx[s.first + min(col + j, s.n - 1)];
                if (id[j] >= a.L) id[j] = -1;
                same &= id[j] == id[0];
            }
            const size_t set = (size_t)a.N * a.r;
            const float *v = static_cast<const float *>(a.v) + (size_t)(s.first + col) * a.r;   // eight rows: as many are behind the last
            if (!same) {
                for (int i = 0; i < a.r; i += 8) {
                    uint4 q[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (id[j] >= 0) q[j] = __ldg(reinterpret_cast<const uint4 *>(b + id[j] * set + i));
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (id[j] >= 0) x[j] = dot(q[j], v + j * a.r + i, x[j]);
                }
            } else if (id[0] >= 0) {   // one adapter: its row of B is read once for the eight
                for (int i = 0; i < a.r; i += 8) {
                    const uint4 q = __ldg(reinterpret_cast<const uint4 *>(b + id[0] * set + i));
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] = dot(q, v + j * a.r + i, x[j]);
                }
            }
        }
    };
    // The adapters' part of the columns that this CTA will add up of a tile that
    // it shares (columns 8 i with i % parts its place among them): worked out
    // while the products run, and left with this CTA's own part.
    struct Ahead {
        static constexpr int kKept = 3;
        Part part;
        int me;
        bool shared;
        float x[kKept][8] = {};
        __device__ Ahead(const RowAdapter &p, const skinny::Segment &s, const skinny::Share<true> &share)
            : part(p, s, share), me(blockIdx.x - s.cta0), shared(!s.whole()) {
            if (!shared) return;
#pragma unroll
            for (int q = 0; q < kKept; ++q)
                if (8 * (me + q * s.parts) < s.n) part.add(8 * (me + q * s.parts), x[q]);
        }
        __device__ void add(int col, float *v) const {
            const int parts = part.s.parts, i = col / 8 - me;
            if (i < 0 || i % parts != 0) return;
            if (i / parts >= kKept) return part.add(col, v);
#pragma unroll
            for (int q = 0; q < kKept; ++q)
                if (i / parts == q)
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] += x[q][j];
        }
    };
    struct Emit {
        Part part;
        bool add;   // a shared tile's parts hold it already
        __device__ Emit(const RowAdapter &p, const skinny::Segment &s, const skinny::Share<true> &me)
            : part(p, s, me), add(s.whole()) {}
        __device__ void operator()(int col, float *x) const {
            if (add) part.add(col, x);
            const AdapterArgs &a = part.a;
            if (part.o >= a.N) return;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (col + j < part.s.n)
                    a.out[(size_t)(part.s.first + col + j) * a.N + part.o] = __float2bfloat16_rn(x[j]);
        }
    };
    __device__ void before_signal(const skinny::Segment &) const {}
    __device__ void tile_done(const skinny::Segment &, uint32_t) const {}
};

// Loads of x and W begin before the shrink kernel has ended: it passed its own
// dependency wait, so all that came before it is complete, and it writes neither.
__global__ void __launch_bounds__(skinny::threads_of<RowAdapter>(), 1)
    adapter_row_kernel(const __grid_constant__ AdapterArgs a) {
    WarpTrace wt(a.trace, MOE_TRACE_ADAPTER);
    if (threadIdx.x == 0)
        for (const CUtensorMap *m : {&a.w, &a.x}) tma_prefetch_map(m);
    skinny::run<false, RowAdapter>([&] {
        if (threadIdx.x >= skinny::ReadersOf<RowAdapter>::first) grid_dependency_wait();   // the counters and v
        return RowAdapter(a);
    }, a.shape, a.tmem_cols);
}

}  // namespace

size_t adapter_workspace_bytes(int T, int K, int N, int L, int r) { return space(T, K, N, L, r, columns(T)).total; }

int launch_adapter_linear(const AdapterLaunch &L) {
    const int T = L.num_tokens, K = L.in_features, N = L.out_features, r = L.rank;
    if (T == 0) return MOE_OK;
    const int cols = columns(T);
    const Space sp = space(T, K, N, L.num_adapters, r, cols);
    char *ws = static_cast<char *>(L.workspace);
    const cudaStream_t s = static_cast<cudaStream_t>(L.stream);
    const bool by_group = grouped(T, N, L.num_adapters, r);

    AdapterArgs a{};
    bool ok = make_tensor_map(&a.w, L.w, false, N, K, kRows) &&
              make_tensor_map(&a.x, by_group ? ws + sp.x : L.x, false, T, K, cols);
    if (by_group)
        ok = ok && make_tensor_map(&a.a_map, L.a, false, (uint64_t)L.num_adapters * r, K, r) &&
             make_tensor_map(&a.b_map, L.b, false, (uint64_t)L.num_adapters * N, r, kRows) &&
             make_tensor_map(&a.v_map, ws + sp.v, false, (uint64_t)2 * T, r, 8);
    if (!ok) return MOE_ERR_CUDA;
    a.idx = L.adapter_idx;
    a.b = static_cast<const __nv_bfloat16 *>(L.b);
    a.scales = L.scales;
    a.words = reinterpret_cast<uint32_t *>(ws + sp.words);
    a.groups = reinterpret_cast<const int4 *>(ws + sp.groups);
    a.order = reinterpret_cast<const int *>(ws + sp.order);
    a.v = ws + sp.v;
    a.partials = reinterpret_cast<float *>(ws + sp.partial);
    a.out = static_cast<__nv_bfloat16 *>(L.out);
    a.status = L.status;
    a.T = T, a.K = K, a.N = N, a.L = L.num_adapters, a.r = r;
    a.shape = skinny::Shape::of(cols, false);
    a.tmem_cols = a.shape.tmem_cols(false);
    a.trace = trace_args();
    const size_t smem = a.shape.smem(false);

    if (by_group) {
        const skinny::PlanArgs<int32_t> plan{L.adapter_idx, T, L.num_adapters, true, cols, a.words, kReady + T,
                                             const_cast<int4 *>(a.groups), const_cast<int *>(a.order),
                                             MOE_ERR_BAD_ADAPTER, L.status, a.trace};
        const int rc = skinny::launch_plan(plan, s);
        if (rc != MOE_OK) return rc;
        const SortArgs so{static_cast<const uint4 *>(L.x), reinterpret_cast<uint4 *>(ws + sp.x), a.order, T, K / 8, a.trace};
        if (launch_kernel(adapter_sort_kernel, dim3(T), dim3(256), 0, s, tuning().overlap != 0, so) != cudaSuccess)
            return MOE_ERR_CUDA;
        return skinny::launch_resident(adapter_grouped_kernel, a, skinny::threads_of<GroupedAdapter>(), smem, s);
    }
    const ShrinkArgs sh{static_cast<const __nv_bfloat16 *>(L.x), static_cast<const __nv_bfloat16 *>(L.a),
                        L.adapter_idx, L.scales, static_cast<float *>(a.v), a.words, T, K, L.num_adapters, r,
                        L.status, a.trace};
    const int64_t ctas = (int64_t)T * ((r + kShrinkRows - 1) / kShrinkRows);
    if (launch_kernel(adapter_shrink_kernel, dim3((unsigned)ctas), dim3(256), 0, s, tuning().overlap != 0, sh) !=
        cudaSuccess)
        return MOE_ERR_CUDA;
    return skinny::launch_resident(adapter_row_kernel, a, skinny::threads_of<RowAdapter>(), smem, s);
}

}  // namespace moe
