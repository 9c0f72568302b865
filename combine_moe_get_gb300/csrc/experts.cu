// experts.cu -- the experts' products of a few tokens (moe_experts).
//
//   h[t, j]  = silu(G x_t) * (U x_t),  [G; U] = w13[e], e = topk_idx[t, j]
//   out[t]   = sum_j topk_weights[t, j] * (w2[e] h[t, j])
//
// The valid entries are sorted by expert and cut into groups of at most `cols` of
// one expert: up to 256 entries by every CTA for itself, more by a plan kernel.
// The experts kernel (one CTA per SM, launched cooperatively) runs skinny.cuh's body
// over two phases of work: phase 0 makes h (a tile is 128 gate and the same 128 up rows,
// so that one thread holds both sums of an element), phase 1 multiplies h by w2
// (a tile is 256 rows) into y, one fp32 row per entry. A group's phase 1 waits
// until all its h tiles are done; the loads of w2 do not wait. The groups go
// through the two phases in up to two waves, phase 0 of a wave before phase 1 of
// the wave before it, so that h is there when its turn comes and the stream of
// weights does not pause. When all of y is there, all CTAs add each token's rows in
// entry order with their weights and round once to bf16.
//
// h is rounded to bf16, or with E4M3 weights to a sum of two codes of the same
// eight bits: it is the operand of a product, and the rounding's effect on an
// output is of the size of that output's own rounding. With E4M3 weights a split
// kernel makes two codes of x before, which is exact for all elements within
// 2^-14 of their block's largest, and off by 2^-22 of that at most for smaller ones:
// channels that are thousands of times the others cost these no bits.
//
// The stream of the chosen experts' weights bounds it. Experts of 7168 x 2048: one
// token, 8 in bf16 (705 MB), 118 us, 6.0 TB/s; 64 tokens' local entries, 32 in E4M3
// (1.46 GB), 265 us, 5.5 TB/s; 128 tokens, 256 in E4M3 (11.4 GB), 1800 us, 6.3 TB/s.
// The rest of a call is set-up (5 us), the wait for the first and the last wave's h
// (6 us each) and the sums over y (3 us): 24 experts of 1160 x 520 and 37 tokens, 86 MB,
// take 30 us where the bytes take 13. In calls this short the kernel's instructions
// come from L2 as well: what runs once for a tile is kept in one short copy.
#include <algorithm>
#include <climits>
#include <cuda_bf16.h>

#include "skinny.cuh"

namespace moe {
namespace {

using skinny::kRows;

// Device workspace: byte offsets.
struct Space {
    size_t words, groups, order, h, h_scales, x_codes, x_scales, y, partial, total;
};
// Two waves from this many K blocks of phase 1 per CTA (32 KB each, some 0.7 us):
// the hand-over of h takes about 6 us after the slowest CTA, and CTAs drift
// apart by about 10. Three or more waves measured slower: over shorter lines
// the CTAs differ by more.
constexpr int kWaveBlocks = 28;
constexpr int kReady = skinny::kWords;   // then a word per group: its finished h tiles

// Columns of a tile: room for more than an expert's even share of the entries. An
// expert with more takes several groups, that is, streams its weights again.
int columns(int T, int k, int E, bool e4m3) {
    const int most = std::min((T + 15) / 16 * 16, e4m3 ? 64 : 128);
    const int64_t want = (3 * (int64_t)T * k / (2 * E) + 8 + 15) / 16 * 16;
    return (int)std::min<int64_t>(most, std::max<int64_t>(want, 16));
}

// Waves of groups at most, 1 or 2 (each is a line of either phase): wider tiles
// have larger partial sums.
int waves_for(int cols) { return cols <= 64 ? 2 : 1; }

Space space(int T, int H, int I, int k, int cols, bool e4m3) {
    Space s{};
    skinny::Cut cut;
    const size_t n = (size_t)T * k;   // groups are at most as many as entries
    s.words = cut.take((kReady + n) * 4);
    s.groups = cut.take(n * sizeof(int4));
    s.order = cut.take(n * 4);
    s.h = cut.take(n * I * 2);   // bf16, or first codes of all entries, then second ones
    s.h_scales = cut.take(e4m3 ? n * (I / 128) * 4 : 0);
    s.x_codes = cut.take(e4m3 ? (size_t)T * H * 2 : 0);
    s.x_scales = cut.take(e4m3 ? (size_t)T * (H / 128) * 4 : 0);
    s.y = cut.take(n * H * 4);
    s.partial = cut.take(skinny::partial_floats(2 * waves_for(cols), cols) * 4);
    s.total = cut.at;
    return s;
}

// ------------------------------------------------------------------ experts

struct ExpertsArgs {
    CUtensorMap w13, w2, x, h_map;   // x and h: bf16, or codes [2 rows]
    const int64_t *topk_idx;
    const float *topk_weights;
    const float *s13, *s2;
    const float *x_scales;   // E4M3: of x and of h, [row][block]
    float *h_scales;
    uint32_t *words;
    const int4 *groups;
    const int *order;
    void *h;
    float *y, *partials;
    __nv_bfloat16 *out;
    int32_t *status;
    int T, H, I, k, E;
    skinny::Shape shape;
    uint32_t tmem_cols;
    int max_waves;
    bool local;   // every CTA makes the plan for itself
    WaitLimits limits;
    TraceArgs trace;
};

// The lines of work in their order: phase 0 of the waves, then their phase 1.
struct Lines {
    skinny::Line line[4];
    int first_group[4];
    int waves;
};

// E4M3: largest magnitudes of 32 rows, [readers' two sides and adders][column][quarter].
struct Most {
    float4 of[3][4];
};

template <bool kE4m3, int kCols>   // kCols: the most columns of a tile
struct ExpertsProblem {
    static constexpr int kSteps = kCols / 8;   // E4M3
    static_assert(kSteps > 0);
    static constexpr bool kHalves = false, kShares = true, kAdders = true, kCodes = kE4m3, kPieces = false;
    static constexpr int kReaders = kE4m3 ? 256 : 512;
    using Readers = skinny::ReadersOf<ExpertsProblem>;
    const ExpertsArgs &a;
    const skinny::LocalPlan *local;   // or null: the plan kernel's
    int G;
    int32_t *status;
    int tiles[2], kbs[2];   // tiles per group and K blocks per tile of the two phases

    const Lines *lines;
    Most *most;

    // All threads of the CTA.
    __device__ ExpertsProblem(const ExpertsArgs &args, const skinny::LocalPlan *plan, Lines &shared_lines, Most &shared_most)
        : a(args), local(plan), status(args.status), lines(&shared_lines), most(&shared_most) {
        G = local ? local->num_groups : (int)args.words[skinny::kGroupsWord];
        constexpr int block = kE4m3 ? 128 : 64;
        tiles[0] = (a.I + kRows - 1) / kRows;
        tiles[1] = (a.H + 2 * kRows - 1) / (2 * kRows);
        kbs[0] = (a.H + block - 1) / block;
        kbs[1] = (a.I + block - 1) / block;
        // Waves of groups, one behind the other: phase 0 of wave 1 comes before phase 1 of wave 0. A
        // line's divisions take the better part of a microsecond: one thread to a line.
        const int64_t work = (int64_t)G * tiles[1] * kbs[1];
        const int waves = a.max_waves == 2 && G > 1 && work >= (int64_t)kWaveBlocks * gridDim.x ? 2 : 1;
        if (threadIdx.x < 2 * waves) {
            const int phase = threadIdx.x >= waves, wave = threadIdx.x - (phase ? waves : 0);
            const int g0 = wave == 0 ? 0 : G / 2, g1 = wave + 1 == waves ? G : G / 2;
            shared_lines.first_group[threadIdx.x] = g0;
            shared_lines.line[threadIdx.x] = skinny::Line((int64_t)(g1 - g0) * tiles[phase], kbs[phase], gridDim.x,
                                                          kE4m3 || a.shape.cols > 32 ? skinny::kSlackWork : skinny::kSlackBytes);
        }
        if (threadIdx.x == 0) shared_lines.waves = waves;
        __syncthreads();
    }

    __device__ int4 group(int g) const {   // {expert, first sorted entry, entries}
        if (local == nullptr) return a.groups[g];
        const uint32_t v = local->groups[g];
        return make_int4(v & 0x1fff, v >> 13 & 0xff, (v >> 21) + 1, 0);
    }
    __device__ int entry(int i) const { return local ? local->order[i] : a.order[i]; }

    template <class F>
    __device__ bool segments(F f) const {
        const int waves = lines->waves;
        for (int i = 0; i < 2 * waves; ++i) {
            const int phase = i >= waves, g0 = lines->first_group[i];
            const bool ok = lines->line[i].each(blockIdx.x, [&](int64_t tile, skinny::Segment &s) {
                s.line = i;
                s.phase = phase;
                const int in_wave = (int)skinny::quotient(tile, tiles[phase]);
                s.group = g0 + in_wave;
                s.f = (int)(tile - (int64_t)in_wave * tiles[phase]);
                const int4 g = group(s.group);
                s.first = g.y;
                s.n = g.z;
                s.two = true;
                if (phase == 0) {
                    s.row0 = g.x * 2 * a.I + s.f * kRows;
                    s.row1 = s.row0 + a.I;
                    s.b_from = INT_MAX;
                } else {
                    s.row0 = g.x * a.H + s.f * 2 * kRows;
                    s.row1 = s.row0 + kRows;
                    s.b_from = 0;
                }
                return f(s);
            });
            if (!ok) return false;
        }
        return true;
    }

    // ---- loads
    __device__ void a_load(const skinny::Segment &s, int kb, uint32_t dst, uint64_t *bar, uint64_t policy) const {
        const CUtensorMap *map = s.phase == 0 ? &a.w13 : &a.w2;
        const int col = kb * (kE4m3 ? 128 : 64);
        mbar_arrive_expect_tx(bar, 2 * skinny::kHalf);
        tma_load(dst, map, col, s.row0, bar, policy);
        tma_load(dst + skinny::kHalf, map, col, s.row1, bar, policy);
    }
    // B: x rows of the group's entries, or their rows of h
    struct Rows {
        int r[4];
    };
    __device__ bool b_ready(const skinny::Segment &s) const {
        return skinny::wait_count(a.words + kReady + s.group, tiles[0] * skinny::kTileWeight, a.limits.wait_ns);
    }
    __device__ Rows b_rows(const skinny::Segment &s, int lane) const {
        Rows rows{};
        if (s.phase == 0)
#pragma unroll
            for (int i = 0; i < 4; ++i) rows.r[i] = entry(s.first + min(4 * lane + i, s.n - 1)) / a.k;
        return rows;
    }
    static constexpr int kParts = kE4m3 ? 2 : 1, kBlock = kE4m3 ? 128 : 64;
    __device__ uint32_t b_bytes(const skinny::Segment &s, int) const {
        return kParts * (s.phase == 0 ? (s.n + 3) / 4 * 512 : (s.n + 7) / 8 * 1024);
    }
    __device__ void b_load(const skinny::Segment &s, const Rows &rows, int kb, uint32_t dst, uint64_t *bar,
                           uint64_t policy, int lane) const {
#pragma unroll
        for (int part = 0; part < kParts; ++part) {   // second codes behind the first ones' rows
            const uint32_t to = dst + part * s.n16() * 128;
            if (s.phase == 0) {
                const int o = part * a.T;
                if (4 * lane < s.n)
                    tma_gather4(to + lane * 512, &a.x, kb * kBlock, o + rows.r[0], o + rows.r[1], o + rows.r[2],
                                o + rows.r[3], bar, policy);
            } else if (8 * lane < s.n) {
                tma_load(to + lane * 1024, &a.h_map, kb * kBlock, part * a.T * a.k + s.first + 8 * lane, bar, policy);
            }
        }
    }
    // the scales of column c's activations, block by block
    __device__ const float *b_scales(const skinny::Segment &s, int c) const {
        return s.phase == 0 ? a.x_scales + (size_t)(entry(s.first + c) / a.k) * kbs[0]
                            : a.h_scales + (size_t)(s.first + c) * kbs[1];
    }

    // ---- sums
    __device__ const float *scales(int phase) const { return phase == 0 ? a.s13 : a.s2; }
    __device__ int weight_rows(int phase) const { return a.E * (phase == 0 ? 2 * a.I : a.H); }
    __device__ float *partial(int line, int cta, int slot) const {
        return a.partials + ((size_t)(line * skinny::kMaxCtas + cta) * 2 + slot) * 2 * a.shape.cols * kRows;
    }
    __device__ uint32_t *arrivals(int line, int cta) const {
        return a.words + skinny::kArrivals + line * skinny::kMaxCtas + cta;
    }
    struct Emit {
        const ExpertsProblem &p;
        const ExpertsArgs &a;
        const skinny::Segment &s;
        int row;
        __device__ Emit(const ExpertsProblem &problem, const skinny::Segment &seg, const skinny::Share<false> &me)
            : p(problem), a(p.a), s(seg), row(me.row) {}
        // Four columns of a block of 128 rows, which the four warps of a side hold:
        // their largest magnitudes go through shared memory.
        __device__ void emit_codes(int col, const float (&h)[4], int i) {
            const int group = (threadIdx.x - Readers::first) / 128, quarter = threadIdx.x / 32 & 3;
            float4 (&most)[4] = p.most->of[group];
            auto side_sync = [&] { asm volatile("barrier.cta.sync %0, 128;" ::"r"(3 + group) : "memory"); };
            side_sync();   // the columns before these are done with it
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float m = lanes_max(fabsf(h[j]));
                if ((threadIdx.x & 31) == 0) reinterpret_cast<float *>(&most[j])[quarter] = m;
            }
            side_sync();
            const size_t pos = s.first + col, second = (size_t)a.T * a.k * a.I;
            uint8_t *to = static_cast<uint8_t *>(a.h) + pos * a.I + i;
            float *scales = a.h_scales + pos * p.kbs[1] + s.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float4 q = most[j];
                const skinny::BlockScale scale(fmaxf(fmaxf(q.x, q.y), fmaxf(q.z, q.w)));   // a NaN's code is one too
                const skinny::Split two(h[j] * scale.inverse);
                if (col + j < s.n) {
                    to[0] = (uint8_t)two.first;
                    to[second] = (uint8_t)two.second;
                    if (row == 0) *scales = scale.scale;
                }
                to += a.I, scales += p.kbs[1];
            }
        }
        __device__ void operator()(int col, const float *v) {
            if (s.phase == 0) {
                float h[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)   // off by some 2^-21 near 0 and 2^-17 at -40: below the eight bits that h keeps
                    h[j] = __fdividef(v[j], 1.0f + __expf(-v[j])) * v[4 + j];
                const int i = s.f * kRows + row;
                if constexpr (kE4m3) {
                    emit_codes(col, h, i);
                } else if (i < a.I) {
                    __nv_bfloat16 *to = static_cast<__nv_bfloat16 *>(a.h) + (size_t)(s.first + col) * a.I + i;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (col + j < s.n) to[(size_t)j * a.I] = __float2bfloat16_rn(h[j]);
                }
            } else {
                const int o = s.f * 2 * kRows + row;
                int e[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) e[j] = p.entry(s.first + min(col + j, s.n - 1));
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (col + j >= s.n) continue;
                    float *y = a.y + (size_t)e[j] * a.H + o;
                    if (o < a.H) y[0] = v[j];
                    if (o + kRows < a.H) y[kRows] = v[4 + j];
                }
            }
        }
    };
    __device__ uint64_t *done() const { return reinterpret_cast<uint64_t *>(a.words + skinny::kDoneWord); }
    __device__ void tile_done(const skinny::Segment &s, uint32_t weight) const {
        if (s.phase == 0) skinny::count_up(a.words + kReady + s.group, weight);
        else skinny::count_up(done(), (uint64_t)weight);
    }

    // out[t] = sum_j w[t, j] y[t, j], eight columns to a thread
    __device__ bool finish() const {
        const int thread = threadIdx.x - Readers::first;
        bool ok = true;
        if (thread == 0) ok = skinny::wait_count(done(), (uint64_t)G * tiles[1] * skinny::kTileWeight, a.limits.wait_ns);
        if (!Readers::agree(ok)) return false;
        const int pieces = a.H / 8;
        const int64_t all = (int64_t)a.T * pieces;
        for (int64_t i = (int64_t)blockIdx.x * kReaders + thread; i < all;
             i += (int64_t)gridDim.x * kReaders) {
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

template <bool kE4m3, int kCols>
__global__ void __launch_bounds__(skinny::threads_of<ExpertsProblem<kE4m3, kCols>>(), 1)
    experts_kernel(const __grid_constant__ ExpertsArgs a) {
    WarpTrace wt(a.trace, MOE_TRACE_EXPERTS);
    if (threadIdx.x == 0)
        for (const CUtensorMap *m : {&a.w13, &a.w2, &a.x, &a.h_map}) tma_prefetch_map(m);
    __shared__ Lines lines;
    __shared__ Most most;
    skinny::run<kE4m3, ExpertsProblem<kE4m3, kCols>>([&](char *ring) {
        grid_dependency_wait();
        skinny::LocalPlan *plan = nullptr;
        if (a.local) {
            plan = reinterpret_cast<skinny::LocalPlan *>(ring + a.shape.used_bytes(kE4m3));
            skinny::local_plan(*plan, a.topk_idx, a.T * a.k, a.E, a.shape.cols, MOE_ERR_BAD_TOPK, a.status);
        }
        return ExpertsProblem<kE4m3, kCols>(a, plan, lines, most);
    }, a.shape, a.tmem_cols);
}

// ------------------------------------------------------------------ x as codes

struct SplitArgs {
    const __nv_bfloat16 *x;
    uint8_t *codes;      // [2T, H]: first codes, then second ones
    float *scales;       // [T, H / 128]
    uint32_t *clear;     // words zeroed for the experts kernel, or null
    int T, H, num_clear;
    TraceArgs trace;
};

// A warp to a block of 128 elements.
__global__ void __launch_bounds__(256) experts_split_kernel(const SplitArgs s) {
    WarpTrace wt(s.trace, MOE_TRACE_EXPERTS_SPLIT);
    grid_dependency_wait();
    grid_launch_dependents();   // the plan, which does not depend on this
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < s.num_clear; i += 256) s.clear[i] = 0;
    const int lane = threadIdx.x & 31;
    const int64_t block = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
    if (block >= (int64_t)s.T * (s.H / 128)) return;
    const size_t at = (size_t)block * 128 + lane * 4;
    const uint2 v = __ldg(reinterpret_cast<const uint2 *>(s.x + at));
    const float x[4] = {__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                        __uint_as_float(v.y & 0xffff0000u)};
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) most = fmaxf(most, fabsf(x[i]));   // a NaN's code is one too
    const skinny::BlockScale scale(lanes_max(most));
    uint32_t first = 0, second = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const skinny::Split two(x[i] * scale.inverse);
        first |= (two.first & 0xff) << (8 * i);
        second |= (two.second & 0xff) << (8 * i);
    }
    *reinterpret_cast<uint32_t *>(s.codes + at) = first;
    *reinterpret_cast<uint32_t *>(s.codes + (size_t)s.T * s.H + at) = second;
    if (lane == 0) s.scales[block] = scale.scale;
}

}  // namespace

size_t experts_workspace_bytes(int T, int H, int I, int k, int E) {
    // one size for both types of weights
    return std::max(space(T, H, I, k, columns(T, k, E, false), false).total,
                    space(T, H, I, k, columns(T, k, E, true), true).total);
}

namespace {
bool is_local(int T, int k, int E) { return T * k <= skinny::kLocalEntries && E <= skinny::kLocalSets; }
}  // namespace

ExpertsWords experts_words(const ExpertsLaunch &L) {
    const int n = L.num_tokens * L.num_topk;
    if (L.num_tokens == 0 || !is_local(L.num_tokens, L.num_topk, L.num_experts)) return ExpertsWords{nullptr, 0};
    return ExpertsWords{static_cast<uint32_t *>(L.workspace), kReady + n};   // the workspace's first piece
}

int launch_experts(const ExpertsLaunch &L, bool words_are_zero) {
    const int T = L.num_tokens, H = L.hidden, I = L.intermediate, k = L.num_topk, E = L.num_experts;
    if (T == 0) return MOE_OK;
    const bool e4m3 = L.w13_scales != nullptr;
    const int cols = columns(T, k, E, e4m3);
    const Space sp = space(T, H, I, k, cols, e4m3);
    char *ws = static_cast<char *>(L.workspace);
    const cudaStream_t s = static_cast<cudaStream_t>(L.stream);

    ExpertsArgs a{};
    if (!make_tensor_map(&a.w13, L.w13, e4m3, (uint64_t)E * 2 * I, H, kRows) ||
        !make_tensor_map(&a.w2, L.w2, e4m3, (uint64_t)E * H, I, kRows) ||
        !make_tensor_map(&a.x, e4m3 ? ws + sp.x_codes : L.x, e4m3, e4m3 ? 2 * T : T, H, 1) ||
        !make_tensor_map(&a.h_map, ws + sp.h, e4m3, (uint64_t)T * k * (e4m3 ? 2 : 1), I, 8))
        return MOE_ERR_CUDA;
    a.topk_idx = L.topk_idx;
    a.topk_weights = L.topk_weights;
    a.s13 = L.w13_scales;
    a.s2 = L.w2_scales;
    a.words = reinterpret_cast<uint32_t *>(ws + sp.words);
    a.groups = reinterpret_cast<const int4 *>(ws + sp.groups);
    a.order = reinterpret_cast<const int *>(ws + sp.order);
    a.h = ws + sp.h;
    a.x_scales = reinterpret_cast<const float *>(ws + sp.x_scales);
    a.h_scales = reinterpret_cast<float *>(ws + sp.h_scales);
    a.y = reinterpret_cast<float *>(ws + sp.y);
    a.partials = reinterpret_cast<float *>(ws + sp.partial);
    a.out = static_cast<__nv_bfloat16 *>(L.out);
    a.status = L.status;
    a.T = T, a.H = H, a.I = I, a.k = k, a.E = E;
    a.local = is_local(T, k, E);
    a.shape = skinny::Shape::of(cols, e4m3, skinny::kSmemBudget - (a.local ? (int)sizeof(skinny::LocalPlan) : 0));
    a.tmem_cols = a.shape.tmem_cols(e4m3);
    a.max_waves = waves_for(cols);
    a.limits = wait_limits();
    a.trace = trace_args();

    const bool overlap = tuning().overlap != 0;
    if (e4m3) {
        const bool clear = a.local && !words_are_zero;
        const SplitArgs split{static_cast<const __nv_bfloat16 *>(L.x), reinterpret_cast<uint8_t *>(ws + sp.x_codes),
                              reinterpret_cast<float *>(ws + sp.x_scales), clear ? a.words : nullptr, T, H,
                              clear ? kReady + T * k : 0, a.trace};
        const int64_t blocks = (int64_t)T * (H / 128);
        if (launch_kernel(experts_split_kernel, dim3((unsigned)((blocks + 7) / 8)), dim3(256), 0, s, overlap, split) !=
            cudaSuccess)
            return MOE_ERR_CUDA;
    }
    if (!a.local) {
        const skinny::PlanArgs<int64_t> plan{L.topk_idx, T * k, E, false, cols, a.words, kReady + T * k,
                                             const_cast<int4 *>(a.groups), const_cast<int *>(a.order), nullptr, nullptr,
                                             MOE_ERR_BAD_TOPK, e4m3 && overlap, L.status, a.trace};
        const int rc = skinny::launch_plan<false>(plan, s);
        if (rc != MOE_OK) return rc;
    } else if (!words_are_zero && !e4m3) {
        if (launch_kernel(skinny::clear_kernel, dim3(1), dim3(1024), 0, s, overlap, a.words, kReady + T * k) != cudaSuccess)
            return MOE_ERR_CUDA;
    }
    const size_t smem = a.shape.smem(e4m3) + (a.local ? sizeof(skinny::LocalPlan) : 0);
    if (!e4m3) return skinny::launch_resident(experts_kernel<false, 128>, a, skinny::threads_of<ExpertsProblem<false, 128>>(), smem, s);
    const int threads = skinny::threads_of<ExpertsProblem<true, 64>>();
    return cols <= 32 ? skinny::launch_resident(experts_kernel<true, 32>, a, threads, smem, s)
                      : skinny::launch_resident(experts_kernel<true, 64>, a, threads, smem, s);
}

}  // namespace moe
