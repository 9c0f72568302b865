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
// rows without one last, each adapter's from a multiple of 16 places on, and the
// sort kernel copies x to those places. The projection runs skinny.cuh's body
// over two lines: phase 0 multiplies the rows of one adapter in a tile (a piece)
// by its A into v; phase 1 multiplies a tile's rows by W, whatever their adapters,
// and then, as more K blocks of the same sums but of the piece's columns alone,
// each piece's v by its B. v is held as the sum of two bf16 (16 bits of it), the
// operands of two products; row by row it stays in fp32, so that a row may round
// otherwise in a batch that goes the other way. (Tiles of one adapter each ran W
// over 1.4 times as many tiles with 4096 rows of 16 adapters in runs: 312 us in all.)
// 4096 rows, 16 adapters of rank 64, 7168 x 4096: 230 us, 1.07 PFLOP/s; the plan takes 10, the copy
// 17, v about 30 and W's two rounds of tiles 175. There a block of 64 KB arrives
// every 1500 cycles where its products take 1024: L2's latency under that load, with
// 160 KB in flight, not its bandwidth (38% of peak).
//
// Row by row (few rows to an adapter): the shrink kernel makes v in fp32, four
// warps to a row of A, the expand kernel B v in fp32, a thread to a row of B, and
// the projection multiplies all rows, in their own order, by W and adds B v to
// its sums. The projection's loads depend on neither, so it is launched to
// overlap them: 128 rows, 48 adapters of rank 16, 7168 x 7168 are bound by the
// 103 MB of W and the 22 MB of adapters, 33 us (3.9 TB/s) of which the exchange of
// sums in clusters and the last stores take 8; one row, 7168 x 2048, takes 11.
#include <algorithm>
#include <climits>
#include <cmath>
#include <mutex>
#include <cuda_bf16.h>

#include "skinny.cuh"

namespace moe {
namespace {

using skinny::kRows;

// Places of the sorted rows: each adapter's (and those without one) begin at a multiple of 16.
int places(int T, int L) { return T + (skinny::kPlaceStep - 1) * std::min(L + 1, T); }

// Which way is faster, and how wide the grouped way's tiles are, by estimates in
// microseconds. They need not know the device: a workspace's size depends on them.
// A block of a tile takes its bytes of A and B at a CTA's share of what L2 gives
// them all, some 12.7 TB/s, or the tensor core's time for its columns.
constexpr double kCtas = 152;
constexpr double kGroupedLeast = 40;   // what the plan and the other launches of the grouped way take
double block_us(double ctas, int cols) {
    return std::max((2 * skinny::kHalf + cols * 128) * ctas / 12.7e6, cols * 2.2e-3);
}
// Row by row: passes over the adapters for every row, of A through the caches
// (some 4 TB/s) and of B (some 10^13 products a second), and W.
double row_us(int T, int K, int N, int r) {
    const double tiles = (double)((T + 127) / 128) * ((N + 2 * kRows - 1) / (2 * kRows)), kbs = (K + 63) / 64;
    return 15 + 1e-7 * T * r * (5.0 * K + N) +
           (tiles < kCtas ? tiles / kCtas : std::ceil(tiles / kCtas)) * kbs * block_us(kCtas, 128);
}
// Grouped: the plan and the copy of x, v by pieces, and then W (whole tiles, or
// few ones shared) with B's blocks for each piece of each tile. Half of the steps
// between adapters is padding.
double grouped_us(int T, int K, int N, int L, int r, int cols) {
    const double sets = std::min(L + 1, T), kbs = (K + 63) / 64, features = (N + 2 * kRows - 1) / (2 * kRows);
    const double rows = std::ceil((T + skinny::kPlaceStep / 2 * sets) / cols), tiles = rows * features;
    const double pieces = sets + rows, extra = pieces * features * 2 * ((r + 63) / 64);
    const double share = 2 * tiles <= kCtas ? std::floor(kCtas / tiles) : 1;
    const double block = block_us(std::min(kCtas, tiles * share), cols);
    const double w = std::ceil(tiles / kCtas) * kbs / share + extra / std::min(kCtas, tiles * share);
    return kGroupedLeast + T * 4e-6 * K / 7 + pieces * kbs / kCtas * 0.4 + w * block + (share > 1 ? 0.05 * cols : 0);
}
int grouped_columns(int T, int K, int N, int L, int r) {
    const int cols = grouped_us(T, K, N, L, r, 256) < grouped_us(T, K, N, L, r, 128) ? 256 : 128;
    return std::min((places(T, L) + 15) / 16 * 16, cols);
}
// Measured with 152 CTAs, row by row against grouped (us): 1024 rows of 8 adapters,
// 4096 x 4096, rank 16 73 : 65, rank 128 353 : 69; of 128 adapters, rank 16 79 : 112.
// Tiles of 128 columns against 256: 4096 rows of 16 adapters, 7168 x 4096 286 : 232;
// 1024 rows of 8 adapters, 4096 x 4096, rank 16 65 : 83. Close to a border either way
// may be taken: 48 adapters of rank 16, 7168 x 7168, 888 rows grouped 136, 889 row by
// row 151 (grouped 134).
constexpr int64_t kMostByRow = (int64_t)1 << 26;   // elements of out: no fp32 copy of a large one
bool grouped(int T, int K, int N, int L, int r) {
    if ((int64_t)T * N > kMostByRow) return true;
    return std::min(grouped_us(T, K, N, L, r, 128), grouped_us(T, K, N, L, r, 256)) < row_us(T, K, N, r);
}

struct Space {
    size_t words, groups, order, place, tiles, v, x, partial, total;   // byte offsets
};
constexpr int kReady = skinny::kWords;   // then a word per tile of rows: its pieces' v are done

Space grouped_space(int T, int K, int L, int r, int cols) {
    Space s{};
    skinny::Cut cut;
    const int P = places(T, L), tiles = (P + cols - 1) / cols;
    s.words = cut.take(((size_t)kReady + tiles) * 4);
    s.groups = cut.take(((size_t)tiles + std::min(L + 1, T)) * sizeof(int4));
    s.order = cut.take((size_t)P * 4);
    s.place = cut.take((size_t)T * 4);
    s.tiles = cut.take(((size_t)tiles + 1) * 4);
    s.v = cut.take((size_t)P * r * 4);               // two bf16
    s.x = cut.take((size_t)P * K * 2);               // rows of x, sorted
    s.partial = cut.take(skinny::partial_floats(2, cols) * 4);
    s.total = cut.at;
    return s;
}
Space row_space(int T, int N, int r) {
    Space s{};
    skinny::Cut cut;
    s.v = cut.take((size_t)T * r * 4);               // fp32
    s.x = cut.take((size_t)T * N * 4);               // each row's B v
    s.total = cut.at;
    return s;
}
Space space(int T, int K, int N, int L, int r) {
    return grouped(T, K, N, L, r) ? grouped_space(T, K, L, r, grouped_columns(T, K, N, L, r)) : row_space(T, N, r);
}

struct AdapterArgs {
    CUtensorMap w, a_map, b_map, x, x16, v_map;   // x: `cols` rows a box (x16: 16), of x or of its sorted copy
    const float *scales;
    uint32_t *words;
    const int4 *groups;   // grouped: pieces
    const int *order, *tile_pieces;
    void *v;   // grouped: v as two bf16; row by row: B v in fp32
    float *partials;
    __nv_bfloat16 *out;
    int32_t *status;
    int T, K, N, L, r;
    int places;  // grouped: rows of the sorted copy
    int split;   // row by row: CTAs that share a tile
    skinny::Shape shape;
    uint32_t tmem_cols;
    WaitLimits limits;
    TraceArgs trace;
};

__device__ __forceinline__ float bf16_low(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_high(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// What both ways share.
struct AdapterBase {
    static constexpr bool kHalves = true, kCodes = false;
    const AdapterArgs &a;
    int32_t *status;
    int tiles, kbs;   // feature tiles of W, K blocks of x
    __device__ explicit AdapterBase(const AdapterArgs &args) : a(args), status(args.status) {
        tiles = (a.N + 2 * kRows - 1) / (2 * kRows);
        kbs = (a.K + 63) / 64;
    }
    __device__ bool finish() const { return true; }
};

// ------------------------------------------------------------------ grouped

struct SortArgs {
    const uint4 *x;
    uint4 *sorted;
    const int *place;
    int pieces;   // 16-byte pieces of a row
    TraceArgs trace;
};

// sorted[place[t]] = x[t], one CTA per row. (Gathering the rows by TMA in the
// products' loads instead, four rows a copy, took 22 cycles a row: 2.5 times the
// whole projection's time at 128 rows to a tile.)
__global__ void __launch_bounds__(256) adapter_sort_kernel(const SortArgs s) {
    WarpTrace wt(s.trace, MOE_TRACE_ADAPTER_SORT);
    grid_dependency_wait();
    grid_launch_dependents();
    const uint4 *from = s.x + (size_t)blockIdx.x * s.pieces;
    uint4 *to = s.sorted + (size_t)s.place[blockIdx.x] * s.pieces;
#pragma unroll 4
    for (int i = threadIdx.x; i < s.pieces; i += 256) to[i] = __ldg(from + i);
}

// Shared tiles cost a CTA a hundred blocks' time or more: 256 KB of partial sums
// and as much to read, and stretches that are not at the same columns of W, so
// that L2 has to hold more of it (4096 rows of 16 adapters, 7168 x 4096: 299 us
// with equal stretches, 234 with whole tiles). Whole tiles cost a tile's blocks less than one at most.
constexpr int kWholeBlocks = 128, kSlackGrouped = 150;

struct GroupedAdapter : AdapterBase {
    static constexpr bool kShares = true, kAdders = false, kPieces = true;
    static constexpr int kReaders = 512, kPhases = 2;
    int pieces, row_tiles, rows;   // pieces with an adapter; tiles of rows, and their places
    int more;                      // K blocks of v's first part

    __device__ explicit GroupedAdapter(const AdapterArgs &args) : AdapterBase(args) {
        pieces = (int)a.words[skinny::kNamedWord];
        row_tiles = (int)a.words[skinny::kTilesWord];
        rows = (int)a.words[skinny::kPlacesWord];
        more = (a.r + 63) / 64;
    }

    __device__ float *partial(int line, int cta, int slot) const {
        return a.partials + ((size_t)(line * skinny::kMaxCtas + cta) * 2 + slot) * 2 * a.shape.cols * kRows;
    }
    __device__ uint32_t *arrivals(int line, int cta) const {
        return a.words + skinny::kArrivals + line * skinny::kMaxCtas + cta;
    }

    // Phase 0: a segment's group is a piece, its set the adapter. Phase 1: its group is
    // a tile of rows, its set the tile's first piece; the pieces' blocks follow W's in
    // the last stretch of the tile.
    template <class F>
    __device__ bool segments(F f, int first_phase = 0, int end_phase = kPhases) const {
        for (int phase = first_phase; phase < end_phase; ++phase) {
            const skinny::Line line(phase == 0 ? pieces : (int64_t)row_tiles * tiles, kbs, gridDim.x,
                                    kbs <= kWholeBlocks ? INT_MAX : kSlackGrouped);
            const bool ok = line.each(blockIdx.x, [&](int64_t tile, skinny::Segment &s) {
                s.line = s.phase = phase;
                if (phase == 0) {
                    const int4 g = a.groups[tile];
                    s.group = (int)tile;
                    s.f = 0;
                    s.set = g.x;
                    s.first = g.y;
                    s.n = g.z;
                    s.row0 = g.x * a.r;
                    s.b_from = INT_MAX;
                } else {
                    s.group = (int)skinny::quotient(tile, tiles);
                    s.f = (int)(tile - (int64_t)s.group * tiles);
                    s.set = a.tile_pieces[s.group];
                    s.first = s.group * a.shape.cols;
                    s.n = min(a.shape.cols, rows - s.first);
                    s.row0 = s.f * 2 * kRows;
                    s.b_from = kbs;
                    const int extra = tile_pieces(s) * 2 * more;
                    if (s.kb1 == kbs) s.kb1 += extra;
                    s.kbs += extra;
                }
                s.two = phase == 1;
                s.row1 = s.row0 + kRows;
                return f(s);
            });
            if (!ok) return false;
        }
        return true;
    }
    __device__ int tile_pieces(const skinny::Segment &s) const {
        return max(0, min(a.tile_pieces[s.group + 1], pieces) - s.set);
    }
    // Block kb of phase 1, behind W's: v's first parts of a piece (more blocks), then its second ones.
    __device__ int4 piece(const skinny::Segment &s, int kb) const { return a.groups[s.set + (kb - kbs) / 2 / more]; }
    __device__ int v_block(int kb) const { return more == 1 ? 0 : (kb - kbs) & 1; }
    __device__ int v_part(int kb) const { return more == 1 ? (kb - kbs) & 1 : (kb - kbs) >> 1 & 1; }

    __device__ void a_load(const skinny::Segment &s, int kb, uint32_t dst, uint64_t *bar, uint64_t policy) const {
        if (s.phase == 0) {
            mbar_arrive_expect_tx(bar, a.r * 128);
            tma_load(dst, &a.a_map, kb * 64, s.row0, bar, policy);
            return;
        }
        const bool is_w = kb < kbs;
        const CUtensorMap *map = is_w ? &a.w : &a.b_map;
        const int col = is_w ? kb * 64 : v_block(kb) * 64, row = is_w ? s.row0 : piece(s, kb).x * a.N + s.row0;
        mbar_arrive_expect_tx(bar, 2 * skinny::kHalf);
        tma_load(dst, map, col, row, bar, policy);
        tma_load(dst + skinny::kHalf, map, col, row + kRows, bar, policy);
    }
    struct Rows {};
    __device__ Rows b_rows(const skinny::Segment &, int) const { return Rows{}; }
    __device__ bool b_ready(const skinny::Segment &s) const {
        return skinny::wait_count(a.words + kReady + s.group, skinny::kTileWeight * tile_pieces(s), a.limits.wait_ns);
    }
    __device__ uint32_t b_bytes(const skinny::Segment &s, int kb) const {
        if (s.phase == 0) return s.n16() * 128;
        return kb < kbs ? a.shape.cols * 128 : (piece(s, kb).z + 7) / 8 * 1024;
    }
    __device__ void b_load(const skinny::Segment &s, const Rows &, int kb, uint32_t dst, uint64_t *bar, uint64_t policy,
                           int lane) const {
        if (s.phase == 0) {
            if (16 * lane < s.n) tma_load(dst + lane * 2048, &a.x16, kb * 64, s.first + 16 * lane, bar, policy);
        } else if (kb < kbs) {
            if (lane == 0) tma_load(dst, &a.x, kb * 64, s.first, bar, policy);
        } else {
            const int4 g = piece(s, kb);   // v's first parts [places, r], then the second ones
            if (8 * lane < g.z)
                tma_load(dst + lane * 1024, &a.v_map, v_block(kb) * 64, v_part(kb) * a.places + g.y + 8 * lane, bar, policy);
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
                    v[(size_t)a.places * a.r + at] = __float2bfloat16_rn(isfinite(rest) ? rest : 0.0f);
                }
                return;
            }
            const int o = s.row0 + half * kRows + row;
            if (o >= a.N) return;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int t = col + j < s.n ? a.order[s.first + col + j] : -1;
                if (t >= 0) a.out[(size_t)t * a.N + o] = __float2bfloat16_rn(sums[j]);
            }
        }
    };
    __device__ void tile_done(const skinny::Segment &s, uint32_t weight) const {
        if (s.phase == 0) skinny::count_up(a.words + kReady + s.first / a.shape.cols, weight);
    }
};

__global__ void __launch_bounds__(skinny::threads_of<GroupedAdapter>(), 1)
    adapter_grouped_kernel(const __grid_constant__ AdapterArgs a) {
    WarpTrace wt(a.trace, MOE_TRACE_ADAPTER);
    if (threadIdx.x == 0)
        for (const CUtensorMap *m : {&a.w, &a.x, &a.x16, &a.a_map, &a.b_map, &a.v_map}) tma_prefetch_map(m);
    skinny::run<false, GroupedAdapter>([&](char *) {
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
    int K, L, r;
    int32_t *status;
    TraceArgs trace;
};

// v = scale * (A x), for every row of x. Rows of A to a CTA: two groups of four
// warps, a quarter of K to a warp, four rows to a warp. The loads of A and x bound
// it, from HBM the first time an adapter's rows are used and from L2 then: 128 rows,
// 48 adapters of rank 16, K = 7168: 10 us with all of it in HBM.
constexpr int kShrinkRows = 8;

__global__ void __launch_bounds__(256) adapter_shrink_kernel(const ShrinkArgs s) {
    WarpTrace wt(s.trace, MOE_TRACE_ADAPTER_SHRINK);
    grid_dependency_wait();
    grid_launch_dependents();   // the projection's loads, of inputs that are complete by now
    __shared__ float sums[8][4];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = (s.r + kShrinkRows - 1) / kShrinkRows;
    const int t = blockIdx.x / per, row0 = (blockIdx.x - t * per) * kShrinkRows;
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

struct ExpandArgs {
    const __nv_bfloat16 *b;
    const int32_t *idx;
    const float *v;      // [T, r]
    float *delta;        // [T, N]
    int T, N, L, r;
    TraceArgs trace;
};

constexpr int kExpandRows = 4;   // rows of x to a CTA, which has 256 rows of B

// delta[t] = B v[t], 0 without an adapter: a thread has one row of B, its loads
// for the CTA's rows of x all at once for every 8 of the rank. Bound by those loads:
// 128 rows, 48 adapters of rank 16, N = 7168: 11 us with all of it in HBM.
__global__ void __launch_bounds__(256) adapter_expand_kernel(const ExpandArgs e) {
    WarpTrace wt(e.trace, MOE_TRACE_ADAPTER_EXPAND);
    __shared__ float v[kExpandRows][MOE_MAX_ADAPTER_RANK];
    const int tiles = (e.N + 255) / 256;
    const int t0 = blockIdx.x / tiles * kExpandRows, o = (blockIdx.x % tiles) * 256 + threadIdx.x;
    grid_launch_dependents();   // the projection's loads, before the shrink kernel ends
    grid_dependency_wait();
    int id[kExpandRows];
#pragma unroll
    for (int j = 0; j < kExpandRows; ++j) {
        id[j] = t0 + j < e.T ? e.idx[t0 + j] : -1;
        if (id[j] >= e.L) id[j] = -1;
    }
    for (int i = threadIdx.x; i < kExpandRows * e.r; i += 256) {
        const int j = i / e.r, c = i - j * e.r;
        if (t0 + j < e.T) v[j][c] = e.v[(size_t)(t0 + j) * e.r + c];
    }
    __syncthreads();
    if (o >= e.N) return;
    const __nv_bfloat16 *b = e.b + (size_t)o * e.r;
    const size_t set = (size_t)e.N * e.r;
    float acc[kExpandRows] = {};
#pragma unroll 2
    for (int c = 0; c < e.r; c += 8) {
        uint4 w[kExpandRows];
#pragma unroll
        for (int j = 0; j < kExpandRows; ++j)
            if (id[j] >= 0) w[j] = __ldg(reinterpret_cast<const uint4 *>(b + id[j] * set + c));
#pragma unroll
        for (int j = 0; j < kExpandRows; ++j) {
            if (id[j] < 0) continue;
            const uint32_t q[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                acc[j] = fmaf(bf16_low(q[k]), v[j][c + 2 * k], acc[j]);
                acc[j] = fmaf(bf16_high(q[k]), v[j][c + 2 * k + 1], acc[j]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < kExpandRows; ++j)
        if (t0 + j < e.T) e.delta[(size_t)(t0 + j) * e.N + o] = acc[j];
}

// Where tiles are fewer than CTAs, a cluster of `split` CTAs shares a tile, each
// with a stretch of K; else CTAs take whole tiles in turn.
struct RowAdapter : AdapterBase {
    static constexpr bool kShares = false, kAdders = false, kPieces = false;
    static constexpr int kReaders = 256;
    int chunks;
    __device__ explicit RowAdapter(const AdapterArgs &args) : AdapterBase(args) {
        chunks = (a.T + a.shape.cols - 1) / a.shape.cols;
    }

    // The one segment of a CTA of a cluster.
    __device__ skinny::Segment of_tile(int64_t tile) const {
        skinny::Segment s;
        s.line = s.phase = s.set = 0;
        s.group = (int)skinny::quotient(tile, tiles);
        s.f = (int)(tile - (int64_t)s.group * tiles);
        s.first = s.group * a.shape.cols;
        s.n = min(a.shape.cols, a.T - s.first);
        s.two = true;
        s.row0 = s.f * 2 * kRows;
        s.row1 = s.row0 + kRows;
        s.b_from = INT_MAX;
        s.kb0 = 0;
        s.kb1 = s.kbs = kbs;
        return s;
    }
    template <class F>
    __device__ bool segments(F f) const {
        if (a.split > 1) {
            const int rank = blockIdx.x % a.split, per = (kbs + a.split - 1) / a.split;
            skinny::Segment s = of_tile(blockIdx.x / a.split);
            s.kb0 = rank * per;
            s.kb1 = min(kbs, s.kb0 + per);
            return f(s);
        }
        for (int64_t tile = blockIdx.x; tile < (int64_t)chunks * tiles; tile += gridDim.x)
            if (!f(of_tile(tile))) return false;
        return true;
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

    struct Emit {
        const AdapterArgs &a;
        const skinny::Segment &s;
        int o;   // this thread's row of W
        __device__ Emit(const RowAdapter &p, const skinny::Segment &seg, const skinny::Share<true> &me)
            : a(p.a), s(seg), o(seg.row0 + (me.side & 1) * kRows + me.row) {}
        __device__ void operator()(int col, const float *sums) const {
            if (o >= a.N) return;
            const size_t at = (size_t)(s.first + col) * a.N + o;
            const float *delta = static_cast<const float *>(a.v) + at;   // complete since the readers' dependency wait
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = col + j < s.n ? delta[(size_t)j * a.N] : 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (col + j < s.n) a.out[at + (size_t)j * a.N] = __float2bfloat16_rn(sums[j] + x[j]);
        }
    };
};

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Sums of a tile whose K a cluster shares: each CTA sends its sums of the
// columns that another will finish to that CTA's shared memory (the ring, which
// no load or product uses any more), and adds up its own in the order of K.
// Through L2 instead (partial sums, a counter, loads of all parts) this took
// 18 us of 44 at 128 rows, 7168 x 7168.
__device__ void finish_in_cluster(const RowAdapter &p, skinny::Control &c, char *ring, const skinny::Segment &s,
                                  uint32_t tmem, bool &ok) {
    using Tm = skinny::ReadersOf<RowAdapter>;
    const AdapterArgs &a = p.a;
    const skinny::Shape sh = a.shape;
    const bool reader = threadIdx.x >= Tm::first;
    const skinny::Share<true> me = skinny::Share<true>::of(Tm::warp());
    const int split = a.split, rank = blockIdx.x % split, half = me.side & 1;
    const int steps = s.n16() / 16, kept = (steps + split - 1) / split;   // steps of 16 columns, and of them one CTA's
    constexpr int kStep = 16 * 2 * kRows;                                 // floats of a step: [column][half][row]
    if (reader) {
        ok = Tm::agree(skinny::wait(&c.sums_full[0], 0, a.limits.wait_ns));
        tc_fence_after();
    }
    cluster_sync();   // every ring of the cluster is free
    if (reader && ok) {
        const uint32_t at = tmem + ((uint32_t)(me.row & ~31) << 16);
        const uint32_t base = smem_addr(ring);
        for (int col = 0; col < s.n16(); col += 8) {
            float v[8];
            me.load(at, sh.cols, col, v);
            const int step = col / 16;
            uint32_t to;   // [part][step of the owner][column][half][row]
            const uint32_t mine = base + (((rank * kept + step / split) * kStep) + ((col & 8) * 2 + half) * kRows + me.row) * 4;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(mine), "r"(step % split));
#pragma unroll
            for (int j = 0; j < 8; ++j)
                asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + j * 2 * kRows * 4), "f"(v[j]) : "memory");
        }
    }
    cluster_sync();   // all parts have arrived
    if (reader && ok) {
        const float *parts = reinterpret_cast<const float *>(ring);
        const RowAdapter::Emit emit(p, s, me);
        for (int step = rank, k = 0; step < steps; step += split, ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int col = step * 16 + h * 8;
                if (col >= s.n) break;
                float v[8] = {};
                for (int i = 0; i < split; ++i) {
                    const float *part = parts + (i * kept + k) * kStep + (h * 16 + half) * kRows + me.row;
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] += part[j * 2 * kRows];
                }
                emit(col, v);
            }
    }
}

// Loads of x and W begin while the two kernels before it run: the shrink kernel
// passed its own dependency wait before it let the next start, so all that came
// before it is complete, and neither writes x or W. At most half of an SM's
// registers, so that their CTAs fit beside it.
template <bool kCluster>
__global__ void __launch_bounds__(skinny::threads_of<RowAdapter>(), 2)
    adapter_row_kernel(const __grid_constant__ AdapterArgs a) {
    WarpTrace wt(a.trace, MOE_TRACE_ADAPTER);
    if (threadIdx.x == 0)
        for (const CUtensorMap *m : {&a.w, &a.x}) tma_prefetch_map(m);
    auto make = [&](char *) {
        if (threadIdx.x >= skinny::ReadersOf<RowAdapter>::first) grid_dependency_wait();   // B v
        return RowAdapter(a);
    };
    if constexpr (kCluster)
        skinny::run_one<RowAdapter>(make, a.shape, a.tmem_cols, [](const RowAdapter &p, skinny::Control &c, char *ring,
                                                                   uint32_t tmem, bool &ok) {
            p.segments([&](const skinny::Segment &s) {
                finish_in_cluster(p, c, ring, s, tmem, ok);
                return true;
            });
        });
    else
        skinny::run<false, RowAdapter>(make, a.shape, a.tmem_cols);
}

// Clusters of n CTAs of the row kernel that fit on the device at once, cached per device.
int clusters_at_once(int n) {
    static std::mutex mu;
    static int known[64][skinny::kMaxSplit + 1];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    std::lock_guard<std::mutex> lock(mu);
    int &v = known[dev][n];   // 0: not asked yet, else the answer + 1
    if (v == 0) {
        const size_t smem = 1024 + skinny::kSmemBudget;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(n);
        cfg.blockDim = dim3(skinny::threads_of<RowAdapter>());
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim = {(unsigned)n, 1, 1};
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int fit = 0;
        if (ensure_dynamic_smem((const void *)adapter_row_kernel<true>, smem) != MOE_OK ||
            cudaOccupancyMaxActiveClusters(&fit, adapter_row_kernel<true>, &cfg) != cudaSuccess) {
            cudaGetLastError();
            fit = 0;
        }
        v = fit + 1;
    }
    return v - 1;
}

// Columns of a tile and the CTAs that share one. Wider tiles stream W less
// often, narrower ones and larger clusters spread the work over more CTAs: about
// 65 KB a microsecond to a CTA, a microsecond for each 16 columns that it
// finishes and three for a cluster's exchange (measured).
void choose_tiles(int T, int K, int N, int &cols, int &split) {
    const int most = std::min((T + 15) / 16 * 16, 128), kbs = (K + 63) / 64;
    const int64_t ctas = std::min(device_sm_count(), skinny::kMaxCtas);
    double least = 0.0;
    for (int c = most; c >= 16; c = c > 16 ? std::max(16, c / 32 * 16) : 0)
        for (int n = 1; n <= skinny::kMaxSplit; n *= 2) {   // five to a cluster came in two waves on these GPCs
            const int64_t tiles = ((int64_t)T + c - 1) / c * ((N + 2 * kRows - 1) / (2 * kRows));
            if (n > 1 && (kbs < 2 * n || tiles > clusters_at_once(n) || (kbs + n - 1) / n * (n - 1) >= kbs)) continue;
            const int64_t rounds = n > 1 ? 1 : (tiles + ctas - 1) / ctas;
            const double us = (double)rounds * ((kbs + n - 1) / n * (2 * skinny::kHalf + c * 128) / 65e3 +
                                                (c / 16 + n - 1) / n) + (n > 1 ? 3.0 : 0.0);
            if (least == 0.0 || us < least) least = us, cols = c, split = n;
        }
}

}  // namespace

size_t adapter_workspace_need(int T, int K, int N, int L, int r) { return space(T, K, N, L, r).total; }

// Room for any number of rows up to T, though the ways and widths change back and
// forth between them: the row by row way's for as many as it may have, and the
// grouped way's in its widest tiles, if it comes into question for any, which it
// does not while row_us, which grows with the rows, is below the least that it takes.
size_t adapter_workspace_bytes(int T, int K, int N, int L, int r) {
    if (T == 0) return 0;
    size_t most = row_space((int)std::min<int64_t>(T, kMostByRow / N), N, r).total;
    if (T * (int64_t)N > kMostByRow || row_us(T, K, N, r) > kGroupedLeast)
        most = std::max(most, grouped_space(T, K, L, r, std::min((places(T, L) + 15) / 16 * 16, 256)).total);
    return most;
}

int launch_adapter_linear(const AdapterLaunch &L) {
    const int T = L.num_tokens, K = L.in_features, N = L.out_features, r = L.rank;
    if (T == 0) return MOE_OK;
    const bool by_group = grouped(T, K, N, L.num_adapters, r);
    const Space sp = space(T, K, N, L.num_adapters, r);
    char *ws = static_cast<char *>(L.workspace);
    const cudaStream_t s = static_cast<cudaStream_t>(L.stream);
    const bool overlap = tuning().overlap != 0;
    const int P = places(T, L.num_adapters);
    int cols = by_group ? grouped_columns(T, K, N, L.num_adapters, r) : 0, split = 1;
    if (!by_group) choose_tiles(T, K, N, cols, split);

    AdapterArgs a{};
    bool ok = make_tensor_map(&a.w, L.w, false, N, K, kRows) &&
              make_tensor_map(&a.x, by_group ? ws + sp.x : L.x, false, by_group ? P : T, K, cols);
    if (by_group)
        ok = ok && make_tensor_map(&a.a_map, L.a, false, (uint64_t)L.num_adapters * r, K, r) &&
             make_tensor_map(&a.b_map, L.b, false, (uint64_t)L.num_adapters * N, r, kRows) &&
             make_tensor_map(&a.x16, ws + sp.x, false, P, K, 16) &&
             make_tensor_map(&a.v_map, ws + sp.v, false, (uint64_t)2 * P, r, 8);
    if (!ok) return MOE_ERR_CUDA;
    a.scales = L.scales;
    a.v = ws + (by_group ? sp.v : sp.x);
    a.out = static_cast<__nv_bfloat16 *>(L.out);
    a.status = L.status;
    a.T = T, a.K = K, a.N = N, a.L = L.num_adapters, a.r = r, a.places = P, a.split = split;
    a.shape = skinny::Shape::of(cols, false);
    a.tmem_cols = a.shape.tmem_cols(false);
    a.limits = wait_limits();
    a.trace = trace_args();
    const size_t smem = a.shape.smem(false);

    if (by_group) {
        a.words = reinterpret_cast<uint32_t *>(ws + sp.words);
        a.groups = reinterpret_cast<const int4 *>(ws + sp.groups);
        a.order = reinterpret_cast<const int *>(ws + sp.order);
        a.tile_pieces = reinterpret_cast<const int *>(ws + sp.tiles);
        a.partials = reinterpret_cast<float *>(ws + sp.partial);
        int *const place = reinterpret_cast<int *>(ws + sp.place);
        const skinny::PlanArgs<int32_t> plan{L.adapter_idx, T, L.num_adapters, true, cols, a.words,
                                             kReady + (P + cols - 1) / cols, const_cast<int4 *>(a.groups),
                                             const_cast<int *>(a.order), place, const_cast<int *>(a.tile_pieces),
                                             MOE_ERR_BAD_ADAPTER, false, L.status, a.trace};
        const int rc = skinny::launch_plan<true>(plan, s);
        if (rc != MOE_OK) return rc;
        const SortArgs so{static_cast<const uint4 *>(L.x), reinterpret_cast<uint4 *>(ws + sp.x), place, K / 8, a.trace};
        if (launch_kernel(adapter_sort_kernel, dim3(T), dim3(256), 0, s, overlap, so) != cudaSuccess) return MOE_ERR_CUDA;
        return skinny::launch_resident(adapter_grouped_kernel, a, skinny::threads_of<GroupedAdapter>(), smem, s);
    }
    const ShrinkArgs sh{static_cast<const __nv_bfloat16 *>(L.x), static_cast<const __nv_bfloat16 *>(L.a),
                        L.adapter_idx, L.scales, reinterpret_cast<float *>(ws + sp.v), K, L.num_adapters, r,
                        L.status, a.trace};
    const ExpandArgs ex{static_cast<const __nv_bfloat16 *>(L.b), L.adapter_idx, sh.v, static_cast<float *>(a.v), T, N,
                        L.num_adapters, r, a.trace};
    const int64_t shrinks = (int64_t)T * ((r + kShrinkRows - 1) / kShrinkRows);
    const int64_t expands = (int64_t)((N + 255) / 256) * ((T + kExpandRows - 1) / kExpandRows);
    const void *kernel = split > 1 ? (const void *)adapter_row_kernel<true> : (const void *)adapter_row_kernel<false>;
    const int rc = ensure_dynamic_smem(kernel, smem);
    if (rc != MOE_OK) return rc;
    if (launch_kernel(adapter_shrink_kernel, dim3((unsigned)shrinks), dim3(256), 0, s, overlap, sh) != cudaSuccess ||
        launch_kernel(adapter_expand_kernel, dim3((unsigned)expands), dim3(256), 0, s, overlap, ex) != cudaSuccess)
        return MOE_ERR_CUDA;
    const int64_t tiles = (int64_t)((T + cols - 1) / cols) * ((N + 2 * kRows - 1) / (2 * kRows));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(split > 1 ? tiles * split : std::min<int64_t>(tiles, device_sm_count())));
    cfg.blockDim = dim3(skinny::threads_of<RowAdapter>());
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (split > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n++].val.clusterDim = {(unsigned)split, 1, 1};
    }
    if (overlap) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    void *args[] = {&a};
    return cudaLaunchKernelExC(&cfg, kernel, args) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe
