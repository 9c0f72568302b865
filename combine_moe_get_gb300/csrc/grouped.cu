// grouped.cu -- matrix products grouped by expert, with ragged numbers of rows:
// the rows of expert e are [prefix[e], prefix[e+1]) (the expand layout's order).
//
//   forward     y[r]  = w[e] x[r]                 D = 128 features of w[e] x n rows, over K
//   gradient    dx[r] = w[e]^T dy[r]              D = 128 columns of w[e] x n rows, over N
//   of weights  dw[e] = sum over r of dy[r] x[r]^T   D = 128 rows of dw[e] x up to 256 columns, over the expert's rows
//
// The ragged side is the tensor core's n, which goes in steps of 16, so that an
// expert with 140 rows costs 144 and not 256; features fill its fixed 128 rows,
// or 256 of a pair of CTAs that work as one (each holds half of both operands, which
// halves what a block takes from L2: 128 x 128 tiles of single CTAs ran at 1.13
// PFLOP/s where pairs' 256 x 256 run at 1.6 to 1.7, 16384 rows, 32 experts, 7168 x 4096;
// one expert 1.8, where a dense library product has 1.9). One persistent CTA per SM;
// each finds its tiles by a scan over the experts' numbers of rows, which stay on
// the device. Few rows to an expert are bound by reading the weights: 128 a piece 6.5
// to 7.0 TB/s, four a piece in E4M3 6.6.
//
// Roles of a CTA's warps: 0 loads both operands by TMA, 1 issues the products,
// 2 owns the tensor memory and finds the tiles, 3 prepares what the products
// need besides (weights' gradients: zeros in place of the next expert's rows;
// E4M3: scales), 4 to 11 (E4M3: to 15) read the sums.
//
// E4M3 has an fp32 scale for each row and feature and 128 of the reduction, so a
// block's sums leave the tensor core unscaled, into registers, where they are
// multiplied by the product of their two scales and added: two operations for each of
// D's elements and block, 128 x n of them while the pair's products take 2 n cycles.
// That is all that the ordinary cores have to give, so these readers bound E4M3 where
// rows are many: 1.77 to 1.86 PFLOP/s (the rate without them 3.2, without their
// arithmetic 2.7), and what helped was fewer instructions and waits around it.
//
// The tensor core's sums are fp32, but of each 16 products what lies below 2^-25 of
// the sum's leading bit is cut off, as in a library's bf16 products: off by 5e-7 of
// their norm over 512 rows, 2e-5 over 16384 (8e-5 where all have one sign), where one
// CTA has them all. fp32 sums of dW show it; bf16's rounding covers it to some 2^17 rows.
#include <algorithm>
#include <atomic>
#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>

#include "umma.cuh"

namespace moe {
namespace grouped {

constexpr int kFirstReader = 4;            // first of the warps that read sums
constexpr int kRows = 128;                 // features of a CTA's tile
constexpr int kTileA = kRows * 128;        // bytes of A in a stage
constexpr int kTileSlots = 4;              // tiles found ahead
constexpr int kSmemBudget = 226 << 10;     // ring, what stands beside it, and 1 KB to align them
constexpr int kScaleSlots = 2;             // E4M3: scales of four blocks each
constexpr int kBoxRows = 32;               // rows of one copy of the ragged operand
constexpr int kDepth = 64;                 // bf16 elements of a block along the reduction (E4M3: 128)
constexpr int kRowGroup = 8;               // row tiles that share a pass over the features

enum Op { kForward, kForwardE4m3, kGradX, kGradW };

struct Tile {
    int e;          // -1: no more
    int a0;         // first feature of the pair's (or CTA's) tile
    int row0;       // first row
    int n;          // rows (weights' gradients: columns) of the tile
    int c0;         // weights' gradients: first column
    int kb0, blocks;   // first block along the reduction, and how many (weights' gradients: the expert's, and this CTA's of them)
    int last;          // weights' gradients: rows in the last block
};

struct Args {
    CUtensorMap a, b;
    CUtensorMap a16, b16, out_map;      // weights' gradients: operands 16 rows at a time, the result in bf16
    const int32_t *prefix;
    const float *a_scales, *b_scales;   // E4M3: [E, N, K/128] and [M, K/128]
    void *out;
    int32_t *status;
    int E, M;
    int features, depth;     // rows of D over all tiles, length of the reduction (weights' gradients: columns of D)
    int feature_tiles, column_tiles;
    int blocks;              // along the whole reduction (rows of scales are this long)
    int split, per_split;    // CTAs of a cluster that share a tile's reduction, and the blocks of each
    bool read_once;          // hardly any expert has rows for two tiles: its weights pass once
    bool accumulate;
    WaitLimits limits;
    TraceArgs trace;
};

// CTAs (pairs) that share a tile's reduction at most, and each one's part of a shared tile's n columns.
constexpr int most_split(int ctas) { return ctas == 2 ? 4 : 8; }
__host__ __device__ constexpr int shared_width(int n, int split) { return ((n + split - 1) / split + 7) & ~7; }
// Bytes of a CTA's sums of n columns with the others' of its own.
constexpr int shared_bytes(int n, int split) { return (n + (split - 1) * shared_width(n, split)) * kRows * 4; }

// kCols: the most columns of a tile. kCtas: CTAs of a cluster that work on one tile of kCtas * 128 features,
// each with its part of the columns' operand.
template <Op kOp, int kCtas, int kCols>
struct Config {
    static constexpr bool kE4m3 = kOp == kForwardE4m3;
    static constexpr int kReaders = kE4m3 ? 12 : 8, kThreads = (kFirstReader + kReaders) * 32;
    static constexpr int kSides = kReaders / 4;   // a quarter of the lanes is read by as many warps, 16 columns in turn
    static constexpr int kTileB = (kCols / kCtas + kBoxRows - 1) / kBoxRows * kBoxRows * 128;
    static constexpr int kSums = kE4m3 ? (512 / kCols < 4 ? 512 / kCols : 4) : 2;
    static constexpr int kScales = kCols + kRows;   // E4M3: scales of a block's rows and features
    static constexpr int kScaleBytes = kE4m3 ? kScaleSlots * 4 * kScales * 4 : 0;
    static constexpr int kStore = kE4m3 ? 16 * 64 : kOp == kGradW ? 32 * 128 : 0;   // what a warp of readers has on its way out
    static constexpr int kBeside = kScaleBytes + kReaders * kStore;
    static constexpr int kFit = (kSmemBudget - 1024 - kBeside) / (kTileA + kTileB);
    static constexpr int kStages = kFit < 12 ? kFit : 12;
    static constexpr int kTmemCols = kSums * kCols <= 64 ? 64 : kSums * kCols <= 128 ? 128 : kSums * kCols <= 256 ? 256 : 512;
    static constexpr int kBlock = kE4m3 ? 128 : kDepth;
    static constexpr size_t smem() { return 1024 + (size_t)kStages * (kTileA + kTileB) + kBeside; }
    static_assert(kStages >= 3 && kSums >= 2);
    // a shared tile's sums take the ring's place, and for 256 columns and four pairs that of what stands beside it too
    static constexpr int kShared = kStages * (kTileA + kTileB) + kBeside;
    static_assert(shared_bytes(kCols, 2) <= kShared && shared_bytes(kCols, 4) <= kShared && shared_bytes(kCols, most_split(kCtas)) <= kShared);
    // who takes a tile from the scan: loads, products (one CTA of a pair), warp 3 (if it has work), readers
    static constexpr bool kHelper = kOp == kGradW || kE4m3;
};

constexpr int kMaxStages = 12, kMaxSums = 4;
struct Control {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t masked_full[kMaxStages];   // a block whose rows past the expert's end are to be zeroed
    uint64_t sums_full[kMaxSums], sums_empty[kMaxSums];
    uint64_t scales_full[kScaleSlots], scales_empty[kScaleSlots];
    uint64_t tile_full[kTileSlots], tile_empty[kTileSlots];
    uint64_t last;
    uint64_t parts;   // a shared tile's sums from the other CTAs
    Tile tiles[kTileSlots];
    uint32_t tmem;
};

// ------------------------------------------------------------------ PTX of pairs

__device__ __forceinline__ uint32_t peer_addr(const void *p, uint32_t rank) {   // of the cluster's CTA `rank`
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr(p)), "r"(rank));
    return r;
}
// ... of the CTA whose products these are: its pair's first (a cluster's neighbours are pairs), or this one.
__device__ __forceinline__ uint32_t first_of_pair() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r & ~1u;
}
template <int kCtas>
__device__ __forceinline__ uint32_t home_addr(const void *p) {
    return kCtas == 2 ? peer_addr(p, first_of_pair()) : smem_addr(p);
}
// Arrivals and waits have the CTA's scope: what they order, tensor memory and shared memory that TMA and the products
// touch, is ordered by those units' own barriers and fences. (With the cluster's scope each wait took L1 with it: 2.5
// times slower.) The zeros of mask_blocks are no exception: fence.proxy.async has them in this CTA's shared memory, where
// its own tensor core reads them, before the arrival leaves (one with the cluster's scope cost a sixth of the kernel's time).
__device__ __forceinline__ void arrive_at(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void arrive_expect_at(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, uint64_t ns) {
    return mbar_wait_bounded(bar, parity, ns);
}
__device__ __forceinline__ bool arrived(uint64_t *bar, uint32_t parity) {
    uint32_t yes;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(yes) : "r"(smem_addr(bar)), "r"(parity) : "memory");
    return yes != 0;
}
// By a whole warp, which goes on or gives up as one. What is waited for has often happened: the rest stays out of the
// way of the code around (E4M3's readers were 4% slower with it in each place).
__device__ __noinline__ bool warp_wait_longer(uint64_t *bar, uint32_t parity, uint64_t ns) {
    return __all_sync(0xffffffffu, wait(bar, parity, ns));
}
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, uint64_t ns) {
    return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) || warp_wait_longer(bar, parity, ns);
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Tiles by TMA; `bar` is a shared::cluster address, of this CTA or its pair's first.
template <int kCtas>
__device__ __forceinline__ void load2(uint32_t dst, const CUtensorMap *map, int c0, int c1, uint32_t bar, uint64_t policy) {
    if constexpr (kCtas == 2)
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
            "[%0], [%1, {%2, %3}], [%4], %5;"
            ::"r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(bar), "l"(policy) : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
            "[%0], [%1, {%2, %3}], [%4], %5;"
            ::"r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(bar), "l"(policy) : "memory");
}
template <int kCtas>
__device__ __forceinline__ void load3(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, uint32_t bar,
                                      uint64_t policy) {
    if constexpr (kCtas == 2)
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
            "[%0], [%1, {%2, %3, %4}], [%5], %6;"
            ::"r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar), "l"(policy) : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
            "[%0], [%1, {%2, %3, %4}], [%5], %6;"
            ::"r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar), "l"(policy) : "memory");
}

template <int kCtas>
__device__ __forceinline__ void tmem_take(uint32_t *slot, uint32_t cols) {
    if constexpr (kCtas == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_addr(slot)), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
        tmem_alloc(slot, cols);
    }
}
template <int kCtas>
__device__ __forceinline__ void tmem_give(uint32_t base, uint32_t cols) {
    if constexpr (kCtas == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols));
    else
        tmem_free(base, cols);
}

// Operand whose rows of 128 bytes are steps of the reduction, 64 bf16 of M or N each (128-byte swizzle): 8 steps are
// 1024 bytes apart (the high word's stride), the next 64 of M or N `chunk` bytes (the low word's).
__device__ __forceinline__ uint32_t operand_low_mn(uint32_t addr, uint32_t chunk) {
    return ((addr >> 4) & 0x3fff) | (chunk >> 4) << 16;
}

template <int kCtas, bool kE4m3>
__device__ __forceinline__ void product(uint32_t d, uint32_t a_low, uint32_t b_low, uint32_t desc, bool add) {
    if constexpr (kCtas == 1) {
        if constexpr (kE4m3) mma_e4m3(d, a_low, b_low, desc, add);
        else mma_ss(d, a_low, b_low, desc, add);
    } else if constexpr (kE4m3) {
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
            ::"r"(d), "l"(operand_desc(a_low)), "l"(operand_desc(b_low)), "r"(desc), "r"((uint32_t)add) : "memory");
    } else {
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
            ::"r"(d), "l"(operand_desc(a_low)), "l"(operand_desc(b_low)), "r"(desc), "r"((uint32_t)add) : "memory");
    }
}
// One arrival on `bar` of each CTA of the tile when the products so far are complete.
template <int kCtas>
__device__ __forceinline__ void commit(uint64_t *bar) {
    if constexpr (kCtas == 2)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
            ::"r"(smem_addr(bar)), "h"((uint16_t)(3u << first_of_pair())) : "memory");
    else
        mma_commit(bar);
}

// ... of this CTA's alone.
template <int kCtas>
__device__ __forceinline__ void commit_here(uint64_t *bar) {
    if constexpr (kCtas == 2)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                     ::"r"(smem_addr(bar)) : "memory");
    else
        mma_commit(bar);
}

__device__ __forceinline__ void tmem_load16(uint32_t addr, float *v) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// ------------------------------------------------------------------ tiles

__device__ __forceinline__ int round16(int n) { return (n + 15) & ~15; }
// Columns of a tile's products: weights' gradients load theirs 64 at a time into each CTA.
template <Op kOp, int kCtas>
__device__ __forceinline__ int columns_of(const Tile &t) {
    return kOp == kGradW ? (t.n + kCtas * 64 - 1) / (kCtas * 64) * (kCtas * 64) : round16(t.n);
}

// Rows of expert e, whatever the prefix holds: inside [0, M], none where it descends.
struct Range {
    int lo, hi;
    bool bad;
};
__device__ __forceinline__ Range rows_of(const Args &a, int e) {
    const int p0 = __ldg(a.prefix + e), p1 = __ldg(a.prefix + e + 1);
    Range r;
    r.lo = min(max(p0, 0), a.M);
    r.hi = min(max(p1, r.lo), a.M);
    r.bad = r.lo != p0 || r.hi != p1;
    return r;
}

// Rows of 32 experts of a wrong prefix, a lane each, without those before the end of earlier experts' rows, so that no row
// has two writers, and there are no more tiles than most_row_tiles (clusters that share tiles take one each). Returns {lo, hi,
// the end of all so far}; `end` is what it was before these 32, kNoEnd behind a prefix without a fault, where the first one's
// start tells if any had rows (`some`).
constexpr int kNoEnd = -1;
static __device__ __noinline__ int3 behind_earlier(int lo, int hi, int end, bool some) {
    const int lane = threadIdx.x & 31, first = __shfl_sync(0xffffffffu, lo, 0);
    if (end == kNoEnd) end = some ? first : 0;
    int most = lo < hi ? hi : 0;   // end of this expert's rows and those before it
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, most, o);
        if (lane >= o) most = max(most, y);
    }
    const int earlier = __shfl_up_sync(0xffffffffu, most, 1);
    lo = max(lo, lane > 0 ? max(end, earlier) : end);
    return make_int3(lo, max(hi, lo), max(end, __shfl_sync(0xffffffffu, most, 31)));
}

struct TileRing {
    int slot = 0;
    uint32_t round = 0;
    __device__ void next() {
        if (++slot == kTileSlots) slot = 0, round ^= 1;
    }
};

// By warp 2: hands every tile of this CTA (or pair) to the others, in order.
template <Op kOp, int kCtas, int kCols>
__device__ bool find_tiles(const Args &a, Control &c) {
    using C = Config<kOp, kCtas, kCols>;
    const int lane = threadIdx.x & 31;
    TileRing ring;
    bool ok = true;
    auto hand = [&](const Tile &t) {   // by lane 0
        if (lane == 0) {
            ok = wait(&c.tile_empty[ring.slot], ring.round ^ 1, a.limits.wait_ns);
            if (ok) {
                c.tiles[ring.slot] = t;
                mbar_arrive(&c.tile_full[ring.slot]);
            }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        ring.next();
        return ok;
    };
    const int share = kCtas * a.split;   // CTAs of a tile
    int64_t t = blockIdx.x / share;
    const int64_t step = gridDim.x / share;
    if constexpr (kOp == kGradW) {
        const int per = a.feature_tiles * a.column_tiles;
        const int64_t total = (int64_t)a.E * per;
        int at = -1;
        Range r{};
        for (; t < total; t += step) {
            const int e = (int)quotient(t, per), i = (int)(t - (int64_t)e * per);
            if (e != at) {
                r = rows_of(a, at = e);
                if (r.bad && lane == 0) report(a.status, MOE_ERR_BAD_PREFIX);
            }
            const int rows = r.hi - r.lo, f = (int)quotient(i, a.column_tiles), col = i - f * a.column_tiles;
            const int all = (rows + kDepth - 1) / kDepth, each = (all + a.split - 1) / a.split;
            const int kb0 = blockIdx.x / kCtas % a.split * each, blocks = max(min(all - kb0, each), 0);
            if (!hand(Tile{e, f * kCtas * kRows, r.lo + kb0 * kDepth, min(kCols, a.depth - col * kCols), col * kCols, all, blocks,
                           kb0 + blocks == all ? rows - (all - 1) * kDepth : kDepth}))
                return false;
            if (a.split > 1) break;   // a tile to a cluster
        }
    } else {
        const int F = a.feature_tiles, kb0 = blockIdx.x / kCtas % a.split * a.per_split;
        const int blocks = min(a.per_split, a.blocks - kb0);
        int64_t before = 0;
        bool wrong = false;      // a fault in this lane's part of the prefix so far
        int end = kNoEnd;        // once there is one: of the rows of the experts before these 32
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            Range r{};
            if (e0 + lane < a.E) r = rows_of(a, e0 + lane);
            if (r.bad && blockIdx.x == 0) report(a.status, MOE_ERR_BAD_PREFIX);
            wrong = wrong || r.bad;
            int rows, R, per;
            int64_t mine, upto, all;
            for (bool flag = wrong;; flag = false) {
                rows = r.hi - r.lo, R = (rows + kCols - 1) / kCols;
                per = R > 1 ? round16((int)quotient(rows + R - 1, R)) : rows;   // row tiles of equal size
                mine = (int64_t)R * F + ((int64_t)flag << 56);   // faults go with the sum: a vote of their own takes 50 ns more
                upto = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= o) upto += y;
                }
                all = __shfl_sync(0xffffffffu, upto, 31);
                if (all >> 56 == 0) break;
                const int3 cut = behind_earlier(r.lo, r.hi, end, before > 0);
                r.lo = cut.x, r.hi = cut.y, end = cut.z;
            }
            while (t < before + all) {
                const int l = __ffs(__ballot_sync(0xffffffffu, before + upto > t)) - 1;
                const int64_t i = t - before - __shfl_sync(0xffffffffu, upto - mine, l);
                const int er = __shfl_sync(0xffffffffu, rows, l), eR = __shfl_sync(0xffffffffu, R, l);
                const int lo = __shfl_sync(0xffffffffu, r.lo, l), size = __shfl_sync(0xffffffffu, per, l);
                // eight row tiles to a pass over the features
                const int64_t pass = (int64_t)kRowGroup * F;
                const int g = eR > kRowGroup ? (int)quotient(i, pass) : 0, width = min(kRowGroup, eR - g * kRowGroup);
                const int in = (int)(i - g * pass), f = width > 1 ? (int)quotient(in, width) : in;
                const int rt = g * kRowGroup + in - f * width;
                if (!hand(Tile{e0 + l, f * kCtas * kRows, lo + rt * size, min(size, er - rt * size), 0, kb0, blocks, 0}))
                    return false;
                t += step;
                if (a.split > 1) {   // a tile to a cluster; the first CTA goes on to see the rest of the prefix
                    if (blockIdx.x != 0) return hand(Tile{-1, 0, 0, 0, 0, 0, 0, 0});
                    t = INT64_MAX;
                }
            }
            before += all;
        }
    }
    return hand(Tile{-1, 0, 0, 0, 0, 0, 0, 0});
}

// f(tile) for each tile, by a whole warp.
template <class F>
__device__ bool each_tile(const Args &a, Control &c, F f) {
    TileRing ring;
    for (;; ring.next()) {
        if (!warp_wait(&c.tile_full[ring.slot], ring.round, a.limits.wait_ns)) return false;
        const Tile t = c.tiles[ring.slot];
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(&c.tile_empty[ring.slot]);
        if (t.e < 0) return true;
        if (!f(t)) return false;
    }
}

struct Ring {
    int slot = 0, stages;
    uint32_t round = 0;
    __device__ explicit Ring(int n) : stages(n) {}
    __device__ void next() {
        if (++slot == stages) slot = 0, round ^= 1;
    }
};

// ------------------------------------------------------------------ roles

template <Op kOp, int kCtas, int kCols>
__device__ bool load(const Args &a, Control &c, uint32_t ring_base, uint32_t rank) {
    using C = Config<kOp, kCtas, kCols>;
    Ring r(C::kStages);
    int issued = 0;
    const bool mine = elect_one();
    // rows are read for every tile of features (weights kept out of L2 where other tiles read them too cost 4%)
    const uint64_t weights = a.read_once ? policy_evict_first() : policy_evict_normal(), often = policy_evict_last();
    bool ok = (int)blockIdx.x != a.limits.withheld_cta;
    ok = ok && each_tile(a, c, [&](const Tile &t) {
        const int a0 = t.a0 + (int)rank * kRows;
        const int part = columns_of<kOp, kCtas>(t) / kCtas;   // columns that this CTA loads
        const int boxes = kOp == kGradW ? part / 64 : (part + kBoxRows - 1) / kBoxRows;
        const uint32_t bytes = kTileA + boxes * (kOp == kGradW ? 64 : kBoxRows) * 128;
        const int steps = round16(t.last) / 16;   // weights' gradients: of the last block, 16 rows each
        for (int kb = 0; kb < t.blocks; ++kb, r.next(), ++issued) {
            if (!warp_wait(&c.empty[r.slot], r.round ^ 1, a.limits.wait_ns)) return false;
            const uint32_t to_a = ring_base + r.slot * (kTileA + C::kTileB), to_b = to_a + kTileA;
            const bool mask = kOp == kGradW && kb == t.blocks - 1 && t.last % 16 != 0;
            const bool part_block = kOp == kGradW && kb == t.blocks - 1 && steps < kDepth / 16;
            if (mine) {
                // what the products wait for lies in the pair's first CTA; a block to be masked is this CTA's affair first
                const uint32_t bar = mask ? smem_addr(&c.masked_full[r.slot]) : home_addr<kCtas>(&c.full[r.slot]);
                arrive_expect_at(bar, part_block ? bytes / (kDepth / 16) * steps : bytes);
                if constexpr (kOp == kForward || kOp == kForwardE4m3) {
                    load3<kCtas>(to_a, &a.a, (t.kb0 + kb) * C::kBlock, a0, t.e, bar, weights);
                } else if constexpr (kOp == kGradX) {
                    for (int i = 0; i < 2; ++i) load3<kCtas>(to_a + i * 8192, &a.a, a0 + i * 64, (t.kb0 + kb) * kDepth, t.e, bar, weights);
                } else {
                    // of the last block, no more rows than the products take
                    const CUtensorMap *map_a = part_block ? &a.a16 : &a.a, *map_b = part_block ? &a.b16 : &a.b;
                    for (int j = 0; j < (part_block ? steps : 1); ++j) {
                        const int row = t.row0 + kb * kDepth + j * 16;
                        for (int i = 0; i < 2; ++i) load2<kCtas>(to_a + i * 8192 + j * 2048, map_a, a0 + i * 64, row, bar, often);
                        for (int i = 0; i < boxes; ++i)
                            load2<kCtas>(to_b + i * 8192 + j * 2048, map_b, t.c0 + (int)rank * part + i * 64, row, bar, often);
                    }
                }
                if constexpr (kOp != kGradW)
                    for (int i = 0; i < boxes; ++i)
                        load2<kCtas>(to_b + i * kBoxRows * 128, &a.b, (t.kb0 + kb) * C::kBlock, t.row0 + (int)rank * part + i * kBoxRows,
                                     bar, often);
            }
            __syncwarp();
        }
        return true;
    });
    // the last fills have been used, so none is in flight; where one is not, no product takes the others either, and each has
    // had a limit's time to land
    for (int fill = max(issued - C::kStages, 0); fill < issued; ++fill)
        if (!warp_wait(&c.empty[fill % C::kStages], (fill / C::kStages) & 1, a.limits.wait_ns)) break;
    return ok;
}

template <Op kOp, int kCtas, int kCols>
__device__ bool multiply(const Args &a, Control &c, uint32_t ring_base, uint32_t tmem) {
    using C = Config<kOp, kCtas, kCols>;
    const bool mine = elect_one();
    Ring r(C::kStages), sums(C::kSums);
    constexpr bool kAmn = kOp == kGradX || kOp == kGradW, kBmn = kOp == kGradW;
    // steps of one product along the reduction, in the descriptors' units of 16 bytes
    constexpr uint32_t kStepA = kAmn ? 2048 >> 4 : 2, kStepB = kBmn ? 2048 >> 4 : 2;
    const bool ok = each_tile(a, c, [&](const Tile &t) {
        const int n = columns_of<kOp, kCtas>(t);
        const uint32_t desc = 1u << 4 | (C::kE4m3 ? 0 : 1u << 7 | 1u << 10) | (uint32_t)kAmn << 15 | (uint32_t)kBmn << 16 |
                              (uint32_t)(n >> 3) << 17 | (uint32_t)(kCtas * kRows >> 4) << 24;
        if (t.blocks == 0) return true;   // weights' gradients of an expert without rows: nothing to wait for
        if (!C::kE4m3 && !warp_wait(&c.sums_empty[sums.slot], sums.round ^ 1, a.limits.wait_ns)) return false;
        for (int kb = 0; kb < t.blocks; ++kb, r.next()) {
            if (C::kE4m3 && !warp_wait(&c.sums_empty[sums.slot], sums.round ^ 1, a.limits.wait_ns)) return false;
            if (!warp_wait(&c.full[r.slot], r.round, a.limits.wait_ns)) return false;
            tc_fence_after();
            const uint32_t d = uniform(tmem + sums.slot * kCols);
            const uint32_t at = ring_base + r.slot * (kTileA + C::kTileB);
            const uint32_t al = uniform(kAmn ? operand_low_mn(at, 8192) : operand_low(at));
            const uint32_t bl = uniform(kBmn ? operand_low_mn(at + kTileA, 8192) : operand_low(at + kTileA));
            if (mine) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (kOp != kGradW || kb + 1 < t.blocks || j * 16 < t.last)   // steps that have a row
                        product<kCtas, C::kE4m3>(d, al + j * kStepA, bl + j * kStepB, desc, j > 0 || (!C::kE4m3 && kb > 0));
                commit<kCtas>(&c.empty[r.slot]);
                if (C::kE4m3 || kb == t.blocks - 1) commit<kCtas>(&c.sums_full[sums.slot]);
            }
            __syncwarp();
            if (C::kE4m3) sums.next();
        }
        if (!C::kE4m3) sums.next();
        return true;
    });
    if (mine) commit_here<kCtas>(&c.last);   // kept waiting or not, no product is in flight behind this
    __syncwarp();
    warp_wait(&c.last, 0, a.limits.wait_ns);
    return ok;
}

// Weights' gradients: the last block of an expert's rows goes on into the next
// expert's. Its steps of 16 without a row of this one are left out, and in one that has
// some, zeros in both operands take the others out (in one alone, an infinity in the
// other would still make NaN).
template <int kCtas, int kCols>
__device__ bool mask_blocks(const Args &a, Control &c, char *ring) {
    using C = Config<kGradW, kCtas, kCols>;
    Ring r(C::kStages);
    uint32_t seen = 0;   // phases of each slot's masked_full, a bit a slot
    const int lane = threadIdx.x & 31;
    return each_tile(a, c, [&](const Tile &t) {
        if (t.blocks == 0) return true;
        for (int kb = 0; kb < t.blocks - 1; ++kb) r.next();
        if (t.last % 16 != 0) {
            if (!warp_wait(&c.masked_full[r.slot], seen >> r.slot & 1, a.limits.wait_ns)) return false;
            seen ^= 1u << r.slot;
            char *at = ring + (size_t)r.slot * (kTileA + C::kTileB);
            const int chunks = 2 + columns_of<kGradW, kCtas>(t) / kCtas / 64;
            for (int chunk = 0; chunk < chunks; ++chunk)
                for (int at16 = t.last * 8 + lane; at16 < round16(t.last) * 8; at16 += 32)   // 16 bytes each
                    *reinterpret_cast<int4 *>(at + chunk * 8192 + at16 * 16) = make_int4(0, 0, 0, 0);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) arrive_at(home_addr<kCtas>(&c.full[r.slot]));
        }
        r.next();
        return true;
    });
}

// Four blocks' scales of one row, from block kb: one load where rows are whole groups of four.
__device__ __forceinline__ float4 four_scales(const float *row, int kb, int blocks, bool whole) {
    if (whole) return __ldg(reinterpret_cast<const float4 *>(row + kb));
    float4 v;
    v.x = __ldg(row + min(kb, blocks - 1)), v.y = __ldg(row + min(kb + 1, blocks - 1));
    v.z = __ldg(row + min(kb + 2, blocks - 1)), v.w = __ldg(row + min(kb + 3, blocks - 1));
    return v;
}
__device__ __forceinline__ float part_of(const float4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
__device__ __forceinline__ bool whole_fours(const float *scales, int blocks) {
    return blocks % 4 == 0 && (reinterpret_cast<uintptr_t>(scales) & 15) == 0;
}

// E4M3: the scales of the blocks' rows and features, four blocks at a time; the loads of the next four are under way
// while the readers use these (a load behind each block would be waited for each time).
template <int kCtas, int kCols>
__device__ bool load_scales(const Args &a, Control &c, float *scales, uint32_t rank) {
    using C = Config<kForwardE4m3, kCtas, kCols>;
    const int lane = threadIdx.x & 31;
    Ring r(kScaleSlots);
    const int all = a.blocks;
    return each_tile(a, c, [&](const Tile &t) {
        constexpr int kPerRow = kCols / 32, kPer = kPerRow + kRows / 32;
        static_assert(kCols % 32 == 0);
        const bool whole = whole_fours(a.b_scales, all) && whole_fours(a.a_scales, all);   // kb0 is a multiple of four
        const int f0 = t.a0 + (int)rank * kRows;
        float4 next[kPer];
        const auto fetch = [&](int kb) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const float *from = i < kPerRow
                                        ? a.b_scales + (size_t)(t.row0 + min(lane + 32 * i, t.n - 1)) * all
                                        : a.a_scales + ((size_t)t.e * a.features + min(f0 + lane + 32 * (i - kPerRow), a.features - 1)) * all;
                if (i >= kPerRow || 32 * i < t.n) next[i] = four_scales(from, t.kb0 + kb, all, whole);
            }
        };
        fetch(0);
        for (int kb = 0; kb < t.blocks; kb += 4, r.next()) {
            if (!warp_wait(&c.scales_empty[r.slot], r.round ^ 1, a.limits.wait_ns)) return false;
            float *to = scales + r.slot * 4 * C::kScales + lane;
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (i >= kPerRow || 32 * i < t.n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) to[j * C::kScales + 32 * i] = part_of(next[i], j);
            __syncwarp();
            if (lane == 0) mbar_arrive(&c.scales_full[r.slot]);
            if (kb + 4 < t.blocks) fetch(kb + 4);
        }
        return true;
    });
}

// Sums of E4M3 blocks are read in the tensor core's own fragments, 32 lanes of tensor memory x 16 columns: register
// 8 h + 4 g + 2 p + i of a lane holds feature 16 h + 8 p + lane / 4 and column 8 g + 2 (lane % 4) + i. A lane then
// needs four features' scales and a quarter of the columns', where lanes that hold whole rows need all of them: their
// loads from shared memory were 60% of the time.
__device__ __forceinline__ void tmem_load_fragments(uint32_t addr, float (&v)[16]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
        asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=f"(v[8 * h]), "=f"(v[8 * h + 1]), "=f"(v[8 * h + 2]), "=f"(v[8 * h + 3]), "=f"(v[8 * h + 4]),
                       "=f"(v[8 * h + 5]), "=f"(v[8 * h + 6]), "=f"(v[8 * h + 7])
                     : "r"(addr + ((uint32_t)(16 * h) << 16)));
}
// Two columns to an instruction: a multiplication and an addition for each pair of sums, as fast as two of each but half
// the instructions, which are what the readers run out of.
__device__ __forceinline__ void scaled_add(float (&sum)[16], const float (&v)[16], const float2 (&columns)[2],
                                           const float (&features)[4]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {   // 4 h + 2 g + p
        const float2 c = columns[j / 2 % 2];
        asm("{\n\t.reg .b64 s, f, v;\n\t"
            "mov.b64 s, {%4, %5};\n\tmov.b64 f, {%6, %6};\n\tmul.rn.f32x2 s, s, f;\n\t"
            "mov.b64 f, {%2, %3};\n\tmov.b64 v, {%0, %1};\n\tfma.rn.f32x2 v, f, s, v;\n\tmov.b64 {%0, %1}, v;\n\t}"
            : "+f"(sum[2 * j]), "+f"(sum[2 * j + 1])
            : "f"(v[2 * j]), "f"(v[2 * j + 1]), "f"(c.x), "f"(c.y), "f"(features[j / 4 * 2 + j % 2]));
    }
}
// One block's sums, kN times 16 columns kStep apart; `read` comes when the last have been read, before they are added.
template <int kN, int kStep, class Read>
__device__ __forceinline__ void add_block(float (*sum)[16], uint32_t from, const float *sx, const float (&features)[4], Read read) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        float v[16];
        tmem_load_fragments(from + i * kStep, v);
        const float2 columns[2] = {*reinterpret_cast<const float2 *>(sx + i * kStep),
                                   *reinterpret_cast<const float2 *>(sx + i * kStep + 8)};
        tmem_load_wait(v);
        if (i == kN - 1) read();
        scaled_add(sum[i], v, columns, features);
    }
    if (kN == 0) read();
}

// 32 features of 16 columns leave through shared memory, transposed on the way in, so that a lane writes eight features of a
// row and four lanes its 64 bytes. (Four bytes a lane, exchanged between neighbours, took 90 us where this takes 78: 27 experts
// of 548 rows, 768 x 3152.) Pieces of 16 bytes lie where neither side meets itself in a bank.
__device__ __forceinline__ void store_fragments(const Args &a, const Tile &t, int f0, int col, const float (&sum)[16], char *buffer) {
    const int lane = threadIdx.x & 31;
    const auto place = [](int column, int piece) { return column * 64 + ((piece ^ (column >> 1 & 3)) * 16); };
    __syncwarp();   // the last columns have been read
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        uint32_t pair[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) {   // features 8 m to 8 m + 7, 2 h + p = m
            const __nv_bfloat162 b = __floats2bfloat162_rn(sum[8 * (m / 2) + 4 * g + 2 * (m % 2)], sum[8 * (m / 2) + 4 * g + 2 * (m % 2) + 1]);
            pair[m] = *reinterpret_cast<const uint32_t *>(&b);
        }
        asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};"
                     ::"r"(smem_addr(buffer + place(8 * g + lane % 8, lane / 8))), "r"(pair[0]), "r"(pair[1]), "r"(pair[2]), "r"(pair[3])
                     : "memory");
    }
    __syncwarp();
    const int f = f0 + lane % 4 * 8;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int column = half * 8 + lane / 4;
        if (f < a.features && col + column < t.n)
            *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + (size_t)(t.row0 + col + column) * a.features + f) =
                *reinterpret_cast<const uint4 *>(buffer + place(column, lane % 4));
    }
}

// Lanes hold features, registers rows: neighbouring lanes exchange halves of two
// rows, so that a lane writes two features of one row (64 bytes of a row a warp).
__device__ __forceinline__ void store_rows(const Args &a, const Tile &t, int f, int col, const float (&v)[16]) {
    const int odd = threadIdx.x & 1;
    uint32_t *out = reinterpret_cast<uint32_t *>(static_cast<__nv_bfloat16 *>(a.out) +
                                                 (size_t)(t.row0 + col + odd) * a.features + (f & ~1));
#pragma unroll
    for (int j = 0; j < 16; j += 2) {
        const float got = __shfl_xor_sync(0xffffffffu, odd ? v[j] : v[j + 1], 1);
        const __nv_bfloat162 pair = odd ? __floats2bfloat162_rn(got, v[j + 1]) : __floats2bfloat162_rn(v[j], got);
        if (f < a.features && col + j + odd < t.n)
            *reinterpret_cast<__nv_bfloat162 *>(out + (size_t)j * (a.features / 2)) = pair;
    }
}

// A warp's 32 rows x 128 bytes of a weight's gradient, through shared memory. (Lanes that stored 16 bytes each to rows of
// their own took 1660 us where this took 1150: 16384 rows, 32 experts, 7168 x 4096, fp32.) fp32 goes out by stores of eight
// lanes to 128 bytes of a row: as TMA tiles, twice bf16's, it keeps TMA from the loads, where issuing one takes 190 cycles,
// 6000 a tile whose products take 4100. bf16 goes out as TMA tiles, which the warps need not wait for. us, stores / TMA: fp32,
// 32 experts of some 512 rows 787 / 853, of some 128 615 / 673, adding to 512 1467 / 1490; bf16 629 / 644, 383 / 312, 930 / 863.
// What a bf16 gradient holds is added in registers, to be rounded once: `before`, asked for as early as the tile is known,
// goes through the same place. (fp32 is added in L2.)
struct Rows {   // 16 bytes of every fourth of 32 rows, from lane / 8
    uint4 v[8];
};
template <typename Out>
__device__ __forceinline__ Out *rows_at(const Args &a, const Tile &t, int f0, int col) {
    const int lane = threadIdx.x & 31;
    return static_cast<Out *>(a.out) + ((size_t)t.e * a.features + f0 + lane / 8) * a.depth + t.c0 + col + (lane & 7) * (int)(16 / sizeof(Out));
}
__device__ __forceinline__ void load_rows(const Args &a, const Tile &t, int f0, int col, Rows &rows) {
    const int lane = threadIdx.x & 31;
    const __nv_bfloat16 *from = rows_at<__nv_bfloat16>(a, t, f0, col);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        rows.v[i] = col + (lane & 7) * 8 < t.n && f0 + i * 4 + lane / 8 < a.features
                        ? *reinterpret_cast<const uint4 *>(from + (size_t)i * 4 * a.depth)
                        : uint4{};
}
template <typename Out, bool kAdd>
__device__ __forceinline__ void store_weights(const Args &a, const Tile &t, int f0, int col, const float (&v)[128 / sizeof(Out)],
                                              const Rows &before, char *buffer) {
    const int lane = threadIdx.x & 31, piece = lane & 7, row = lane / 8;
    const auto place = [&](int r, int p) { return reinterpret_cast<uint4 *>(buffer + r * 128 + ((p ^ (r & 7)) * 16)); };
    constexpr bool kTma = sizeof(Out) == 2, add = kAdd && kTma;
    if (kTma && lane == 0) bulk_wait_read<0>();
    __syncwarp();   // the last ones have been read
    if constexpr (add) {
#pragma unroll
        for (int i = 0; i < 8; ++i) *place(i * 4 + row, piece) = before.v[i];
        __syncwarp();
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint4 x;
        if constexpr (sizeof(Out) == 4) {
            x = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                           __float_as_uint(v[4 * i + 3]));
        } else {
            if constexpr (add) x = *place(lane, i);
            __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&x);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 y = add ? __bfloat1622float2(h[j]) : make_float2(0.0f, 0.0f);
                h[j] = __floats2bfloat162_rn(v[8 * i + 2 * j] + y.x, v[8 * i + 2 * j + 1] + y.y);
            }
        }
        *place(lane, i) = x;
    }
    if constexpr (kTma) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];"
                         ::"l"(&a.out_map), "r"(t.c0 + col), "r"(f0), "r"(t.e), "r"(smem_addr(buffer)) : "memory");
            bulk_commit();
        }
    } else {
        __syncwarp();
        if (col + piece * 4 >= t.n) return;
        float *out = rows_at<float>(a, t, f0, col);
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
            const uint4 x = *place(i + row, piece);
            if (f0 + i + row < a.features) {
                uint4 *to = reinterpret_cast<uint4 *>(out + (size_t)i * a.depth);
                if constexpr (kAdd)
                    asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};"
                                 ::"l"(to), "f"(__uint_as_float(x.x)), "f"(__uint_as_float(x.y)), "f"(__uint_as_float(x.z)),
                                   "f"(__uint_as_float(x.w)) : "memory");
                else
                    *to = x;
            }
        }
    }
}

// A tile whose reduction a cluster shares: each of its CTAs (of a pair's two, each for its own features) adds up the
// sums of as many columns. Every CTA lays its sums out in its ring and in the space beside it (scales, or readers'
// buffers, idle like the ring: a cluster that shares has one tile), which no copy or product uses any more once every CTA's
// roles have ended, and bulk copies take each column's to the CTA that adds them, in the order of the reduction.
// (Sums stored into the other CTAs' memory four bytes a lane took some 10 us longer for 256 x 256.) `put` hands this
// thread's sums to f(column, feature, value); take(first column, columns, sum) stores this CTA's, where sum(i, f) is
// what the i-th of them has for features f and f + 1. All warps of all CTAs of the cluster come here, or through
// cluster_sync() of their own: before the rings are written, before they are copied, and behind the last copy.
template <int kCtas, class Put, class Take>
__device__ bool share_tile(const Args &a, Control &c, const Tile &t, char *ring, int tid, Put put, Take take) {
    const int split = a.split, side = blockIdx.x % kCtas, part = blockIdx.x / kCtas % split;
    const int width = shared_width(t.n, split), mine = max(min(width, t.n - part * width), 0);
    float *sums = reinterpret_cast<float *>(ring), *others = sums + t.n * kRows;   // [column][feature]; the others' of mine
    cluster_sync();
    put([&](int col, int feature, float v) { sums[col * kRows + feature] = v; });
    fence_proxy_async_smem();
    cluster_sync();
    if (tid == 0) {
        if (mine > 0) mbar_arrive_expect_tx(&c.parts, (split - 1) * mine * kRows * 4);
        for (int p = 0; p < split; ++p) {
            const int cols = min(width, t.n - p * width);
            if (p == part || cols <= 0) continue;
            const uint32_t to = peer_addr(others + (part < p ? part : part - 1) * cols * kRows, p * kCtas + side);
            asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                         ::"r"(to), "r"(smem_addr(sums + p * width * kRows)), "r"(cols * kRows * 4),
                           "r"(peer_addr(&c.parts, p * kCtas + side)) : "memory");
        }
    }
    __syncwarp();
    const bool ok = mine == 0 || warp_wait(&c.parts, 0, a.limits.wait_ns);
    if (ok)
        take(part * width, mine, [&](int i, int f) {
            float2 sum = make_float2(0.0f, 0.0f);
            for (int p = 0; p < split; ++p) {
                const float *from = p == part ? sums + (part * width + i) * kRows : others + ((p < part ? p : p - 1) * mine + i) * kRows;
                const float2 v = *reinterpret_cast<const float2 *>(from + f);
                sum.x += v.x, sum.y += v.y;
            }
            return sum;
        });
    __syncwarp();
    cluster_sync();
    return ok;
}

// A shared tile's part of the result's rows: two features a thread, 64 threads to a row.
template <int kCtas, class Sum>
__device__ void store_shared_rows(const Args &a, const Tile &t, int readers, int tid, int col0, int cols, Sum sum) {
    const int f = tid % 64 * 2, feature = t.a0 + (int)(blockIdx.x % kCtas) * kRows + f;
    if (feature >= a.features) return;
    for (int i = tid / 64; i < cols; i += readers * 32 / 64) {
        const float2 v = sum(i, f);
        *reinterpret_cast<__nv_bfloat162 *>(static_cast<__nv_bfloat16 *>(a.out) + (size_t)(t.row0 + col0 + i) * a.features + feature) =
            __floats2bfloat162_rn(v.x, v.y);
    }
}
// ... of a weight's gradient: eight columns of two of its rows a thread.
template <int kCtas, typename Out, class Sum>
__device__ void store_shared_weights(const Args &a, const Tile &t, int readers, int tid, int col0, int cols, Sum sum) {
    const int f = tid % 64 * 2, feature = t.a0 + (int)(blockIdx.x % kCtas) * kRows + f;
    if (feature >= a.features || (t.kb0 == 0 && a.accumulate)) return;
    for (int i = tid / 64 * 8; i < cols; i += readers * 32 / 64 * 8) {   // columns come in eights
        float v[2][8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 x = sum(i + j, f);
            v[0][j] = x.x, v[1][j] = x.y;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            Out *out = static_cast<Out *>(a.out) + ((size_t)t.e * a.features + feature + h) * a.depth + t.c0 + col0 + i;
            if constexpr (sizeof(Out) == 4) {
                float4 *to = reinterpret_cast<float4 *>(out);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float4 x = make_float4(v[h][4 * j], v[h][4 * j + 1], v[h][4 * j + 2], v[h][4 * j + 3]);
                    if (a.accumulate) {
                        const float4 y = to[j];
                        x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
                    }
                    to[j] = x;
                }
            } else {
                uint4 *to = reinterpret_cast<uint4 *>(out);
                uint4 x = {};
                __nv_bfloat162 *b = reinterpret_cast<__nv_bfloat162 *>(&x);
                if (a.accumulate) {
                    x = *to;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 y = __bfloat1622float2(b[j]);
                        v[h][2 * j] += y.x, v[h][2 * j + 1] += y.y;
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) b[j] = __floats2bfloat162_rn(v[h][2 * j], v[h][2 * j + 1]);
                *to = x;
            }
        }
    }
}

// The warps from the fourth on, eight or (E4M3) twelve: a quarter of tensor memory's lanes each, every second or third 16
// columns (weights' gradients: 128 bytes of the result).
template <Op kOp, int kCtas, int kCols, typename Out>
__device__ bool read_sums(const Args &a, Control &c, char *ring, char *beside, uint32_t tmem, uint32_t rank, bool &shared) {
    using C = Config<kOp, kCtas, kCols>;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, q = warp % 4, side = (warp - kFirstReader) / 4;
    const int tid = threadIdx.x - kFirstReader * 32;
    const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
    Ring sums(C::kSums), fours(kScaleSlots);
    bool ready = false;   // E4M3: the next block's sums are there
    constexpr int kStep = 16 * C::kSides, kChunks = (kCols + kStep - 1) / kStep;
    const float *scales = reinterpret_cast<const float *>(beside);
    char *const buffer = beside + C::kScaleBytes + (warp - kFirstReader) * C::kStore;
    const bool ok = each_tile(a, c, [&](const Tile &t) {
        const int f = t.a0 + (int)rank * kRows + q * 32 + lane;
        if constexpr (C::kE4m3) {
            float sum[kChunks][16] = {};
            const uint32_t empty = home_addr<kCtas>(&c.sums_empty[0]);
            const auto blocks = [&](auto chunks) {   // straight code for each number of chunks: branches cost as much as sums
                constexpr int kN = decltype(chunks)::value;
                for (int kb = 0; kb < t.blocks; kb += 4, fours.next()) {
                    if (!warp_wait(&c.scales_full[fours.slot], fours.round, a.limits.wait_ns)) return false;
                    const float *four = scales + fours.slot * 4 * C::kScales;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (kb + i >= t.blocks) break;
                        const float *sx = four + i * C::kScales;
                        float features[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) features[j] = sx[kCols + q * 32 + j * 8 + lane / 4];
                        if (!ready && !warp_wait(&c.sums_full[sums.slot], sums.round, a.limits.wait_ns)) return false;
                        tc_fence_after();
                        // the block's place is given back and the next one looked for while the last sums are added: 4% and 2%
                        add_block<kN, kStep>(sum, lanes + sums.slot * kCols + side * 16, sx + side * 16 + (lane & 3) * 2, features, [&] {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) arrive_at(empty + sums.slot * 8);
                            sums.next();
                            ready = __all_sync(0xffffffffu, arrived(&c.sums_full[sums.slot], sums.round));
                        });
                    }
                    if (lane == 0) mbar_arrive(&c.scales_empty[fours.slot]);   // behind the last block's __syncwarp
                }
                return true;
            };
            const int chunks = t.n <= side * 16 ? 0 : (t.n - side * 16 + kStep - 1) / kStep;
            bool done;
            switch (chunks) {
                case 0: done = blocks(std::integral_constant<int, 0>()); break;
                case 1: done = blocks(std::integral_constant<int, 1>()); break;
                case 2: done = blocks(std::integral_constant<int, 2>()); break;
                case 3: done = blocks(std::integral_constant<int, 3>()); break;
                default: done = blocks(std::integral_constant<int, kChunks>()); break;
            }
            if (!done) return false;
            if (a.split > 1) {
                shared = true;
                const bool all = share_tile<kCtas>(a, c, t, ring, tid, [&](auto f) {
#pragma unroll
                    for (int i = 0; i < kChunks; ++i)
#pragma unroll
                        for (int j = 0; j < 16; ++j) {   // 8 h + 4 g + 2 p + i
                            const int col = i * kStep + side * 16 + j / 4 % 2 * 8 + (lane & 3) * 2 + j % 2;
                            if (col < t.n) f(col, q * 32 + j / 8 * 16 + j / 2 % 2 * 8 + lane / 4, sum[i][j]);
                        }
                }, [&](int col0, int cols, auto total) { store_shared_rows<kCtas>(a, t, C::kReaders, tid, col0, cols, total); });
                return all;
            }
#pragma unroll
            for (int i = 0; i < kChunks; ++i) {
                const int col = i * kStep + side * 16;
                if (col < t.n) store_fragments(a, t, t.a0 + (int)rank * kRows + q * 32, col, sum[i], buffer);
            }
        } else {
            const bool some = t.blocks > 0;
            Rows before;
            if constexpr (kOp == kGradW && sizeof(Out) == 2)
                if (some && a.accumulate && a.split == 1)
                    load_rows(a, t, t.a0 + (int)rank * kRows + q * 32, side * 64, before);
            if (some && !warp_wait(&c.sums_full[sums.slot], sums.round, a.limits.wait_ns)) return false;
            tc_fence_after();
            if (a.split > 1) {
                shared = true;
                const auto put_all = [&](auto put) {
                    for (int col = side * 16; col < t.n; col += kStep) {
                        float v[16] = {};
                        if (some) {
                            tmem_load16(lanes + sums.slot * kCols + col, v);
                            tmem_load_wait(v);
                        }
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (col + j < t.n) put(col + j, q * 32 + lane, v[j]);
                    }
                };
                const bool all = share_tile<kCtas>(a, c, t, ring, tid, put_all, [&](int col0, int cols, auto total) {
                    if constexpr (kOp == kGradW) store_shared_weights<kCtas, Out>(a, t, C::kReaders, tid, col0, cols, total);
                    else store_shared_rows<kCtas>(a, t, C::kReaders, tid, col0, cols, total);
                });
                if (!all) return false;
            } else if constexpr (kOp == kGradW) {
                constexpr int kWide = 128 / sizeof(Out);
                const int f0 = t.a0 + (int)rank * kRows + q * 32;
                for (int col = side * kWide; col < t.n; col += C::kSides * kWide) {
                    float v[kWide] = {};
                    if (some) {
#pragma unroll
                        for (int i = 0; i < kWide; i += 16)
                            tmem_load16(lanes + sums.slot * kCols + col + i, v + i);
                        tmem_load_wait(v);
                    }
                    if (f0 >= a.features || (!some && a.accumulate)) continue;
                    if (a.accumulate) {
                        store_weights<Out, true>(a, t, f0, col, v, before, buffer);
                        if (sizeof(Out) == 2 && col + C::kSides * kWide < t.n) load_rows(a, t, f0, col + C::kSides * kWide, before);
                    } else {
                        store_weights<Out, false>(a, t, f0, col, v, before, buffer);
                    }
                }
            } else {
                for (int col = side * 16; col < t.n; col += kStep) {
                    float v[16];
                    tmem_load16(lanes + sums.slot * kCols + col, v);
                    tmem_load_wait(v);
                    store_rows(a, t, f, col, v);
                }
            }
            if (some) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_at(home_addr<kCtas>(&c.sums_empty[sums.slot]));
                sums.next();
            }
        }
        return true;
    });
    if (kOp == kGradW && sizeof(Out) == 2 && lane == 0) bulk_wait_read<0>();
    __syncwarp();
    return ok;
}

template <Op kOp, int kCtas, int kCols, typename Out>
__global__ __launch_bounds__((Config<kOp, kCtas, kCols>::kThreads), 1) void grouped_kernel(const __grid_constant__ Args a) {
    using C = Config<kOp, kCtas, kCols>;
    const WarpTrace trace(a.trace, MOE_TRACE_GROUPED);
    extern __shared__ char smem_raw[];
    __shared__ Control c;
    char *ring = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    char *beside = ring + C::kStages * (kTileA + C::kTileB);
    const uint32_t ring_base = smem_addr(ring);
    const int warp = threadIdx.x / 32;
    const uint32_t rank = kCtas == 1 ? 0 : blockIdx.x % kCtas;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&c.full[i], kCtas);
            mbar_init(&c.empty[i], 1);
            mbar_init(&c.masked_full[i], 1);
        }
        for (int i = 0; i < C::kSums; ++i) {
            mbar_init(&c.sums_full[i], 1);
            mbar_init(&c.sums_empty[i], kCtas * C::kReaders);
        }
        for (int i = 0; i < kScaleSlots; ++i) {
            mbar_init(&c.scales_full[i], 1);
            mbar_init(&c.scales_empty[i], C::kReaders);
        }
        for (int i = 0; i < kTileSlots; ++i) {
            mbar_init(&c.tile_full[i], 1);
            mbar_init(&c.tile_empty[i], 1 + (rank == 0) + C::kHelper + C::kReaders);
        }
        mbar_init(&c.last, 1);
        mbar_init(&c.parts, 1);
        fence_barrier_init();
        tma_prefetch_map(&a.a);
        tma_prefetch_map(&a.b);
    }
    if (warp == 2) tmem_take<kCtas>(&c.tmem, C::kTmemCols);
    tc_fence_before();
    __syncthreads();
    if constexpr (kCtas == 2) cluster_sync();
    tc_fence_after();
    const uint32_t tmem = c.tmem;
    grid_dependency_wait();
    grid_launch_dependents();

    bool ok = true, shared = false;
    if (warp == 0) {
        ok = load<kOp, kCtas, kCols>(a, c, ring_base, rank);
    } else if (warp == 1) {
        if (rank == 0) ok = multiply<kOp, kCtas, kCols>(a, c, ring_base, tmem);
    } else if (warp == 2) {
        ok = find_tiles<kOp, kCtas, kCols>(a, c);
    } else if (warp == 3) {
        if constexpr (kOp == kGradW) ok = mask_blocks<kCtas, kCols>(a, c, ring);
        if constexpr (C::kE4m3) ok = load_scales<kCtas, kCols>(a, c, reinterpret_cast<float *>(beside), rank);
    } else {
        ok = read_sums<kOp, kCtas, kCols, Out>(a, c, ring, beside, tmem, rank, shared);
    }
    if (!ok && (threadIdx.x & 31) == 0) report(a.status, MOE_ERR_TIMEOUT);
    __syncwarp();
    if (a.split > 1 && !shared) {   // beside share_tile
        cluster_sync();
        cluster_sync();
        if (!ok) warp_wait(&c.parts, 0, a.limits.wait_ns);   // the others' copies may be on their way here all the same
        cluster_sync();
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (kCtas == 2) cluster_sync();   // no arrival or product of the other CTA is under way
    tc_fence_after();
    if (warp == 2) tmem_give<kCtas>(tmem, C::kTmemCols);
}

// ------------------------------------------------------------------ host

// CTA pairs that are resident at once (0: none): GPCs with an odd number of SMs leave one over.
template <Op kOp, int kCtas, int kCols, typename Out>
int resident() {
    auto kernel = grouped_kernel<kOp, kCtas, kCols, Out>;
    if (kCtas == 1) return device_sm_count();
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) dev = 0;
    int n = known[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(device_sm_count() / kCtas * kCtas);
        cfg.blockDim = dim3(Config<kOp, kCtas, kCols>::kThreads);
        cfg.dynamicSmemBytes = Config<kOp, kCtas, kCols>::smem();
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim = {kCtas, 1, 1};
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) n = 1;
        known[dev].store(n, std::memory_order_relaxed);
    }
    return n * kCtas;
}

template <Op kOp, int kCtas, int kCols, typename Out = __nv_bfloat16>
int launch(Args &a, int64_t most_tiles, cudaStream_t s) {
    using C = Config<kOp, kCtas, kCols>;
    auto kernel = grouped_kernel<kOp, kCtas, kCols, Out>;
    const int rc = ensure_dynamic_smem((const void *)kernel, C::smem());
    if (rc != MOE_OK) return rc;
    const int64_t ctas = a.split > 1 ? most_tiles * a.split * kCtas   // a cluster each, that wait for no other
                                     : std::min<int64_t>(resident<kOp, kCtas, kCols, Out>(), most_tiles * kCtas);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::smem();
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (kCtas * a.split > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n++].val.clusterDim = {(unsigned)(kCtas * a.split), 1, 1};
    }
    if (tuning().overlap) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace grouped

namespace {
using namespace grouped;

constexpr int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Row tiles that M rows in E groups make at most.
int64_t most_row_tiles(int M, int E, int cols) { return (int64_t)M / cols + std::min(M, E); }

template <Op kOp, int kCtas, int kCols>
int launch_rows(Args &a, int split, cudaStream_t s) {
    a.feature_tiles = ceil_div(a.features, kCtas * kRows);
    a.split = split;
    a.per_split = Config<kOp, kCtas, kCols>::kE4m3 ? ceil_div(a.blocks, 4 * split) * 4 : ceil_div(a.blocks, split);
    a.read_once = a.M <= (int64_t)a.E * kCols;
    return launch<kOp, kCtas, kCols>(a, most_row_tiles(a.M, a.E, kCols) * a.feature_tiles, s);
}

// Pairs of CTAs with 256 features to a tile, or single CTAs with 128 features and at most 128 rows, either alone or up to
// four (eight) to a tile's reduction, in a cluster: whichever an estimate finds faster, from rows that are spread evenly.
// A block takes the tensor core 2 n cycles and its loads a cycle for 64 bytes (70 for single CTAs); a tile's ends cost
// some 2000 cycles and a shared tile's exchange 1000 and 55 a column. Captured calls, us, launch and flush (7) included, as
// pairs / 2 / 4 of them / single / 2 / 4 / 8: 100 rows, 7168 x 512: 34 / 26 / 22 / 36 / 28 / 22 / 20; 4 x 32 rows, 7168 x 512:
// 32 / 26 / 20 / 34 / 26 / 20 / 28; 2048 rows, 7168 x 512: 40 / 36 / 48 / 36 / 30 / 40 / 73; 2 x 700 rows, 4096 x 1024:
// 30 / 30 / 44 / 26 / 40 / 46 / 84; 8 x 128 rows, 2048 x 2048: 24 / 38 / 67 / 28 / 44 / 63 / 128.
struct Way {
    bool pair;
    int split;
};
Way way_for(const Args &a, int block_cells, int pair_cols) {
    const int groups = std::min(a.M, a.E), sms = device_sm_count();
    const double rows = (double)a.M / groups;
    Way best{true, 1};
    double least = 0;
    for (int pair = 1; pair >= 0; --pair) {
        const int cols = pair ? pair_cols : 128, per = (int)((rows + cols - 1) / cols);
        const double n = rows / per, features = pair ? 256 : 128;
        const int64_t tiles = (int64_t)groups * per * ceil_div(a.features, (int)features);
        const int64_t most = most_row_tiles(a.M, a.E, cols) * ceil_div(a.features, (int)features);
        const double block = std::max(2.0 * n, (128 * 128 + (pair ? n / 2 : n) * 128) / (pair ? 64.0 : 70.0));
        for (int split = 1; split <= most_split(pair ? 2 : 1); split *= 2) {
            const int step = block_cells == 128 ? 4 : 1, of = ceil_div(a.blocks, split * step) * step;
            const int size = split * (pair ? 2 : 1);
            // the grid has a cluster for every tile there may be; four fifths of the SMs take clusters of eight at once
            if (split > 1 && (most * size > (size == 8 ? sms * 4 / 5 : sms) || (split - 1) * of >= a.blocks)) break;
            const int64_t at_once = sms / size;
            const double cycles = (double)((tiles + at_once - 1) / at_once) * (of * block + 2000) + (split > 1 ? 1000 + 55 * n : 0);
            if (least == 0 || cycles < least) least = cycles, best = Way{pair != 0, split};
        }
    }
    return best;
}

// Weights' gradients, likewise: pairs with 256 x 256 of a weight to a tile or single CTAs with 128 x 128, alone or in
// clusters that share an expert's rows. us as above: 16384 rows, 1024 x 512: 81 / 57 / 41 / 79 / 52 / 36 / 67; 4096 rows,
// 2048 x 512: 30 / 32 / 46 / 28 / 26 / 36 / 72; 8 x 16384 rows, 512 x 512: 89 / 74 / 121 / 83 / 103 / 123 / 188; 100 rows,
// 7168 x 512: 14 / 39 / 71 / 13 / 40 / 77 / 174; 4096 rows, 7168 x 2048: 79 / 190 / 323 / 124 / 247 / 375 / 788.
Way way_for_weights(const Args &a) {
    const int sms = device_sm_count(), rows = ceil_div(a.M, a.E), blocks = ceil_div(rows, kDepth);
    Way best{true, 1};
    double least = 0;
    for (int pair = 1; pair >= 0; --pair) {
        const int edge = pair ? 256 : 128;
        const int64_t tiles = (int64_t)a.E * ceil_div(a.features, edge) * ceil_div(a.depth, edge);
        const double block = pair ? 512 : 468;
        for (int split = 1; split <= most_split(pair ? 2 : 1); split *= 2) {
            const int size = split * (pair ? 2 : 1), of = ceil_div(blocks, split);
            if (split > 1 && (tiles * size > (size == 8 ? sms * 4 / 5 : sms) || (split - 1) * of >= blocks)) break;
            const int64_t at_once = sms / size;
            const double cycles = (double)((tiles + at_once - 1) / at_once) * (of * block + 2000) + (split > 1 ? 1000 + 55 * edge : 0);
            if (least == 0 || cycles < least) least = cycles, best = Way{pair != 0, split};
        }
    }
    return best;
}
template <int kCtas, int kCols, typename Out>
int launch_weights(Args &a, int split, cudaStream_t s) {
    a.split = split;
    a.feature_tiles = ceil_div(a.features, kCtas * kRows);
    a.column_tiles = ceil_div(a.depth, kCols);
    return launch<kGradW, kCtas, kCols, Out>(a, (int64_t)a.E * a.feature_tiles * a.column_tiles, s);
}
template <typename Out>
int launch_weights(Args &a, cudaStream_t s) {
    const Way w = way_for_weights(a);
    return w.pair ? launch_weights<2, 256, Out>(a, w.split, s) : launch_weights<1, 128, Out>(a, w.split, s);
}

template <Op kOp, int kPairCols>
int launch_best(Args &a, cudaStream_t s) {
    constexpr int cells = kOp == kForwardE4m3 ? 128 : kDepth;
    a.blocks = ceil_div(a.depth, cells);
    const Way w = way_for(a, cells, kPairCols);
    return w.pair ? launch_rows<kOp, 2, kPairCols>(a, w.split, s) : launch_rows<kOp, 1, 128>(a, w.split, s);
}
}  // namespace

int launch_grouped_linear(const GroupedLaunch &L) {
    const bool e4m3 = L.x_scales != nullptr;
    Args a{};
    if (!make_tensor_map3(&a.a, L.w, e4m3 ? 1 : 2, L.num_experts, L.out_features, L.in_features, kRows) ||
        !make_tensor_map(&a.b, L.x, e4m3, L.num_rows, L.in_features, kBoxRows))
        return MOE_ERR_CUDA;
    a.prefix = L.expert_prefix;
    a.a_scales = L.w_scales, a.b_scales = L.x_scales;
    a.out = L.out;
    a.status = L.status;
    a.E = L.num_experts, a.M = L.num_rows;
    a.features = L.out_features, a.depth = L.in_features;
    a.limits = wait_limits();
    a.trace = trace_args();
    const cudaStream_t s = static_cast<cudaStream_t>(L.stream);
    return e4m3 ? launch_best<kForwardE4m3, 160>(a, s) : launch_best<kForward, 256>(a, s);
}

int launch_grouped_grad_x(const GroupedLaunch &L) {
    Args a{};
    if (!make_tensor_map3(&a.a, L.w, 2, L.num_experts, L.out_features, L.in_features, kDepth) ||
        !make_tensor_map(&a.b, L.x, false, L.num_rows, L.out_features, kBoxRows))
        return MOE_ERR_CUDA;
    a.prefix = L.expert_prefix;
    a.out = L.out;
    a.status = L.status;
    a.E = L.num_experts, a.M = L.num_rows;
    a.features = L.in_features, a.depth = L.out_features;
    a.limits = wait_limits();
    a.trace = trace_args();
    return launch_best<kGradX, 256>(a, static_cast<cudaStream_t>(L.stream));
}

int launch_grouped_grad_w(const GroupedGradWLaunch &L) {
    const cudaStream_t s = static_cast<cudaStream_t>(L.stream);
    const size_t cell = L.out_type == MOE_GRAD_F32 ? 4 : 2;
    if (L.num_rows == 0) {
        if (L.accumulate) return MOE_OK;
        const size_t bytes = (size_t)L.num_experts * L.out_features * L.in_features * cell;
        return cudaMemsetAsync(L.out, 0, bytes, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
    }
    Args a{};
    if (!make_tensor_map(&a.a, L.grad, false, L.num_rows, L.out_features, kDepth) ||
        !make_tensor_map(&a.b, L.x, false, L.num_rows, L.in_features, kDepth) ||
        !make_tensor_map(&a.a16, L.grad, false, L.num_rows, L.out_features, 16) ||
        !make_tensor_map(&a.b16, L.x, false, L.num_rows, L.in_features, 16) ||
        (cell == 2 && !make_tensor_map3(&a.out_map, L.out, 2, L.num_experts, L.out_features, L.in_features, 32)))
        return MOE_ERR_CUDA;
    a.prefix = L.expert_prefix;
    a.out = L.out;
    a.status = L.status;
    a.E = L.num_experts, a.M = L.num_rows;
    a.features = L.out_features, a.depth = L.in_features;
    a.accumulate = L.accumulate;
    a.limits = wait_limits();
    // One wait may cover all of a tile's reduction (its sums, its last block, the tile after next): 2^22 rows of one expert
    // take 16 ms, so that 2^30 took four times the limit of 1 s. A limit more for every 2^22 rows.
    a.limits.wait_ns *= 1 + (uint64_t)(L.num_rows >> 22);
    a.trace = trace_args();
    return L.out_type == MOE_GRAD_F32 ? launch_weights<float>(a, s) : launch_weights<__nv_bfloat16>(a, s);
}

}  // namespace moe
