// skinny.cuh -- matrix products of long weight matrices with few rows of
// activations, as one persistent kernel body: D[256 weight rows x n columns] =
// A[256 x K] B[n x K]^T, the weights as the tensor core's 128-row operand (twice,
// over one B tile) and the activations as its n columns (16..128).
//
// What bounds it is the stream of weights, so the work is cut by bytes: all
// tiles' K blocks stand in one line, each CTA takes an equal stretch of it
// (tiles may begin and end inside a stretch), and a CTA's loads run ahead of
// its products across tile and phase borders. CTAs that share a tile leave
// fp32 partial sums in the workspace, and each of them adds up its share of the
// tile's columns, in the order of K, once all partial sums are there: the
// result does not depend on the arrival order.
//
// Roles of a CTA's warps: 0 loads A (weights), 1 loads B (activations), 2 issues
// the products, 3 owns the tensor memory and announces results to other CTAs, and
// the next 8 or 16 (P::kReaders) read the sums. Tiles shared through the workspace
// (P::kShares) are added up by 4 more warps while the others go on (P::kAdders), or
// by the readers at the end of each phase.
//   bf16 weights: A and B from shared memory; sums stay in tensor memory for a
//     whole stretch of K, double-buffered, so that the readers' work on one
//     tile runs under the next tile's products.
//   E4M3 weights: the activations come as the sum of two E4M3 codes, the second
//     one's 32nd, under a power of two per row and block (Split, below), the second
//     codes as further columns, so that the codes go to the tensor core as they are. A block of 128
//     along K has its own fp32 scale per weight row, so the readers scale each
//     block's sums and add them in registers (n <= 64); four blocks' sums in
//     tensor memory let the products run ahead. (Turning the codes into bf16 in
//     tensor memory, by 8 more warps, was bound by that memory's ports: 2.01 ms for
//     256 experts of 7168 x 2048 where this took 1.83, and now takes 1.80.)
//
// The problem P gives the segments, the loads of B and what becomes of the sums.
#pragma once

#include <algorithm>

#include "umma.cuh"

namespace moe {
namespace skinny {

constexpr int kFirstReader = 128;      // first thread of the reading warps
constexpr int kAdders = 128;           // threads of the adding warps
constexpr int kMaxLines = 8;
constexpr int kMaxSplit = 8;           // CTAs of a cluster that share a tile
constexpr uint32_t kTileWeight = 1024;   // what the finished parts of a tile count together
// Two thirds of the SMs draw all of HBM's bandwidth where a block costs little
// besides its bytes (100 SMs: within 1% of 152, one token); a tile that no other
// CTA shares saves some 10 us of hand-over. Blocks that keep an SM busy, E4M3
// ones or products of many columns, want equal stretches.
constexpr int kSlackBytes = 140, kSlackWork = 110;
constexpr int kRows = 128;             // weight rows of one product; a tile has two
constexpr int kHalf = kRows * 128;     // bytes of one A tile of a stage
constexpr int kMaxCtas = 160;
constexpr int kMaxStages = 8;
constexpr int kMaxSums = 4;            // tiles' or blocks' sums in tensor memory
constexpr int kSmemBudget = 224 << 10;
constexpr int kMinBlocks = MOE_TUNE_SKINNY_MIN_BLOCKS;          // K blocks a CTA takes at least (or a whole tile)

// One CTA's stretch of one tile.
struct Segment {
    int row0, row1;       // weight rows of the two products
    bool two;             // both products (else the first alone)
    int kb0, kb1, kbs;    // K blocks [kb0, kb1) of the tile's kbs
    int b_from;           // first K block whose B the problem has to wait for (P::kPieces: and that is a piece's)
    int n;                // columns in use
    int line, phase, f, group, set, first;   // which tile: line and phase, feature tile, group, its weight set and first row
    int cta0, parts;      // the CTAs that share the tile: cta0 .. cta0 + parts - 1
    __device__ int n16() const { return (n + 15) & ~15; }
    __device__ bool whole() const { return kb0 == 0 && kb1 == kbs; }
};

// a / b for a >= 0 and b > 0. An integer division takes 250 cycles or more, and
// a small call waits for a dozen of them before its first load; below 2^20 a
// float one is exact: (a + 1/2) / b is at least 1 / (2 b) from the next integer,
// its error at most 3 units of 2^-24 of a / b.
static __device__ __noinline__ int64_t long_quotient(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    if ((a | b) >> 20) return long_quotient(a, b);
    return (int)__fdividef((float)(int)a + 0.5f, (float)(int)b);
}

// A line of K blocks: `tiles` tiles of `kbs` blocks, cut for the CTAs in one of
// three ways. With room for two CTAs or more to a tile, each tile goes to the
// same number of neighbours (`span` blocks of the line, some of them past the
// tile's end). Else whole tiles, where that makes the longest stretch at most
// `slack` percent of an equal one; else equal stretches.
struct Line {
    int64_t tiles, units, per;
    int kbs, span;
    Line() = default;
    __device__ Line(int64_t n, int k_blocks, int ctas, int slack) : tiles(n), kbs(k_blocks), span(k_blocks) {
        const int least = min(kbs, kMinBlocks);
        if (tiles > 0 && 2 * tiles <= ctas) {
            const int share = (int)min(quotient(ctas, tiles), quotient(kbs, least));
            per = quotient(kbs + share - 1, share);
            span = (int)per * share;
        } else {
            const int64_t whole = quotient(tiles + ctas - 1, ctas) * kbs;
            per = quotient(tiles * kbs + ctas - 1, ctas);
            if (per < least) per = least;
            if (whole * 100 <= per * slack) per = whole;
        }
        units = tiles * span;
    }
    // Each segment of CTA `cta`, in order: f(tile, segment with K range and sharing CTAs filled in).
    template <class F>
    __device__ bool each(int cta, F f) const {
        int64_t u = cta * per;
        const int64_t end = u + per < units ? u + per : units;
        while (u < end) {
            const int64_t tile = quotient(u, span), begin = tile * span;
            Segment s;
            s.kbs = kbs;
            s.kb0 = (int)(u - begin);
            s.kb1 = (int)(end - begin < kbs ? end - begin : kbs);
            s.cta0 = (int)quotient(begin, per);
            s.parts = (int)quotient(begin + kbs - 1, per) - s.cta0 + 1;
            if (s.kb0 < s.kb1 && !f(tile, s)) return false;
            u = end - begin < span ? end : begin + span;
        }
        return true;
    }
};

struct Control {
    uint64_t full_a[kMaxStages], empty_a[kMaxStages], full_b[kMaxStages], empty_b[kMaxStages];
    uint64_t sums_full[kMaxSums], sums_empty[kMaxSums];
    uint64_t last;
    uint32_t tmem;
    uint32_t written;        // reader warps that have written a segment's results, over all segments
};

// E4M3: the scales of a block's activations, a place for each column and block.
// Loads run at most kMaxStages blocks ahead of the products, those kMaxSums ahead
// of the readers.
constexpr int kScaleSlots = 16, kScaleBytes = kScaleSlots * 64 * 4;
static_assert(kMaxStages + kMaxSums < kScaleSlots, "a place may be in use when its turn comes");

// A and B have a ring each: the loads of A in flight are what keeps HBM busy (five
// or six blocks of 32 KB; with four the stream was 10% slower), those of B come
// from L2 and are smaller.
struct Shape {
    int cols;      // columns a tile may have: a multiple of 16, at most 256 (E4M3: 64)
    int a_stages, b_stages;
    __host__ __device__ static constexpr int b_bytes(int cols, bool e4m3) { return cols * (e4m3 ? 256 : 128); }
    static Shape of(int cols, bool e4m3, int budget = kSmemBudget) {
        if (e4m3) budget -= kScaleBytes;
        const int b = b_bytes(cols, e4m3);
        const int a_stages = 3 * b <= budget - 6 * 2 * kHalf ? 6 : cols <= 128 ? 5 : 4;
        const int b_stages = (budget - a_stages * 2 * kHalf) / b;
        return Shape{cols, a_stages, b_stages < kMaxStages ? b_stages : kMaxStages};
    }
    __host__ __device__ int ring_bytes(bool e4m3) const { return a_stages * 2 * kHalf + b_stages * b_bytes(cols, e4m3); }
    // the ring, and for E4M3 the activations' scales behind it
    __host__ __device__ int used_bytes(bool e4m3) const { return ring_bytes(e4m3) + (e4m3 ? kScaleBytes : 0); }
    size_t smem(bool e4m3) const { return 1024 + (size_t)used_bytes(e4m3); }
    __device__ uint32_t a_at(int slot) const { return slot * 2 * kHalf; }
    __device__ uint32_t b_at(int slot, bool e4m3) const { return a_stages * 2 * kHalf + slot * b_bytes(cols, e4m3); }
    // bf16: two tiles' sums of 2 `cols` columns, or one's where two do not fit; E4M3: kMaxSums blocks' of twice as many, or two
    __host__ __device__ int sums() const { return cols <= 128 ? 2 : 1; }
    int tmem_cols(bool e4m3) const {
        if (e4m3) return 512;
        int c = 32;
        while (c < 2 * sums() * cols) c *= 2;
        return c;
    }
};

// Counts fills of the ring: slot and the parity of its barriers.
struct Ring {
    int slot = 0, stages;
    uint32_t round = 0;
    __device__ explicit Ring(int n) : stages(n) {}
    __device__ void next() {
        if (++slot == stages) slot = 0, round ^= 1;
    }
};

// Every wait has a limit of `ns`. A role whose wait runs out gives up; the others run
// out of theirs in turn. Gave up or not, the roles that start copies and products
// wait for their own last ones, so that none is in flight when the CTA gives up
// its tensor memory and its shared memory.
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, uint64_t ns) {
    return mbar_wait_bounded(bar, parity, ns);
}

// ... by a whole warp, which goes on or gives up as one.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, uint64_t ns) {
    return __all_sync(0xffffffffu, wait(bar, parity, ns));
}

// The last fills of a ring have landed.
__device__ __forceinline__ void wait_fills(uint64_t *full, int stages, int issued, uint64_t ns) {
    for (int fill = max(issued - stages, 0); fill < issued; ++fill) wait(&full[fill % stages], (fill / stages) & 1, ns);
}

// The readers (barrier 1) or the adders (barrier 2) as a team of kCount threads from kFirst.
template <int kBarrier, int kFirst, int kCount>
struct Team {
    static constexpr int count = kCount;
    static constexpr int first = kFirst;
    __device__ static bool leader() { return threadIdx.x == first; }
    __device__ static int warp() { return (threadIdx.x - first) / 32; }
    __device__ static void sync() { asm volatile("barrier.cta.sync %0, %1;" ::"n"(kBarrier), "n"(kCount) : "memory"); }
    // true if every thread of the team says so
    __device__ static bool agree(bool ok) {
        uint32_t r;
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
            "barrier.cta.red.and.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
            : "=r"(r) : "r"((uint32_t)ok), "n"(kBarrier), "n"(kCount) : "memory");
        return r != 0;
    }
};
template <class P>
using ReadersOf = Team<1, kFirstReader, P::kReaders>;
template <class P>
using AddersOf = Team<2, ReadersOf<P>::first + P::kReaders, kAdders>;

// Wait (bounded) until a counter reaches `want`; release/acquire with count_up.
__device__ __forceinline__ uint32_t ld_acquire(const uint32_t *p) { return ld_acquire_gpu_u32(p); }
__device__ __forceinline__ uint64_t ld_acquire(const uint64_t *p) {
    uint64_t v;
    asm volatile("ld.acquire.gpu.global.b64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
    return v;
}
template <typename U>
__device__ __forceinline__ bool wait_count(const U *p, U want, uint64_t ns) {
    if (ld_acquire(p) >= want) return true;
    const uint64_t deadline = globaltimer_ns() + ns;
    while (ld_acquire(p) < want)
        if (globaltimer_ns() > deadline) return false;
    return true;
}
__device__ __forceinline__ void count_up(uint32_t *p, uint32_t v) {
    asm volatile("red.release.gpu.global.add.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ void count_up(uint64_t *p, uint64_t v) {
    asm volatile("red.release.gpu.global.add.u64 [%0], %1;" ::"l"(p), "l"(v) : "memory");
}

// ------------------------------------------------------------------ roles

template <class P>
__device__ bool load_a(const P &p, Control &c, uint32_t ring_base, const Shape sh) {
    const uint64_t policy = policy_evict_first();
    const int lane = threadIdx.x & 31;
    Ring r(sh.a_stages);
    int issued = 0;
    bool ok = true;
    if (lane == 0) {
        ok = p.segments([&](const Segment &s) {
            for (int kb = s.kb0; kb < s.kb1; ++kb, r.next(), ++issued) {
                if (!wait(&c.empty_a[r.slot], r.round ^ 1, p.a.limits.wait_ns)) return false;
                const uint32_t dst = ring_base + sh.a_at(r.slot);
                p.a_load(s, kb, dst, &c.full_a[r.slot], policy);
            }
            return true;
        });
        wait_fills(c.full_a, sh.a_stages, issued, p.a.limits.wait_ns);
    }
    return ok;
}

template <bool kE4m3, class P>
__device__ bool load_b(const P &p, Control &c, uint32_t ring_base, float *scales, const Shape sh) {
    const int lane = threadIdx.x & 31;
    Ring r(sh.b_stages);
    int issued = 0;
    const uint64_t policy = policy_evict_last();
    const bool ok = p.segments([&](const Segment &s) {
        typename P::Rows rows = p.b_rows(s, lane);
        bool waited = false;
        // E4M3: scales of this lane's columns, of this block and the next two
        const float *from[2] = {};
        float ahead[3][2] = {};
        if constexpr (kE4m3)
#pragma unroll
            for (int h = 0; h < 2; ++h) from[h] = p.b_scales(s, min(lane + 32 * h, s.n - 1));
        auto load_scales = [&](int kb, float (&x)[2]) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (lane + 32 * h < s.n) x[h] = __ldcg(from[h] + min(kb, s.kb1 - 1));
        };
        for (int kb = s.kb0; kb < s.kb1; ++kb, r.next(), ++issued) {
            bool go = true;
            if (lane == 0) {
                if (kb >= s.b_from && !waited) go = p.b_ready(s);
                if (go) go = wait(&c.empty_b[r.slot], r.round ^ 1, p.a.limits.wait_ns);
            }
            if (!__shfl_sync(0xffffffffu, go, 0)) return false;
            if (kb >= s.b_from && !waited) {   // other CTAs' ordinary stores, about to be read by TMA
                waited = true;
                __syncwarp();
                fence_proxy_async();
            }
            if constexpr (kE4m3) {
                if (kb == s.kb0)
#pragma unroll
                    for (int i = 0; i < 3; ++i) load_scales(kb + i, ahead[i]);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    scales[(issued % kScaleSlots) * 64 + lane + 32 * h] = ahead[0][h];
                    ahead[0][h] = ahead[1][h];
                    ahead[1][h] = ahead[2][h];
                }
                load_scales(kb + 3, ahead[2]);
                __syncwarp();
            }
            if (lane == 0) mbar_arrive_expect_tx(&c.full_b[r.slot], p.b_bytes(s, kb));
            __syncwarp();
            p.b_load(s, rows, kb, ring_base + sh.b_at(r.slot, kE4m3), &c.full_b[r.slot], policy, lane);
        }
        return true;
    });
    if (lane == 0) wait_fills(c.full_b, sh.b_stages, issued, p.a.limits.wait_ns);
    return ok;
}

// A whole warp waits and works out the operands; the same lane of it issues
// every product and commit.
//
// Products of bf16 weights.
template <class P>
__device__ bool multiply(const P &p, Control &c, uint32_t ring_base, const Shape sh, uint32_t tmem) {
    const bool mine = elect_one();
    Ring ra(sh.a_stages), rb(sh.b_stages), sums(sh.sums());
    const bool ok = p.segments([&](const Segment &s) {
        const uint32_t buf = sums.slot;
        const uint32_t desc = uniform(product_desc(s.n16())), d0 = uniform(tmem + buf * 2 * sh.cols);
        const uint32_t d1 = uniform(d0 + sh.cols);
        const bool two = uniform(s.two) != 0;
        if (!warp_wait(&c.sums_empty[buf], sums.round ^ 1, p.a.limits.wait_ns)) return false;
        tc_fence_after();
        for (int kb = s.kb0; kb < s.kb1; ++kb, ra.next(), rb.next()) {
            if (!warp_wait(&c.full_a[ra.slot], ra.round, p.a.limits.wait_ns) ||
                !warp_wait(&c.full_b[rb.slot], rb.round, p.a.limits.wait_ns))
                return false;
            tc_fence_after();
            const uint32_t a = uniform(operand_low(ring_base + sh.a_at(ra.slot)));
            const uint32_t b = uniform(operand_low(ring_base + sh.b_at(rb.slot, false)));
            const bool more = uniform(kb > s.kb0) != 0;
            uint32_t columns = desc, at = 0;
            if constexpr (P::kPieces)
                if (kb >= s.b_from) {   // a block of some of the tile's columns
                    const int4 piece = p.piece(s, kb);
                    columns = uniform(product_desc((piece.z + 15) & ~15));
                    at = uniform(piece.y - s.first);
                }
            if (mine) {
#pragma unroll
                for (int k = 0; k < 4; ++k) mma_ss(d0 + at, a + 2 * k, b + 2 * k, columns, more || k > 0);
                if (two)
#pragma unroll
                    for (int k = 0; k < 4; ++k) mma_ss(d1 + at, a + (kHalf >> 4) + 2 * k, b + 2 * k, columns, more || k > 0);
                mma_commit(&c.empty_a[ra.slot]);
                mma_commit(&c.empty_b[rb.slot]);
            }
            __syncwarp();
        }
        if (mine) mma_commit(&c.sums_full[buf]);
        __syncwarp();
        sums.next();
        return true;
    });
    if (mine) {
        mma_commit(&c.last);
        wait(&c.last, 0, p.a.limits.wait_ns);
    }
    return ok;
}

// E4M3: blocks' sums in tensor memory, 4 columns of it for each of a tile's.
constexpr int sum_buffers(int most_cols) { return most_cols <= 32 ? 4 : 2; }

// Products of E4M3 weights with activations split in two: first codes in columns
// [0, n16), second ones in [n16, 2 n16). Each block's sums start from zero.
template <class P>
__device__ bool multiply_e4m3(const P &p, Control &c, uint32_t ring_base, const Shape sh, uint32_t tmem) {
    const bool mine = elect_one();
    Ring ra(sh.a_stages), rb(sh.b_stages), sums(sum_buffers(8 * P::kSteps));
    const bool ok = p.segments([&](const Segment &s) {
        const uint32_t desc = uniform(product_desc(2 * s.n16(), true));
        for (int kb = s.kb0; kb < s.kb1; ++kb, ra.next(), rb.next(), sums.next()) {
            if (!warp_wait(&c.full_a[ra.slot], ra.round, p.a.limits.wait_ns) ||
                !warp_wait(&c.full_b[rb.slot], rb.round, p.a.limits.wait_ns) ||
                !warp_wait(&c.sums_empty[sums.slot], sums.round ^ 1, p.a.limits.wait_ns))
                return false;
            tc_fence_after();
            const uint32_t a = uniform(operand_low(ring_base + sh.a_at(ra.slot)));
            const uint32_t b = uniform(operand_low(ring_base + sh.b_at(rb.slot, true)));
            const uint32_t d0 = uniform(tmem + sums.slot * 4 * sh.cols), d1 = uniform(d0 + 2 * sh.cols);
            if (mine) {
#pragma unroll
                for (int k = 0; k < 4; ++k) mma_e4m3(d0, a + 2 * k, b + 2 * k, desc, k > 0);
#pragma unroll
                for (int k = 0; k < 4; ++k) mma_e4m3(d1, a + (kHalf >> 4) + 2 * k, b + 2 * k, desc, k > 0);
                mma_commit(&c.empty_a[ra.slot]);
                mma_commit(&c.empty_b[rb.slot]);
                mma_commit(&c.sums_full[sums.slot]);
                mbar_arrive(&c.sums_full[sums.slot]);   // hands the readers the scales that came with B
            }
            __syncwarp();
        }
        return true;
    });
    if (mine) {
        mma_commit(&c.last);
        wait(&c.last, 0, p.a.limits.wait_ns);
    }
    return ok;
}

// y scaled to |y| < 256 as a + b / 32, a and b E4M3 codes: what a leaves of y is 8 at
// most, half a step of the largest codes, so 32 times that stays below 448 and has
// five bits more to go before b's smallest step. a holds four bits, what is left
// has at most four more of a bf16's eight: the sum is y exactly for |y| >= 2^-7,
// and off by 2^-15 at most below, which is 2^-22 of a block's largest. Of an fp32
// it is within 2^-9 of y, or those 2^-15. (With b taken as it is, a block with one
// element 4096 times the others held these to six bits.)
constexpr float kSecond = 1.0f / 32;
struct Split {
    uint32_t first, second;   // low bytes
    __device__ __forceinline__ explicit Split(float y) {
        first = code(y);
        second = code((y - value(first)) * (1.0f / kSecond));
    }
    __device__ __forceinline__ static uint32_t code(float v) {
        uint16_t r;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(v));
        return r;
    }
    __device__ __forceinline__ static float value(uint32_t code) {
        float f;
        asm("{\n\t.reg .b16 t, lo, hi;\n\t.reg .b32 h;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 h, t;\n\t"
            "mov.b32 {lo, hi}, h;\n\tcvt.f32.f16 %0, lo;\n\t}"
            : "=f"(f) : "r"(code));
        return f;
    }
};

// The power of two under which a block with this largest magnitude stays below
// 256, and its inverse. A block with an infinity gets NaN for its scale: so does
// all that it is multiplied with.
struct BlockScale {
    float scale, inverse;
    __device__ __forceinline__ explicit BlockScale(float most) {
        const int e = max((int)(__float_as_uint(most) >> 23) - 7, 7);
        scale = most < INFINITY ? __uint_as_float((uint32_t)e << 23) : __uint_as_float(0x7fc00000u);
        inverse = __uint_as_float((uint32_t)(254 - e) << 23);
    }
};

// A thread's share of a tile's sums: one row, and eight values at a time.
// P::kHalves: eight columns of one half (side % 2), every second eight of them
// (side / 2) where four sides share the tile; else four columns of both halves,
// the first half's first, so that a thread holds both sums of a pair of weight
// rows. A step is 8 columns with two sides and 16 with four.
template <bool kHalves>
struct Share {
    int row, side;   // 0..127, 0..3
    __device__ static constexpr int step(int sides) { return sides == 2 ? 8 : 16; }
    __device__ static Share of(int warp) { return Share{(warp & 3) * 32 + (int)(threadIdx.x & 31), warp / 4}; }
    __device__ int first_col() const { return kHalves ? (side >> 1) * 8 : side * 4; }
    __device__ int half_of(int j) const { return kHalves ? side & 1 : j / 4; }
    __device__ static int col_of(int j) { return kHalves ? j : j & 3; }
    __device__ void load(uint32_t at, int cols, int col, float (&v)[8]) const {
        if (kHalves) {
            tmem_load8(at + (side & 1) * cols + col, v);
        } else {
            tmem_load4(at + col, v);
            tmem_load4(at + cols + col, v + 4);
        }
        tmem_load_wait(v);
    }
};

// This CTA's part of a tile that it shares: fp32 partial sums to the workspace, [half][column][row].
template <class P, class Each>
__device__ void leave_part(const P &p, const Shape sh, const Segment &s, const Share<P::kHalves> me, Each each) {
    if (P::kHalves && !s.two && (me.side & 1)) return;
    const size_t half = (size_t)sh.cols * kRows;
    float *mine = p.partial(s.line, blockIdx.x, s.kb0 > 0 ? 0 : 1) + me.row;
    each([&](int col, const float *v) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int at = col + me.col_of(j);
            if (at < s.n) mine[me.half_of(j) * half + at * kRows] = v[j];
        }
    });
}

// This CTA's share of the columns of such a tile, in steps of 16, once all parts are there.
template <class Tm, class P>
__device__ bool add_up(const P &p, const Shape sh, const Segment &s) {
    constexpr int kSides = Tm::count / 128;
    const int skip = P::kHalves && !s.two ? 2 : 1;   // the first half's units alone
    const int units = P::kHalves ? (s.n + 7) / 8 * 2 / skip : (s.n + 3) / 4;
    const int shares = min(s.parts, (units + kSides - 1) / kSides), me = blockIdx.x - s.cta0;
    if (me >= shares) return true;
    bool ok = true;
    if (Tm::leader()) ok = wait_count(p.arrivals(s.line, s.cta0), (uint32_t)s.parts, p.a.limits.wait_ns);
    if (!Tm::agree(ok)) return false;
    const size_t half = (size_t)sh.cols * kRows;
    // unit: side unit % 4 of the 16 columns unit / 4; each of the team's groups of 128 threads takes one at a time
    for (int unit = me * kSides + Tm::warp() / 4; unit < units; unit += s.parts * kSides) {
        Share<P::kHalves> share = Share<P::kHalves>::of(Tm::warp());
        share.side = unit * skip & 3;
        const int col = (unit * skip >> 2) * 16 + share.first_col();
        // 32 loads at once, of four parts: a trip to another SM's sums in L2 takes about a microsecond.
        // (Twice as many for two units were no faster: code that runs once waits for its instructions.)
        float v[8] = {};
#pragma unroll 1
        for (int i0 = 0; i0 < s.parts; i0 += 4) {
            float x[4][8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // the stretch that begins the tile is its CTA's last, the others their CTA's first
                const float *part = p.partial(s.line, s.cta0 + i0 + i, i0 + i == 0 ? 1 : 0) + share.row;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int at = col + share.col_of(j);
                    x[i][j] = i0 + i < s.parts && at < s.n ? __ldcg(part + share.half_of(j) * half + at * kRows) : 0.0f;
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] += x[i][j];
        }
        typename P::Emit emit(p, s, share);
        emit(col, v);
    }
    __threadfence();
    Tm::sync();
    // the shares' weights add up to kTileWeight
    if (Tm::leader()) p.tile_done(s, kTileWeight * (me + 1) / shares - kTileWeight * me / shares);
    return true;
}

// What the reader threads do with a segment's sums. `each(f)` calls f(column,
// 8 values) for all of the thread's columns, `release()` gives up the sums' place.
// Where others wait for the results the announcing warp tells them: its fences
// take microseconds that the readers have not.
template <class P, class Each, class Release>
__device__ bool take(const P &p, Control &c, const Shape sh, const Segment &s, const Share<P::kHalves> me, Each each,
                     Release release) {
    if (P::kShares && !s.whole()) {
        if constexpr (P::kShares) leave_part(p, sh, s, me, each);
    } else {
        typename P::Emit emit(p, s, me);
        each([&](int col, const float *v) { emit(col, v); });
    }
    release();
    if constexpr (P::kShares) {
        __syncwarp();
        if ((threadIdx.x & 31) == 0)
            asm volatile("red.release.cta.shared::cta.add.u32 [%0], 1;" ::"r"(smem_addr(&c.written)) : "memory");
    }
    return true;
}

// One lane: announces each segment once all reader warps have written its results
// (but for a test's withheld one).
template <class P>
__device__ bool announce(const P &p, Control &c) {
    uint32_t want = 0;
    bool withheld = blockIdx.x == p.a.limits.withheld_cta;
    return p.segments([&](const Segment &s) {
        want += P::kReaders / 32;
        const uint64_t deadline = globaltimer_ns() + p.a.limits.wait_ns;
        while (true) {
            uint32_t now;
            asm volatile("ld.acquire.cta.shared::cta.u32 %0, [%1];" : "=r"(now) : "r"(smem_addr(&c.written)) : "memory");
            if (now >= want) break;
            if (globaltimer_ns() > deadline) return false;
            __nanosleep(100);
        }
        if (withheld) {
            withheld = false;
            return true;
        }
        __threadfence();
        if (s.whole()) p.tile_done(s, kTileWeight);
        else count_up(p.arrivals(s.line, s.cta0), 1u);
        return true;
    });
}

// A CTA's shared tiles (of one phase, by the readers), all of whose parts it has left or will leave.
template <class Tm, class P, class... Phase>
__device__ bool add_shared(const P &p, const Shape sh, Phase... phase) {
    return p.segments([&](const Segment &s) { return s.whole() || add_up<Tm>(p, sh, s); }, phase...);
}

// Readers of bf16 weights' sums.
template <class P>
__device__ bool read_sums(const P &p, Control &c, const Shape sh, uint32_t tmem) {
    using Tm = ReadersOf<P>;
    const int lane = threadIdx.x & 31;
    const Share<P::kHalves> me = Share<P::kHalves>::of(Tm::warp());
    Ring sums(sh.sums());
    constexpr bool kAdd = P::kShares && !P::kAdders;
    int phase = 0;
    bool ok = p.segments([&](const Segment &s) {
        if constexpr (kAdd)
            for (; phase < s.phase; ++phase)
                if (!add_shared<Tm>(p, sh, phase, phase + 1)) return false;
        const uint32_t buf = sums.slot;
        if (!Tm::agree(wait(&c.sums_full[buf], sums.round, p.a.limits.wait_ns))) return false;
        tc_fence_after();
        const uint32_t at = tmem + ((uint32_t)(me.row & ~31) << 16) + buf * 2 * sh.cols;
        auto each = [&](auto f) {
            for (int col = me.first_col(); col < s.n16(); col += me.step(Tm::count / 128)) {
                float v[8];
                me.load(at, sh.cols, col, v);
                if (col < s.n) f(col, v);
            }
        };
        auto release = [&] {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&c.sums_empty[buf]);
        };
        sums.next();
        return take(p, c, sh, s, me, each, release);
    });
    if constexpr (kAdd)
        for (; ok && phase < P::kPhases; ++phase) ok = add_shared<Tm>(p, sh, phase, phase + 1);
    return ok;
}

// Readers of E4M3 weights' sums: each block's, scaled, into registers; tiles of up to 8 kSteps columns.
template <int kSteps, class P>
__device__ bool read_sums_e4m3(const P &p, Control &c, const float *b_scales, const Shape sh, uint32_t tmem) {
    using Tm = ReadersOf<P>;
    static_assert(!P::kHalves && P::kReaders == 256, "a thread scales both halves, two sides share the columns");
    const int lane = threadIdx.x & 31;
    const Share<false> me = Share<false>::of(Tm::warp());
    const uint32_t at0 = tmem + ((uint32_t)(me.row & ~31) << 16);
    Ring sums(sum_buffers(8 * kSteps));
    uint32_t block = 0;
    return p.segments([&](const Segment &s) {
        float acc[kSteps][8] = {};
        const float *scales = p.scales(s.phase);
        const int rows = p.weight_rows(s.phase);
        const float *s0 = scales + (size_t)min(s.row0 + me.row, rows - 1) * s.kbs;
        const float *s1 = scales + (size_t)min(s.row1 + me.row, rows - 1) * s.kbs;
        bool ok = true;
        // weights' scales come four blocks ahead: every eighth block's are in a new sector
        float w0[4], w1[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) w0[u] = __ldg(s0 + min(s.kb0 + u, s.kb1 - 1)), w1[u] = __ldg(s1 + min(s.kb0 + u, s.kb1 - 1));
#pragma unroll 1
        for (int kb = s.kb0; kb < s.kb1; ++kb) {
            const float now0 = w0[0], now1 = w1[0];
#pragma unroll
            for (int u = 0; u < 3; ++u) w0[u] = w0[u + 1], w1[u] = w1[u + 1];
            const int later = min(kb + 4, s.kb1 - 1);
            w0[3] = __ldg(s0 + later), w1[3] = __ldg(s1 + later);
            if (!warp_wait(&c.sums_full[sums.slot], sums.round, p.a.limits.wait_ns)) { ok = false; break; }
            tc_fence_after();
            const float *of_block = b_scales + (block++ % kScaleSlots) * 64 + me.first_col();
            const uint32_t at = at0 + sums.slot * 4 * sh.cols + me.first_col();
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                if (i * 8 >= s.n16()) break;
                float v[16];   // first and second codes' sums of half 0, then of half 1
                tmem_load4(at + i * 8, v);
                tmem_load4(at + s.n16() + i * 8, v + 4);
                tmem_load4(at + 2 * sh.cols + i * 8, v + 8);
                tmem_load4(at + 2 * sh.cols + s.n16() + i * 8, v + 12);
                tmem_load_wait(v);
                if ((i + 1) * 8 >= s.n16()) {   // all of the block's sums are in registers
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&c.sums_empty[sums.slot]);
                }
                const float4 bs = *reinterpret_cast<const float4 *>(of_block + i * 8);
                const float scale[4] = {bs.x, bs.y, bs.z, bs.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    acc[i][j] = fmaf(now0 * scale[j], fmaf(v[4 + j], kSecond, v[j]), acc[i][j]);
                    acc[i][4 + j] = fmaf(now1 * scale[j], fmaf(v[12 + j], kSecond, v[8 + j]), acc[i][4 + j]);
                }
            }
            sums.next();
        }
        if (!Tm::agree(ok)) return false;
        // One copy of f's code: a tile runs it once, and with a copy for every step the
        // instructions came from L2 at some 2 us a step.
        auto each = [&](auto f) {
#pragma unroll 1
            for (int col = me.first_col(); col < s.n; col += 8) {
                f(col, acc[0]);
#pragma unroll
                for (int i = 0; i + 1 < kSteps; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) acc[i][j] = acc[i + 1][j];
            }
        };
        return take(p, c, sh, s, me, each, [] {});
    });
}

template <class P>
constexpr int threads_of() {
    return ReadersOf<P>::first + P::kReaders + (P::kAdders ? kAdders : 0);
}

// Barriers and tensor memory, then `roles(problem, ring, tensor memory, warp, ok)`
// on every thread; `problem(ring)` makes the problem after the set-up, when the
// ring is still unused.
template <class P, class Make, class Roles>
__device__ void with_set_up(Make problem, Control &c, const uint32_t tmem_cols, Roles roles) {
    extern __shared__ char smem_raw[];
    const int warp = (int)uniform(threadIdx.x / 32);
    char *ring = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    if (threadIdx.x == 0) {
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(&c.full_a[i], 1);
            mbar_init(&c.full_b[i], 1);
            mbar_init(&c.empty_a[i], 1);
            mbar_init(&c.empty_b[i], 1);
        }
        for (int i = 0; i < kMaxSums; ++i) {
            mbar_init(&c.sums_full[i], P::kCodes ? 2 : 1);
            mbar_init(&c.sums_empty[i], P::kReaders / 32);
        }
        mbar_init(&c.last, 1);
        c.written = 0;
        fence_barrier_init();
    }
    if (warp == 3) tmem_alloc(&c.tmem, tmem_cols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = c.tmem;
    const P p = problem(ring);
    bool ok = true;
    roles(p, ring, tmem, warp, ok);
    if (!ok) report(p.status, MOE_ERR_TIMEOUT);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 3) tmem_free(tmem, tmem_cols);
}

// The whole kernel body, threads_of<P>() threads; P::finish runs on the reader
// threads after the last segment.
template <bool kE4m3, class P, class Make>
__device__ void run(Make problem, const Shape sh, const uint32_t tmem_cols) {
    __shared__ Control c;
    with_set_up<P>(problem, c, tmem_cols, [&](const P &p, char *ring, uint32_t tmem, int warp, bool &ok) {
        float *scales = reinterpret_cast<float *>(ring + sh.ring_bytes(kE4m3));   // E4M3
        if (warp == 0) ok = load_a(p, c, smem_addr(ring), sh);
        else if (warp == 1) ok = load_b<kE4m3>(p, c, smem_addr(ring), scales, sh);
        else if (warp == 2) {
            if constexpr (kE4m3) ok = multiply_e4m3(p, c, smem_addr(ring), sh, tmem);
            else ok = multiply(p, c, smem_addr(ring), sh, tmem);
        } else if (warp == 3) {
            if constexpr (P::kShares)
                if ((threadIdx.x & 31) == 0) ok = announce(p, c);
        } else if (threadIdx.x >= AddersOf<P>::first) {
            if constexpr (P::kAdders) ok = add_shared<AddersOf<P>>(p, sh);
        } else if (threadIdx.x >= ReadersOf<P>::first) {
            if constexpr (kE4m3) ok = read_sums_e4m3<P::kSteps>(p, c, scales, sh, tmem);
            else ok = read_sums(p, c, sh, tmem);
            if (ok) ok = p.finish();
        }
    });
}

// bf16 weights, one segment: `finish(problem, control, ring, tensor memory, ok)`
// on every thread once the other roles are through (it waits for the sums itself).
template <class P, class Make, class Finish>
__device__ void run_one(Make problem, const Shape sh, const uint32_t tmem_cols, Finish finish) {
    __shared__ Control c;
    with_set_up<P>(problem, c, tmem_cols, [&](const P &p, char *ring, uint32_t tmem, int warp, bool &ok) {
        if (warp == 0) ok = load_a(p, c, smem_addr(ring), sh);
        else if (warp == 1) ok = load_b<false>(p, c, smem_addr(ring), nullptr, sh);
        else if (warp == 2) ok = multiply(p, c, smem_addr(ring), sh, tmem);
        __syncwarp();
        finish(p, c, ring, tmem, ok);
    });
}

// Words at the head of a workspace: the numbers of groups and of those with a set
// that is named; the count of finished tiles (64 bits), or of a plan in tiles their
// number and that of its places; arrivals of parts by line and CTA.
constexpr int kGroupsWord = 0, kNamedWord = 1, kDoneWord = 2, kTilesWord = 2, kPlacesWord = 3, kArrivals = 4,
              kWords = 4 + kMaxLines * kMaxCtas;

// ------------------------------------------------------------------ plan

// Sorts entries by the weight set that they name and cuts each set's into groups
// of at most `cols`; clears the counters of the kernel behind it. In tiles
// (kTiles): each set begins at a multiple of 16 places, and groups end where
// tiles of `cols` places do, so that a tile consists of whole groups.
constexpr int kPlaceStep = 16;   // the tensor core's step of columns
template <typename Index>
struct PlanArgs {
    const Index *idx;        // [n], -1: none
    int n, sets;
    bool rest;               // entries that name none make up a last set of their own
    int cols;
    uint32_t *words;         // the numbers of groups and of those with a set that is named; the rest become 0
    int num_words;
    int4 *groups;            // {set, first sorted entry, entries, 0}
    int *order;              // sorted entries, in tiles -1 in the places between them
    int *place;              // in tiles: each entry's place
    int *tiles;              // in tiles: each tile's first group, then the number of groups
    int bad;                 // status of an index out of range
    bool beside;             // runs beside the kernel before it, which began after all that idx depends on was complete
    int32_t *status;
    TraceArgs trace;
};

constexpr int kPlanThreads = 1024;

// Warps that sort, each a stretch of the entries with counters of its own, and
// the shared memory that they and the three sums over the sets take.
inline int plan_warps(int sets) { return std::max(1, std::min(kPlanThreads / 32, (220 << 10) / (4 * (sets + 1)) - 3)); }
inline size_t plan_smem(int sets) { return ((size_t)plan_warps(sets) + 3) * (sets + 1) * 4; }

// Sets in order, entries of a set in their own order: where entries change
// places between groups, their sums are cut elsewhere and may round otherwise, so
// the same choice has to give the same groups. One CTA, bound by the latency of its
// passes: 512 entries of 32 sets 7 us, 4096 entries of 17 sets in tiles 10 us.
template <typename Index, bool kTiles>
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanArgs<Index> a, const int warps) {
    WarpTrace wt(a.trace, MOE_TRACE_PLAN);
    if (!a.beside) grid_dependency_wait();
    grid_launch_dependents();   // the next kernel's set-up
    extern __shared__ int32_t plan_memory[];
    const int sets = a.sets + (a.rest ? 1 : 0);
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    int32_t *start = plan_memory, *first_group = start + sets + 1, *entries = first_group + sets + 1;
    int32_t *counts = entries + sets + 1, *mine = counts + (size_t)warp * sets;   // [warps][sets]
    auto set_of = [&](Index e) { return e >= 0 && e < a.sets ? (int)e : a.rest ? a.sets : -1; };
    for (int i = threadIdx.x; i < warps * sets; i += kPlanThreads) counts[i] = 0;
    for (int i = threadIdx.x; i < a.num_words; i += kPlanThreads) a.words[i] = 0;
    __syncthreads();
    const int per = ((a.n + warps - 1) / warps + 31) / 32 * 32;   // entries of a warp
    const int64_t first = (int64_t)warp * per;
    const int begin = warp < warps && first < a.n ? (int)first : a.n, end = min(a.n, begin + per);
    for (int i = begin + lane; i < end; i += 32) {
        const Index e = a.idx[i];
        if (e < -1 || e >= a.sets) report(a.status, a.bad);
        if (set_of(e) >= 0) atomicAdd(&mine[set_of(e)], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < sets; e += kPlanThreads) {   // each warp's first place in a set
        int total = 0;
        for (int w = 0; w < warps; ++w) {
            const int c = counts[(size_t)w * sets + e];
            counts[(size_t)w * sets + e] = total;
            total += c;
        }
        entries[e] = total;
        start[e] = kTiles ? (total + kPlaceStep - 1) / kPlaceStep * kPlaceStep : total;
        if (!kTiles) first_group[e] = (total + a.cols - 1) / a.cols;
    }
    __syncthreads();
    if (warp == 0) warp_exclusive_scan(start, sets, lane);
    if constexpr (kTiles) {
        __syncthreads();
        for (int e = threadIdx.x; e < sets; e += kPlanThreads)
            first_group[e] = entries[e] > 0 ? (start[e] + entries[e] - 1) / a.cols - start[e] / a.cols + 1 : 0;
        __syncthreads();
    }
    if (warp == 1) warp_exclusive_scan(first_group, sets, lane);
    __syncthreads();
    for (int e = threadIdx.x; e < sets; e += kPlanThreads) {
        const int last = start[e] + entries[e];
        for (int g = first_group[e], b = start[e]; b < last; ++g) {
            const int end = min(last, kTiles ? (b / a.cols + 1) * a.cols : b + a.cols);
            a.groups[g] = make_int4(e, b, end - b, 0);
            // the first group of a tile begins it: a set that begins elsewhere follows another's last entries
            if (kTiles && b % a.cols == 0) a.tiles[b / a.cols] = g;
            b = end;
        }
        if constexpr (kTiles)
            for (int b = last; b < start[e + 1]; ++b) a.order[b] = -1;
    }
    if (threadIdx.x == 0) {
        a.words[kGroupsWord] = first_group[sets];
        a.words[kNamedWord] = first_group[a.sets];
        if constexpr (kTiles) {
            const int tiles = (start[sets] + a.cols - 1) / a.cols;
            a.words[kTilesWord] = tiles;
            a.words[kPlacesWord] = start[sets];
            a.tiles[tiles] = first_group[sets];
        }
    }
    for (int i0 = begin; i0 < end; i0 += 32) {
        const int i = i0 + lane, e = i < end ? set_of(a.idx[i]) : -1;
        const uint32_t same = __match_any_sync(0xffffffffu, e);
        if (e >= 0) {
            const int place = start[e] + mine[e] + __popc(same & ((1u << lane) - 1));
            a.order[place] = i;
            if constexpr (kTiles) a.place[i] = place;
        }
        __syncwarp();
        if (e >= 0 && same >> lane == 1) mine[e] += __popc(same);   // the last of them
        __syncwarp();
    }
    if (a.beside) grid_dependency_wait();   // the next kernel waits for this one alone
}

// The same for few entries, by every CTA for itself in its shared memory: no
// launch before, and no chain of loads from its results. CTAs have to agree, so an
// entry's place is fixed: by set, then in the order of the entries. A few threads
// to a set look through the entries for its own, 32 to a word of a mask. (By
// counters in shared memory this took 2.8 us, by matching a warp's entries 4, and
// the plan kernel with its launch takes 5.)
constexpr int kLocalEntries = 256, kLocalSets = 512;
struct LocalPlan {
    uint32_t groups[kLocalEntries];    // set | first sorted entry << 13 | (entries - 1) << 21
    uint16_t order[kLocalEntries];
    uint16_t set_of[kLocalEntries];    // 0xffff: none
    uint32_t totals[kLocalSets / 32];  // entries | groups << 16 of a warp's sets
    int num_groups;
};

// All threads of the CTA, at least kLocalSets.
template <typename Index>
__device__ void local_plan(LocalPlan &plan, const Index *idx, int n, int sets, int cols, int bad, int32_t *status) {
    const int tid = threadIdx.x, lane = threadIdx.x & 31;
    if (tid < kLocalEntries) {
        const Index e = tid < n ? idx[tid] : (Index)-1;
        const bool named = e >= 0 && e < sets;
        if (!named && e != -1 && blockIdx.x == 0) report(status, bad);
        plan.set_of[tid] = named ? (uint16_t)e : (uint16_t)0xffff;
    }
    __syncthreads();
    // 2^split threads to a set, each with `words` words of 32 entries
    constexpr int kWords = kLocalEntries / 32;
    const int split = min(3, 31 - __clz(kLocalSets / sets)), part = tid & ((1 << split) - 1), set = tid >> split;
    const int words = (((n + 31) / 32) + (1 << split) - 1) >> split;
    uint32_t mine[kWords] = {};
    uint32_t count = 0;
    if (set < sets)
#pragma unroll
        for (int j = 0; j < kWords; ++j) {
            const int w = part * words + j;
            if (j >= words || w * 32 >= n) break;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint4 v = *reinterpret_cast<const uint4 *>(&plan.set_of[w * 32 + q * 8]);
                const uint32_t two[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    if ((two[h] & 0xffff) == (uint32_t)set) mine[j] |= 1u << (q * 8 + 2 * h);
                    if (two[h] >> 16 == (uint32_t)set) mine[j] |= 2u << (q * 8 + 2 * h);
                }
            }
            count += __popc(mine[j]);
        }
    uint32_t all = count, groups = 0, before = 0, here = 0;   // entries of the set; before the set and in it before this thread
    if (tid < kLocalSets) {
        for (int o = 1; o < 1 << split; o <<= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
        groups = (uint32_t)quotient(all + cols - 1, cols);
        // entries | groups << 16 of the warp's sets, the groups by a set's first thread
        const uint32_t both = count | (part == 0 ? groups << 16 : 0);
        uint32_t sum = both;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += v;
        }
        if (lane == 31) plan.totals[tid / 32] = sum;
        here = sum - both;
    }
    __syncthreads();
    if (set < sets && tid < kLocalSets) {
        for (int w = 0; w < tid / 32; ++w) before += plan.totals[w];
        before += here;
        int at = before & 0xffff;
        if (part == 0) {
            int g = before >> 16;
            for (int b = 0; b < (int)all; b += cols, ++g)
                plan.groups[g] = (uint32_t)set | (uint32_t)(at + b) << 13 | (uint32_t)(min(cols, (int)all - b) - 1) << 21;
            if (set == sets - 1) plan.num_groups = g;
        }
#pragma unroll
        for (int j = 0; j < kWords; ++j)
            for (uint32_t m = mine[j]; m != 0; m &= m - 1)
                plan.order[at++] = (uint16_t)((part * words + j) * 32 + __ffs(m) - 1);
    }
    __syncthreads();
}

// Zeroes the counters where no plan kernel does.
static __global__ void __launch_bounds__(1024) clear_kernel(uint32_t *words, int n) {
    grid_dependency_wait();
    for (int i = threadIdx.x; i < n; i += 1024) words[i] = 0;
}

template <bool kTiles, typename Index>
int launch_plan(const PlanArgs<Index> &a, cudaStream_t s) {
    const int sets = a.sets + (a.rest ? 1 : 0);
    const size_t smem = plan_smem(sets);
    const int rc = ensure_dynamic_smem((const void *)plan_kernel<Index, kTiles>, smem);
    if (rc != MOE_OK) return rc;
    return launch_kernel(plan_kernel<Index, kTiles>, dim3(1), dim3(kPlanThreads), smem, s, tuning().overlap != 0, a,
                         plan_warps(sets)) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// One CTA per SM, all of them resident at once (they wait for one another).
template <class Args>
int launch_resident(void (*kernel)(Args), Args &a, int threads, size_t smem, cudaStream_t s) {
    const int rc = ensure_dynamic_smem((const void *)kernel, smem);
    if (rc != MOE_OK) return rc;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(device_sm_count() < kMaxCtas ? device_sm_count() : kMaxCtas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = tuning().overlap ? 2 : 1;
    void *args[] = {&a};
    return cudaLaunchKernelExC(&cfg, (const void *)kernel, args) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// Partial sums of `lines` lines: two tiles per CTA and line.
constexpr size_t partial_floats(int lines, int cols) { return (size_t)lines * kMaxCtas * 2 * 2 * cols * kRows; }

// Byte offsets of the pieces of a workspace, each 256-byte aligned.
struct Cut {
    size_t at = 0;
    size_t take(size_t bytes) {
        const size_t o = at;
        at += (bytes + 255) / 256 * 256;
        return o;
    }
};

}  // namespace skinny
}  // namespace moe
