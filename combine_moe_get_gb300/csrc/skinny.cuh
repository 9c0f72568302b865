// skinny.cuh -- matrix products of long weight matrices with few rows of
// activations, as one persistent kernel body: D[256 weight rows x n columns] =
// A[256 x K] B[n x K]^T, the weights as the tensor core's 128-row operand (twice,
// over one B tile) and the activations as its n columns (16..128).
//
// What bounds it is the stream of weights, so the work is cut by bytes: all
// tiles' K blocks stand in one line, each CTA takes an equal stretch of it
// (tiles may begin and end inside a stretch), and a CTA's loads run ahead of
// its products across tile and phase borders. A tile that several CTAs share
// is summed by the last of them to arrive, in the order of K, from fp32
// partial sums in the workspace: the result does not depend on the arrival
// order.
//
// Roles of a CTA's 12 warps: 0 loads A (weights), 1 loads B (activations), 2
// issues the products, 3 owns the tensor memory, 4..11 read the sums.
//   bf16 weights: A and B from shared memory; sums stay in tensor memory for a
//     whole stretch of K, double-buffered, so that the readers' work on one
//     tile runs under the next tile's products.
//   E4M3 weights: the reader warps also turn each block's codes into bf16 (exact)
//     in tensor memory, from where the products take A; a block of 128 along K
//     has its own fp32 scale per weight row, so the block's sums are scaled and
//     added in registers (n <= 64).
//
// The problem P gives the segments, the loads of B and what becomes of the sums.
#pragma once

#include "umma.cuh"

namespace moe {
namespace skinny {

constexpr int kThreads = 384;
constexpr int kReaders = 256;          // threads of warps 4..11
constexpr int kRows = 128;             // weight rows of one product; a tile has two
constexpr int kHalf = kRows * 128;     // bytes of one A tile of a stage
constexpr int kMaxCtas = 160;
constexpr int kMaxStages = 8;
constexpr int kSmemBudget = 224 << 10;
constexpr int kMinBlocks = 8;          // K blocks a CTA takes at least (or a whole tile)

// One CTA's stretch of one tile.
struct Segment {
    const CUtensorMap *a_map;
    int row0, row1;       // weight rows of the two products
    int row_end;          // rows of the whole weight matrix
    int a_bytes;          // bytes of A that a K block loads for one product
    bool two;             // both products (else the first alone)
    int kb0, kb1, kbs;    // K blocks [kb0, kb1) of the tile's kbs
    int n;                // columns in use
    int phase, f, group, first;   // which tile: phase, feature tile, group and its first row
    int cta0, parts;      // the CTAs that share the tile: cta0 .. cta0 + parts - 1
    __device__ int n16() const { return (n + 15) & ~15; }
    __device__ bool whole() const { return kb0 == 0 && kb1 == kbs; }
};

// The line of K blocks of one phase: `tiles` tiles of `kbs` blocks, `per` blocks to a CTA.
struct Line {
    int64_t units, per;
    int kbs;
    __device__ Line(int64_t tiles, int k_blocks, int ctas) {
        kbs = k_blocks;
        units = tiles * kbs;
        per = (units + ctas - 1) / ctas;
        const int64_t least = kbs < kMinBlocks ? kbs : kMinBlocks;
        if (per < least) per = least;
    }
    // Each segment of CTA `cta`, in order: f(tile, segment with K range and sharing CTAs filled in).
    template <class F>
    __device__ bool each(int cta, F f) const {
        int64_t u = cta * per;
        const int64_t end = u + per < units ? u + per : units;
        while (u < end) {
            const int64_t tile = u / kbs, begin = tile * kbs;
            Segment s;
            s.kbs = kbs;
            s.kb0 = (int)(u - begin);
            s.kb1 = end - begin < kbs ? (int)(end - begin) : kbs;
            s.cta0 = (int)(begin / per);
            s.parts = (int)((begin + kbs - 1) / per) - s.cta0 + 1;
            if (!f(tile, s)) return false;
            u = begin + s.kb1;
        }
        return true;
    }
};

struct Control {
    uint64_t full_a[kMaxStages], full_b[kMaxStages], empty[kMaxStages];
    uint64_t sums_full[2], sums_empty[2];
    uint64_t a_ready[2];     // E4M3: converted block in tensor memory
    uint64_t last;
    uint32_t tmem;
    int vote;
};

struct Shape {
    int cols;      // columns a tile may have: a multiple of 16, at most 128 (E4M3: 64)
    int stages;
    static constexpr int b_bytes(int cols, bool e4m3) { return cols * (e4m3 ? 256 : 128); }
    static constexpr int stage_bytes(int cols, bool e4m3) { return 2 * kHalf + b_bytes(cols, e4m3); }
    static int stages_for(int cols, bool e4m3) {
        const int s = kSmemBudget / stage_bytes(cols, e4m3);
        return s < kMaxStages ? s : kMaxStages;
    }
    static size_t smem(int cols, bool e4m3) { return 1024 + (size_t)stages_for(cols, e4m3) * stage_bytes(cols, e4m3); }
    static int tmem_cols(int cols, bool e4m3) {
        if (e4m3) return 512;
        int c = 32;
        while (c < 4 * cols) c *= 2;
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

__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity) {
    return mbar_wait_bounded(bar, parity, kDefaultWaitNs);
}

// ... by a whole warp, which goes on or gives up as one.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait(bar, parity));
}

// All reader threads agree: true if every one of them says so.
__device__ __forceinline__ bool readers_agree(bool ok) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.and.pred q, 1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r) : "r"((uint32_t)ok) : "memory");
    return r != 0;
}
__device__ __forceinline__ void readers_sync() { asm volatile("barrier.cta.sync 1, 256;" ::: "memory"); }

// Wait (bounded) until the word reaches `want`; release/acquire with add_release.
__device__ __forceinline__ bool wait_count(const uint32_t *p, uint32_t want) {
    if (ld_acquire_gpu_u32(p) >= want) return true;
    const uint64_t deadline = globaltimer_ns() + kDefaultWaitNs;
    while (ld_acquire_gpu_u32(p) < want)
        if (globaltimer_ns() > deadline) return false;
    return true;
}
__device__ __forceinline__ uint32_t add_acq_rel(uint32_t *p, uint32_t v) {
    uint32_t old;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
    return old;
}

// ------------------------------------------------------------------ roles

template <bool kE4m3, class P>
__device__ bool load_a(const P &p, Control &c, uint32_t ring_base, const Shape sh) {
    const uint64_t policy = policy_evict_first();
    const int lane = threadIdx.x & 31;
    Ring r(sh.stages);
    int issued = 0;
    bool ok = true;
    if (lane == 0) {
        ok = p.segments([&](const Segment &s) {
            for (int kb = s.kb0; kb < s.kb1; ++kb, r.next(), ++issued) {
                if (!wait(&c.empty[r.slot], r.round ^ 1)) return false;
                const uint32_t dst = ring_base + r.slot * Shape::stage_bytes(sh.cols, kE4m3);
                const int col = kb * (kE4m3 ? 128 : 64);
                mbar_arrive_expect_tx(&c.full_a[r.slot], s.two ? 2 * s.a_bytes : s.a_bytes);
                tma_load(dst, s.a_map, col, s.row0, &c.full_a[r.slot], policy);
                if (s.two) tma_load(dst + kHalf, s.a_map, col, s.row1, &c.full_a[r.slot], policy);
            }
            return true;
        });
        if (!ok)   // leave only when the loads in flight have landed
            for (int i = 0; i < sh.stages && i < issued; ++i) {
                const int fill = issued - 1 - i;
                wait(&c.full_a[fill % sh.stages], (fill / sh.stages) & 1);
            }
    }
    return ok;
}

template <bool kE4m3, class P>
__device__ bool load_b(const P &p, Control &c, uint32_t ring_base, const Shape sh) {
    const int lane = threadIdx.x & 31;
    Ring r(sh.stages);
    int issued = 0;
    const bool ok = p.segments([&](const Segment &s) {
        bool ready = true;
        if (lane == 0) ready = p.b_ready(s);
        if (!__shfl_sync(0xffffffffu, ready, 0)) return false;
        typename P::Rows rows = p.b_rows(s, lane);
        for (int kb = s.kb0; kb < s.kb1; ++kb, r.next(), ++issued) {
            bool free = true;
            if (lane == 0) {
                free = wait(&c.empty[r.slot], r.round ^ 1);
                if (free) mbar_arrive_expect_tx(&c.full_b[r.slot], p.b_bytes(s) * (kE4m3 ? 2 : 1));
            }
            if (!__shfl_sync(0xffffffffu, free, 0)) return false;
            const uint32_t dst = ring_base + r.slot * Shape::stage_bytes(sh.cols, kE4m3) + 2 * kHalf;
#pragma unroll
            for (int h = 0; h < (kE4m3 ? 2 : 1); ++h)
                p.b_load(s, rows, (kb * (kE4m3 ? 2 : 1) + h) * 64, dst + h * sh.cols * 128, &c.full_b[r.slot], lane);
        }
        return true;
    });
    if (!ok && lane == 0)
        for (int i = 0; i < sh.stages && i < issued; ++i) {
            const int fill = issued - 1 - i;
            wait(&c.full_b[fill % sh.stages], (fill / sh.stages) & 1);
        }
    return ok;
}

// Products of bf16 weights: lane 0 of one warp.
template <class P>
__device__ bool multiply(const P &p, Control &c, uint32_t ring_base, const Shape sh, uint32_t tmem) {
    Ring r(sh.stages);
    uint32_t seq = 0;
    const bool ok = p.segments([&](const Segment &s) {
        const uint32_t buf = seq & 1, desc = product_desc(s.n16());
        const uint32_t d0 = tmem + buf * 2 * sh.cols, d1 = d0 + sh.cols;
        if (!wait(&c.sums_empty[buf], (seq >> 1 & 1) ^ 1)) return false;
        tc_fence_after();
        for (int kb = s.kb0; kb < s.kb1; ++kb, r.next()) {
            if (!wait(&c.full_a[r.slot], r.round) || !wait(&c.full_b[r.slot], r.round)) return false;
            tc_fence_after();
            const uint32_t at = ring_base + r.slot * Shape::stage_bytes(sh.cols, false);
            const uint64_t a0 = operand_desc(at), a1 = operand_desc(at + kHalf), b = operand_desc(at + 2 * kHalf);
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_ss(d0, a0 + 2 * k, b + 2 * k, desc, kb > s.kb0 || k > 0);
            if (s.two)
#pragma unroll
                for (int k = 0; k < 4; ++k) mma_ss(d1, a1 + 2 * k, b + 2 * k, desc, kb > s.kb0 || k > 0);
            mma_commit(&c.empty[r.slot]);
        }
        mma_commit(&c.sums_full[buf]);
        ++seq;
        return true;
    });
    if (!ok) {
        mma_commit(&c.last);
        wait(&c.last, 0);
    }
    return ok;
}

constexpr int kTmemCodes = 256;   // E4M3: first tensor-memory column of the converted blocks

// Products of converted E4M3 blocks: lane 0 of one warp. Each block's sums start from zero.
template <class P>
__device__ bool multiply_e4m3(const P &p, Control &c, uint32_t ring_base, const Shape sh, uint32_t tmem) {
    Ring r(sh.stages);
    uint32_t seq = 0;
    const bool ok = p.segments([&](const Segment &s) {
        const uint32_t desc = product_desc(s.n16());
        for (int kb = s.kb0; kb < s.kb1; ++kb, r.next(), ++seq) {
            const uint32_t buf = seq & 1;
            if (!wait(&c.full_b[r.slot], r.round) || !wait(&c.a_ready[buf], seq >> 1 & 1)) return false;
            tc_fence_after();
            const uint32_t at = ring_base + r.slot * Shape::stage_bytes(sh.cols, true) + 2 * kHalf;
            const uint32_t a = tmem + kTmemCodes + buf * 128, d = tmem + buf * 2 * sh.cols;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    mma_ts(d + h * sh.cols, a + h * 64 + k * 8,
                           operand_desc(at + (k >> 2) * sh.cols * 128) + 2 * (k & 3), desc, k > 0);
            mma_commit(&c.empty[r.slot]);
            mma_commit(&c.sums_full[buf]);
        }
        return true;
    });
    if (!ok) {
        mma_commit(&c.last);
        wait(&c.last, 0);
    }
    return ok;
}

// Two E4M3 codes (the low 16 bits) as two bf16, exactly.
__device__ __forceinline__ uint32_t codes_to_bf16(uint32_t two) {
    uint32_t h, out;
    asm("{\n\t.reg .b16 t, lo, hi;\n\t.reg .f32 x, y;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}"
        : "=r"(h) : "r"(two));
    asm("{\n\t.reg .b16 lo, hi;\n\t.reg .f32 x, y;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 x, lo;\n\t"
        "cvt.f32.f16 y, hi;\n\tcvt.rn.bf16x2.f32 %0, y, x;\n\t}"
        : "=r"(out) : "r"(h));
    return out;
}

// What a reader thread does with its sums of a segment: row `row` of both
// halves, columns 16 i + 8 side + 0..7. `each(f)` calls f(column, sums of half
// 0, sums of half 1) for all of them.
template <class P, class Each, class Release>
__device__ bool hand_over(const P &p, Control &c, const Shape sh, const Segment &s, int row, Each each, Release release) {
    if (s.whole()) {
        if (!p.emit_ready(s)) return false;
        typename P::Emit emit(p, s, row);
        each([&](int col, const float *v0, const float *v1) { emit(col, v0, v1); });
        release();
    } else {
        const size_t half = (size_t)sh.cols * kRows;
        float *mine = p.partial(s.phase, blockIdx.x, s.kb0 > 0 ? 0 : 1);
        each([&](int col, const float *v0, const float *v1) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                mine[(col + j) * kRows + row] = v0[j];
                mine[half + (col + j) * kRows + row] = v1[j];
            }
        });
        release();
        __threadfence();
        readers_sync();
        if (threadIdx.x == kThreads - kReaders) {
            uint32_t *arrived = p.arrivals(s.phase, s.cta0);
            const uint32_t before = add_acq_rel(arrived, 1);
            c.vote = before + 1 == (uint32_t)s.parts;
        }
        readers_sync();
        const bool last = c.vote != 0;
        readers_sync();
        if (!last) return true;
        __threadfence();
        if (!p.emit_ready(s)) return false;
        typename P::Emit emit(p, s, row);
        const int side = (threadIdx.x - (kThreads - kReaders)) / 128;
        for (int col = side * 8; col < s.n; col += 16) {
            float v0[8] = {}, v1[8] = {};
            for (int i = 0; i < s.parts; ++i) {
                // a stretch that begins inside the tile is its CTA's first, the one that begins the tile its last
                const float *part = p.partial(s.phase, s.cta0 + i, i == 0 ? 1 : 0);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    v0[j] += __ldcg(part + (col + j) * kRows + row);
                    v1[j] += __ldcg(part + half + (col + j) * kRows + row);
                }
            }
            emit(col, v0, v1);
        }
    }
    p.tile_done(s);
    return true;
}

// Readers of bf16 weights' sums.
template <class P>
__device__ bool read_sums(const P &p, Control &c, const Shape sh, uint32_t tmem) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, quarter = warp & 3, side = (warp - 4) / 4;
    const int row = quarter * 32 + lane;
    uint32_t seq = 0;
    return p.segments([&](const Segment &s) {
        const uint32_t buf = seq & 1;
        if (!readers_agree(wait(&c.sums_full[buf], seq >> 1 & 1))) return false;
        tc_fence_after();
        const uint32_t at = tmem + ((uint32_t)(quarter * 32) << 16) + buf * 2 * sh.cols;
        auto each = [&](auto f) {
            for (int col = side * 8; col < s.n16(); col += 16) {
                float v[16];
                tmem_load8(at + col, v);
                tmem_load8(at + sh.cols + col, v + 8);
                tmem_load_wait(v);
                if (col < s.n) f(col, v, v + 8);
            }
        };
        auto release = [&] {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&c.sums_empty[buf]);
        };
        ++seq;
        return hand_over(p, c, sh, s, row, each, release);
    });
}

// Readers of E4M3 weights: convert block i, then add block i - 1's scaled sums.
template <class P>
__device__ bool read_sums_e4m3(const P &p, Control &c, const char *ring, const Shape sh, uint32_t tmem) {
    constexpr int kChunks = 4;   // of 8 columns to a thread: 64 columns over two sides
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, quarter = warp & 3, side = (warp - 4) / 4;
    const int row = quarter * 32 + lane;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    Ring r(sh.stages);
    uint32_t seq = 0;
    return p.segments([&](const Segment &s) {
        float acc0[kChunks * 8] = {}, acc1[kChunks * 8] = {};
        const float *scales = p.scales(s.phase);
        const float *s0 = scales + (size_t)min(s.row0 + row, s.row_end - 1) * s.kbs;
        const float *s1 = scales + (size_t)min(s.row1 + row, s.row_end - 1) * s.kbs;
        float was0 = 0.0f, was1 = 0.0f;
        bool ok = true;
        auto add = [&](uint32_t q, float w0, float w1) {   // block q's sums
            const uint32_t buf = q & 1;
            if (!warp_wait(&c.sums_full[buf], q >> 1 & 1)) return false;
            tc_fence_after();
            const uint32_t at = tmem + lanes + buf * 2 * sh.cols;
#pragma unroll
            for (int i = 0; i < kChunks; ++i) {
                const int col = i * 16 + side * 8;
                if (col >= s.n16()) break;
                float v[16];
                tmem_load8(at + col, v);
                tmem_load8(at + sh.cols + col, v + 8);
                tmem_load_wait(v);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    acc0[i * 8 + j] = fmaf(w0, v[j], acc0[i * 8 + j]);
                    acc1[i * 8 + j] = fmaf(w1, v[8 + j], acc1[i * 8 + j]);
                }
            }
            return true;
        };
        for (int kb = s.kb0; kb < s.kb1; ++kb, r.next(), ++seq) {
            const float now0 = __ldg(s0 + kb), now1 = __ldg(s1 + kb);
            if (!warp_wait(&c.full_a[r.slot], r.round)) { ok = false; break; }
            // this thread's row of its side's half: 128 codes, 16-byte pieces swizzled by the row
            const char *codes = ring + (size_t)r.slot * Shape::stage_bytes(sh.cols, true) + side * kHalf + row * 128;
            const uint32_t dst = tmem + lanes + kTmemCodes + (seq & 1) * 128 + side * 64;
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const uint4 w = *reinterpret_cast<const uint4 *>(codes + ((q ^ (row & 7)) << 4));
                uint32_t b[8];
                b[0] = codes_to_bf16(w.x), b[1] = codes_to_bf16(w.x >> 16);
                b[2] = codes_to_bf16(w.y), b[3] = codes_to_bf16(w.y >> 16);
                b[4] = codes_to_bf16(w.z), b[5] = codes_to_bf16(w.z >> 16);
                b[6] = codes_to_bf16(w.w), b[7] = codes_to_bf16(w.w >> 16);
                tmem_store8(dst + q * 8, b);
            }
            tmem_store_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&c.empty[r.slot]);
                mbar_arrive(&c.a_ready[seq & 1]);
            }
            if (kb > s.kb0 && !add(seq - 1, was0, was1)) { ok = false; break; }
            was0 = now0, was1 = now1;
        }
        if (ok) ok = add(seq - 1, was0, was1);
        if (!readers_agree(ok)) return false;
        auto each = [&](auto f) {
#pragma unroll
            for (int i = 0; i < kChunks; ++i)
                if (i * 16 + side * 8 < s.n) f(i * 16 + side * 8, acc0 + i * 8, acc1 + i * 8);
        };
        return hand_over(p, c, sh, s, row, each, [] {});
    });
}

// The whole kernel body; P::finish runs on the reader threads after the last segment.
template <bool kE4m3, class P>
__device__ void run(const P &p, const Shape sh, const uint32_t tmem_cols) {
    extern __shared__ char smem_raw[];
    __shared__ Control c;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    char *ring = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    const uint32_t ring_base = smem_addr(ring);
    if (threadIdx.x == 0) {
        for (int i = 0; i < sh.stages; ++i) {
            mbar_init(&c.full_a[i], 1);
            mbar_init(&c.full_b[i], 1);
            mbar_init(&c.empty[i], kE4m3 ? 9 : 1);   // the products, and the 8 converting warps
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&c.sums_full[i], 1);
            mbar_init(&c.sums_empty[i], 8);
            mbar_init(&c.a_ready[i], 8);
        }
        mbar_init(&c.last, 1);
        fence_barrier_init();
    }
    if (warp == 3) tmem_alloc(&c.tmem, tmem_cols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = c.tmem;

    bool ok = true;
    if (warp == 0) ok = load_a<kE4m3>(p, c, ring_base, sh);
    else if (warp == 1) ok = load_b<kE4m3>(p, c, ring_base, sh);
    else if (warp == 2) {
        if (lane == 0) {
            if constexpr (kE4m3) ok = multiply_e4m3(p, c, ring_base, sh, tmem);
            else ok = multiply(p, c, ring_base, sh, tmem);
        }
    } else if (warp >= 4) {
        if constexpr (kE4m3) ok = read_sums_e4m3(p, c, ring, sh, tmem);
        else ok = read_sums(p, c, sh, tmem);
        if (ok) ok = p.finish();
    }
    if (!ok) report(p.status, MOE_ERR_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 3) tmem_free(tmem, tmem_cols);
}

// ------------------------------------------------------------------ plan

// Sorts entries by the weight set that they name and cuts each set's into groups
// of at most `cols`; clears the counters of the kernel behind it.
template <typename Index>
struct PlanArgs {
    const Index *idx;        // [n], -1: none
    int n, sets, cols;
    uint32_t *words;         // [0] becomes the number of groups, the rest 0
    int num_words;
    int4 *groups;            // {set, first sorted entry, entries, 0}
    int *order;              // sorted entries
    int bad;                 // status of an index out of range
    int32_t *status;
    TraceArgs trace;
};

constexpr int kPlanThreads = 1024;

// The order of a set's entries is the arrival order of the counters: it says
// only which column of a product an entry takes, and columns do not depend on
// one another.
template <typename Index>
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanArgs<Index> a) {
    WarpTrace wt(a.trace, MOE_TRACE_PLAN);
    grid_dependency_wait();
    extern __shared__ int32_t plan_smem[];
    int32_t *start = plan_smem, *first_group = plan_smem + a.sets + 1;
    for (int i = threadIdx.x; i <= a.sets; i += kPlanThreads) start[i] = 0;
    for (int i = threadIdx.x; i < a.num_words; i += kPlanThreads) a.words[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < a.n; i += kPlanThreads) {
        const Index e = a.idx[i];
        if (e >= 0 && e < a.sets) atomicAdd(&start[e], 1);
        else if (e != -1) report(a.status, a.bad);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.sets; e += kPlanThreads) first_group[e] = (start[e] + a.cols - 1) / a.cols;
    __syncthreads();
    if (threadIdx.x < 32) warp_exclusive_scan(start, a.sets, threadIdx.x);
    else if (threadIdx.x < 64) warp_exclusive_scan(first_group, a.sets, threadIdx.x - 32);
    __syncthreads();
    for (int e = threadIdx.x; e < a.sets; e += kPlanThreads) {
        const int end = start[e + 1];
        for (int g = first_group[e], b = start[e]; b < end; ++g, b += a.cols)
            a.groups[g] = make_int4(e, b, min(a.cols, end - b), 0);
    }
    if (threadIdx.x == 0) a.words[0] = first_group[a.sets];
    __syncthreads();
    for (int i = threadIdx.x; i < a.n; i += kPlanThreads) {
        const Index e = a.idx[i];
        if (e >= 0 && e < a.sets) a.order[atomicAdd(&start[e], 1)] = i;
    }
}

template <typename Index>
int launch_plan(const PlanArgs<Index> &a, cudaStream_t s) {
    const size_t smem = (size_t)2 * (a.sets + 1) * 4;
    const int rc = ensure_dynamic_smem((const void *)plan_kernel<Index>, smem);
    if (rc != MOE_OK) return rc;
    return launch_kernel(plan_kernel<Index>, dim3(1), dim3(kPlanThreads), smem, s, tuning().overlap != 0, a) ==
                   cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// One CTA per SM, all of them resident at once (they wait for one another).
template <class Args>
int launch_resident(void (*kernel)(Args), Args &a, size_t smem, cudaStream_t s) {
    const int rc = ensure_dynamic_smem((const void *)kernel, smem);
    if (rc != MOE_OK) return rc;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(device_sm_count() < kMaxCtas ? device_sm_count() : kMaxCtas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void *args[] = {&a};
    return cudaLaunchKernelExC(&cfg, (const void *)kernel, args) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// Words of the workspace that both sides share.
constexpr int kGroupsWord = 0, kDoneWord = 1, kArrivals = 2, kWords = 2 + 2 * kMaxCtas;
constexpr size_t partial_floats(int cols) { return (size_t)2 * kMaxCtas * 2 * 2 * cols * kRows; }

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
