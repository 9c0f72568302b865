// gate.cu -- the router's gate: scores, top-k choice and weights from logits
// (moe_topk_gate), and the gradient of the weights with respect to the logits
// (moe_topk_gate_backward).
//
// Mathematics. The chosen experts are the k largest logits (softmax and
// sigmoid keep their order), or the k largest score + bias; ties go to the
// lowest index. Logits are compared as they are, so a choice is exact: no
// rounding takes part unless a bias is given. Exponentials are taken of
// differences to the largest logit (0 at the maximum even when that is +inf), sums
// are fp32.
//
// A warp handles a token: 32 lanes hold the row's E logits in registers (up to
// 64 each), so that a row is read once (and a gradient's written once), each
// choice is one max over the warp's keys and one min over the indices that reach
// it (redux.sync), and lane j keeps entry j (k <= 32). Rows longer than 2048 take
// one CTA per token with the keys in shared memory, and in the backward pass a
// warp that reads the row three times. 128 tokens, 256 experts, top 8 take 2.0 us,
// which is a launch and a row's latency; rows are bound by the instructions of a
// choice (forward) and by HBM (backward), see there. A choice by score + bias takes a
// score for every expert: 16384 rows of 2048 fp32 logits 76 us (sigmoid, top 8), of 256
// 19 us where the choice by logits takes 16.
#include <algorithm>
#include <cfloat>
#include <cuda_bf16.h>

#include "moe_common.cuh"

namespace moe {
namespace {

constexpr int kWarpsPerCta = 4;
constexpr int kWideThreads = 256;      // CTA of a row with more experts than a warp holds
constexpr int kMaxPerLane = 64;
constexpr uint32_t kFull = 0xffffffffu;

struct GateArgs {
    const void *logits;
    const float *bias;
    int T, k, E;
    int mode;
    float scale;
    int64_t *idx;
    float *w;
    int32_t *status;
    uint32_t *clear;   // words zeroed for the kernel behind this one, or null
    int num_clear;
    bool early;
    TraceArgs trace;
};

struct GateBackArgs {
    const void *logits;
    const int64_t *idx;
    const float *gw;
    int T, k, E;
    int mode;
    float scale;
    void *gl;
    int32_t *status;
    TraceArgs trace;
};

// By the first CTA.
__device__ __forceinline__ void clear_words(const GateArgs &a) {
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < a.num_clear; i += blockDim.x) a.clear[i] = 0;
}

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void store(float *p, float v) { *p = v; }
__device__ __forceinline__ void store(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// The wide kernel's keys: unsigned order of the key = order of the float, -0 as +0; 0 (never chosen)
// for -inf and NaN.
__device__ __forceinline__ uint32_t order_key(float v) {
    if (!(v > -INFINITY)) return 0;
    const uint32_t u = __float_as_uint(v + 0.0f);   // -0 + 0 = +0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
    return v;
}

// exp(l - m) for l <= m, 1 at l == m also when both are infinite.
__device__ __forceinline__ float exp_below(float l, float m) { return l == m ? 1.0f : expf(l - m); }

// The same for a row's softmax sum and its gradient's elements, m finite: __expf is
// off by 2 + 1.16 |l - m| units in the last place, about what the rounding of l - m
// itself does. Terms that count are off by a few units; an element of the
// gradient e^-20 times the largest by 3e-6 of itself. It takes a third of
// expf's instructions (16384 rows of 2048 fp32 logits: 35.9 us against 36.7
// forward, 44.5 against 46.2 backward; bf16 36.9 against 39.8 backward).
__device__ __forceinline__ float exp_term(float l, float m) { return __expf(l - m); }

struct Sigmoid {
    float s, not_s;   // sigmoid(l) and 1 - sigmoid(l), each without cancellation
};
__device__ __forceinline__ Sigmoid sigmoid(float l) {
    const float t = expf(-fabsf(l)), a = 1.0f / (1.0f + t), b = t / (1.0f + t);
    return l >= 0.0f ? Sigmoid{a, b} : Sigmoid{b, a};
}

// The normalised weights q_j of the chosen logits, one per lane (`on`: this
// lane has one). The sigmoids are taken relative to exp(min(max l, 0)), so that
// their sum does not vanish when every chosen logit is far below zero.
__device__ __forceinline__ float normalised(float l, bool on, bool is_sigmoid) {
    const float m = warp_max(on ? l : -INFINITY);
    float q = 0.0f;
    if (on) {
        if (is_sigmoid)
            q = exp_below(fminf(l, 0.0f), fminf(m, 0.0f)) / (1.0f + expf(-fabsf(l)));
        else
            q = exp_below(l, m);
    }
    const float sum = warp_sum(q);
    return on ? q / sum : 0.0f;
}

// Lane j: the weight of entry j with logit l; m and z the row's maximum and
// softmax sum (used only by the softmax that is not normalised).
__device__ __forceinline__ float entry_weight(int mode, float l, bool on, float m, float z) {
    const bool is_sigmoid = (mode & 0xff) == MOE_GATE_SIGMOID;
    if (mode & MOE_GATE_NORMALIZE) return normalised(l, on, is_sigmoid);
    if (!on) return 0.0f;
    return is_sigmoid ? sigmoid(l).s : exp_below(l, m) / z;
}

// ------------------------------------------------------------------ a row in a warp's registers

// Element i of a lane is expert_of(i, lane): four neighbours to a lane and load
// where the rows allow it (kVec), else one.
template <bool kVec>
__device__ __forceinline__ int expert_of(int i, int lane) {
    return kVec ? ((i >> 2) * 32 + lane) * 4 + (i & 3) : i * 32 + lane;
}
template <bool kVec, int kPerLane>
__device__ __forceinline__ void load_row(const float *row, int E, int lane, float (&v)[kPerLane]) {
#pragma unroll
    for (int i = 0; i < kPerLane; i += kVec ? 4 : 1) {
        const int e = expert_of<kVec>(i, lane);
        if (kVec) {
            const float4 f = e < E ? __ldg(reinterpret_cast<const float4 *>(row + e))
                                   : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            v[i] = f.x, v[i + 1] = f.y, v[i + 2] = f.z, v[i + 3] = f.w;
        } else {
            v[i] = e < E ? row[e] : -INFINITY;
        }
    }
}
template <bool kVec, int kPerLane>
__device__ __forceinline__ void load_row(const __nv_bfloat16 *row, int E, int lane, float (&v)[kPerLane]) {
#pragma unroll
    for (int i = 0; i < kPerLane; i += kVec ? 4 : 1) {
        const int e = expert_of<kVec>(i, lane);
        if (kVec) {
            const uint2 f = e < E ? __ldg(reinterpret_cast<const uint2 *>(row + e)) : make_uint2(0xff80ff80u, 0xff80ff80u);
            v[i] = __uint_as_float(f.x << 16), v[i + 1] = __uint_as_float(f.x & 0xffff0000u);
            v[i + 2] = __uint_as_float(f.y << 16), v[i + 3] = __uint_as_float(f.y & 0xffff0000u);
        } else {
            v[i] = e < E ? to_float(row[e]) : -INFINITY;
        }
    }
}
template <bool kVec, int kPerLane>
__device__ __forceinline__ void store_row(float *row, int E, int lane, const float (&v)[kPerLane]) {
#pragma unroll
    for (int i = 0; i < kPerLane; i += kVec ? 4 : 1) {
        const int e = expert_of<kVec>(i, lane);
        if (e >= E) continue;
        if (kVec) *reinterpret_cast<float4 *>(row + e) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        else row[e] = v[i];
    }
}
template <bool kVec, int kPerLane>
__device__ __forceinline__ void store_row(__nv_bfloat16 *row, int E, int lane, const float (&v)[kPerLane]) {
#pragma unroll
    for (int i = 0; i < kPerLane; i += kVec ? 4 : 1) {
        const int e = expert_of<kVec>(i, lane);
        if (e >= E) continue;
        if (kVec) {
            __nv_bfloat162 b[2] = {__floats2bfloat162_rn(v[i], v[i + 1]), __floats2bfloat162_rn(v[i + 2], v[i + 3])};
            *reinterpret_cast<uint2 *>(row + e) = *reinterpret_cast<const uint2 *>(b);
        } else {
            row[e] = __float2bfloat16_rn(v[i]);
        }
    }
}

// ------------------------------------------------------------------ forward, a warp per token

// Takes the lowest expert whose value is `top` out of the warp's group number
// `group`, one of [kFrom, kTo), and renews the group's maximum; returns the expert.
// The groups' code is kept apart by the asm: merged, it would index the values in
// memory.
template <bool kVec, int kGroup, int kFrom, int kTo, int kHeld, int kGroups>
__device__ __forceinline__ uint32_t take_out(float (&v)[kHeld], float (&group_top)[kGroups], uint32_t group, float top,
                                             int lane) {
    if constexpr (kTo - kFrom > 1) {
        constexpr int kMid = (kFrom + kTo) / 2;
        return group < kMid ? take_out<kVec, kGroup, kFrom, kMid>(v, group_top, group, top, lane)
                            : take_out<kVec, kGroup, kMid, kTo>(v, group_top, group, top, lane);
    } else {
        asm volatile("" ::"n"(kFrom));
        int first = kGroup;   // of this lane's values
#pragma unroll
        for (int i = kGroup - 1; i >= 0; --i)
            if (v[kFrom * kGroup + i] == top) first = i;
        const uint32_t e = first < kGroup ? expert_of<kVec>(kFrom * kGroup + first, lane) : kFull;
        const uint32_t win = __reduce_min_sync(kFull, e);
        if (e != win) first = kGroup;
        float rest = -INFINITY;
#pragma unroll
        for (int i = 0; i < kGroup; ++i) {
            if (i == first) v[kFrom * kGroup + i] = -INFINITY;
            rest = fmaxf(rest, v[kFrom * kGroup + i]);
        }
        group_top[kFrom] = rest;
        return win;
    }
}

// A choice looks at the maxima of groups of eight values a lane, and only the
// winner's group is gone through again (its number is made the same in every lane).
// Groups of four are faster for 32 values a lane (16384 rows of 1024 logits: 24 us
// against 26) and slower for 64. Five CTAs' registers to an SM: with what the
// compiler takes for 64 values a lane it would be three, and four took 38 us for
// 16384 rows of 2048 fp32 logits (softmax over all, top 8) where five take 36. That
// is 3.8 TB/s: eight choices of some hundred instructions and three reductions over
// the warp bound it, not the 134 MB; bf16 logits take as long. (Fetching a warp's
// next row into shared memory meanwhile gained nothing.)
template <typename L, int kPerLane, bool kVec>
__global__ void __launch_bounds__(kWarpsPerCta * 32, kPerLane > 32 ? 5 : 8) gate_kernel(const GateArgs a) {
    WarpTrace wt(a.trace, MOE_TRACE_GATE);
    grid_dependency_wait();
    // A layer's plan or split is set up meanwhile (1 us of a small layer); after a gate alone the
    // next kernel's CTAs would take room (4096 rows of 512 logits: 8.0 us against 7.2).
    if (a.early) grid_launch_dependents();
    clear_words(a);
    constexpr int kGroup = kPerLane == 32 ? 4 : 8, kGroups = kPerLane / kGroup;
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * kWarpsPerCta + (threadIdx.x >> 5);
    if (t >= a.T) return;
    const L *row = static_cast<const L *>(a.logits) + (size_t)t * a.E;
    const bool is_sigmoid = (a.mode & 0xff) == MOE_GATE_SIGMOID;

    float v[kPerLane], group_top[kGroups];   // -inf: never chosen
    load_row<kVec>(row, a.E, lane, v);
    bool nan = false;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
        group_top[g] = -INFINITY;
#pragma unroll
        for (int i = g * kGroup; i < (g + 1) * kGroup; ++i) {
            nan |= v[i] != v[i];
            v[i] = fmaxf(v[i], -INFINITY);   // NaN becomes -inf
            group_top[g] = fmaxf(group_top[g], v[i]);
        }
    }
    if (nan) report(a.status, MOE_ERR_BAD_LOGIT);

    // the row's maximum and softmax sum, where the weights or the choice need them
    float m = 0.0f, z = 1.0f;
    const bool whole_row = !is_sigmoid && (!(a.mode & MOE_GATE_NORMALIZE) || a.bias != nullptr);
    if (whole_row) {
        m = -INFINITY;
#pragma unroll
        for (int g = 0; g < kGroups; ++g) m = fmaxf(m, group_top[g]);
        m = lanes_max(m);
        if (!(m > -INFINITY)) m = 0.0f;
        float s[4] = {};
        if (m < INFINITY) {
#pragma unroll
            for (int i = 0; i < kPerLane; ++i) s[i & 3] += exp_term(v[i], m);
        } else {
#pragma unroll
            for (int i = 0; i < kPerLane; ++i) s[i & 3] += v[i] == INFINITY ? 1.0f : 0.0f;
        }
        z = warp_sum((s[0] + s[1]) + (s[2] + s[3]));
    }
    if (a.bias != nullptr) {   // choose by score + bias; the logits are read again for the chosen
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
            group_top[g] = -INFINITY;
#pragma unroll
            for (int i = g * kGroup; i < (g + 1) * kGroup; ++i) {
                if (v[i] > -INFINITY) {
                    const float s = is_sigmoid ? sigmoid(v[i]).s : exp_below(v[i], m) / z;
                    v[i] = fmaxf(s + a.bias[expert_of<kVec>(i, lane)], -INFINITY);
                }
                group_top[g] = fmaxf(group_top[g], v[i]);
            }
        }
    }

    float mine = 0.0f;      // lane j: entry j's logit
    int mine_e = -1;        // ... and expert
    for (int j = 0; j < a.k; ++j) {
        float best = -INFINITY;
#pragma unroll
        for (int g = 0; g < kGroups; ++g) best = fmaxf(best, group_top[g]);
        const float top = lanes_max(best);
        if (!(top > -INFINITY)) break;
        // the lowest expert with that value is in the lowest group that has it
        uint32_t group = kFull;
#pragma unroll
        for (int g = kGroups - 1; g >= 0; --g)
            if (group_top[g] == top) group = g;
        group = __reduce_min_sync(kFull, group);
        const uint32_t win = take_out<kVec, kGroup, 0, kGroups>(v, group_top, group, top, lane);
        if (lane == j) mine = a.bias == nullptr ? top : to_float(row[win]), mine_e = (int)win;
    }
    const float w = entry_weight(a.mode, mine, mine_e >= 0, m, z);
    if (lane < a.k) {
        a.idx[(size_t)t * a.k + lane] = mine_e;
        a.w[(size_t)t * a.k + lane] = mine_e >= 0 ? a.scale * w : 0.0f;
    }
}

// ------------------------------------------------------------------ forward, a CTA per token

// Rows of more experts than a warp holds: keys in shared memory, of which a thread
// has every 256th, and each choice two barriers and a look at the warps' best ones.
// Only the thread whose key was taken goes through its own again.
struct Top {
    uint32_t key;
    int e;
};
__device__ __forceinline__ Top better(Top x, Top y) {
    return y.key > x.key || (y.key == x.key && y.e < x.e) ? y : x;
}

template <typename L>
__global__ void __launch_bounds__(kWideThreads) gate_wide_kernel(const GateArgs a) {
    WarpTrace wt(a.trace, MOE_TRACE_GATE);
    grid_dependency_wait();
    clear_words(a);
    extern __shared__ uint32_t keys[];
    __shared__ Top tops[kWideThreads / 32];
    __shared__ float sums[kWideThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t = blockIdx.x;
    const L *row = static_cast<const L *>(a.logits) + (size_t)t * a.E;
    const bool is_sigmoid = (a.mode & 0xff) == MOE_GATE_SIGMOID;

    auto block_top = [&](Top v) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            v = better(v, Top{__shfl_xor_sync(kFull, v.key, o), __shfl_xor_sync(kFull, v.e, o)});
        __syncthreads();
        if (lane == 0) tops[warp] = v;
        __syncthreads();
        v = tops[0];
        for (int i = 1; i < kWideThreads / 32; ++i) v = better(v, tops[i]);
        return v;
    };

    bool nan = false;
    Top local{0, a.E};
    for (int e = threadIdx.x; e < a.E; e += kWideThreads) {
        const float v = to_float(row[e]);
        nan |= v != v;
        keys[e] = order_key(v);
        local = better(local, Top{keys[e], e});
    }
    if (nan) report(a.status, MOE_ERR_BAD_LOGIT);
    float m = 0.0f, z = 1.0f;
    if (!is_sigmoid && (!(a.mode & MOE_GATE_NORMALIZE) || a.bias != nullptr)) {
        const Top top = block_top(local);
        m = top.key ? key_value(top.key) : 0.0f;
        float s = 0.0f;
        for (int e = threadIdx.x; e < a.E; e += kWideThreads)
            if (keys[e]) s += exp_below(key_value(keys[e]), m);
        s = warp_sum(s);
        if (lane == 0) sums[warp] = s;
        __syncthreads();
        z = 0.0f;
        for (int i = 0; i < kWideThreads / 32; ++i) z += sums[i];
    }
    if (a.bias != nullptr) {
        local = Top{0, a.E};
        for (int e = threadIdx.x; e < a.E; e += kWideThreads) {
            if (keys[e] != 0) {
                const float l = key_value(keys[e]);
                const float s = is_sigmoid ? sigmoid(l).s : exp_below(l, m) / z;
                keys[e] = order_key(s + a.bias[e]);
            }
            local = better(local, Top{keys[e], e});
        }
    }
    float mine = 0.0f;
    int mine_e = -1;
    for (int j = 0; j < a.k; ++j) {
        const Top top = block_top(local);
        if (top.key == 0) break;
        if (top.e % kWideThreads == threadIdx.x) {   // the thread that holds it looks for its next
            keys[top.e] = 0;
            local = Top{0, a.E};
            for (int e = threadIdx.x; e < a.E; e += kWideThreads) local = better(local, Top{keys[e], e});
        }
        if (threadIdx.x == j) mine = a.bias == nullptr ? key_value(top.key) : to_float(row[top.e]), mine_e = top.e;
    }
    if (warp != 0) return;
    const float w = entry_weight(a.mode, mine, mine_e >= 0, m, z);
    if (lane < a.k) {
        a.idx[(size_t)t * a.k + lane] = mine_e;
        a.w[(size_t)t * a.k + lane] = mine_e >= 0 ? a.scale * w : 0.0f;
    }
}

// ------------------------------------------------------------------ backward, a warp per token

// kPerLane: the row fits into the warp's registers (E <= 32 kPerLane) and is read
// and written once; 0: longer rows, read again for each use. The softmax's gradient
// without normalisation is bound by HBM: 16384 rows of 2048 fp32 logits, 268 MB, take
// 44 us (6.0 TB/s); the others write only zeros and the chosen entries.
template <typename L, int kPerLane, bool kVec>
__global__ void __launch_bounds__(kWarpsPerCta * 32, kPerLane > 32 ? 4 : 8) gate_backward_kernel(const GateBackArgs a) {
    WarpTrace wt(a.trace, MOE_TRACE_GATE_BACKWARD);
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * kWarpsPerCta + (threadIdx.x >> 5);
    if (t >= a.T) return;
    const L *row = static_cast<const L *>(a.logits) + (size_t)t * a.E;
    L *out = static_cast<L *>(a.gl) + (size_t)t * a.E;
    const bool is_sigmoid = (a.mode & 0xff) == MOE_GATE_SIGMOID;
    const bool norm = (a.mode & MOE_GATE_NORMALIZE) != 0;
    const bool dense = !is_sigmoid && !norm;

    constexpr int kHeld = kPerLane > 0 ? kPerLane : 1;
    float x[kHeld];
    if (kPerLane > 0 && dense) load_row<kVec>(row, a.E, lane, x);

    // lane j: entry j
    int e = -1;
    float g = 0.0f, l = 0.0f;
    if (lane < a.k) {
        const int64_t v = a.idx[(size_t)t * a.k + lane];
        if (v < -1 || v >= a.E) report(a.status, MOE_ERR_BAD_TOPK);
        else e = (int)v;
        g = a.gw[(size_t)t * a.k + lane] * a.scale;
        if (e >= 0) l = to_float(row[e]);
        if (!(l > -INFINITY)) e = -1;   // a masked logit has no weight
    }
    const bool on = e >= 0;
    if (!on) g = 0.0f;

    // d: the entry's own part of its logit's gradient; every other logit gets -p * dot
    float d = 0.0f, dot = 0.0f, m = 0.0f, rz = 0.0f;
    if (norm) {
        const float q = normalised(l, on, is_sigmoid);
        d = q * (g - warp_sum(g * q));
        if (is_sigmoid) d *= sigmoid(l).not_s;
    } else if (is_sigmoid) {
        const Sigmoid s = sigmoid(l);
        d = g * s.s * s.not_s;
    } else {
        m = -INFINITY;
        float z = 0.0f;
        if (kPerLane > 0) {
#pragma unroll
            for (int i = 0; i < kHeld; ++i) m = fmaxf(m, x[i]);   // fmaxf passes over NaN
            m = warp_max(m);
            float s[4] = {};
            if (m < INFINITY) {
                const float from = fmaxf(m, -FLT_MAX);   // a row that is masked whole
#pragma unroll
                for (int i = 0; i < kHeld; ++i) {
                    x[i] = exp_term(fmaxf(x[i], -INFINITY), from);   // NaN becomes -inf, and that 0
                    s[i & 3] += x[i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < kHeld; ++i) {
                    x[i] = x[i] == INFINITY ? 1.0f : 0.0f;
                    s[i & 3] += x[i];
                }
            }
            z = (s[0] + s[1]) + (s[2] + s[3]);
        } else {
            for (int i = lane; i < a.E; i += 32) m = fmaxf(m, to_float(row[i]));
            m = warp_max(m);
            for (int i = lane; i < a.E; i += 32) {
                const float v = to_float(row[i]);
                if (v > -INFINITY) z += exp_below(v, m);
            }
        }
        z = warp_sum(z);
        rz = z > 0.0f ? 1.0f / z : 0.0f;
        const float p = on ? exp_below(l, m) * rz : 0.0f;
        dot = warp_sum(g * p);
        d = p * (g - dot);
    }
    if (!on) d = 0.0f;
    if (kPerLane > 0) {
        const float c = -rz * dot;
#pragma unroll
        for (int i = 0; i < kHeld; ++i) x[i] = dense ? x[i] * c : 0.0f;
        store_row<kVec>(out, a.E, lane, x);
    } else {
        for (int i = lane; i < a.E; i += 32) {
            float v = 0.0f;
            if (dense) {
                const float y = to_float(row[i]);
                if (y > -INFINITY) v = -exp_below(y, m) * rz * dot;
            }
            store(out + i, v);
        }
    }
    // an expert named by several entries gets the sum of their parts, in entry order
    const uint32_t same = __match_any_sync(kFull, e);
    float sum = 0.0f;
    int n = 0;
    for (int j = 0; j < a.k; ++j) {
        const float dj = __shfl_sync(kFull, d, j);
        if (same >> j & 1) sum += dj, ++n;
    }
    // ... and its -p * dot once
    if (dense && n > 1) sum += (float)(n - 1) * exp_below(l, m) * rz * dot;
    __syncwarp();
    if (on && (same & ((1u << lane) - 1)) == 0) store(out + e, sum);
}

// Rows whose every fourth element is aligned for a load of four.
template <typename L>
bool rows_of_four(const void *p, int E) { return E % 4 == 0 && reinterpret_cast<uintptr_t>(p) % (4 * sizeof(L)) == 0; }

template <typename L, int kPerLane>
cudaError_t launch_rows(const GateArgs &a, cudaStream_t s) {
    const dim3 grid((a.T + kWarpsPerCta - 1) / kWarpsPerCta), block(kWarpsPerCta * 32);
    const bool overlap = tuning().overlap != 0;
    return rows_of_four<L>(a.logits, a.E) ? launch_kernel(gate_kernel<L, kPerLane, true>, grid, block, 0, s, overlap, a)
                                          : launch_kernel(gate_kernel<L, kPerLane, false>, grid, block, 0, s, overlap, a);
}

template <typename L>
int launch_gate_typed(const GateArgs &a, cudaStream_t s) {
    cudaError_t e;
    if (a.E <= 256) e = launch_rows<L, 8>(a, s);
    else if (a.E <= 1024) e = launch_rows<L, 32>(a, s);
    else if (a.E <= 32 * kMaxPerLane) e = launch_rows<L, kMaxPerLane>(a, s);
    else
        e = launch_kernel(gate_wide_kernel<L>, dim3(a.T), dim3(kWideThreads), a.E * sizeof(uint32_t), s,
                          tuning().overlap != 0, a);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

template <typename L, int kPerLane>
cudaError_t launch_back_rows(const GateBackArgs &a, cudaStream_t s) {
    const dim3 grid((a.T + kWarpsPerCta - 1) / kWarpsPerCta), block(kWarpsPerCta * 32);
    const bool overlap = tuning().overlap != 0;
    return rows_of_four<L>(a.logits, a.E) && rows_of_four<L>(a.gl, a.E)
               ? launch_kernel(gate_backward_kernel<L, kPerLane, true>, grid, block, 0, s, overlap, a)
               : launch_kernel(gate_backward_kernel<L, kPerLane, false>, grid, block, 0, s, overlap, a);
}

template <typename L>
int launch_back_typed(const GateBackArgs &a, cudaStream_t s) {
    cudaError_t e;
    if (a.E <= 256) e = launch_back_rows<L, 8>(a, s);
    else if (a.E <= 1024) e = launch_back_rows<L, 32>(a, s);
    else if (a.E <= 32 * kMaxPerLane) e = launch_back_rows<L, kMaxPerLane>(a, s);
    else
        e = launch_kernel(gate_backward_kernel<L, 0, false>, dim3((a.T + kWarpsPerCta - 1) / kWarpsPerCta),
                          dim3(kWarpsPerCta * 32), 0, s, tuning().overlap != 0, a);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace

int launch_gate(const GateLaunch &L) {
    if (L.num_tokens == 0) return MOE_OK;
    const GateArgs a{L.logits, L.bias, L.num_tokens, L.num_topk, L.num_experts, L.mode, L.scale,
                     L.topk_idx, L.topk_weights, L.status, L.clear, L.num_clear, L.early, trace_args()};
    const cudaStream_t s = static_cast<cudaStream_t>(L.stream);
    return L.logits_type == MOE_LOGITS_BF16 ? launch_gate_typed<__nv_bfloat16>(a, s) : launch_gate_typed<float>(a, s);
}

int launch_gate_backward(const GateBackwardLaunch &L) {
    if (L.num_tokens == 0) return MOE_OK;
    const GateBackArgs a{L.logits, L.topk_idx, L.grad_weights, L.num_tokens, L.num_topk, L.num_experts, L.mode,
                         L.scale, L.grad_logits, L.status, trace_args()};
    const cudaStream_t s = static_cast<cudaStream_t>(L.stream);
    return L.logits_type == MOE_LOGITS_BF16 ? launch_back_typed<__nv_bfloat16>(a, s) : launch_back_typed<float>(a, s);
}

}  // namespace moe
