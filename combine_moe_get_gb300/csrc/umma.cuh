// umma.cuh -- tensor-core and tensor-copy building blocks for sm_103a as inline
// PTX: tensor maps (host), TMA tile and gather loads, tensor memory, and
// tcgen05 matrix products with operands in shared memory.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "moe_common.cuh"

namespace moe {

// ------------------------------------------------------------------ tensor maps (host)

// Map of a row-major matrix [rows, cols] whose tiles are [box_rows, box_cols],
// box_cols covering 128 bytes, laid out in shared memory with the 128-byte
// swizzle. Elements outside the matrix read as 0. False if the driver refuses.
inline bool make_tensor_map(CUtensorMap *map, const void *base, bool bytes, uint64_t rows, uint64_t cols,
                            uint32_t box_rows) {
    using Encode = decltype(&cuTensorMapEncodeTiled);
    static const Encode encode = [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) !=
                cudaSuccess || found != cudaDriverEntryPointSuccess)
            fn = nullptr;
        return reinterpret_cast<Encode>(fn);
    }();
    if (encode == nullptr) return false;
    const cuuint64_t size = bytes ? 1 : 2;
    const cuuint64_t dims[2] = {cols, rows}, strides[1] = {cols * size};
    const cuuint32_t box[2] = {(cuuint32_t)(128 / size), box_rows}, step[2] = {1, 1};
    return encode(map, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                  const_cast<void *>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// ------------------------------------------------------------------ TMA loads

// Tile at (col, row); col times the element size is a multiple of 16 bytes.
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap *map, int col, int row, uint64_t *bar,
                                         uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
        "[%0], [%1, {%2, %3}], [%4], %5;"
        ::"r"(dst), "l"(map), "r"(col), "r"(row), "r"(smem_addr(bar)), "l"(policy) : "memory");
}

// Four rows of a matrix whose map has a box one row high, at the same columns.
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap *map, int col, int r0, int r1, int r2,
                                            int r3, uint64_t *bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes.L2::cache_hint "
        "[%0], [%1, {%2, %3, %4, %5, %6}], [%7], %8;"
        ::"r"(dst), "l"(map), "r"(col), "r"(r0), "r"(r1), "r"(r2), "r"(r3), "r"(smem_addr(bar)), "l"(policy)
        : "memory");
}

__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// Order this thread's (and, after a barrier, its CTA's) generic accesses of any
// state space and later accesses by TMA.
__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async;" ::: "memory"); }

__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// ------------------------------------------------------------------ tensor memory

// `cols`: a power of two from 32 to 512. Called by one whole warp; the base
// address lands in *slot (shared memory).
__device__ __forceinline__ void tmem_alloc(uint32_t *slot, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 ::"r"(smem_addr(slot)), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols));
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// This warp's 32 lanes (of tensor memory's 128: lanes 32 * (warp % 4) up) x 4 or 8 columns from `addr`.
__device__ __forceinline__ void tmem_load4(uint32_t addr, float *v) {
    uint32_t r[4];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_load8(uint32_t addr, float *v) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(addr));
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
// The loads above have arrived; `v` keeps the compiler from using them earlier.
template <int N>
__device__ __forceinline__ void tmem_load_wait(float (&v)[N]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));
}

// ------------------------------------------------------------------ matrix products

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}

// The same value in every lane, and known to be: products take their operands
// from uniform registers, and moving each there from a lane's own costs more
// than a small product (80 cycles each, measured).
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }

// Shared-memory operand: rows of 128 bytes (64 bf16 or 128 E4M3 along K) under the
// 128-byte swizzle, groups of 8 rows 1024 bytes apart; the steps of one product
// along K (16 bf16, 32 E4M3) are 32 bytes apart. The low word holds the address, the high one is constant.
__device__ __forceinline__ uint32_t operand_low(uint32_t addr) { return ((addr >> 4) & 0x3fff) | 1u << 16; }
__device__ __forceinline__ uint64_t operand_desc(uint32_t low) {
    constexpr uint32_t kHigh = (1024 >> 4) | 1u << 14 | 2u << 29;
    return (uint64_t)kHigh << 32 | low;
}

// bf16 x bf16 or E4M3 x E4M3 -> fp32, 128 rows of A, n rows of B (a multiple of 16, 16..256), both K-major.
__device__ __forceinline__ uint32_t product_desc(int n, bool e4m3 = false) {
    return 1u << 4 | (e4m3 ? 0 : 1u << 7 | 1u << 10) | (uint32_t)(n >> 3) << 17 | (uint32_t)(128 >> 4) << 24;
}

// d (+)= A B^T over 16 columns of bf16. By one lane of the warp.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_low, uint32_t b_low, uint32_t desc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(operand_desc(a_low)), "l"(operand_desc(b_low)), "r"(desc), "r"((uint32_t)add) : "memory");
}
// ... over 32 columns of E4M3.
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint32_t a_low, uint32_t b_low, uint32_t desc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(operand_desc(a_low)), "l"(operand_desc(b_low)), "r"(desc), "r"((uint32_t)add) : "memory");
}
// One arrival on `bar` when this lane's products so far are complete.
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                 ::"r"(smem_addr(bar)) : "memory");
}

}  // namespace moe
