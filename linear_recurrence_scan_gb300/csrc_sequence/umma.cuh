// umma.cuh -- thin wrappers of what a matrix product on the 5th-generation
// tensor cores needs (PTX tcgen05, tensor-map copies, barriers of a pair of
// blocks), and descriptors of operands in shared memory.
#pragma once

#include "async_copy.cuh"

namespace rlscan {
namespace umma {

// ---- addresses and barriers of the pair's blocks ------------------------------
__device__ __forceinline__ uint32_t of_rank(uint32_t smem, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem), "r"(rank));
    return r;
}
__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// one arrival at a barrier of any block of the cluster
__device__ __forceinline__ void arrive_cluster(uint32_t bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// ---- copies ---------------------------------------------------------------------
// A box of a tensor map into this block's shared memory; its bytes count on a
// barrier of any block of the pair.
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
        ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// ---- tensor memory ----------------------------------------------------------------
__device__ __forceinline__ void tmem_alloc(uint32_t at_smem, uint32_t columns)
{
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(at_smem), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t tmem, uint32_t columns)
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(columns));
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 columns of the warp's 32 lanes: v[i] is column i of the lane's row
__device__ __forceinline__ void tmem_load(uint32_t (&v)[32], uint32_t tmem)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(tmem));
}
__device__ __forceinline__ void tmem_loaded() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// ---- products -----------------------------------------------------------------------
// Operands are tiles of 128-byte rows with the 128-byte swizzle, as a tensor
// map writes them; a tile starts on a 1024-byte boundary.
//  - K-major: a row is 64 values of K of one row of the matrix; groups of
//    eight rows are 1024 bytes apart.  16 values of K further is 32 bytes.
//  - MN-major: a row is 64 neighbouring rows of the matrix at one K; groups of
//    eight K are 1024 bytes apart, the next 64 rows of the matrix `chunk`
//    bytes.  16 values of K further is 2048 bytes.
// Fields: address and both distances in units of 16 bytes (bits 0, 16, 32),
// 1 at bit 46, the swizzle (2: 128 bytes) at bit 61.
__device__ __forceinline__ uint64_t descriptor(uint32_t smem, uint32_t chunk)
{
    return static_cast<uint64_t>((smem & 0x3ffffu) >> 4) | static_cast<uint64_t>(chunk >> 4) << 16 |
           static_cast<uint64_t>(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
}

// bfloat16 operands, float32 sums: types at bits 4, 7 and 10, MN-major flags at
// 15 (A) and 16 (B), N / 8 at 17, M / 16 at 24.
__host__ __device__ constexpr uint32_t instruction(bool a_mn, bool b_mn, uint32_t m, uint32_t n)
{
    return 1u << 4 | 1u << 7 | 1u << 10 | (a_mn ? 1u : 0u) << 15 | (b_mn ? 1u : 0u) << 16 | (n >> 3) << 17 | (m >> 4) << 24;
}

// D[tmem] (+)= A B^T over 16 values of K, by the pair
__device__ __forceinline__ void multiply(uint32_t tmem, uint64_t a, uint64_t b, uint32_t instruction, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(tmem), "l"(a), "l"(b), "r"(instruction), "r"(add ? 1u : 0u)
        : "memory");
}
// When all products so far are done, one arrival at the barrier at this
// address in each block of the pair
__device__ __forceinline__ void commit(uint32_t bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

// ---- host ---------------------------------------------------------------------------
// A map of a [rows, columns] array of bfloat16, its rows `pitch` values apart,
// copied in boxes of 64 columns x `box` rows with the 128-byte swizzle; what
// lies outside the array reads 0.
inline bool encode(CUtensorMap *map, const void *p, int64_t rows, int64_t columns, int64_t pitch, uint32_t box)
{
    const int64_t extents[2] = {columns, rows}, strides[1] = {pitch * 2};
    const uint32_t boxes[2] = {64, box};
    return seq::encode_map(map, p, true, 2, extents, strides, boxes, true);
}

}  // namespace umma
}  // namespace rlscan
