// Fifth-generation tensor cores (internal): tensor memory, tcgen05 matrix steps
// of bf16 operands in shared memory, and the operands' layout.
//
// An operand tile is rows of 128 bytes (64 bf16 of K), eight rows to an atom of 1024
// bytes, with the 16-byte pieces of row r in the order piece ^ (r & 7) (the
// 128-byte swizzle).  Tiles start 1024-byte aligned; a step of 16 of K is 32 bytes
// further in the tile.
#pragma once

#include <cuda.h>

#include "ep_device.cuh"

namespace ep {

__device__ __forceinline__ uint32_t tile_offset(int row, int piece) { return row * 128 + ((piece ^ (row & 7)) << 4); }

// The descriptor of a tile at shared-memory address `at` (its own address or a step of K further).
__device__ __forceinline__ uint64_t tile_descriptor(uint32_t at)
{
    // address / 16; 1 (not used with a swizzle); 1024 bytes from atom to atom; version 1; 128-byte swizzle
    return (uint64_t)(at >> 4 & 0x3fff) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// bf16 operands with K contiguous in both, fp32 sums, 128 x N.
__device__ __forceinline__ uint32_t step_kind(int N)
{
    return 1u << 4 | 1u << 7 | 1u << 10 | (uint32_t)(N >> 3) << 17 | (uint32_t)(128 >> 4) << 24;
}

// Tensor memory (a whole warp): `columns` is a power of two, 32 to 512.  The address goes to *to in shared memory.
__device__ __forceinline__ void tensor_alloc(uint32_t *to, int columns)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(to)), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}

__device__ __forceinline__ void tensor_free(uint32_t at, int columns)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns));
}

// D (+)= A B^T, one step of 16 of K; one thread.
__device__ __forceinline__ void tensor_step(uint32_t d, uint64_t a, uint64_t b, uint32_t kind, bool add)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 ::"r"(d), "l"(a), "l"(b), "r"(kind), "r"((uint32_t)add)
                 : "memory");
}

// Arrives at `bar` once this thread's steps so far are done.
__device__ __forceinline__ void tensor_commit(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void tensor_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tensor_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// A box of a tensor map from (x, y, z) on to a tile at shared-memory address `to`, completing its bytes on `bar`; one
// thread.  x * 2 is a multiple of 16 bytes.
__device__ __forceinline__ void tensor_copy(uint32_t to, const CUtensorMap *map, int x, int y, int z, uint64_t *bar)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
                 ::"r"(to), "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
                 : "memory");
}

// A box from a tile at shared-memory address `from` to (x, y, z) on of a tensor map, what lies past its edges left out; one
// thread, which then commits it to a group of its own.  No coordinate is negative.
__device__ __forceinline__ void tensor_store(const CUtensorMap *map, uint32_t from, int x, int y, int z)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(x),
                 "r"(y), "r"(z), "r"(from)
                 : "memory");
}

__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }

// All but this thread's last N groups of stores have been read from shared memory; or are done.
template <int N>
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory"); }
template <int N>
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group %0;" ::"n"(N) : "memory"); }

// Makes this thread's writes to shared memory visible to matrix steps (and bulk copies) that are ordered behind it.
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// N columns of the warp's 32 lanes of tensor memory; a lane gets its own, once
// they are there (one block of assembly, so that no use moves ahead of the wait).
template <int N>
__device__ __forceinline__ void tensor_load(float (&f)[N], uint32_t at)
{
    static_assert(N == 16 || N == 32, "columns of a load");
    uint32_t r[N];
    __syncwarp();   // the warp is together for an .aligned instruction
    if constexpr (N == 32)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                     "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
                     "tcgen05.wait::ld.sync.aligned;"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                       "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
                       "=r"(r[16 % N]), "=r"(r[17 % N]), "=r"(r[18 % N]), "=r"(r[19 % N]), "=r"(r[20 % N]), "=r"(r[21 % N]),
                       "=r"(r[22 % N]), "=r"(r[23 % N]), "=r"(r[24 % N]), "=r"(r[25 % N]), "=r"(r[26 % N]), "=r"(r[27 % N]),
                       "=r"(r[28 % N]), "=r"(r[29 % N]), "=r"(r[30 % N]), "=r"(r[31 % N])
                     : "r"(at)
                     : "memory");
    else
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
                     "tcgen05.wait::ld.sync.aligned;"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                       "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                     : "r"(at)
                     : "memory");
#pragma unroll
    for (int i = 0; i < N; ++i)
        f[i] = __uint_as_float(r[i]);
}

}  // namespace ep
