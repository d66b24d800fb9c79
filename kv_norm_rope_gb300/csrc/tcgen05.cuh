// The fifth-generation tensor core: tensor memory, matrix instructions on
// shared-memory operands, and their completion.
//
// Operands are bf16 in shared memory in the 128-byte swizzle: rows of 128 bytes
// (64 elements), 8 rows to a 1024-byte atom, the 16-byte chunk c of row r stored
// at chunk c ^ (r % 8).  The same bytes serve both ways round: read along the
// rows (K-major: 64 elements of the product's inner dimension) or across them
// (MN-major: 64 elements of an outer dimension, the rows being the inner one).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "bulkcopy.cuh"

namespace dsv4 {
namespace {

// Byte offset of 16-byte chunk c of row r in a swizzled operand.
__device__ __forceinline__ uint32_t swizzled(uint32_t r, uint32_t c)
{
    return r * 128u + ((c ^ (r & 7u)) << 4);
}

// All columns of the CTA's tensor memory (one warp calls it; the address is
// written to shared memory).
__device__ __forceinline__ void tmem_alloc512(uint32_t *address)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_addr(address))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}

__device__ __forceinline__ void tmem_free512(uint32_t address)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(address));
}

// Order this thread's tensor-memory accesses before a barrier / after one.
__device__ __forceinline__ void tmem_fence_before()
{
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_fence_after()
{
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// Descriptor of a swizzled operand: `low` has the address, `high` the stride.
// K-major: `stride` is the distance of the 8-row groups.  MN-major: `stride` is that
// of the 8-row groups along the inner dimension, `lead` that of the blocks of 64
// outer elements.  Addresses are below 2^18, so adding bytes / 16 to `low` moves it.
struct Operand {
    uint32_t low, high;
};

__device__ __forceinline__ Operand operand(uint32_t address, uint32_t lead, uint32_t stride)
{
    return Operand{(address >> 4) | (lead >> 4 << 16), (stride >> 4) | (1u << 14) | (2u << 29)};
}

__device__ __forceinline__ Operand operator+(Operand o, uint32_t bytes)
{
    return Operand{o.low + (bytes >> 4), o.high};
}

// Instruction descriptor: bf16 operands, fp32 accumulator, M = 128, N = n;
// `across` marks MN-major operands (both).
__device__ __forceinline__ uint32_t instruction(uint32_t n, bool across)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | (across ? 3u << 15 : 0u) | ((n >> 3) << 17) |
           ((128u >> 4) << 24);
}

// The matrix instructions take their operands from uniform registers, so a whole
// warp runs the code that issues them, with values the same in every lane, and
// one elected lane issues: `elected` is 1 there.  (Issued from a branch that only
// one lane takes, each cost 110 cycles of moving descriptors, three times what the
// product takes.)
__device__ __forceinline__ uint32_t elect_one()
{
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(e));
    return e;
}

// d[128, n] (+)= a[128, 16] b[16, n]
__device__ __forceinline__ void mma_bf16(uint32_t d, Operand a, Operand b, uint32_t inst,
                                         bool accumulate, uint32_t elected)
{
    asm volatile("{\n\t.reg .pred p, e;\n\t.reg .b64 x, y;\n\t"
                 "setp.ne.u32 p, %6, 0;\n\tsetp.ne.u32 e, %7, 0;\n\t"
                 "mov.b64 x, {%1, %2};\n\tmov.b64 y, {%3, %4};\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %5, p;\n\t}" ::"r"(d),
                 "r"(a.low), "r"(a.high), "r"(b.low), "r"(b.high), "r"(inst),
                 "r"(accumulate ? 1u : 0u), "r"(elected)
                 : "memory");
}

// the same with a in tensor memory: 8 columns, two bf16 each, of the 128 lanes
__device__ __forceinline__ void mma_bf16_staged(uint32_t d, uint32_t a, Operand b, uint32_t inst,
                                                bool accumulate, uint32_t elected)
{
    asm volatile("{\n\t.reg .pred p, e;\n\t.reg .b64 y;\n\t"
                 "setp.ne.u32 p, %5, 0;\n\tsetp.ne.u32 e, %6, 0;\n\tmov.b64 y, {%2, %3};\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n\t}" ::"r"(d),
                 "r"(a), "r"(b.low), "r"(b.high), "r"(inst), "r"(accumulate ? 1u : 0u), "r"(elected)
                 : "memory");
}

// arrive on *bar once every matrix instruction the elected lane has issued is done
__device__ __forceinline__ void mma_commit(uint64_t *bar, uint32_t elected)
{
    asm volatile("{\n\t.reg .pred e;\n\tsetp.ne.u32 e, %1, 0;\n\t"
                 "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::
                     "r"(smem_addr(bar)),
                 "r"(elected)
                 : "memory");
}

// 16 columns from `address` on of the calling thread's lane (warp w of a
// warpgroup: lanes 32w..); finished after tmem_wait_load
__device__ __forceinline__ void tmem_load16(uint32_t address, float *v)
{
    uint32_t *u = reinterpret_cast<uint32_t *>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]),
          "=r"(u[7]), "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]),
          "=r"(u[14]), "=r"(u[15])
        : "r"(address));
}

__device__ __forceinline__ void tmem_wait_load()
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_store16(uint32_t address, const float *v)
{
    const uint32_t *u = reinterpret_cast<const uint32_t *>(v);
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(address),
        "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]),
        "r"(u[8]), "r"(u[9]), "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15])
        : "memory");
}

// 16 columns from 4 vectors
__device__ __forceinline__ void tmem_store16(uint32_t address, const uint4 *v)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(address),
        "r"(v[0].x), "r"(v[0].y), "r"(v[0].z), "r"(v[0].w), "r"(v[1].x), "r"(v[1].y), "r"(v[1].z),
        "r"(v[1].w), "r"(v[2].x), "r"(v[2].y), "r"(v[2].z), "r"(v[2].w), "r"(v[3].x), "r"(v[3].y),
        "r"(v[3].z), "r"(v[3].w)
        : "memory");
}

__device__ __forceinline__ void tmem_wait_store()
{
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// A warpgroup's registers a thread, out of what the CTA was launched with: up waits
// until others went down by as much.
template <int n>
__device__ __forceinline__ void registers_up()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(n));
}
template <int n>
__device__ __forceinline__ void registers_down()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(n));
}

// 2^x, flushing subnormal results
__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// barrier `id` over `threads` threads that also returns whether any of them brought `v`
__device__ __forceinline__ bool named_barrier_any(int id, int threads, bool v)
{
    uint32_t any;
    __syncwarp();
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
                 "barrier.cta.red.or.aligned.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(any)
                 : "r"(v ? 1u : 0u), "r"(id), "r"(threads)
                 : "memory");
    return any != 0u;
}

__device__ __forceinline__ void named_barrier(int id, int threads)
{
    __syncwarp();
    asm volatile("barrier.cta.sync.aligned %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

}  // namespace
}  // namespace dsv4
