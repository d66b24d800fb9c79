// Reading the 4-bit paged cache back out: out[n, :] = the 512 dims stored at
// slot slots[n], as bf16 (exact: fp4.cuh).  A negative slot gives a zero row, a
// slot past the cache a zero row and an error bit, as the 8-bit reader does.
//
// HBM-bound: per row 368 bytes read and 1024 written.  One warp per row with
// the insert's lane layout (lane l: dims [8l, 8l+8) and [256+8l, 256+8l+8)):
// the codes go in as one 4-byte word per lane and half (128 contiguous bytes a
// warp), the rope lanes 24..31 take 16 bytes of bf16 instead, and every store
// covers 512 contiguous bytes.  The next row's loads are in flight while a row
// is converted, its slot id one row ahead of that.  100003 rows: 23.6 us, 5.9 TB/s (a
// list of launches with a cold L2; 25.1 a call among others).

#include <cuda_runtime.h>
#include <stdint.h>

#include "fp4.cuh"
#include "launch_status.h"
#include "ops.h"

namespace dsv4 {
namespace {

constexpr int kThreads = 128;

struct GParams {
    const uint8_t *cache;
    int64_t num_slots;
    uint32_t block_size;
    uint64_t slot_div;
    const int64_t *slots;
    int64_t rows;
    uint16_t *out;
    int32_t *err;
};

__device__ __forceinline__ Span cache_span(const GParams &p)
{
    return Span{p.cache, uint64_t(p.num_slots) * kFp4Slot};
}
__device__ __forceinline__ Span slots_span(const GParams &p)
{
    return Span{p.slots, uint64_t(p.rows) * 8u};
}
__device__ __forceinline__ Span out_span(const GParams &p)
{
    return Span{p.out, uint64_t(p.rows) * DSV4_HEAD_DIM * 2u};
}

// what a lane holds of one row
struct Row {
    int64_t slot;
    uint32_t lo, e0, e1;
    uint4 hi;  // .x: the second code word (lanes 0..23), or 8 rope dims (lanes 24..31)
};

__device__ __forceinline__ Row load_row(const GParams &p, int lane, int64_t slot)
{
    Row r;
    r.slot = slot;
    r.lo = r.e0 = r.e1 = 0u;
    r.hi = make_uint4(0u, 0u, 0u, 0u);
    if (slot >= 0 && slot < p.num_slots) {
        const uint32_t s32 = static_cast<uint32_t>(slot);
        const uint32_t blk = fastdiv(s32, p.slot_div);
        const Fp4Row at = fp4_row(p.cache, blk, s32 - blk * p.block_size, p.block_size);
        const Span cs = cache_span(p);
        r.lo = ldg4_in(at.data + 4 * lane, cs, p.err);
        r.e0 = ldg_byte_in(at.scale + (lane >> 2), cs, p.err);
        if (lane < 24) {
            r.hi.x = ldg4_in(at.data + 128 + 4 * lane, cs, p.err);
            r.e1 = ldg_byte_in(at.scale + 8 + (lane >> 2), cs, p.err);
        } else {
            r.hi = ldg16_in(at.data + kFp4Codes + 16 * (lane - 24), cs, p.err);
        }
    }
    return r;
}

__device__ __forceinline__ int64_t load_slot(const GParams &p, int64_t n)
{
    return n < p.rows ? ldg_i64_in(p.slots + n, slots_span(p), p.err) : -1;
}

__global__ void __launch_bounds__(kThreads, 12) fp4_gather_kernel(const GParams p)
{
    wait_for_kernel_before();
    const int lane = threadIdx.x & 31;
    const int64_t stride = int64_t(gridDim.x) * (kThreads / 32);
    int64_t n = int64_t(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    if (n >= p.rows)
        return;
    Row cur = load_row(p, lane, load_slot(p, n));
    int64_t ahead = load_slot(p, n + stride);
    for (; n < p.rows; n += stride) {
        const Row nxt = load_row(p, lane, ahead);
        ahead = load_slot(p, n + 2 * stride);
        uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
        if (cur.slot >= p.num_slots) {
            if (lane == 0 && p.err != nullptr)
                atomicOr(p.err, DSV4_DEVERR_SLOT_RANGE);
        } else if (cur.slot >= 0) {
            a = fp4x8_to_bf16(cur.lo, fp4_scale_bf16x2(cur.e0));
            b = lane < 24 ? fp4x8_to_bf16(cur.hi.x, fp4_scale_bf16x2(cur.e1)) : cur.hi;
        }
        uint16_t *row = p.out + n * DSV4_HEAD_DIM;
        st16_in(row + 8 * lane, a, out_span(p), p.err);
        st16_in(row + 256 + 8 * lane, b, out_span(p), p.err);
        cur = nxt;
    }
}

}  // namespace

int fp4_gather_ctas_per_sm(int *ctas_per_sm)
{
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(ctas_per_sm, fp4_gather_kernel, kThreads,
                                                         0) == cudaSuccess
               ? DSV4_OK
               : DSV4_ERR_CUDA;
}

int launch_fp4_gather(const uint8_t *cache, int64_t num_blocks, int32_t block_size,
                      const int64_t *slots, int64_t rows, uint16_t *out, int32_t *err,
                      int64_t max_ctas, cudaStream_t stream)
{
    GParams p;
    p.cache = cache;
    p.num_slots = num_blocks * int64_t(block_size);
    p.block_size = static_cast<uint32_t>(block_size);
    p.slot_div = fastdiv_magic(p.block_size);
    p.slots = slots;
    p.rows = rows;
    p.out = out;
    p.err = err;
    const int64_t need = (rows + kThreads / 32 - 1) / (kThreads / 32);
    return launch_after(fp4_gather_kernel, dim3(unsigned(need < max_ctas ? need : max_ctas)),
                        dim3(kThreads), stream, p);
}

}  // namespace dsv4

DSV4_BOUNDS_FLAG_READER(bounds_flag_fp4_gather)
