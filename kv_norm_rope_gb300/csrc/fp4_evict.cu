// Eviction from the 4-bit cache by accumulated attention weight: select, then move.
//
// A weight becomes an unsigned key that orders as the number does (NaN as
// -infinity, -0 as 0).  The threshold T is the `need`-th highest key of the
// candidates, found by radix selection, 8 bits a pass: a histogram of the
// keys that agree with T's bits so far says which 8 bits come next.  A row is
// then kept when it is recent, when its key is above T, or when it equals T and
// is among the first of those that are still needed; positions come from a
// prefix sum in index order, so ties go to the lower index and nothing depends
// on the order in which threads run.

#include <cuda_runtime.h>
#include <stdint.h>

#include "fp4.cuh"
#include "launch_status.h"
#include "ops.h"

namespace dsv4 {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kSelectThreads = 1024;
constexpr int kMoveThreads = 256;

struct EParams {
    Fp4EvictArgs a;
    uint64_t block_div;
};

__device__ __forceinline__ void flag(int32_t *err, int bit)
{
    if (err != nullptr)
        atomicOr(err, bit);
}

__device__ __forceinline__ Span weights_span(const Fp4EvictArgs &a)
{
    return Span{a.weights, (uint64_t(a.b.batch - 1) * a.weights_stride + a.weights_width) * 4u};
}
__device__ __forceinline__ Span kept_span(const Fp4EvictArgs &a)
{
    return Span{a.kept, uint64_t(a.b.batch) * uint32_t(a.budget) * 4u};
}

__device__ __forceinline__ uint32_t order_key(float w)
{
    if (w != w)
        w = -INFINITY;
    const uint32_t b = __float_as_uint(w + 0.0f);  // -0 + 0 = 0
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// inclusive prefix sum over the CTA; *total gets the sum
__device__ __forceinline__ uint32_t cta_scan(uint32_t v, uint32_t *warp_sums, uint32_t *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t o = __shfl_up_sync(kFull, v, d);
        if (lane >= d)
            v += o;
    }
    __syncthreads();
    if (lane == 31)
        warp_sums[warp] = v;
    __syncthreads();
    if (warp == 0) {
        uint32_t s = warp_sums[lane];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t o = __shfl_up_sync(kFull, s, d);
            if (lane >= d)
                s += o;
        }
        warp_sums[lane] = s;
    }
    __syncthreads();
    *total = warp_sums[31];
    return v + (warp > 0 ? warp_sums[warp - 1] : 0u);
}

__global__ void __launch_bounds__(kSelectThreads) fp4_select_kernel(const EParams p)
{
    __shared__ uint32_t hist[256], warp_sums[32], chosen[2];
    const Fp4EvictArgs &a = p.a;
    const int r = blockIdx.x;
    int64_t limit = int64_t(a.b.width) * a.b.block_size;
    limit = limit < a.weights_width ? limit : a.weights_width;
    int n = int(ldg4_in(a.b.lens + r, Span{a.b.lens, uint64_t(a.b.batch) * 4u}, a.b.err));
    __syncthreads();  // new_lens may be lens
    if (n > limit) {
        if (threadIdx.x == 0)
            flag(a.b.err, DSV4_DEVERR_SLOT_RANGE);
        n = int(limit);
    }
    n = n < 0 ? 0 : n;
    const int keep = n < a.budget ? n : a.budget;
    int32_t *kept = a.kept + int64_t(r) * a.budget;
    if (threadIdx.x == 0)
        st_i32_in(a.new_lens + r, keep, Span{a.new_lens, uint64_t(a.b.batch) * 4u}, a.b.err);
    if (n <= a.budget) {
        for (int i = threadIdx.x; i < a.budget; i += kSelectThreads)
            st_i32_in(kept + i, i < n ? i : -1, kept_span(a), a.b.err);
        return;
    }
    const float *w = a.weights + r * a.weights_stride;
    const int candidates = n - a.recent;
    uint32_t need = uint32_t(a.budget - a.recent), prefix = 0u;
    if (need > 0u) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            if (threadIdx.x < 256)
                hist[threadIdx.x] = 0u;
            __syncthreads();
            for (int i = threadIdx.x; i < candidates; i += kSelectThreads) {
                const uint32_t k = order_key(ldg_f32_in(w + i, weights_span(a), a.b.err));
                if (shift == 24 || ((k ^ prefix) >> (shift + 8)) == 0u)
                    atomicAdd(&hist[(k >> shift) & 255u], 1u);
            }
            __syncthreads();
            // thread i holds digit 255 - i: the running count from the top
            uint32_t total;
            const uint32_t mine = threadIdx.x < 256 ? hist[255 - threadIdx.x] : 0u;
            const uint32_t upto = cta_scan(mine, warp_sums, &total);
            if (threadIdx.x < 256 && upto >= need && upto - mine < need) {
                chosen[0] = 255u - threadIdx.x;
                chosen[1] = need - (upto - mine);
            }
            __syncthreads();
            prefix |= chosen[0] << shift;
            need = chosen[1];
            __syncthreads();
        }
    }
    // `need` rows whose key is the threshold `prefix` are kept, the first ones
    const bool any = a.budget > a.recent;
    uint32_t equal_before = 0u, out = 0u;
    for (int i0 = 0; i0 < n; i0 += kSelectThreads) {
        const int i = i0 + threadIdx.x;
        const bool candidate = any && i < candidates;
        const uint32_t k = candidate ? order_key(ldg_f32_in(w + i, weights_span(a), a.b.err)) : 0u;
        const bool equal = candidate && k == prefix;
        uint32_t equals;
        const uint32_t rank = equal_before + cta_scan(equal ? 1u : 0u, warp_sums, &equals);
        const bool take = (i >= candidates && i < n) || (candidate && k > prefix) ||
                          (equal && rank <= need);
        uint32_t taken;
        const uint32_t at = out + cta_scan(take ? 1u : 0u, warp_sums, &taken);
        if (take)
            st_i32_in(kept + at - 1, i, kept_span(a), a.b.err);
        equal_before += equals;
        out += taken;
    }
}

// One warp per kept row: 22 lanes move its data, one its scales, and lane 0 its weight.
__global__ void __launch_bounds__(kMoveThreads) fp4_move_kernel(const EParams p)
{
    const Fp4EvictArgs &a = p.a;
    const int lane = threadIdx.x & 31;
    const int64_t rows = int64_t(a.b.batch) * a.budget;
    const uint32_t bs = uint32_t(a.b.block_size);
    uint8_t *cache = const_cast<uint8_t *>(a.b.cache);
    const Span cs{cache, uint64_t(a.b.num_blocks) * bs * kFp4Slot};
    const Span old_span{a.b.table, (uint64_t(a.b.batch - 1) * a.b.table_stride + a.b.width) * 4u};
    const Span new_span{a.new_table, (uint64_t(a.b.batch - 1) * a.new_table_stride + a.new_width) * 4u};
    const Span out_span{a.new_weights, uint64_t(rows) * 4u};
    for (int64_t i = int64_t(blockIdx.x) * (kMoveThreads / 32) + (threadIdx.x >> 5); i < rows;
         i += int64_t(gridDim.x) * (kMoveThreads / 32)) {
        const int64_t r = i / a.budget;
        const uint32_t to = uint32_t(i - r * a.budget);
        const int from = int(ldg4_in(a.kept + i, kept_span(a), a.b.err));
        if (from < 0) {
            if (lane == 0)
                st_f32_in(a.new_weights + i, 0.0f, out_span, a.b.err);
            continue;
        }
        const uint32_t from_at = fastdiv(uint32_t(from), p.block_div), to_at = fastdiv(to, p.block_div);
        const uint32_t src = ldg4_in(a.b.table + r * a.b.table_stride + from_at, old_span, a.b.err);
        const uint32_t dst = ldg4_in(a.new_table + r * a.new_table_stride + to_at, new_span, a.b.err);
        if (lane == 0)
            st_f32_in(a.new_weights + i,
                      ldg_f32_in(a.weights + r * a.weights_stride + from, weights_span(a), a.b.err),
                      out_span, a.b.err);
        if (int64_t(src) >= a.b.num_blocks || int64_t(dst) >= a.b.num_blocks) {
            if (lane == 0)
                flag(a.b.err, DSV4_DEVERR_SLOT_RANGE);
            continue;
        }
        const Fp4Row s = fp4_row(cache, src, uint32_t(from) - from_at * bs, bs);
        const Fp4Row d = fp4_row(cache, dst, to - to_at * bs, bs);
        if (lane < 23) {
            const uint8_t *at = lane < 22 ? s.data + 16 * lane : s.scale;
            uint8_t *put = const_cast<uint8_t *>(lane < 22 ? d.data + 16 * lane : d.scale);
            st16_in(put, ldg16_in(at, cs, a.b.err), cs, a.b.err);
        }
    }
}

}  // namespace

int launch_fp4_evict(const Fp4EvictArgs &a, cudaStream_t stream)
{
    EParams p{a, fastdiv_magic(uint32_t(a.b.block_size))};
    const int st = launch_kernel(fp4_select_kernel, dim3(unsigned(a.b.batch)), dim3(kSelectThreads), 0,
                                 stream, p);
    if (st != DSV4_OK)
        return st;
    const int64_t warps = int64_t(a.b.batch) * a.budget, ctas = (warps + 7) / 8;
    return launch_kernel(fp4_move_kernel, dim3(unsigned(ctas < 152 * 8 ? ctas : 152 * 8)),
                         dim3(kMoveThreads), 0, stream, p);
}

}  // namespace dsv4

DSV4_BOUNDS_FLAG_READER(bounds_flag_fp4_evict)
