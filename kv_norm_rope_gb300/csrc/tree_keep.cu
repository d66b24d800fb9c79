// Keeping the accepted path of a tree of drafted tokens: the path's rows move together
// behind the context, in whichever paged cache they lie.
//
// Row path[i] of the drafted ones goes to place i <= path[i].  Places are sources of later
// moves too, so one CTA has a request: it loads all rows that move (64 of 1 KB at most, in the
// registers of 512 threads), waits, and stores them.  A row is a data row and a scale row of
// its block; they are moved as bytes.
//
// A chain of dependent loads (length and path, table, rows) and one exchange: latency, not
// bandwidth, bounds it.  In a graph 2.2 us for 32 requests of 16 drafted FP8 rows, 4.0 for 256
// of 64 bf16 rows; a launch from the host takes longer than either.

#include <cuda_runtime.h>
#include <stdint.h>

#include "bounds.cuh"
#include "fastdiv.h"
#include "launch_status.h"
#include "ops.h"

namespace dsv4 {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kKeepWarps = 16;
constexpr int kWarpRows = kMaxDrafted / kKeepWarps;  // 4
static_assert(kMaxDrafted == 64, "a path is two ballots");

struct KeepParams {
    TreeKeepArgs a;
    uint64_t block_div;
};

__device__ __forceinline__ void flag(int32_t *err, int bit)
{
    if (err != nullptr)
        atomicOr(err, bit);
}

__device__ __forceinline__ uint4 load_unit(const uint4 *p, Span s, int32_t *err) { return ld16_in(p, s, err); }
__device__ __forceinline__ uint2 load_unit(const uint2 *p, Span s, int32_t *err) { return ld8_in(p, s, err); }
__device__ __forceinline__ uint32_t load_unit(const uint32_t *p, Span s, int32_t *err) { return ld4_in(p, s, err); }
__device__ __forceinline__ void store_unit(uint4 *p, uint4 v, Span s, int32_t *err) { st16_in(p, v, s, err); }
__device__ __forceinline__ void store_unit(uint2 *p, uint2 v, Span s, int32_t *err) { st8_in(p, v, s, err); }
__device__ __forceinline__ void store_unit(uint32_t *p, uint32_t v, Span s, int32_t *err) { st4_in(p, v, s, err); }

// A slot's data row and its scale row (kScale bytes, one unit S; kScale 0: none).
template <int kData, int kScale>
struct Slot {
    uint8_t *data, *scale;
};

template <int kData, int kScale>
__device__ __forceinline__ Slot<kData, kScale> slot_at(const TreeKeepArgs &a, uint32_t block, uint32_t off)
{
    const uint64_t bs = uint32_t(a.b.block_size);
    uint8_t *page = const_cast<uint8_t *>(a.b.cache) + block * bs * (kData + kScale);
    return Slot<kData, kScale>{page + uint64_t(off) * kData, page + bs * kData + uint64_t(off) * kScale};
}

// kData, kScale: bytes of the rows; D, S: the units they are moved in
template <int kData, typename D, int kScale, typename S>
__global__ void __launch_bounds__(kKeepWarps * 32) tree_keep_kernel(const KeepParams p)
{
    constexpr int kUnits = kData / int(sizeof(D)), kLaneUnits = (kUnits + 31) / 32;
    const TreeKeepArgs &a = p.a;
    int32_t *err = a.b.err;
    const int b = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    wait_for_kernel_before();
    const int32_t *path = a.path + int64_t(b) * a.q_len;
    const Span path_span{a.path, uint64_t(a.b.batch) * uint32_t(a.q_len) * 4u};
    const auto entry = [&](int i) { return i < a.q_len ? int(ld4_in(path + i, path_span, err)) : -1; };
    const int e0 = entry(lane), e1 = entry(lane + 32);
    int n = int(ld4_in(a.b.lens + b, Span{a.b.lens, uint64_t(a.b.batch) * 4u}, err));
    const int asked = int(ld4_in(a.path_lens + b, Span{a.path_lens, uint64_t(a.b.batch) * 4u}, err));
    const int limit = a.b.width * a.b.block_size;
    bool bad = n > limit;
    n = n < 0 ? 0 : n > limit ? limit : n;
    // the entries up to the first that does not rise or is none of the drafted
    const int last0 = __shfl_sync(kFull, e0, 31);
    int before0 = __shfl_up_sync(kFull, e0, 1), before1 = __shfl_up_sync(kFull, e1, 1);
    before0 = lane == 0 ? -1 : before0;
    before1 = lane == 0 ? last0 : before1;
    const unsigned wrong0 = __ballot_sync(kFull, e0 <= before0 || e0 >= a.q_len);
    const unsigned wrong1 = __ballot_sync(kFull, e1 <= before1 || e1 >= a.q_len);
    const int rising = wrong0 != 0u ? __ffs(wrong0) - 1 : wrong1 != 0u ? 31 + __ffs(wrong1) : 64;
    int count = asked < 0 ? 0 : asked < rising ? asked : rising;
    const int context = n - a.q_len;
    bad = bad || (n > 0 && (count != asked || context < 0));
    if (n == 0 || context < 0)
        count = 0;
    if (bad && threadIdx.x == 0)
        flag(err, DSV4_DEVERR_SLOT_RANGE);
    // row i of the path is the i % kKeepWarps-th warp's; its lane j < kWarpRows has row j's places
    const int row = (lane & (kWarpRows - 1)) * kKeepWarps + warp;
    // (by the whole warp: some of its lanes have rows below 32, some above)
    const int from0 = __shfl_sync(kFull, e0, row & 31), from1 = __shfl_sync(kFull, e1, row & 31);
    const int from = row < 32 ? from0 : from1;
    uint32_t src_block = UINT32_MAX, src_off = 0u, dst_block = 0u, dst_off = 0u;
    if (row < count && from != row) {
        const int32_t *table = a.b.table + b * a.b.table_stride;
        const Span table_span{a.b.table, (uint64_t(a.b.batch - 1) * a.b.table_stride + a.b.width) * 4u};
        const uint32_t src = uint32_t(context + from), dst = uint32_t(context + row);
        const uint32_t at = fastdiv(src, p.block_div), to = fastdiv(dst, p.block_div);
        src_off = src - at * uint32_t(a.b.block_size);
        dst_off = dst - to * uint32_t(a.b.block_size);
        src_block = ld4_in(table + at, table_span, err);
        dst_block = ld4_in(table + to, table_span, err);
        if (int64_t(src_block) >= a.b.num_blocks || int64_t(dst_block) >= a.b.num_blocks) {
            flag(err, DSV4_DEVERR_SLOT_RANGE);
            src_block = UINT32_MAX;
        }
    }
    const Span cache{a.b.cache, uint64_t(a.b.num_blocks) * uint32_t(a.b.block_size) * (kData + kScale)};
    D data[kWarpRows][kLaneUnits];
    S scale;
    Slot<kData, kScale> to[kWarpRows];
#pragma unroll
    for (int j = 0; j < kWarpRows; ++j) {
        const uint32_t block = __shfl_sync(kFull, src_block, j);
        const Slot<kData, kScale> at = slot_at<kData, kScale>(a, block, __shfl_sync(kFull, src_off, j));
        to[j] = slot_at<kData, kScale>(a, __shfl_sync(kFull, dst_block, j), __shfl_sync(kFull, dst_off, j));
        if (block == UINT32_MAX)
            to[j].data = nullptr;
#pragma unroll
        for (int u = 0; u < kLaneUnits; ++u)
            if (to[j].data != nullptr && u * 32 + lane < kUnits)
                data[j][u] = load_unit(reinterpret_cast<const D *>(at.data) + u * 32 + lane, cache, err);
        if (kScale > 0 && to[j].data != nullptr && lane == j)
            scale = load_unit(reinterpret_cast<const S *>(at.scale), cache, err);
    }
    __syncthreads();  // all that this request moves is read, its length too
#pragma unroll
    for (int j = 0; j < kWarpRows; ++j) {
        if (to[j].data == nullptr)
            continue;
#pragma unroll
        for (int u = 0; u < kLaneUnits; ++u)
            if (u * 32 + lane < kUnits)
                store_unit(reinterpret_cast<D *>(to[j].data) + u * 32 + lane, data[j][u], cache, err);
        if (kScale > 0 && lane == j)
            store_unit(reinterpret_cast<S *>(to[j].scale), scale, cache, err);
    }
    if (threadIdx.x == 0)
        st_i32_in(a.new_lens + b, context < 0 ? n : context + count, Span{a.new_lens, uint64_t(a.b.batch) * 4u}, err);
}

}  // namespace

int launch_tree_keep(int store_mode, const TreeKeepArgs &a, cudaStream_t stream)
{
    const KeepParams p{a, fastdiv_magic(uint32_t(a.b.block_size))};
    const dim3 grid(unsigned(a.b.batch)), block(kKeepWarps * 32);
    // FP8 rows stand on 16-byte boundaries in caches of an even block size, indexer rows on
    // 4-byte ones in any
    const bool wide = ((reinterpret_cast<uintptr_t>(a.b.cache) | (8u * uint32_t(a.b.block_size))) & 15u) == 0u;
    switch (store_mode) {
    case DSV4_STORE_FP8:
        return launch_after(wide ? tree_keep_kernel<DSV4_FP8_DATA_BYTES, uint4, DSV4_FP8_SCALE_BYTES, uint2>
                                 : tree_keep_kernel<DSV4_FP8_DATA_BYTES, uint2, DSV4_FP8_SCALE_BYTES, uint2>,
                            grid, block, stream, p);
    case DSV4_STORE_BF16:
        return launch_after(tree_keep_kernel<DSV4_BF16_SLOT_BYTES, uint4, 0, uint32_t>, grid, block, stream, p);
    case DSV4_STORE_FP4:
        return launch_after(tree_keep_kernel<DSV4_FP4_DATA_BYTES, uint4, DSV4_FP4_SCALE_BYTES, uint4>, grid, block,
                            stream, p);
    default:
        return launch_after(tree_keep_kernel<DSV4_INDEXER_DIM, uint32_t, 4, uint32_t>, grid, block, stream, p);
    }
}

}  // namespace dsv4

DSV4_BOUNDS_FLAG_READER(bounds_flag_tree_keep)
