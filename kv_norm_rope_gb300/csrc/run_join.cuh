// Attention in runs: each CTA of a persistent attention kernel takes a run of tiles of
// keys (key_tiles.cuh) and leaves the unnormalised outputs of row tiles that it shares
// with other runs in a workspace; the kernel here joins them.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include "convert.cuh"
#include "key_tiles.cuh"
#include "launch_status.h"
#include "ops.h"

namespace dsv4 {
namespace {

constexpr int kRows = 64;            // query rows of a CTA
constexpr int kMaxCtas = 160;        // of a launch: what the workspace is for
constexpr float kUnset = -3.402823466e38f;  // m of a row that has seen no key: below any score
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Workspace: two partial results a CTA, O [64, 512] then m [64] and sum [64]; after all
// of them, a RunEnds a CTA.
constexpr size_t kPartialFloats = size_t(kRows) * DSV4_HEAD_DIM + 2 * kRows;

// The units whose partial results a run left, for the join; -1 for none.
struct alignas(16) RunEnds {
    int continued;  // one that an earlier run began, in slot 0
    int left_open;  // one that this run began and later ones go on with
    int slot;       // of left_open
    int unused;
};

struct WParams {
    AParams p;
    float *partials;
    RunEnds *ends;
    int runs;    // CTAs
    int splits;  // columns of the join's blocks that join; the others serve rows without keys
    float unit;  // of the accumulated O: what it is multiplied by for the output
};

__device__ __forceinline__ float *partial_at(const WParams &w, int x, int slot)
{
    return w.partials + (size_t(x) * 2 + slot) * kPartialFloats;
}
__device__ __forceinline__ Span partial_span(const WParams &w)
{
    return Span{w.partials, uint64_t(w.runs) * 2u * kPartialFloats * 4u};
}
__device__ __forceinline__ Span ends_span(const WParams &w)
{
    return Span{w.ends, uint64_t(w.runs) * sizeof(RunEnds)};
}

// What the join has to know of a run (its first place is c), found by following it from unit
// to unit by one warp.
template <typename Cursor>
__device__ void note_ends(const WParams &w, Cursor c)
{
    int continued = -1, left_open = -1, slot = 0;
    if (c.left > 0 && c.tile > c.range.first())
        continued = c.unit;
    while (c.left > 0) {
        const int rest = c.range.stop() - c.tile;  // of the unit's tiles
        if (c.left < rest && c.tile == c.range.first())
            left_open = c.unit;
        if (c.left <= rest)
            break;
        slot = 1;  // of any but the first unit
        c.left -= rest - 1;
        c.tile = c.range.stop() - 1;
        c.advance(w.p);
    }
    if ((threadIdx.x & 31) == 0)
        st16_in(w.ends + blockIdx.x, make_uint4(uint32_t(continued), uint32_t(left_open), uint32_t(slot), 0u),
                ends_span(w), w.p.a.b.err);
}

__device__ __forceinline__ float sink_of(const AttentionArgs &a, int row)
{
    return a.sinks == nullptr ? -INFINITY
                              : kLog2e * ldg_f32_in(a.sinks + row % a.heads,
                                                    Span{a.sinks, uint64_t(a.heads) * 4u}, a.b.err);
}

// From a row's m and sum (both without the sink): the factor that makes its O the
// output, and its lse.
__device__ __forceinline__ float finish(float m, float sum, float sink, float unit, float *lse)
{
    if (sum == 0.0f)
        m = -INFINITY;
    const float top = fmaxf(m, sink);
    if (top == -INFINITY) {
        *lse = -INFINITY;
        return 0.0f;
    }
    const float w = exp2_approx(m - top), total = sum * w + exp2_approx(sink - top);
    *lse = (top + log2f(total)) * kLn2;
    return w / total * unit;
}

// Joins the partial results of the units whose tiles more than one run took, and
// writes the rows of units that see no key.  A row goes to one warp, or, where a few long
// requests are spread over many runs, to the eight warps of a block (kSplit), each
// with every eighth run.  It is launched while the attention ends.
//
// Column x < splits of the blocks joins the x-th unit that some run left open, which the
// runs have noted, so the cost goes by the runs and not by the units.  The other columns
// look through the units for those without keys, each at its share of them.  (A column a
// unit, each finding its runs by a look at all lengths, took 6.1 ms for 64000 idle
// requests, against 0.3.)  What the first two runs left of a row is loaded before the maximum
// is known: 17.3 us instead of 18.4 for two requests of 8 heads, 41.0 instead of 42.8 for
// 48 of 64.
constexpr int kJoinWarps = 8;
constexpr int kIdleColumns = 64;
static_assert(kMaxCtas % 32 == 0, "the join's lanes hold the ends of kMaxCtas / 32 runs each");

__device__ __forceinline__ int row_of_block(bool split)
{
    return split ? blockIdx.y : blockIdx.y * kJoinWarps + (threadIdx.x >> 5);
}

// Row r of a unit from its m, its sum and the unnormalised o (kSplit: o[0] is dims 128
// times the warp on).
template <bool kSplit>
__device__ __forceinline__ void write_row(const WParams &w, int unit, int r, float m, float sum,
                                          const float4 *o)
{
    const AParams &p = w.p;
    const AttentionArgs &a = p.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int request = int(fastdiv(uint32_t(unit), p.tile_div));
    const int in_request = (unit - request * p.row_tiles) * kRows + r;
    const int64_t row = int64_t(request) * p.all_rows + in_request;
    const Span os{a.out, rows_of(a) * (DSV4_HEAD_DIM * 2u)};
    float lse;
    const float f = finish(m, sum, sink_of(a, in_request), w.unit, &lse);
    const int first = kSplit ? warp : 0, last = kSplit ? warp : 3;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (k < first || k > last)
            continue;
        const float4 v = kSplit ? o[0] : o[k];
        st8_in(a.out + row * DSV4_HEAD_DIM + 128 * k + 4 * lane,
               f == 0.0f ? make_uint2(0u, 0u)
                         : make_uint2(bf16x2_rn(v.x * f, v.y * f), bf16x2_rn(v.z * f, v.w * f)),
               os, a.b.err);
    }
    if (lane == 0 && first == 0 && a.lse != nullptr)
        st_f32_in(a.lse + row, lse, Span{a.lse, rows_of(a) * 4u}, a.b.err);
}

// whether row r of the unit is one of its request's
__device__ __forceinline__ bool has_row(const AParams &p, int unit, int r)
{
    return (unit - int(fastdiv(uint32_t(unit), p.tile_div)) * p.row_tiles) * kRows + r < p.all_rows;
}

template <bool kSplit, typename Tiles>
__device__ __forceinline__ void rows_without_keys(const WParams &w, int column, int columns)
{
    const AParams &p = w.p;
    const int lane = threadIdx.x & 31, r = row_of_block(kSplit);
    if (kSplit && (threadIdx.x >> 5) >= 4)
        return;
    const float4 none[4] = {};
    for (int base = column; base < p.units; base += 32 * columns) {
        const int mine = base + lane * columns;
        unsigned idle = __ballot_sync(kFull, mine < p.units && Tiles::tiles_of(p, mine) == 0);
        for (; idle != 0u; idle &= idle - 1u) {
            const int unit = base + (__ffs(idle) - 1) * columns;
            if (has_row(p, unit, r))
                write_row<kSplit>(w, unit, r, kUnset, 0.0f, none);
        }
    }
}

template <bool kSplit, typename Tiles>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const __grid_constant__ WParams w)
{
    __shared__ float4 o_s[kSplit ? kJoinWarps : 1][4][32];
    __shared__ float sum_s[kJoinWarps];
    const AParams &p = w.p;
    int32_t *err = p.a.b.err;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    wait_for_kernel_before();
    if (int(blockIdx.x) >= w.splits) {
        rows_without_keys<kSplit, Tiles>(w, int(blockIdx.x) - w.splits, int(gridDim.x) - w.splits);
        return;
    }
    // the run that left this block's unit open, and the last one that goes on with it
    int continued[kMaxCtas / 32], unit = -1, x0 = 0, slot0 = 0, count = 0;
#pragma unroll
    for (int i = 0; i < kMaxCtas / 32; ++i) {
        const int x = 32 * i + lane;
        const uint4 e = x < w.runs ? ld16_in(w.ends + x, ends_span(w), err)
                                   : make_uint4(~0u, ~0u, 0u, 0u);
        continued[i] = int(e.x);
        const unsigned open = __ballot_sync(kFull, int(e.y) >= 0);
        const int nth = int(blockIdx.x) - count;
        count += __popc(open);
        if (nth >= 0 && nth < __popc(open)) {
            const unsigned before = open & ((1u << lane) - 1u);
            const int from = __ffs(__ballot_sync(kFull, ((open >> lane) & 1u) && __popc(before) == nth)) - 1;
            x0 = 32 * i + from;
            unit = __shfl_sync(kFull, int(e.y), from);
            slot0 = __shfl_sync(kFull, int(e.z), from);
        }
    }
    const int r = row_of_block(kSplit);
    // fewer units are open, or no row (with kSplit the same for the whole block)
    if (unit < 0 || !has_row(p, unit, r))
        return;
    int x1 = x0;
#pragma unroll
    for (int i = 0; i < kMaxCtas / 32; ++i)
        x1 = continued[i] == unit ? max(x1, 32 * i + lane) : x1;
    x1 = __reduce_max_sync(kFull, x1);
    const Span ps = partial_span(w);
    const auto part = [&](int x) {
        return w.partials + (size_t(x) * 2 + (x == x0 ? slot0 : 0)) * kPartialFloats;
    };
    // a run's m and sum for the row, and the lane's share of its O
    struct Part {
        float m, n;
        float4 o[4];
    };
    const auto load = [&](int x) {
        const float *from = x <= x1 ? part(x) : nullptr;
        Part q;
        q.m = q.n = 0.0f;
        if (from != nullptr) {
            q.m = ld_f32_in(from + kRows * DSV4_HEAD_DIM + r, ps, err);
            q.n = ld_f32_in(from + kRows * DSV4_HEAD_DIM + kRows + r, ps, err);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            q.o[k] = from != nullptr ? ld_f4_in(from + r * DSV4_HEAD_DIM + 4 * lane + 128 * k, ps, err)
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
        return q;
    };
    const int step = kSplit ? kJoinWarps : 1;
    int x = x0 + (kSplit ? warp : 0);
    // what most rows need, on its way before the maximum is known
    const Part a = load(x), b = load(x + step);
    float m = kUnset;
    for (int y = x0 + lane; y <= x1; y += 32) {
        const float *at = part(y) + kRows * DSV4_HEAD_DIM + r;
        const float own = ld_f32_in(at, ps, err);
        if (ld_f32_in(at + kRows, ps, err) != 0.0f)
            m = fmaxf(m, own);
    }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1)
        m = fmaxf(m, __shfl_xor_sync(kFull, m, d));
    float sum = 0.0f;
    float4 o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
        o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    const auto add = [&](const Part &q) {
        const float f = q.n == 0.0f ? 0.0f : exp2_approx(q.m - m);
        sum += q.n * f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            o[k].x += q.o[k].x * f;
            o[k].y += q.o[k].y * f;
            o[k].z += q.o[k].z * f;
            o[k].w += q.o[k].w * f;
        }
    };
    add(a);
    add(b);
    x += 2 * step;
#pragma unroll 4
    for (; x <= x1; x += step)
        add(load(x));
    if constexpr (kSplit) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            o_s[warp][k][lane] = o[k];
        if (lane == 0)
            sum_s[warp] = sum;
        __syncthreads();
        if (warp >= 4)
            return;
        // warp k finishes dims 128k..
        sum = 0.0f;
        o[0] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kJoinWarps; ++i) {
            const float4 v = o_s[i][warp][lane];
            sum += sum_s[i];
            o[0].x += v.x;
            o[0].y += v.y;
            o[0].z += v.z;
            o[0].w += v.w;
        }
    }
    write_row<kSplit>(w, unit, r, m, sum, o);
}

// The current device's SMs, and the kernel's shared memory allowed on it; `sm_count` is the
// kernel's own.
template <typename P>
inline int configure_runs(void (*kernel)(P), size_t smem, std::atomic<int> (&sm_count)[64], int *sms)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return DSV4_ERR_CUDA;
    const bool cached = dev >= 0 && dev < 64;
    *sms = cached ? sm_count[dev].load(std::memory_order_relaxed) : 0;
    if (*sms > 0)
        return DSV4_OK;
    if (cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || *sms < 1 ||
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)) != cudaSuccess)
        return DSV4_ERR_CUDA;
    if (cached)
        sm_count[dev].store(*sms, std::memory_order_relaxed);
    return DSV4_OK;
}

inline size_t run_workspace()
{
    return size_t(kMaxCtas) * (2 * kPartialFloats * sizeof(float) + sizeof(RunEnds));
}

// What an attention kernel of w.runs CTAs is launched with.
template <typename Tiles>
inline WParams plan_runs(const AttentionArgs &a, float unit, int sms, void *workspace)
{
    WParams w;
    w.p = tile_params(a, kRows);
    w.partials = static_cast<float *>(workspace);
    w.ends = reinterpret_cast<RunEnds *>(w.partials + size_t(kMaxCtas) * 2 * kPartialFloats);
    w.unit = unit;
    const int64_t most =
        (int64_t(a.b.width) * a.b.block_size + Tiles::keys - 1) / Tiles::keys * w.p.units;
    int runs = sms < kMaxCtas ? sms : kMaxCtas;
    runs = most < runs ? int(most) : runs;
    w.runs = runs;
    // each is begun by a run that is not the last
    w.splits = w.p.units < runs - 1 ? w.p.units : runs - 1;
    return w;
}

// The join, after that kernel.
template <typename Tiles>
inline int launch_join(const WParams &w, cudaStream_t stream)
{
    const int idle = w.p.units < kIdleColumns ? w.p.units : kIdleColumns;
    const unsigned columns = unsigned(w.splits + idle);
    const unsigned rows = unsigned(w.p.all_rows < kRows ? w.p.all_rows : kRows);
    // a unit spans runs / units of them and at most two more
    if (w.runs / w.p.units >= kJoinWarps)
        return launch_after(join_kernel<true, Tiles>, dim3(columns, rows), dim3(kJoinWarps * 32), stream, w);
    return launch_after(join_kernel<false, Tiles>, dim3(columns, (rows + kJoinWarps - 1) / kJoinWarps),
                        dim3(kJoinWarps * 32), stream, w);
}

}  // namespace
}  // namespace dsv4
