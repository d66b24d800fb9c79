// What the attention kernels over paged caches share: which keys a tile of query rows
// sees, and how the tiles of keys of all requests are dealt out to CTAs.
//
// A tile is kKeys keys, aligned in the request.  The tiles that some row of a row
// tile sees, over all requests in order, form one line; each CTA takes a run of it of
// equal cost (start_cost() below).  So a long request is shared by many CTAs and short ones share a
// CTA, whatever the lengths, which only the device knows.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "bounds.cuh"
#include "fastdiv.h"
#include "ops.h"
#include "tcgen05.cuh"

namespace dsv4 {
namespace {

constexpr unsigned kFull = 0xffffffffu;

struct AParams {
    AttentionArgs a;
    uint64_t block_div, head_div, tile_div;  // fastdiv_magic of block_size, heads, row_tiles
    int all_rows;        // q_len * heads
    int tile_rows;       // of a row tile
    int row_tiles;       // of a request
    int units;           // row tiles of the batch
};

__device__ __forceinline__ Span table_span(const PagedBatch &b)
{
    return Span{b.table, (uint64_t(b.batch - 1) * b.table_stride + b.width) * 4u};
}
__device__ __forceinline__ uint64_t rows_of(const AttentionArgs &a)
{
    return uint64_t(a.b.batch) * uint32_t(a.q_len) * uint32_t(a.heads);
}

__device__ __forceinline__ void flag(int32_t *err, int bit)
{
    if (err != nullptr)
        atomicOr(err, bit);
}

// the keys of request r, as many as its row of the table can name
__device__ __forceinline__ int length_of(const PagedBatch &b, int r)
{
    const int limit = b.width * b.block_size;
    const int n = int(ldg4_in(b.lens + r, Span{b.lens, uint64_t(b.batch) * 4u}, b.err));
    if (n > limit)
        flag(b.err, DSV4_DEVERR_SLOT_RANGE);
    return n < 0 ? 0 : n > limit ? limit : n;
}

constexpr int kDealThreads = 512;
constexpr int kDealWarps = kDealThreads / 32;
constexpr int kDealWords = 4 * kDealWarps + 4;
static_assert(kDealWarps <= 32, "a lane has a warp's sums");

// kStartCost: start_cost() below.  kTrees: the arguments may hold trees of drafted tokens.
template <int kKeys, int kStartCost, bool kTrees>
struct KeyTiles {
    static constexpr int keys = kKeys;

    // The keys [lo, hi) that some of the rows [row0, row1) of a request of n keys sees,
    // and the tiles they lie in.  Row r is head r % heads of token r / heads.
    struct Range {
        int lo, hi;
        __device__ __forceinline__ int first() const { return lo / kKeys; }
        __device__ __forceinline__ int stop() const { return (hi + kKeys - 1) / kKeys; }
        __device__ __forceinline__ int tiles() const { return stop() - first(); }
    };

    static __device__ __forceinline__ Range range_of(const AParams &p, int n, int row0, int row1)
    {
        const AttentionArgs &a = p.a;
        if (kTrees && a.tree != nullptr) {
            // the context from where a first drafted token's window begins, and all drafted keys
            const int from = a.window > 0 ? n - a.q_len + 1 - a.window : 0;
            return Range{from > 0 ? from : 0, n};
        }
        const int hi = n - a.q_len + 1 + int(fastdiv(uint32_t(row1 - 1), p.head_div));
        if (hi <= 0)
            return Range{0, 0};
        const int from =
            a.window > 0 ? n - a.q_len + 1 + int(fastdiv(uint32_t(row0), p.head_div)) - a.window : 0;
        return Range{from > 0 ? from : 0, hi};
    }

    // A place on a CTA's run of tiles.  A unit is one row tile of one request.
    struct Cursor {
        int unit, request, tile, left, n, row0, row1;
        Range range;

        // the unit's numbers, for a place inside it
        __device__ __forceinline__ void enter(const AParams &p)
        {
            request = int(fastdiv(uint32_t(unit), p.tile_div));
            row0 = (unit - request * p.row_tiles) * p.tile_rows;
            row1 = row0 + p.tile_rows < p.all_rows ? row0 + p.tile_rows : p.all_rows;
            n = length_of(p.a.b, request);
            range = range_of(p, n, row0, row1);
        }

        // true when this tile is the last of the run or of its unit
        __device__ __forceinline__ bool ends_segment() const
        {
            return left == 1 || tile + 1 == range.stop();
        }

        // to the next tile; true when that is in another unit
        __device__ __forceinline__ bool advance(const AParams &p)
        {
            if (--left == 0)
                return false;
            if (++tile < range.stop())
                return false;
            do {
                if (++unit >= p.units) {  // only if the lengths changed under the launch
                    left = 0;
                    return false;
                }
                enter(p);
            } while (range.tiles() == 0);
            tile = range.first();
            return true;
        }
    };

    static __device__ __forceinline__ int tiles_of(const AParams &p, int unit)
    {
        Cursor c;
        c.unit = unit;
        c.enter(p);
        return c.range.tiles();
    }

    // The line that is dealt to the CTAs: the units' tiles, and before those of each
    // start_cost() positions without one, for what it takes to begin a unit (its queries,
    // its first reference, its results), so that a run of many short units has fewer tiles.
    // With fewer tiles than CTAs, or few units, a run has one or two units anyway, and the
    // positions would only make some runs a tile longer.
    static __device__ __forceinline__ int start_cost(const AParams &p, int total, int X)
    {
        return total > X && p.units > X / 8 ? kStartCost : 0;
    }

    // Places c at the start of CTA x's run.  All threads of the CTA (at least
    // kDealThreads) call it.  scratch: kDealWords words of shared memory.
    static __device__ __forceinline__ void deal(const AParams &p, int x, int X, int *scratch, Cursor &c)
    {
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
        // the units from `base` on, one a thread: their tiles up to and with the thread's
        // own, and all of them, and of the units themselves those with tiles; `half` of the
        // scratch words, so that calls in turn need one barrier each
        int upto = 0, mine = 0, all = 0, units_upto = 0, units_all = 0, half = 0;
        const auto scan = [&](int base) {
            mine = tid < kDealThreads && base + tid < p.units ? tiles_of(p, base + tid) : 0;
            upto = mine;
#pragma unroll
            for (int s = 1; s < 32; s <<= 1) {
                const int o = __shfl_up_sync(kFull, upto, s);
                if (lane >= s)
                    upto += o;
            }
            units_upto = __popc(__ballot_sync(kFull, mine > 0) & (kFull >> (31 - lane)));
            int *sums = scratch + half * 2 * kDealWarps;
            if (lane == 31 && warp < kDealWarps) {
                sums[warp] = upto;
                sums[kDealWarps + warp] = units_upto;
            }
            __syncthreads();
            const int tiles = lane < kDealWarps ? sums[lane] : 0;
            const int with_tiles = lane < kDealWarps ? sums[kDealWarps + lane] : 0;
            all = __reduce_add_sync(kFull, tiles);
            units_all = __reduce_add_sync(kFull, with_tiles);
            upto += __reduce_add_sync(kFull, lane < warp ? tiles : 0);
            units_upto += __reduce_add_sync(kFull, lane < warp ? with_tiles : 0);
            half ^= 1;
        };
        int total = 0, units = 0;
        for (int base = 0; base < p.units; base += kDealThreads) {
            scan(base);
            total += all;
            units += units_all;
        }
        const int cost = start_cost(p, total, X), positions = total + cost * units;
        const int share = (positions + X - 1) / X;
        const int64_t from = int64_t(x) * share;
        c.left = 0;
        if (from >= positions)
            return;
        const int begin = int(from), end = positions - begin < share ? positions : begin + share;
        int *found = scratch + 4 * kDealWarps;  // unit, tile in it, tiles before the run, and with it
        for (int base = 0, before = 0, units_before = 0;
             base < p.units && before + cost * units_before < end; base += kDealThreads) {
            if (p.units > kDealThreads)
                scan(base);
            const int tiles = before + upto - mine;  // before the thread's unit
            const int first = tiles + cost * (units_before + units_upto), last = first + mine;
            if (mine > 0 && first - cost <= begin && begin < last) {
                const int in = begin > first ? begin - first : 0;
                found[0] = base + tid;
                found[1] = in;
                found[2] = tiles + in;
            }
            if (mine > 0 && first - cost < end && end <= last)
                found[3] = tiles + (end > first ? end - first : 0);
            before += all;
            units_before += units_all;
        }
        __syncthreads();
        c.left = found[3] - found[2];
        if (c.left == 0)
            return;
        c.unit = found[0];
        c.enter(p);
        c.tile = c.range.first() + found[1];
    }
};

// Query rows row0.. of a request into the K-major operand of `rows` rows (chunk j:
// dims 64j.., rows * 128 bytes), zeros past the request's last.  `threads` threads.
__device__ __forceinline__ void load_query(const AParams &p, int request, int row0, uint8_t *to,
                                           int rows, int tid, int threads)
{
    const AttentionArgs &a = p.a;
    const int real = p.all_rows - row0;
    const uint16_t *q = a.q + (int64_t(request) * p.all_rows + row0) * DSV4_HEAD_DIM;
    const Span qs{a.q, rows_of(a) * (DSV4_HEAD_DIM * 2u)};
#pragma unroll 8
    for (int i = tid; i < rows * 64; i += threads) {
        const int r = i >> 6, c = i & 63;
        const uint4 v = r < real ? ldg16_in(q + r * DSV4_HEAD_DIM + c * 8, qs, a.b.err)
                                 : make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4 *>(to + (c >> 3) * rows * 128 + swizzled(r, c & 7)) = v;
    }
}

inline AParams tile_params(const AttentionArgs &a, int tile_rows)
{
    AParams p;
    p.a = a;
    p.block_div = fastdiv_magic(uint32_t(a.b.block_size));
    p.head_div = fastdiv_magic(uint32_t(a.heads));
    p.all_rows = a.q_len * a.heads;
    p.tile_rows = tile_rows;
    p.row_tiles = (p.all_rows + tile_rows - 1) / tile_rows;
    p.tile_div = fastdiv_magic(uint32_t(p.row_tiles));
    p.units = p.row_tiles * a.b.batch;
    return p;
}

}  // namespace
}  // namespace dsv4
