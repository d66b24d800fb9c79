// What the attention over the 4-bit cache and the attention weights share: which
// keys a tile of query rows sees, how the tiles of keys of all requests are
// dealt out to CTAs, and how a tile of cache rows becomes a bf16 matrix operand.
//
// A tile is 128 keys, aligned in the request.  The tiles that some row of a row
// tile sees, over all requests in order, form one line; each CTA takes a run of it of
// equal cost (start_cost() below).  So a long request is shared by many CTAs and short ones share a
// CTA, whatever the lengths, which only the device knows.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "bounds.cuh"
#include "fp4.cuh"
#include "ops.h"
#include "tcgen05.cuh"

namespace dsv4 {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kTileKeys = 128;
constexpr int kChunks = 8;                    // a row in chunks of 64 dims: 7 of codes, 1 of rope
constexpr uint32_t kChunkBytes = kTileKeys * 128;

struct AParams {
    Fp4AttentionArgs a;
    uint64_t block_div, head_div, tile_div;  // fastdiv_magic of block_size, heads, row_tiles
    int all_rows;        // q_len * heads
    int tile_rows;       // of a row tile
    int row_tiles;       // of a request
    int units;           // row tiles of the batch
};

__device__ __forceinline__ Span cache_span(const Fp4Batch &b)
{
    return Span{b.cache, uint64_t(b.num_blocks) * uint32_t(b.block_size) * kFp4Slot};
}
__device__ __forceinline__ Span table_span(const Fp4Batch &b)
{
    return Span{b.table, (uint64_t(b.batch - 1) * b.table_stride + b.width) * 4u};
}
__device__ __forceinline__ uint64_t rows_of(const Fp4AttentionArgs &a)
{
    return uint64_t(a.b.batch) * uint32_t(a.q_len) * uint32_t(a.heads);
}

__device__ __forceinline__ void flag(int32_t *err, int bit)
{
    if (err != nullptr)
        atomicOr(err, bit);
}

// the keys of request r, as many as its row of the table can name
__device__ __forceinline__ int length_of(const Fp4Batch &b, int r)
{
    const int limit = b.width * b.block_size;
    const int n = int(ldg4_in(b.lens + r, Span{b.lens, uint64_t(b.batch) * 4u}, b.err));
    if (n > limit)
        flag(b.err, DSV4_DEVERR_SLOT_RANGE);
    return n < 0 ? 0 : n > limit ? limit : n;
}

// The keys [lo, hi) that some of the rows [row0, row1) of a request of n keys sees,
// and the tiles they lie in.  Row r is head r % heads of token r / heads.
struct Range {
    int lo, hi;
    __device__ __forceinline__ int first() const { return lo / kTileKeys; }
    __device__ __forceinline__ int stop() const { return (hi + kTileKeys - 1) / kTileKeys; }
    __device__ __forceinline__ int tiles() const { return stop() - first(); }
};

__device__ __forceinline__ Range range_of(const AParams &p, int n, int row0, int row1)
{
    const Fp4AttentionArgs &a = p.a;
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

__device__ __forceinline__ int tiles_of(const AParams &p, int unit)
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
// positions would only make some runs a tile longer.  0, 1, 2, 3, 4, 6 positions:
// attention over 48 requests of 64 to 4096 keys 47.9, 47.3, 41.0, 40.3, 40.1, 43.3 us;
// 24 of 1 to 6000 in windows of 2048 with three tokens 68, 47, 43, 46, 47, 51; 128 of
// 1024 to 8192 258, 252, 240, 245, 246, 248; the weights over the first gain
// nothing (24.2 without and 23.4 with it on one resident input, 24.9 and 25.3 on changing ones).
constexpr int kStartCost = kFp4StartCost;

__device__ __forceinline__ int start_cost(const AParams &p, int total, int X)
{
    return total > X && p.units > X / 8 ? kStartCost : 0;
}

// Places c at the start of CTA x's run.  All threads of the CTA (at least
// kDealThreads) call it.  scratch: kDealWords words of shared memory.
constexpr int kDealThreads = 512;
constexpr int kDealWarps = kDealThreads / 32;
constexpr int kDealWords = 4 * kDealWarps + 4;

__device__ __forceinline__ void deal(const AParams &p, int x, int X, int *scratch, Cursor &c)
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
        all = units_all = 0;
#pragma unroll
        for (int w = 0; w < kDealWarps; ++w) {
            if (w < warp) {
                upto += sums[w];
                units_upto += sums[kDealWarps + w];
            }
            all += sums[w];
            units_all += sums[kDealWarps + w];
        }
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

// ---- Cache rows -> operand
//
// Two teams of 256 threads: team 0 converts the pairs of chunks 0 1 and 4 5, team 1
// those of 2 3 and 6 7.  Thread i of a team owns half (i & 1) of each chunk of key
// i / 2 of the tile, that is one scale group (16 bytes of codes) or 64 bytes of rope.
// Codes come through a slot in shared memory by asynchronous copies into the thread's
// own bytes, issued a pair ahead, half a tile; scales and block numbers are loaded a
// tile ahead, and rope dims, after a prefetch into L2, when the pair before is done.

constexpr int kTeam = 256;
constexpr uint32_t kRingSlot = kTeam * 32;

// where a thread's key of a tile is
struct KeyPlace {
    uint32_t block, off;  // off = UINT32_MAX: not seen by any row
    int unit;             // its complement on the first tile of a unit
};

// the block's number is on its way when this returns
__device__ __forceinline__ KeyPlace key_place(const AParams &p, const Cursor &c, bool new_unit,
                                              int key)
{
    KeyPlace k;
    const int i = c.tile * kTileKeys + key;
    k.unit = new_unit ? ~c.unit : c.unit;
    k.block = 0u;
    k.off = UINT32_MAX;
    if (c.left > 0 && i >= c.range.lo && i < c.range.hi) {
        const uint32_t at = fastdiv(uint32_t(i), p.block_div);
        k.off = uint32_t(i) - at * uint32_t(p.a.b.block_size);
        k.block = ldg4_now_in(p.a.b.table + c.request * p.a.b.table_stride + at, table_span(p.a.b),
                              p.a.b.err);
    }
    return k;
}

// the row of a placed key; data = null for none (not seen, or a bad block, which is flagged)
__device__ __forceinline__ Fp4Row row_at(const AParams &p, const KeyPlace &k)
{
    if (k.off == UINT32_MAX)
        return Fp4Row{nullptr, nullptr};
    if (int64_t(k.block) >= p.a.b.num_blocks) {
        flag(p.a.b.err, DSV4_DEVERR_SLOT_RANGE);
        return Fp4Row{nullptr, nullptr};
    }
    return fp4_row(p.a.b.cache, k.block, k.off, uint32_t(p.a.b.block_size));
}

// 16 bytes to shared memory, zeros for none
__device__ __forceinline__ void copy16(const AParams &p, uint32_t to, const uint8_t *from, bool ok)
{
    ok = ok && in_span(from, 16, cache_span(p.a.b), p.a.b.err);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(ok ? from : p.a.b.cache),
                 "r"(ok ? 16 : 0)
                 : "memory");
}

// the thread's codes of pair i of chunks on their way into its place of a slot
__device__ __forceinline__ void copy_codes(const AParams &p, uint32_t slot, int tid, const Fp4Row &row, int i)
{
    const uint8_t *from = row.data + 64 * i + 16 * (tid & 1);
    copy16(p, slot + tid * 16, from, row.data != nullptr);
    copy16(p, slot + 4096 + tid * 16, from + 32, row.data != nullptr && i < 3);
}

// the thread's copies have landed
__device__ __forceinline__ void copy_wait()
{
    asm volatile("cp.async.wait_all;" ::: "memory");
}

__device__ __forceinline__ uint4 load_raw(const AParams &p, const uint8_t *at, bool ok)
{
    return ok ? ldg16_now_in(at, cache_span(p.a.b), p.a.b.err) : make_uint4(0u, 0u, 0u, 0u);
}

__device__ __forceinline__ void prefetch64(const AParams &p, const uint8_t *at, bool ok)
{
    if (ok && in_span(at, 64, cache_span(p.a.b), p.a.b.err))
        asm volatile("prefetch.global.L2 [%0];\n\tprefetch.global.L2 [%0 + 32];" ::"l"(at));
}

// 32 dims of a key: 16 bytes of codes with their scale.  kMarked: an exponent past
// the operands' range gives zeros, for the caller to mark the row
template <bool kMarked>
__device__ __forceinline__ void convert_group(uint4 codes, uint32_t scale, uint4 *out)
{
    const uint32_t scale2 = fp4_operand_scale(scale & 255u, kMarked ? 0u : 0x7F80u);
    out[0] = mul_bf16x8(fp4x8_small(codes.x), scale2);
    out[1] = mul_bf16x8(fp4x8_small(codes.y), scale2);
    out[2] = mul_bf16x8(fp4x8_small(codes.z), scale2);
    out[3] = mul_bf16x8(fp4x8_small(codes.w), scale2);
}

// keeps values from being computed later than here
__device__ __forceinline__ void computed(uint4 &v)
{
    asm volatile("" : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w));
}

// 16 bytes of shared memory by 32-bit address: the converting warps have no registers
// to spare for generic ones
__device__ __forceinline__ uint4 load_shared16(uint32_t at)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
}

__device__ __forceinline__ void store_shared1(uint32_t at, uint32_t v)
{
    asm volatile("st.shared.u8 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}

__device__ __forceinline__ void store_shared16(uint32_t at, uint4 v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z),
                 "r"(v.w)
                 : "memory");
}

// the thread's half of a chunk's row into the operand at `chunk`; `place` = swizzled(key,
// 4 * half), so that 16-byte chunk k of the half is at place ^ 16k
__device__ __forceinline__ void store_half(uint32_t chunk, uint32_t place, const uint4 *v)
{
#pragma unroll
    for (int k = 0; k < 4; ++k)
        store_shared16(chunk + (place ^ (k << 4)), v[k]);
}

// Query rows row0.. of a request into the K-major operand of `rows` rows (chunk j:
// dims 64j.., rows * 128 bytes), zeros past the request's last.  `threads` threads.
__device__ __forceinline__ void load_query(const AParams &p, int request, int row0, uint8_t *to,
                                           int rows, int tid, int threads)
{
    const Fp4AttentionArgs &a = p.a;
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

inline AParams tile_params(const Fp4AttentionArgs &a, int tile_rows)
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
