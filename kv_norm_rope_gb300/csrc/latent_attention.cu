// Attention over the FP8 and bf16 caches: out = softmax(scale * q k^T [sink]) k, where a
// request's latent rows are keys and values in one, for chains of new tokens and for trees
// of drafted ones.
//
// Per (query row, key) it takes 2 * 512 multiplications for the score and as many for the
// value; a key's 584 or 1024 bytes are read once for all rows of its request.  With one
// token of 64 heads that is 224 or 128 operations a byte where the card has 290, so ordinary
// decoding is bound by memory and several tokens at once by the matrix units.
//
//  * A CTA holds 64 query rows (the heads of one or more tokens of a request) and walks its
//    run of tiles of 64 keys (key_tiles.cuh).  Two tiles fit shared memory beside the
//    queries, so the scores of the next tile are computed while the softmax works on this one.
//  * Scores are S[row, key] = q K^T with M = 64: rows in 16 lanes of each quarter of the
//    tensor memory.  Outputs are computed transposed, O^T[dim, row] = K^T P^T with M = 128, so
//    512 dims take 4 x 64 columns and any number of rows costs in proportion.  By
//    measurement an instruction with 64 x 64 results takes 32 cycles, one with 128 x 64 takes
//    48 (6 KB of operands at 128 bytes a cycle): 1024 and 768 cycles a tile, and 512 more of
//    shared memory's time to write the rows.
//  * Warps 0..7 do the softmax: a warp has 16 rows and half of the keys; what a row needs
//    (its reference, sum, range, tree bits) is in the registers of 8 threads.
//  * The warps from 8 on bring the rows: 16 that convert FP8 rows, 8 that copy bf16 rows.
//  * The last four: one issues the products, one notes what the run leaves for the join
//    (run_join.cuh), one copies queries, one finds where FP8 rows are.
//  * The softmax needs no maximum per tile.  Each row has a reference m, the largest score of
//    the first tile it saw; p = 2^(x - m) is taken against that, and only when some x exceeds m
//    by more than kSlack is m moved and everything rescaled (fp32 and bf16 have the same
//    range, so a p of 2^kSlack loses nothing).  Sums stay per thread, in fp32, until the segment ends.
//
// What it takes (with the results joined), and what bounds it:
//  * 128 requests of 1024 to 8192 FP8 keys, 128 heads: 253 us, 573 TFLOP/s; 32 requests of up to 4096,
//    16 drafted tokens of 64 heads: 291 us.  About 3900 cycles a tile.  Counters give the data pipe of
//    shared memory 91% busy (42% the products' operands, 49% loads and stores) and 60% of all issue
//    slots: each row tile converts its keys for itself.
//  * 6 requests of up to 4096 bf16 keys in a window, 61 drafted tokens of 128 heads: 598 us, 545 TFLOP/s;
//    one of 262147 keys, 128 heads: 107 us.  About 3000 cycles a tile: a tile's copy, product, softmax
//    and product follow one another, with two tiles to fill the gaps.
//  * 48 requests of up to 4096 FP8 keys, 64 heads: 37.9 us in a graph, two requests of 130 keys: 12.3 us.
//    A run's first product comes after 9000 to 14000 cycles (the deal, the lengths, tables, rows and
//    queries, one load behind the other), a whole row tile's results take 7500, a part's 4200.
//
// (Not built: products that two SMs issue together, cta_group::2, with a row tile each.)
//
// Slower, each beside the best of its time (us, the first case unless another is named):
//  * 8 converting warps of 8 keys, all rows in registers: 311 to 252; 16 warps so: 259;
//  * two teams of converting warps, each with every second tile: 308 to 264;
//  * pairs of CTAs that convert half a tile each for both: 386 by remote stores, 296 by bulk copies, to 264;
//  * the FP8 tile in two halves like the bf16 one: 286 to 257;
//  * the next kernel let in from the start: 39.8 to 38.2 for the 48 requests;
//  * three bf16 tiles of 48 keys in flight: 665 to 616 for the trees (what lands waits for the products'
//    operands, and 48 keys a product take 28 cycles to 32 of 64);
//  * half of the queries in tensor memory, so that the first product reads a quarter less of shared memory:
//    269 to 252, and 613 to 614 for the trees;
//  * rows put in L2 by the copy unit; the two products in a fixed order.
// Without the look at the codes for NaN it was 247 to 260, and without any conversion 232.
//
// A key whose row is not finite may be masked for some rows of the tile, and 0 times an
// infinity is NaN in the second product.  So such a row enters the operands as zeros and the key
// is marked: rows that see it get NaN as its score, whose P makes all of their dims NaN, and
// the others are left alone.
//
// P is rounded to bf16 as an operand (half a step, at most 2^-8 of the value, to either side);
// the sum that divides it is of the unrounded p.

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "bounds.cuh"
#include "convert.cuh"
#include "fp8_rows.cuh"
#include "key_tiles.cuh"
#include "launch_status.h"
#include "ops.h"
#include "run_join.cuh"
#include "tcgen05.cuh"
#include "tensor_copy.cuh"

namespace dsv4 {
namespace {

constexpr int kTileKeys = kLatentTileKeys;
using Tiles = KeyTiles<kTileKeys, kLatentStartCost, true>;
using Cursor = Tiles::Cursor;

constexpr int kChunks = 8;  // a row in chunks of 64 dims: a tile is 8 chunks of 64 keys
constexpr uint32_t kChunkBytes = kTileKeys * 128;
constexpr uint32_t kTileBytes = kChunks * kChunkBytes;
constexpr uint32_t kQueryBytes = kChunks * kRows * 128;
constexpr uint32_t kProbBytes = kRows * 128;  // 64 rows of 64 keys
constexpr int kSoftmaxWarps = 8, kRowWarp = kSoftmaxWarps;  // warps from kRowWarp on see to the rows
constexpr float kSlack = 16.0f;
constexpr float kLargeScore = 16777216.0f;  // half a step there is 1
static_assert(kRows == 64 && kTileKeys == 64, "the lanes are dealt for these");

// What differs with the store.
template <bool kFp8>
struct Kind;
template <>
struct Kind<true> {
    static constexpr int row_warps = 16;
    static constexpr int prob_slots = 1;  // the second one's place is the ring's
    static constexpr int parts = 1;       // of the dims, that a tile is filled and freed in
    static constexpr uint32_t ring_bytes = row_warps * 3 * DSV4_NOPE_DIM;  // three rows of codes a warp
    // registers a thread: 72 at launch (896 * 72 = 64512), then
    static constexpr int softmax_regs = 88, row_regs = 72, other_regs = 40;
};
template <>
struct Kind<false> {
    static constexpr int row_warps = 8;
    static constexpr int prob_slots = 2;
    static constexpr int parts = 2;
    static constexpr uint32_t ring_bytes = 0;
};
constexpr int kPlaceSlots = 3;  // FP8
template <bool kFp8>
constexpr int kMultiplyWarp = kRowWarp + Kind<kFp8>::row_warps;  // then the run's ends, the queries, FP8: places
template <bool kFp8>
constexpr int kThreads = (kMultiplyWarp<kFp8> + 4) * 32;
static_assert(128 * (2 * Kind<true>::softmax_regs + 4 * Kind<true>::row_regs + Kind<true>::other_regs) <=
                  kThreads<true> * 72,
              "the shares exceed what the CTA was launched with");

// Shared memory (from a 1024-byte boundary).
constexpr uint32_t kKeys = 0;                        // two tiles
constexpr uint32_t kQuery = kKeys + 2 * kTileBytes;  // 8 chunks of 64 rows
constexpr uint32_t kProbs = kQuery + kQueryBytes;    // P
template <bool kFp8>
constexpr uint32_t kRing = kProbs + Kind<kFp8>::prob_slots * kProbBytes;
template <bool kFp8>
constexpr uint32_t kShared = kRing<kFp8> + Kind<kFp8>::ring_bytes;

// Tensor memory: O^T in 4 blocks of 128 dims by 64 rows, then two S of 64 keys.
constexpr uint32_t kScoresAt = 4 * kRows;

struct Shared {
    uint64_t full[2][2], free[2][2];  // of the two tiles, and their parts
    uint64_t scores[2], probs[2];     // of the two tiles
    uint64_t query, query_free, output;
    uint32_t tmem;
    int scratch[kDealWords];
    float m[kRows];
    alignas(16) float factor[kRows];
    // maxima and sums over the keys of either half: apart, for in a segment of one tile no barrier
    // stands between the last look at the maxima and the sums
    float half_max[2][kRows], half_sum[2][kRows];
    alignas(4) uint8_t state[2][kTileKeys];
    Cursor place[kSoftmaxWarps];
};
template <bool kFp8>
struct KindShared;
template <>
struct KindShared<true> {
    // where a tile's keys are (null: not there), and their exponents
    uint64_t placed[kPlaceSlots], taken[kPlaceSlots];
    const uint8_t *row[kPlaceSlots][kTileKeys];
    uint2 exponents[kPlaceSlots][kTileKeys];
};
template <>
struct KindShared<false> {};
template <bool kFp8>
constexpr uint32_t kKindShared = kShared<kFp8> + (sizeof(Shared) + 15) / 16 * 16;
template <bool kFp8>
constexpr size_t kSmemBytes = kKindShared<kFp8> + sizeof(KindShared<kFp8>);
enum : uint8_t { kMissing = 0, kTaken = 1, kNotFinite = 2 };  // of a key
static_assert(kSmemBytes<true> <= 227 * 1024 && kSmemBytes<false> <= 227 * 1024, "too much shared memory");

struct LParams {
    WParams w;
    CUtensorMap q;  // boxes of 64 rows
};

__device__ __forceinline__ void store_shared16(uint32_t at, uint4 v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z),
                 "r"(v.w)
                 : "memory");
}

__device__ __forceinline__ void store_shared4(uint32_t at, uint32_t v)
{
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}

__device__ __forceinline__ uint4 load_shared16(uint32_t at)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
}

// where 16 bytes of a key are in a tile: piece 0..7 of a chunk
__device__ __forceinline__ uint32_t piece_of(int key, int chunk, int piece)
{
    return chunk * kChunkBytes + swizzled(key, piece);
}

// a wait by the whole warp
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity)
{
    return __all_sync(kFull, mbar_wait(bar, parity));
}

// ---- Queries, by the copying warp

__device__ __forceinline__ void copy_query(const LParams &l, Shared &s, uint32_t smem, int request, int row0,
                                           uint32_t elected)
{
    if (elected != 0u)
        mbar_arrive_expect_tx(&s.query, kQueryBytes);
    __syncwarp();
    // rows past the unit's last are another request's, or zeros past the batch's: their scores
    // go nowhere
    copy_rows(smem + kQuery, &l.q, request * l.w.p.all_rows + row0, &s.query, elected);
}

__device__ __forceinline__ void query_role(const LParams &l, Shared &s, uint32_t smem, Cursor c)
{
    const uint32_t elected = elect_one();
    int segment = 0;
    bool alive = c.left > 0;
    while (alive && c.left > 0) {
        alive = segment == 0 || warp_wait(&s.query_free, (segment - 1) & 1);
        if (!alive)
            break;
        copy_query(l, s, smem, c.request, c.row0, elected);
        ++segment;
        // to the next unit
        const int rest = c.range.stop() - c.tile;
        if (c.left <= rest)
            break;
        c.left -= rest - 1;
        c.tile = c.range.stop() - 1;
        c.advance(l.w.p);
    }
    // nothing of this CTA's is on its way when it ends
    if (segment > 0 && !warp_wait(&s.query, (segment - 1) & 1))
        alive = false;
    if (!alive && segment > 0)
        flag(l.w.p.a.b.err, DSV4_DEVERR_TIMEOUT);
}

// keeps values from being computed later than here
__device__ __forceinline__ void computed(uint4 &v)
{
    asm volatile("" : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w));
}

// ---- FP8 rows into operands: warps 8..23, a warp 4 keys of each tile
//
// Of a row lanes 0..27 have 16 codes; of the rope dims of all four rows each lane has 8.  The codes of
// the first three rows come through the warp's part of a ring in shared memory (asynchronous copies
// into each lane's own bytes), those of the fourth and the rope dims in registers: what is on its way
// to registers takes lines of the L1 that shared memory leaves, about 28 KB, and a load that
// finds none waits.  Where the rows are, one warp finds for all, and puts them on their way to L2.
// Rows on 16-byte boundaries have a kernel of their own: chosen at each load it took 264 us, not 256.

constexpr int kWarpKeys = 4, kRingRows = 3;

__device__ __forceinline__ Span fp8_span(const PagedBatch &b)
{
    return Span{b.cache, uint64_t(b.num_blocks) * uint32_t(b.block_size) * DSV4_FP8_SLOT_BYTES};
}

// Where a key of a tile is: its block (on its way when this returns) and the offset in it,
// UINT32_MAX for a key that no row of the unit may see.
struct KeyPlace {
    uint32_t block, off;
};

__device__ __forceinline__ KeyPlace key_place(const AParams &p, const Cursor &c, int key)
{
    KeyPlace k{0u, UINT32_MAX};
    const int i = c.tile * kTileKeys + key;
    if (c.left > 0 && i >= c.range.lo && i < c.range.hi) {
        const uint32_t at = fastdiv(uint32_t(i), p.block_div);
        k.off = uint32_t(i) - at * uint32_t(p.a.b.block_size);
        k.block = ldg4_now_in(p.a.b.table + c.request * p.a.b.table_stride + at, table_span(p.a.b),
                              p.a.b.err);
    }
    return k;
}

// a bad block is flagged and counts as no key
__device__ __forceinline__ void check_place(const AParams &p, KeyPlace &k)
{
    if (k.off != UINT32_MAX && int64_t(k.block) >= p.a.b.num_blocks) {
        flag(p.a.b.err, DSV4_DEVERR_SLOT_RANGE);
        k.off = UINT32_MAX;
    }
}

// Rows are 16-byte aligned in aligned caches with an even block size (kWide), else 8-byte.
template <bool kWide>
__device__ __forceinline__ uint4 load_fp8_16(const AParams &p, const uint8_t *at)
{
    const Span cs = fp8_span(p.a.b);
    if constexpr (kWide)
        return ldg16_now_in(at, cs, p.a.b.err);
    const uint2 lo = ldg8_now_in(at, cs, p.a.b.err), hi = ldg8_now_in(at + 8, cs, p.a.b.err);
    return make_uint4(lo.x, lo.y, hi.x, hi.y);
}

// 16 bytes to shared memory, zeros for none
template <bool kWide>
__device__ __forceinline__ void copy_fp8_16(const AParams &p, uint32_t to, const uint8_t *from, bool ok)
{
    ok = ok && in_span(from, 16, fp8_span(p.a.b), p.a.b.err);
    const uint8_t *at = ok ? from : p.a.b.cache;
    if constexpr (kWide) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(at), "r"(ok ? 16 : 0) : "memory");
    } else {
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(to), "l"(at), "r"(ok ? 8 : 0) : "memory");
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(to + 8), "l"(at + 8), "r"(ok ? 8 : 0)
                     : "memory");
    }
}

// A lane has keys `lane` and `lane + 32` of a tile: their addresses and exponents, kPlaceSlots tiles
// ahead of the converting warps at most, found two tiles and loaded one tile ahead of that.
__device__ __forceinline__ void place_role(const AParams &p, KindShared<true> &ks, Cursor c)
{
    const int lane = threadIdx.x & 31, count = c.left;
    struct Two {
        KeyPlace k[2];
    };
    struct Rows {
        const uint8_t *data[2];
        uint2 exponents[2];
    };
    const auto place_and_advance = [&] {
        Two a;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            a.k[h] = key_place(p, c, lane + 32 * h);
        if (c.left > 0)
            c.advance(p);
        return a;
    };
    const auto load = [&](Two a) {
        const Span cs = fp8_span(p.a.b);
        const uint32_t bs = uint32_t(p.a.b.block_size);
        Rows r;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            check_place(p, a.k[h]);
            r.data[h] = nullptr;
            r.exponents[h] = make_uint2(0u, 0u);
            if (a.k[h].off == UINT32_MAX)
                continue;
            const uint8_t *page = p.a.b.cache + uint64_t(a.k[h].block) * bs * DSV4_FP8_SLOT_BYTES;
            r.data[h] = page + uint64_t(a.k[h].off) * DSV4_FP8_DATA_BYTES;
            r.exponents[h] = ldg8_now_in(page + uint64_t(bs) * DSV4_FP8_DATA_BYTES +
                                             uint64_t(a.k[h].off) * DSV4_FP8_SCALE_BYTES, cs, p.a.b.err);
            if (in_span(r.data[h], DSV4_FP8_DATA_BYTES, cs, p.a.b.err))
#pragma unroll
                for (int i = 0; i < DSV4_FP8_DATA_BYTES; i += 128)
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(r.data[h] + i));
        }
        return r;
    };
    Rows now = load(place_and_advance());
    Two next = place_and_advance();
    for (int t = 0, slot = 0, round = 0; t < count; ++t) {
        if (round > 0 && !warp_wait(&ks.taken[slot], (round - 1) & 1)) {
            flag(p.a.b.err, DSV4_DEVERR_TIMEOUT);
            return;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            ks.row[slot][lane + 32 * h] = now.data[h];
            ks.exponents[slot][lane + 32 * h] = now.exponents[h];
        }
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&ks.placed[slot]);
        now = load(next);
        next = place_and_advance();
        if (++slot == kPlaceSlots) {
            slot = 0;
            ++round;
        }
    }
}

// what a lane holds of its warp's keys of a tile, beside the ring
struct Raw {
    uint4 last, rope;
};

// the warp's rows on their way (zeros for keys that are not there); ring: the lane's first bytes
template <bool kWide>
__device__ __forceinline__ void load_rows(const AParams &p, const uint8_t *const *rows, uint32_t ring, Raw &raw)
{
    const int lane = threadIdx.x & 31;
    const uint8_t *own = rows[lane >> 3];
    raw.rope = own != nullptr ? load_fp8_16<kWide>(p, own + DSV4_NOPE_DIM + 16 * (lane & 7)) : make_uint4(0u, 0u, 0u, 0u);
    raw.last = make_uint4(0u, 0u, 0u, 0u);
    if (lane < 28) {
        const uint8_t *row[kWarpKeys];
#pragma unroll
        for (int i = 0; i < kWarpKeys; ++i)
            row[i] = rows[i];
        if (row[kRingRows] != nullptr)
            raw.last = load_fp8_16<kWide>(p, row[kRingRows] + 16 * lane);
#pragma unroll
        for (int i = 0; i < kRingRows; ++i)
            copy_fp8_16<kWide>(p, ring + DSV4_NOPE_DIM * i, row[i] + 16 * lane, row[i] != nullptr);
    }
}

// 16 codes times their block's scale as two pieces of an operand, the second first where `swap`;
// nonzero if one of them is not finite.
__device__ __forceinline__ uint32_t convert_codes(uint4 c, uint32_t e, bool swap, uint4 &first, uint4 &second)
{
    const uint32_t scale2 = fp8_operand_scale(e);
    first = e4m3x8_scaled(swap ? c.z : c.x, swap ? c.w : c.y, scale2);
    second = e4m3x8_scaled(swap ? c.x : c.z, swap ? c.y : c.w, scale2);
    return e4m3x16_nan(c) | (e > kFp8OperandTop ? 1u : 0u);
}

template <bool kWide>
__device__ __forceinline__ void convert_role(const AParams &p, Shared &s, KindShared<true> &ks, uint32_t smem, int count)
{
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) - kRowWarp, key0 = warp * kWarpKeys;
    const uint32_t ring = smem + kRing<true> + warp * (kRingRows * DSV4_NOPE_DIM) + 16 * lane;
    // lanes 0..27: chunk lane / 4 of a row's codes, a quarter of it.  Odd chunks store their two pieces
    // the other way round: no two of 8 lanes meet in a bank.
    const bool odd = ((lane >> 2) & 1) != 0;
    uint32_t place[kWarpKeys];
#pragma unroll
    for (int i = 0; i < kWarpKeys; ++i)
        place[i] = smem + kKeys + piece_of(key0 + i, lane >> 2, 2 * (lane & 3) + (odd ? 1 : 0));
    const uint32_t rope_place = smem + kKeys + piece_of(key0 + (lane >> 3), kChunks - 1, lane & 7);
    Raw raw;
    bool alive = warp_wait(&ks.placed[0], 0);
    if (alive)
        load_rows<kWide>(p, ks.row[0] + key0, ring, raw);
    int slot = 0, round = 0;  // of the tile's place
    for (int t = 0; alive && t < count; ++t) {
        // Converted before the wait for its place: that way only the stores stand between the product
        // that frees it and the one that reads it.  (Lanes without codes take the last block's exponent:
        // byte 7 of a scale row is padding and may hold anything.)
        uint32_t e[kWarpKeys];
#pragma unroll
        for (int i = 0; i < kWarpKeys; ++i)
            e[i] = reinterpret_cast<const uint8_t *>(&ks.exponents[slot][key0 + i])[lane < 28 ? lane >> 2 : 6];
        const bool there = ks.row[slot][key0 + (lane & (kWarpKeys - 1))] != nullptr;
        copies_wait();
        uint4 first[kWarpKeys], second[kWarpKeys];
#pragma unroll
        for (int i = 0; i < kRingRows; ++i)
            first[i] = lane < 28 ? load_shared16(ring + DSV4_NOPE_DIM * i) : make_uint4(0u, 0u, 0u, 0u);
        first[kRingRows] = raw.last;
        uint32_t bad = bf16x8_not_finite(raw.rope) != 0u ? 1u << (lane >> 3) : 0u;
        uint4 rope = fp8_rope_operand(raw.rope);
#pragma unroll
        for (int i = 0; i < kWarpKeys; ++i)
            bad |= convert_codes(first[i], e[i], odd, first[i], second[i]) != 0u ? 1u << i : 0u;
        bad = __reduce_or_sync(kFull, bad);
        if (bad != 0u) {
            // rows that are not finite enter as zeros
            const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int i = 0; i < kWarpKeys; ++i)
                if (((bad >> i) & 1u) != 0u)
                    first[i] = second[i] = zero;
            if (((bad >> (lane >> 3)) & 1u) != 0u)
                rope = zero;
        }
#pragma unroll
        for (int i = 0; i < kWarpKeys; ++i) {
            computed(first[i]);
            computed(second[i]);
        }
        if (t >= 2 && !warp_wait(&s.free[t & 1][0], ((t >> 1) - 1) & 1)) {
            alive = false;
            break;
        }
        const uint32_t tile = uint32_t(t & 1) * kTileBytes;
        if (lane < 28) {
#pragma unroll
            for (int i = 0; i < kWarpKeys; ++i) {
                store_shared16(place[i] + tile, first[i]);
                store_shared16((place[i] + tile) ^ 16u, second[i]);
            }
        }
        store_shared16(rope_place + tile, rope);
        if (lane < kWarpKeys)
            s.state[t & 1][key0 + lane] = !there ? kMissing : ((bad >> lane) & 1u) ? kNotFinite : kTaken;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(&s.full[t & 1][0]);
            mbar_arrive(&ks.taken[slot]);
        }
        if (++slot == kPlaceSlots) {
            slot = 0;
            ++round;
        }
        // Every load stands behind the fence, which waits for those before it (128 heads, 262147
        // bf16 keys, when those rows came this way too: 243 us with the next rows' loads before it, 188 so).
        if (t + 1 < count) {
            alive = warp_wait(&ks.placed[slot], round & 1);
            if (alive)
                load_rows<kWide>(p, ks.row[slot] + key0, ring, raw);
        }
    }
    copies_wait();
    if (!alive)
        flag(p.a.b.err, DSV4_DEVERR_TIMEOUT);
}

// ---- bf16 rows into operands: warps 8..15, a warp 8 keys of each tile
//
// Copied as they are, asynchronously, half a row an instruction.  The halves of the dims are filled and
// freed apart, so that the first product begins on one while the other is on its way, and the copies
// arrive at the tile's barrier by themselves (together 653 us to 626 for wide trees; in quarters
// it took 735).  By the copy unit, in boxes of up to 64 rows, a tile took no less: its copies wait for the
// products' use of shared memory as these do.  Gathering single rows it took 3400 cycles a tile.
//
// A tile that is not seen whole by all rows of the unit, or lacks keys, is looked through for rows
// that are not finite; in a tile that every row sees whole, such a row makes scores that are not
// finite in every row of S, and the softmax makes NaN of those.

// the keys that all rows of the unit see, but those of tokens that see nothing
__device__ __forceinline__ Tiles::Range whole_range(const AParams &p, const Cursor &c)
{
    const AttentionArgs &a = p.a;
    const int context = c.n - a.q_len;
    if (a.tree != nullptr)
        return Tiles::Range{a.window > 0 ? context + a.q_len - a.window : INT32_MIN, context};
    const int first = int(fastdiv(uint32_t(c.row0), p.head_div)), last = int(fastdiv(uint32_t(c.row1 - 1), p.head_div));
    return Tiles::Range{a.window > 0 ? context + 1 + last - a.window : INT32_MIN, context + 1 + first};
}

// a lane's key of a tile, and whether some row of the unit does not see all of the tile
struct Bf16Place {
    KeyPlace k;
    bool partly;
};

__device__ __forceinline__ Bf16Place bf16_place(const AParams &p, const Cursor &c, int key)
{
    const int i = c.tile * kTileKeys;
    const Tiles::Range whole = whole_range(p, c);
    return Bf16Place{key_place(p, c, key), i < whole.lo || i + kTileKeys > whole.hi};
}

// the key's row of the cache; row 0 for none, whose bytes the tile then has instead
__device__ __forceinline__ uint32_t resolve(const AParams &p, Bf16Place &a)
{
    check_place(p, a.k);
    return a.k.off != UINT32_MAX ? a.k.block * uint32_t(p.a.b.block_size) + a.k.off : 0u;
}

// Zeros for a key of the tile whose row is not finite: `at` is the first of the lane's two pieces, half a
// row apart.  True if it is none.
__device__ __forceinline__ bool clean_key(uint32_t at)
{
    const uint32_t bad = bf16x8_not_finite(load_shared16(at)) | bf16x8_not_finite(load_shared16(at + 4 * kChunkBytes));
    if (!__any_sync(kFull, bad != 0u))
        return true;
    store_shared16(at, make_uint4(0u, 0u, 0u, 0u));
    store_shared16(at + 4 * kChunkBytes, make_uint4(0u, 0u, 0u, 0u));
    return false;
}

constexpr int kCopyKeys = kTileKeys / Kind<false>::row_warps;
static_assert(kCopyKeys == 8, "a key and half a lane for its place");

// 16 bytes to shared memory
__device__ __forceinline__ void copy16(const AParams &p, uint32_t to, const uint8_t *from)
{
    const bool ok = in_span(from, 16, Span{p.a.b.cache, uint64_t(p.a.b.num_blocks) * uint32_t(p.a.b.block_size) *
                                                            DSV4_BF16_SLOT_BYTES}, p.a.b.err);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(ok ? from : p.a.b.cache),
                 "r"(ok ? 16 : 0)
                 : "memory");
}

__device__ __forceinline__ void copy_role(const AParams &p, Shared &s, uint32_t smem, Cursor c)
{
    const int lane = threadIdx.x & 31, key0 = ((threadIdx.x >> 5) - kRowWarp) * kCopyKeys, key = key0 + (lane & 7);
    const int count = c.left;
    const auto place_and_advance = [&] {
        const Bf16Place a = bf16_place(p, c, key);
        if (c.left > 0)
            c.advance(p);
        return a;
    };
    Bf16Place now = place_and_advance(), next = place_and_advance();
    uint32_t row = resolve(p, now);
    for (int t = 0; t < count; ++t) {
        const bool there = now.k.off != UINT32_MAX, look = now.partly || __any_sync(kFull, !there);
        const uint32_t group = smem + kKeys + uint32_t(t & 1) * kTileBytes + piece_of(key0, lane >> 3, 0);
        bool alive = true;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            alive = alive && (t < 2 || warp_wait(&s.free[t & 1][h], ((t >> 1) - 1) & 1));
            if (!alive)
                break;
#pragma unroll
            for (int i = 0; i < kCopyKeys; ++i)
                copy16(p, group + swizzled(i, lane & 7) + h * 4 * kChunkBytes,
                       p.a.b.cache + uint64_t(__shfl_sync(kFull, row, i)) * DSV4_BF16_SLOT_BYTES + 16 * lane + 512 * h);
            if (!look) {
                if (h == 1 && lane < kCopyKeys)
                    s.state[t & 1][key] = kTaken;
                copies_arrive(&s.full[t & 1][h]);
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&s.full[t & 1][h]);
            }
        }
        if (!alive) {
            flag(p.a.b.err, DSV4_DEVERR_TIMEOUT);
            break;
        }
        // the next tile's rows on their way to L2 meanwhile, 8 lanes a row
        now = next;
        row = resolve(p, now);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint8_t *at = p.a.b.cache + 128 * (lane & 7) +
                                uint64_t(__shfl_sync(kFull, row, 4 * i + (lane >> 3))) * DSV4_BF16_SLOT_BYTES;
            asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
        }
        next = place_and_advance();
        if (look) {
            copies_wait();
            __syncwarp();
            uint32_t finite = 0xffu;
#pragma unroll 2
            for (int i = 0; i < kCopyKeys; ++i)
                if (!clean_key(group + swizzled(i, lane & 7)))
                    finite &= ~(1u << i);
            if (lane < kCopyKeys)
                s.state[t & 1][key] = !there ? kMissing : ((finite >> lane) & 1u) ? kTaken : kNotFinite;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                copies_arrive(&s.full[t & 1][h]);
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&s.full[t & 1][h]);
            }
        }
    }
    copies_wait();
}

// ---- The products, by one warp

// What they take their operands from.  Slots of the two tiles are template arguments, so that
// every descriptor is a constant away from these, in uniform registers.
struct Operands {
    Operand keys, query, values, probs;
    uint32_t tmem, scores_inst, elected;
};

// part kPart of kParts of the sum of the first product, of the tile in slot kSlot
template <int kSlot, int kPart, int kParts>
__device__ __forceinline__ void multiply_scores(const Operands &o)
{
#pragma unroll
    for (int i = kPart * kChunks / kParts; i < (kPart + 1) * kChunks / kParts; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k)
            mma_bf16(o.tmem + kScoresAt + kSlot * kTileKeys, o.query + (i * kRows * 128 + 32 * k),
                     o.keys + (kSlot * kTileBytes + i * kChunkBytes + 32 * k), o.scores_inst, i > 0 || k > 0,
                     o.elected);
}

// and of the dims of the second
template <int kSlot, int kProbSlot, int kPart, int kParts>
__device__ __forceinline__ void multiply_values(const Operands &o, uint32_t inst, bool first)
{
    constexpr int kBlocks = kChunks / 2;
#pragma unroll
    for (int i = kPart * kBlocks / kParts; i < (kPart + 1) * kBlocks / kParts; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k)
            mma_bf16(o.tmem + i * kRows, o.values + (kSlot * kTileBytes + 2 * i * kChunkBytes + 2048 * k),
                     o.probs + (kProbSlot * kProbBytes + 32 * k), inst, !first || k > 0, o.elected);
}

// What other threads wrote of P and of bf16 rows is ordered before the products here, by one fence after
// the barrier; a writer's own, before it, waits for the writer's loads as well.
//
// Tile t's first product runs as soon as its rows are there, the second one of tile t - 1 as soon as
// its P is there, whichever is first, and the second if both are.  (In a fixed order each waited for the
// other's operands.)  Each stands in the code once a slot: the warp fetches most of it anew for each tile.
template <bool kFp8>
__device__ void multiply_role(const AParams &p, Shared &s, uint32_t smem, Cursor c)
{
    constexpr int kParts = Kind<kFp8>::parts;
    Operands o;
    o.keys = operand(smem + kKeys, 16, 1024);
    o.query = operand(smem + kQuery, 16, 1024);
    o.values = operand(smem + kKeys, kChunkBytes, 1024);
    o.probs = operand(smem + kProbs, 16, 1024);
    o.tmem = s.tmem;
    o.scores_inst = instruction_of(kRows, kTileKeys, false, false);
    o.elected = elect_one();
    const int count = c.left;
    int t = 0, segment = 0;  // the tile of the first product, and its segment
    bool pending = false;    // the second product of tile t - 1 has not been issued
    bool first = true;       // t begins its segment
    uint32_t inst = 0u;      // of the pending product
    bool begins = false, ends = false;
    const auto ready = [&](uint64_t *bar, uint32_t parity) { return __all_sync(kFull, mbar_test(bar, parity)); };
    const auto multiply_pending = [&](auto slot) {
        constexpr int kSlot = decltype(slot)::value;
        tmem_fence_after();
        fence_proxy_async_smem();
        multiply_values<kSlot, kFp8 ? 0 : kSlot, 0, kParts>(o, inst, begins);
        mma_commit(&s.free[kSlot][0], o.elected);
        if constexpr (kParts == 2) {
            multiply_values<kSlot, kFp8 ? 0 : kSlot, 1, kParts>(o, inst, begins);
            mma_commit(&s.free[kSlot][1], o.elected);
        }
        if (ends)
            mma_commit(&s.output, o.elected);
        pending = false;
    };
    // tile t, in slot kSlot; the pending one is in the other
    const auto step = [&](auto slot) {
        constexpr int kSlot = decltype(slot)::value;
        constexpr std::integral_constant<int, 1 - kSlot> other;
        bool last = false, issued = false;
        long long since = clock64();
        for (;;) {
            if (pending && ready(&s.probs[1 - kSlot], ((t - 1) >> 1) & 1)) {
                multiply_pending(other);
                if (issued)
                    break;
                since = clock64();
            } else if (!issued && ready(&s.full[kSlot][0], (t >> 1) & 1) && (!first || ready(&s.query, segment & 1))) {
                tmem_fence_after();
                if constexpr (!kFp8)
                    fence_proxy_async_smem();
                multiply_scores<kSlot, 0, kParts>(o);
                if constexpr (kParts == 2) {
                    // (the pending product waits as well: with its code here too 613 us to 601 for wide trees)
                    if (!warp_wait(&s.full[kSlot][1], (t >> 1) & 1))
                        return false;
                    tmem_fence_after();
                    fence_proxy_async_smem();
                    multiply_scores<kSlot, 1, kParts>(o);
                }
                mma_commit(&s.scores[kSlot], o.elected);
                last = c.ends_segment();
                if (last)
                    mma_commit(&s.query_free, o.elected);
                if (!pending)
                    break;
                issued = true;
                // asleep until then beside the converting warps (298 us to 290 for drafted trees), polling beside
                // copying ones (107.8 to 106.3 for a long request)
                if (kFp8 && !warp_wait(&s.probs[1 - kSlot], ((t - 1) >> 1) & 1))
                    return false;
                since = clock64();
            } else if (__any_sync(kFull, clock64() - since > kWaitCycles)) {
                return false;
            }
        }
        inst = instruction_of(128, uint32_t((c.row1 - c.row0 + 15) & ~15), true, false);
        begins = first;
        ends = last;
        pending = true;
        segment += first ? 1 : 0;
        first = last;
        c.advance(p);
        ++t;
        return true;
    };
    bool alive = true;
    while (alive && t < count) {
        alive = step(std::integral_constant<int, 0>());
        if (alive && t < count)
            alive = step(std::integral_constant<int, 1>());
    }
    if (alive && pending) {
        const int slot = (t - 1) & 1;
        alive = warp_wait(&s.probs[slot], ((t - 1) >> 1) & 1);
        if (alive && slot == 0)
            multiply_pending(std::integral_constant<int, 0>());
        else if (alive)
            multiply_pending(std::integral_constant<int, 1>());
    }
    if (!alive)
        flag(p.a.b.err, DSV4_DEVERR_TIMEOUT);
}

// ---- Warps 0..7: softmax and results

// What a query row sees: keys [from, to), and those from `to` on that bits name.
struct RowView {
    int to, from;
    uint64_t bits;
    __device__ __forceinline__ bool sees(int i) const
    {
        const uint32_t d = uint32_t(i - to);
        return (i < to && i >= from) || (d < 64u && ((bits >> d) & 1u) != 0u);
    }
};

__device__ __forceinline__ RowView view_of(const AParams &p, const Cursor &c, int r)
{
    const AttentionArgs &a = p.a;
    // the results of a row past the unit's last go nowhere
    RowView v{INT32_MAX, INT32_MIN, 0u};
    if (c.row0 + r >= c.row1)
        return v;
    const int token = int(fastdiv(uint32_t(c.row0 + r), p.head_div));
    if (a.tree == nullptr) {
        v.to = c.n - a.q_len + 1 + token;
        if (a.window > 0)
            v.from = v.to - a.window;
        return v;
    }
    const uint64_t *at = a.tree + int64_t(c.request) * a.q_len + token;
    v.bits = uint64_t(ldg_i64_in(reinterpret_cast<const int64_t *>(at),
                                 Span{a.tree, uint64_t(a.b.batch) * uint32_t(a.q_len) * 8u}, a.b.err));
    if (a.q_len < 64)
        v.bits &= (1ull << a.q_len) - 1u;
    v.to = c.n - a.q_len;
    if (v.bits == 0u)
        v.from = INT32_MAX;
    else if (a.window > 0)
        v.from = v.to + __popcll(v.bits) - a.window;
    return v;
}

// 16 rows of 32 dims of the output from O^T: each lane brings the dim `dim` + lane of the rows, times
// their factors, and stores 8 dims of two rows, after three exchanges with the lanes 1, 2 and 4
// away.  (Stores of two dims took 7400 cycles a row tile, four times as many.)
__device__ __forceinline__ void store_rows16(const float *o, const float *factor, bool some_idle,
                                             const AttentionArgs &a, int64_t row0, int rows, int dim)
{
    const int lane = threadIdx.x & 31;
    uint32_t x[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const float4 f = *reinterpret_cast<const float4 *>(factor + 2 * i);
        float v[4] = {o[2 * i] * f.x, o[2 * i + 1] * f.y, o[2 * i + 2] * f.z, o[2 * i + 3] * f.w};
        if (some_idle) {
            v[0] = f.x == 0.0f ? 0.0f : v[0];
            v[1] = f.y == 0.0f ? 0.0f : v[1];
            v[2] = f.z == 0.0f ? 0.0f : v[2];
            v[3] = f.w == 0.0f ? 0.0f : v[3];
        }
        x[i] = bf16x2_rn(v[0], v[1]);
        x[i + 1] = bf16x2_rn(v[2], v[3]);
    }
    // x[i]: rows 2i, 2i + 1 of one dim -> row 2i + lane % 2 of two dims
    const uint32_t pick = (lane & 1) ? 0x3276u : 0x5410u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t other = __shfl_xor_sync(kFull, x[i], 1);
        x[i] = __byte_perm(x[i], other, pick);
    }
    // -> rows 4q + lane % 4 of four dims
    const bool second = (lane & 2) != 0, third = (lane & 4) != 0;
    uint2 y[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint32_t keep = second ? x[2 * q + 1] : x[2 * q];
        const uint32_t got = __shfl_xor_sync(kFull, second ? x[2 * q] : x[2 * q + 1], 2);
        y[q] = second ? make_uint2(got, keep) : make_uint2(keep, got);
    }
    // -> rows 8u + lane % 8 of eight dims
    const Span os{a.out, rows_of(a) * (DSV4_HEAD_DIM * 2u)};
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const uint2 keep = third ? y[2 * u + 1] : y[2 * u], give = third ? y[2 * u] : y[2 * u + 1];
        const uint2 got = make_uint2(__shfl_xor_sync(kFull, give.x, 4), __shfl_xor_sync(kFull, give.y, 4));
        const int row = 8 * u + (lane & 7);
        if (row < rows)
            st16_in(a.out + (row0 + row) * DSV4_HEAD_DIM + dim + (lane >> 3) * 8,
                    third ? make_uint4(got.x, got.y, keep.x, keep.y) : make_uint4(keep.x, keep.y, got.x, got.y), os,
                    a.b.err);
    }
}

template <bool kFp8>
__device__ void softmax_role(const WParams &w, Shared &s, uint32_t smem, const Cursor &start)
{
    const AParams &p = w.p;
    const AttentionArgs &a = p.a;
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3, half = threadIdx.x >> 7;
    // rows r and r + 8; of each 8 keys of the half, the two from `pair` on
    const int r = 16 * warp + (lane >> 2), pair = 2 * (lane & 3), key0 = 32 * half;
    // the warp's place lives in shared memory: the rest fills the registers
    Cursor &c = s.place[threadIdx.x >> 5];
    if (lane == 0)
        c = start;
    __syncwarp();
    const uint32_t tmem = s.tmem + (uint32_t(warp * 32) << 16);
    const float scale = a.scale * (kLog2e * w.unit);
    const uint32_t probs = smem + kProbs + 2 * pair;
    RowView lo{0, 0, 0u}, hi{0, 0, 0u};
    int whole_to = 0, whole_from = 0;  // keys that all of the warp's rows see
    float m0 = 0.0f, m1 = 0.0f, sum0 = 0.0f, sum1 = 0.0f;
    // A reference is a rounded product.  Its error is a factor that all keys of the row have in common, but
    // one outside any range for scores this large: there the scores are rounded alike.  (Looked up where
    // references move: FP8 as before, wide trees 598.5 to 601 us.  Looked up at each tile 292 to 294 and 604.)
    bool large = false;
    bool first = true, valid_lo = true, valid_hi = true;  // of rows r and r + 8: of the unit
    int segment = 0, from_tile = 0;
    for (uint32_t t = 0; c.left > 0; ++t) {
        if (first) {
            from_tile = c.tile;
            lo = view_of(p, c, r);
            hi = view_of(p, c, r + 8);
            valid_lo = c.row0 + r < c.row1;
            valid_hi = c.row0 + r + 8 < c.row1;
            whole_to = __reduce_min_sync(kFull, min(lo.to, hi.to));
            whole_from = __reduce_max_sync(kFull, max(lo.from, hi.from));
            m0 = m1 = kUnset;
            large = false;
            sum0 = sum1 = 0.0f;
        }
        const bool last = c.ends_segment();
        bool failed = !mbar_wait(&s.scores[t & 1], (t >> 1) & 1);
        tmem_fence_after();
        const int begin = c.tile * kTileKeys + key0;
        const bool whole = begin + 32 <= whole_to && begin >= whole_from;
        const int state = s.state[t & 1][key0 + lane];
        const uint32_t missing = __ballot_sync(kFull, state == kMissing) >> pair;
        const uint32_t marked = __ballot_sync(kFull, state == kNotFinite) >> pair;
        float v[16];
        // v = the scores less a reference, -infinity where unseen
        const auto load_scores = [&](float ref0, float ref1, bool alike) {
            tmem_load16_rows16(tmem + kScoresAt + (t & 1) * kTileKeys + key0, v);
            tmem_wait_load();
            float by = scale;
            if (alike) {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    v[j] *= scale;
                by = 1.0f;
            }
            if constexpr (!kFp8) {
                // an infinite score is one of a row that is not finite, or outside fp32 (looked for here: a
                // score's distance from the reference may be infinite where both are finite)
                float least = v[0];
#pragma unroll
                for (int j = 1; j < 16; ++j)
                    least = fminf(least, v[j]);
                if (least * by == -INFINITY) {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        v[j] = v[j] * by == -INFINITY ? __int_as_float(0x7FFFFFFF) : v[j];
                }
            }
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
                v[j] = __fmaf_rn(v[j], by, -ref0);
                v[j + 1] = __fmaf_rn(v[j + 1], by, -ref0);
                v[j + 2] = __fmaf_rn(v[j + 2], by, -ref1);
                v[j + 3] = __fmaf_rn(v[j + 3], by, -ref1);
            }
            if (__any_sync(kFull, (missing | marked) != 0u) || !whole) {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int at = 8 * (j >> 2) + (j & 1);  // the key, less `pair`
                    const bool seen = ((j & 2) ? hi : lo).sees(begin + pair + at);
                    if (((marked >> at) & 1u) != 0u)
                        v[j] = __int_as_float(0x7FFFFFFF);
                    if (!seen || ((missing >> at) & 1u) != 0u)
                        v[j] = -INFINITY;
                }
            }
        };
        __syncwarp();
        load_scores(m0, m1, large);
        // (rows past the unit's last move nothing)
        float over = -INFINITY;
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (((j & 2) ? valid_hi : valid_lo))
                over = fmaxf(over, v[j]);
        if (named_barrier_any(1, 256, failed || over > kSlack)) {
            if (!first)  // the second product of the tile before is done with O
                failed = !mbar_wait(&s.free[(t - 1) & 1][Kind<kFp8>::parts - 1], ((t - 1) >> 1) & 1) || failed;
            if (named_barrier_any(1, 256, failed)) {
                flag(a.b.err, DSV4_DEVERR_TIMEOUT);
                return;
            }
            tmem_fence_after();
            // move the references up to this tile's scores and rescale what was taken before
            load_scores(0.0f, 0.0f, false);
            float top0 = fmaxf(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[4], v[5])), fmaxf(fmaxf(v[8], v[9]), fmaxf(v[12], v[13])));
            float top1 = fmaxf(fmaxf(fmaxf(v[2], v[3]), fmaxf(v[6], v[7])), fmaxf(fmaxf(v[10], v[11]), fmaxf(v[14], v[15])));
#pragma unroll
            for (int d = 1; d <= 2; d <<= 1) {
                top0 = fmaxf(top0, __shfl_xor_sync(kFull, top0, d));
                top1 = fmaxf(top1, __shfl_xor_sync(kFull, top1, d));
            }
            if ((lane & 3) == 0) {
                s.half_max[half][r] = top0;
                s.half_max[half][r + 8] = top1;
            }
            named_barrier(1, 256);
            // (fmaxf takes the number of a NaN and a number)
            const float new0 = fmaxf(m0, fmaxf(s.half_max[0][r], s.half_max[1][r]));
            const float new1 = fmaxf(m1, fmaxf(s.half_max[0][r + 8], s.half_max[1][r + 8]));
            const float factor0 = exp2_approx(m0 - new0), factor1 = exp2_approx(m1 - new1);
            m0 = new0;
            m1 = new1;
            large = fmaxf(fabsf(m0), fabsf(m1)) > kLargeScore;
            sum0 *= factor0;
            sum1 *= factor1;
            if (!first) {
                if (half == 0 && (lane & 3) == 0) {
                    s.factor[r] = factor0;
                    s.factor[r + 8] = factor1;
                }
                named_barrier(1, 256);
#pragma unroll 1
                for (int i = 0; i < 8; ++i) {
                    const int col = key0 + (i & 1) * 16;  // a row of O, here a column
                    float o[16];
                    tmem_load16(tmem + (i >> 1) * kRows + col, o);
                    tmem_wait_load();
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        o[j] *= s.factor[col + j];
                    tmem_store16(tmem + (i >> 1) * kRows + col, o);
                }
                tmem_wait_store();
            }
            load_scores(m0, m1, large);
        }
        uint32_t packed[8];
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const float a0 = exp2_approx(v[2 * j]), a1 = exp2_approx(v[2 * j + 1]);
            const float b0 = exp2_approx(v[2 * j + 2]), b1 = exp2_approx(v[2 * j + 3]);
            sum0 += a0 + a1;
            sum1 += b0 + b1;
            packed[j] = bf16x2_rn(a0, a1);
            packed[j + 1] = bf16x2_rn(b0, b1);
        }
        if (Kind<kFp8>::prob_slots == 1 && t > 0 && !mbar_wait(&s.free[(t - 1) & 1][Kind<kFp8>::parts - 1], ((t - 1) >> 1) & 1)) {
            // (P of the tile before was not taken; the others of the CTA run out of time as well)
            flag(a.b.err, DSV4_DEVERR_TIMEOUT);
        }
        const uint32_t p_at = probs + (Kind<kFp8>::prob_slots == 1 ? 0u : (t & 1) * kProbBytes);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            store_shared4(p_at + swizzled(r, 4 * half + j), packed[2 * j]);
            store_shared4(p_at + swizzled(r + 8, 4 * half + j), packed[2 * j + 1]);
        }
        tmem_fence_before();
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&s.probs[t & 1]);
        if (last) {
            // the segment's result
            const int row0 = c.row0, rows = c.row1 - c.row0;
#pragma unroll
            for (int d = 1; d <= 2; d <<= 1) {
                sum0 += __shfl_xor_sync(kFull, sum0, d);
                sum1 += __shfl_xor_sync(kFull, sum1, d);
            }
            if ((lane & 3) == 0) {
                s.half_sum[half][r] = sum0;
                s.half_sum[half][r + 8] = sum1;
                if (half == 0) {
                    s.m[r] = m0;
                    s.m[r + 8] = m1;
                }
            }
            const float sink = threadIdx.x < rows ? sink_of(a, c.row0 + threadIdx.x) : 0.0f;
            failed = !mbar_wait(&s.output, segment & 1);
            ++segment;
            if (named_barrier_any(1, 256, failed)) {
                flag(a.b.err, DSV4_DEVERR_TIMEOUT);
                return;
            }
            tmem_fence_after();
            const bool whole_range = from_tile == c.range.first() && c.tile + 1 == c.range.stop();
            const int64_t out_row = int64_t(c.request) * p.all_rows + row0;
            // the run's first segment or its last
            float *part = partial_at(w, blockIdx.x, t + 1 == uint32_t(c.tile + 1 - from_tile) ? 0 : 1);
            const Span ps = partial_span(w);
            if (threadIdx.x < kRows) {
                const int i = threadIdx.x;
                const float total = s.half_sum[0][i] + s.half_sum[1][i];
                if (whole_range) {
                    float lse = 0.0f;
                    s.factor[i] = 1.0f;
                    if (i < rows)
                        s.factor[i] = finish(s.m[i], total, sink, w.unit, &lse);
                    if (i < rows && a.lse != nullptr)
                        st_f32_in(a.lse + out_row + i, lse, Span{a.lse, rows_of(a) * 4u}, a.b.err);
                } else {
                    st_f32_in(part + kRows * DSV4_HEAD_DIM + i, s.m[i], ps, a.b.err);
                    st_f32_in(part + kRows * DSV4_HEAD_DIM + kRows + i, total, ps, a.b.err);
                }
            }
            named_barrier(1, 256);
            const int mine = rows - key0;  // of the half's 32 rows, which are columns here
            if (mine > 0 && whole_range) {
                // (rows without keys have factor 0, and may have anything in O)
                const bool some_idle = __any_sync(kFull, s.factor[key0 + lane] == 0.0f);
#pragma unroll 1
                for (int k = 0; k < 4; ++k) {
                    float o[32];
                    tmem_load16(tmem + k * kRows + key0, o);
                    tmem_load16(tmem + k * kRows + key0 + 16, o + 16);
                    tmem_wait_load();
#pragma unroll
                    for (int i = 0; i < 32; i += 16)
                        store_rows16(o + i, s.factor + key0 + i, some_idle, a, out_row + key0 + i, mine - i,
                                     k * 128 + warp * 32);
                }
            } else if (mine > 0) {
#pragma unroll 1
                for (int k = 0; k < 4; ++k) {
                    float o[32];
                    tmem_load16(tmem + k * kRows + key0, o);
                    tmem_load16(tmem + k * kRows + key0 + 16, o + 16);
                    tmem_wait_load();
                    float *to = part + key0 * DSV4_HEAD_DIM + k * 128 + warp * 32 + lane;
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (j < mine)
                            st_f32_in(to + j * DSV4_HEAD_DIM, o[j], ps, a.b.err);
                }
            }
            tmem_fence_before();
            named_barrier(1, 256);  // m, factor and the halves' sums are free for the next segment
        }
        first = last;
        __syncwarp();
        if (lane == 0)
            c.advance(p);
        __syncwarp();
    }
}

template <bool kFp8, bool kWide>
__global__ void __launch_bounds__(kThreads<kFp8>, 1) latent_attention_kernel(const __grid_constant__ LParams l)
{
    extern __shared__ __align__(1024) uint8_t smem_bytes[];
    Shared &s = *reinterpret_cast<Shared *>(smem_bytes + kShared<kFp8>);
    KindShared<kFp8> &ks = *reinterpret_cast<KindShared<kFp8> *>(smem_bytes + kKindShared<kFp8>);
    const uint32_t smem = smem_addr(smem_bytes);
    const AParams &p = l.w.p;
    const int warp = threadIdx.x >> 5;
    wait_for_kernel_before();
    if ((smem & 1023u) != 0u) {  // never: there is no static shared memory
        flag(p.a.b.err, DSV4_DEVERR_TIMEOUT);
        return;
    }
    if (warp == kMultiplyWarp<kFp8>) {
        tmem_alloc512(&s.tmem);
        if ((threadIdx.x & 31) == 0) {
            for (int i = 0; i < 2; ++i) {
                for (int h = 0; h < Kind<kFp8>::parts; ++h) {
                    mbar_init(&s.free[i][h], 1);
                    // bf16: each thread when its copies have landed, too
                    mbar_init(&s.full[i][h], Kind<kFp8>::row_warps * (kFp8 ? 1 : 33));
                }
                mbar_init(&s.scores[i], 1);
                mbar_init(&s.probs[i], kSoftmaxWarps);
            }
            mbar_init(&s.query, 1);
            mbar_init(&s.query_free, 1);
            mbar_init(&s.output, 1);
            if constexpr (kFp8) {
                for (int i = 0; i < kPlaceSlots; ++i) {
                    mbar_init(&ks.placed[i], 1);
                    mbar_init(&ks.taken[i], Kind<true>::row_warps);
                }
            }
            mbar_init_fence();
        }
        tmem_fence_before();
    }
    Cursor c;
    Tiles::deal(p, blockIdx.x, gridDim.x, s.scratch, c);  // with barriers for the CTA
    tmem_fence_after();
    if (warp >= kMultiplyWarp<kFp8>) {
        if constexpr (kFp8)
            registers_down<Kind<true>::other_regs>();
        if (warp == kMultiplyWarp<kFp8>)
            multiply_role<kFp8>(p, s, smem, c);
        else if (warp == kMultiplyWarp<kFp8> + 1)
            note_ends(l.w, c);
        else if (warp == kMultiplyWarp<kFp8> + 2)
            query_role(l, s, smem, c);
        else if constexpr (kFp8)
            place_role(p, ks, c);
    } else if (c.left == 0) {
        // more CTAs than tiles
    } else if (warp < kSoftmaxWarps) {
        if constexpr (kFp8)
            registers_up<Kind<true>::softmax_regs>();
        softmax_role<kFp8>(l.w, s, smem, c);
    } else {
        if constexpr (kFp8) {
            convert_role<kWide>(p, s, ks, smem, c.left);
        } else {
            copy_role(p, s, smem, c);
        }
    }
    tmem_fence_before();
    __syncthreads();
    if (warp == kMultiplyWarp<kFp8>) {
        tmem_fence_after();
        tmem_free512(s.tmem);
    }
}

template <bool kFp8, bool kWide>
int launch(const AttentionArgs &a, void *workspace, cudaStream_t stream)
{
    static std::atomic<int> sm_count[64];
    int sms = 0;
    if (configure_runs(latent_attention_kernel<kFp8, kWide>, kSmemBytes<kFp8>, sm_count, &sms) != DSV4_OK)
        return DSV4_ERR_CUDA;
    LParams l;
    l.w = plan_runs<Tiles>(a, kFp8 ? kFp8OperandUnit : 1.0f, sms, workspace);
    int st = encode_rows(&l.q, a.q, uint64_t(a.b.batch) * uint32_t(l.w.p.all_rows), kRows);
    if (st != DSV4_OK)
        return st;
    st = launch_after(latent_attention_kernel<kFp8, kWide>, dim3(unsigned(l.w.runs)), dim3(kThreads<kFp8>), stream, l,
                      kSmemBytes<kFp8>);
    return st != DSV4_OK ? st : launch_join<Tiles>(l.w, stream);
}

}  // namespace

size_t latent_attention_workspace()
{
    return run_workspace();
}

int launch_latent_attention(int store_mode, const AttentionArgs &a, void *workspace, cudaStream_t stream)
{
    if (store_mode != DSV4_STORE_FP8)
        return launch<false, true>(a, workspace, stream);
    const bool wide = ((reinterpret_cast<uintptr_t>(a.b.cache) | (8u * uint32_t(a.b.block_size))) & 15u) == 0u;
    return wide ? launch<true, true>(a, workspace, stream) : launch<true, false>(a, workspace, stream);
}

}  // namespace dsv4

DSV4_BOUNDS_FLAG_READER(bounds_flag_latent_attention)
