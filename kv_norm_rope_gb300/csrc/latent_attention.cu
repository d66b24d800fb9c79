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
//  * Warps 8..23 load: a warp has 4 keys of each tile, one row a load instruction, in
//    registers while the tile before is computed; a row becomes bf16 on its way to shared memory.
//    One tile of bytes is in flight a SM.
//  * Warps 0..7 do the softmax: a warp has 16 rows and half of the keys; what a row needs
//    (its reference, sum, range, tree bits) is in the registers of 8 threads.
//  * The softmax needs no maximum per tile.  Each row has a reference m, the largest score of
//    the first tile it saw; p = 2^(x - m) is taken against that, and only when some x exceeds m
//    by more than kSlack is m moved and everything rescaled (fp32 and bf16 have the same
//    range, so a p of 2^kSlack loses nothing).  Sums stay per thread, in fp32, until the segment ends.
//  * Warp 24 issues the products, warp 25 notes what the run leaves for the join (run_join.cuh).
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

// A tile lies in groups of 8 keys, a group in 8 chunks of 64 dims, each an atom of the swizzle
// (tcgen05.cuh): a copy can bring whole groups, and both products read them as they are.
constexpr int kChunks = 8;
constexpr uint32_t kGroupBytes = kChunks * 1024;
constexpr uint32_t kTileBytes = kTileKeys / 8 * kGroupBytes;
constexpr uint32_t kQueryBytes = kChunks * kRows * 128;
constexpr uint32_t kProbBytes = kRows * 128;  // 64 rows of 64 keys
constexpr int kSoftmaxWarps = 8, kRowWarp = kSoftmaxWarps;  // warps from kRowWarp on see to the rows
constexpr float kSlack = 16.0f;
static_assert(kRows == 64 && kTileKeys == 64, "the lanes are dealt for these");

// What differs with the store.
template <bool kFp8>
struct Kind;
template <>
struct Kind<true> {
    static constexpr int row_warps = 16;
    static constexpr int prob_slots = 1;  // the second one's place is the ring's
    static constexpr uint32_t ring_bytes = row_warps * 1536;
    // registers a thread: 72 at launch (896 * 72 = 64512), then
    static constexpr int softmax_regs = 88, row_regs = 72, other_regs = 40;
};
template <>
struct Kind<false> {
    static constexpr int row_warps = 8;
    static constexpr int prob_slots = 2;
    static constexpr uint32_t ring_bytes = 0;
};
constexpr int kCopyWarps = 4;  // bf16
template <bool kFp8>
constexpr int kMultiplyWarp = kRowWarp + Kind<kFp8>::row_warps;  // then the run's ends, the queries, none
template <bool kFp8>
constexpr int kThreads = (kMultiplyWarp<kFp8> + 4 + (kFp8 ? 0 : kCopyWarps)) * 32;
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
    uint64_t landed[2];                              // bf16: of the copies of the two tiles in flight
    uint64_t full[2], free[2], scores[2], probs[2];  // of the two tiles
    uint64_t query, query_free, output;
    uint32_t tmem;
    int scratch[kDealWords];
    float m[kRows];
    alignas(16) float factor[kRows];
    float half_rows[2][kRows];  // maxima or sums over the keys of either half
    alignas(4) uint8_t state[2][kTileKeys];
    alignas(16) uint32_t dirty[2][kCopyWarps];  // bf16: the tile has to be looked through before the products
    Cursor place[kSoftmaxWarps];
};
template <bool kFp8>
constexpr size_t kSmemBytes = kShared<kFp8> + sizeof(Shared);
enum : uint8_t { kMissing = 0, kTaken = 1, kNotFinite = 2 };  // of a key
static_assert(kSmemBytes<true> <= 227 * 1024 && kSmemBytes<false> <= 227 * 1024, "too much shared memory");

struct LParams {
    WParams w;
    CUtensorMap q;     // boxes of 64 rows
    CUtensorMap rows;  // bf16: the cache, in boxes of `box` rows, or by single rows
    int box;           // 64, 32, 16, 8, or 1: single rows, gathered by fours
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
    return (key >> 3) * kGroupBytes + chunk * 1024 + swizzled(key & 7, piece);
}

// a wait by the whole warp
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity)
{
    return __all_sync(kFull, mbar_wait(bar, parity));
}

// ---- Queries, by the copying warp

// (Copies are issued by one elected lane of code that the whole warp runs with the same values:
// from lanes of their own each took about 80 cycles.)
__device__ __forceinline__ void copy_query(const LParams &l, Shared &s, uint32_t smem, int request, int row0,
                                           uint32_t elected)
{
    if (elected != 0u)
        mbar_arrive_expect_tx(&s.query, kQueryBytes);
    __syncwarp();
    // rows past the unit's last are another request's, or zeros past the batch's: their scores
    // go nowhere
    copy_rows3(smem + kQuery, &l.q, request * l.w.p.all_rows + row0, &s.query, elected);
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

// ---- FP8 rows into operands: warps 8..23, a warp 4 keys of each tile
//
// Of a row lanes 0..27 have 16 codes and lanes 28..31 eight rope dims; the other 32 rope dims of
// the four rows are with lanes 0..15.  The first three rows come through the warp's part of a ring in
// shared memory (asynchronous copies into each lane's own bytes), the fourth, the rest of the
// rope dims and the exponents in registers: what is on its way to registers takes lines of the
// L1 that shared memory leaves, about 28 KB, and a load that finds none waits.

constexpr int kWarpKeys = 4, kRingRows = 3;

__device__ __forceinline__ Span fp8_span(const PagedBatch &b)
{
    return Span{b.cache, uint64_t(b.num_blocks) * uint32_t(b.block_size) * DSV4_FP8_SLOT_BYTES};
}

// Where a key is: its block (on its way when this returns) and the offset in it, UINT32_MAX
// for a key outside [lo, hi).
struct KeyPlace {
    uint32_t block, off;
};

__device__ __forceinline__ KeyPlace key_place(const AParams &p, const Cursor &c, int key, int lo, int hi)
{
    KeyPlace k{0u, UINT32_MAX};
    const int i = c.tile * kTileKeys + key;
    if (c.left > 0 && i >= lo && i < hi) {
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

// The place as addresses, found once by the lanes that have the key: null for none.  A row's
// exponents stand `scale` bytes after its data.
struct Fp8Row {
    const uint8_t *data;
    uint32_t scale;
};

__device__ __forceinline__ Fp8Row fp8_row(const AParams &p, const KeyPlace &k)
{
    if (k.off == UINT32_MAX)
        return Fp8Row{nullptr, 0u};
    const uint32_t bs = uint32_t(p.a.b.block_size);
    return Fp8Row{p.a.b.cache + uint64_t(k.block) * bs * DSV4_FP8_SLOT_BYTES + uint64_t(k.off) * DSV4_FP8_DATA_BYTES,
                  (bs - k.off) * DSV4_FP8_DATA_BYTES + k.off * DSV4_FP8_SCALE_BYTES};
}

__device__ __forceinline__ Fp8Row row_of_lane(const Fp8Row &mine, int lane)
{
    const uint64_t at = reinterpret_cast<uint64_t>(mine.data);
    const uint32_t low = __shfl_sync(kFull, uint32_t(at), lane), high = __shfl_sync(kFull, uint32_t(at >> 32), lane);
    return Fp8Row{reinterpret_cast<const uint8_t *>(uint64_t(high) << 32 | low), __shfl_sync(kFull, mine.scale, lane)};
}

// Rows are 16-byte aligned in caches with an even block size (wide), else 8-byte.
__device__ __forceinline__ uint4 load_fp8_16(const AParams &p, const uint8_t *at, bool wide)
{
    const Span cs = fp8_span(p.a.b);
    if (wide)
        return ldg16_now_in(at, cs, p.a.b.err);
    const uint2 lo = ldg8_now_in(at, cs, p.a.b.err), hi = ldg8_now_in(at + 8, cs, p.a.b.err);
    return make_uint4(lo.x, lo.y, hi.x, hi.y);
}

// 16 bytes to shared memory, zeros for none
__device__ __forceinline__ void copy_fp8_16(const AParams &p, uint32_t to, const uint8_t *from, bool ok, bool wide)
{
    ok = ok && in_span(from, 16, fp8_span(p.a.b), p.a.b.err);
    const uint8_t *at = ok ? from : p.a.b.cache;
    if (wide) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(at), "r"(ok ? 16 : 0) : "memory");
    } else {
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(to), "l"(at), "r"(ok ? 8 : 0) : "memory");
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(to + 8), "l"(at + 8), "r"(ok ? 8 : 0)
                     : "memory");
    }
}

// what a lane holds of its warp's keys of a tile, beside the ring
struct Raw {
    uint4 last, tail;
    uint32_t e[kWarpKeys];
};

// the warp's rows on their way (zeros for keys that are not there); ring: the lane's first bytes
__device__ __forceinline__ void load_rows(const AParams &p, const Fp8Row &mine, uint32_t ring, bool wide, Raw &raw)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < kWarpKeys; ++i) {
        const Fp8Row row = row_of_lane(mine, i);
        const bool ok = row.data != nullptr;
        if (i < kRingRows)
            copy_fp8_16(p, ring + 512 * i, row.data + 16 * lane, ok, wide);
        else
            raw.last = ok ? load_fp8_16(p, row.data + 16 * lane, wide) : make_uint4(0u, 0u, 0u, 0u);
        raw.e[i] = ok && lane < 28
                       ? ldg_byte_now_in(row.data + row.scale + (lane >> 2), fp8_span(p.a.b), p.a.b.err)
                       : 0u;
    }
    const Fp8Row row = row_of_lane(mine, (lane >> 2) & 3);
    raw.tail = lane < 16 && row.data != nullptr
                   ? load_fp8_16(p, row.data + DSV4_NOPE_DIM + 64 + 16 * (lane & 3), wide)
                   : make_uint4(0u, 0u, 0u, 0u);
}

// the same on their way to L2: 8 lanes a row, five of them for its data and one for its exponents
__device__ __forceinline__ void prefetch_rows(const AParams &p, const Fp8Row &mine)
{
    const int lane = threadIdx.x & 31, part = lane & 7;
    const Fp8Row row = row_of_lane(mine, lane >> 3);
    const uint8_t *at = row.data + (part < 5 ? 128u * part : row.scale);
    if (row.data != nullptr && part < 6 && in_span(at, 1, fp8_span(p.a.b), p.a.b.err))
        asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
}

// Row i of the warp's four, whose bytes are `bits`, into the operand at `tile` (key: its place there);
// true where it is not finite: it is then zeros.  tail_marks: of the rows' other rope dims, by lane.
__device__ __forceinline__ bool store_row(uint4 bits, uint32_t e, int i, uint32_t tile, int key, uint32_t tail_marks)
{
    const int lane = threadIdx.x & 31, chunk = lane >> 2, quarter = lane & 3;
    uint4 first, second;
    uint32_t bad;
    if (lane < 28) {
        bad = e4m3x16_nan(bits) | (e > kFp8OperandTop ? 1u : 0u);
        const uint32_t scale2 = fp8_operand_scale(e);
        const uint4 lo = e4m3x8_scaled(bits.x, bits.y, scale2);
        const uint4 hi = e4m3x8_scaled(bits.z, bits.w, scale2);
        // odd chunks store their pieces the other way round: no two of 8 lanes meet in a bank
        first = (chunk & 1) ? hi : lo;
        second = (chunk & 1) ? lo : hi;
    } else {
        bad = bf16x8_not_finite(bits);
        first = second = fp8_rope_operand(bits);
    }
    const bool not_finite = __any_sync(kFull, bad != 0u) || ((tail_marks >> (4 * i)) & 15u) != 0u;
    if (not_finite)
        first = second = make_uint4(0u, 0u, 0u, 0u);
    const uint32_t at = tile + piece_of(key, chunk, lane < 28 ? 2 * quarter + (chunk & 1) : quarter);
    store_shared16(at, first);
    if (lane < 28)
        store_shared16(at ^ 16u, second);
    return not_finite;
}

__device__ __forceinline__ void convert_role(const AParams &p, Shared &s, uint32_t smem, Cursor c)
{
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) - kRowWarp;
    const int key0 = warp * kWarpKeys, key = key0 + (lane & (kWarpKeys - 1));
    const bool wide = ((reinterpret_cast<uintptr_t>(p.a.b.cache) | (8u * uint32_t(p.a.b.block_size))) & 15u) == 0u;
    const uint32_t ring = smem + kRing<true> + warp * (kRingRows * 512) + 16 * lane;
    const int count = c.left;
    // A key's block number is loaded three tiles ahead of its conversion, its row put on its way to
    // L2 two and to the SM one tile ahead.
    const auto place_and_advance = [&] {
        const KeyPlace k = key_place(p, c, key, c.range.lo, c.range.hi);
        if (c.left > 0)
            c.advance(p);
        return k;
    };
    const auto row_at = [&](KeyPlace k) {
        check_place(p, k);
        return fp8_row(p, k);
    };
    KeyPlace third = place_and_advance();
    Fp8Row next = row_at(third);
    Raw raw;
    load_rows(p, next, ring, wide, raw);
    bool now = next.data != nullptr;  // the tile's key is there
    third = place_and_advance();
    next = row_at(third);
    prefetch_rows(p, next);
    third = place_and_advance();
    bool alive = true;
    for (int t = 0; t < count; ++t) {
        if (t >= 2 && !warp_wait(&s.free[t & 1], ((t >> 1) - 1) & 1)) {
            alive = false;
            break;
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        const uint32_t tile = smem + kKeys + uint32_t(t & 1) * kTileBytes;
        const uint32_t marks = __ballot_sync(kFull, bf16x8_not_finite(raw.tail) != 0u);
        uint32_t bad = 0u;
#pragma unroll
        for (int i = 0; i < kWarpKeys; ++i) {
            const uint4 bits = i < kRingRows ? load_shared16(ring + 512 * i) : raw.last;
            bad |= store_row(bits, raw.e[i], i, tile, key0 + i, marks) ? 1u << i : 0u;
        }
        if (lane < 16)
            store_shared16(tile + piece_of(key0 + (lane >> 2), 7, 4 + (lane & 3)),
                           ((bad >> (lane >> 2)) & 1u) ? make_uint4(0u, 0u, 0u, 0u) : fp8_rope_operand(raw.tail));
        if (lane < kWarpKeys)
            s.state[t & 1][key] = !now ? kMissing : ((bad >> lane) & 1u) ? kNotFinite : kTaken;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&s.full[t & 1]);
        // Every load stands behind the fence, which waits for those before it (128 heads, 262147
        // bf16 keys, when those rows came this way too: 243 us with the next rows' loads before it, 188 so).
        load_rows(p, next, ring, wide, raw);
        now = next.data != nullptr;
        next = row_at(third);
        prefetch_rows(p, next);
        third = place_and_advance();
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (!alive)
        flag(p.a.b.err, DSV4_DEVERR_TIMEOUT);
}

// ---- bf16 rows: copied as they are, and, where a tile is not seen whole by all rows of the unit
// or lacks keys, looked through by warps 8..15
//
// In a tile that every row sees whole, a row that is not finite makes scores that are not finite
// in every row of S, and the softmax makes NaN of those.

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

// Copy warp j has keys 16j.. of each tile, one a lane of its first half.  In boxes of more keys
// the warp of the first one copies; a box is copied if a row of the unit may see a key of it.
constexpr int kCopyKeys = kTileKeys / kCopyWarps;

__device__ __forceinline__ void copy_role(const LParams &l, Shared &s, uint32_t smem, Cursor c)
{
    const AParams &p = l.w.p;
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) - (kMultiplyWarp<false> + 4);
    const int count = c.left, box = l.box, key0 = kCopyKeys * warp, key = key0 + (lane & (kCopyKeys - 1));
    const uint32_t elected = elect_one();
    // what the warp copies of a tile
    const int boxes = box > kCopyKeys ? (key0 % box == 0 ? 1 : 0) : box >= 8 ? kCopyKeys / box : 0;
    const uint32_t bytes = (box >= 8 ? boxes * box : kCopyKeys) * DSV4_BF16_SLOT_BYTES;
    struct Place {
        KeyPlace k;
        bool seen, dirty;
    };
    const auto place_and_advance = [&] {
        const int lo = c.range.lo & ~(box - 1), hi = (c.range.hi + box - 1) & ~(box - 1), i = c.tile * kTileKeys;
        const Tiles::Range whole = whole_range(p, c);
        Place a;
        a.k = key_place(p, c, key, lo, hi);
        a.seen = i + key >= c.range.lo && i + key < c.range.hi;
        a.dirty = i < whole.lo || i + kTileKeys > whole.hi;
        if (c.left > 0)
            c.advance(p);
        return a;
    };
    // the key's row of the cache; row 0 for none, whose bytes the tile then has instead
    const auto resolve = [&](Place &a) {
        check_place(p, a.k);
        const bool there = a.k.off != UINT32_MAX;
        a.seen = a.seen && there;
        a.dirty = a.dirty || __any_sync(kFull, !a.seen);
        return there ? int(a.k.block * uint32_t(p.a.b.block_size) + a.k.off) : 0;
    };
    Place now = place_and_advance(), next = place_and_advance();
    int row = resolve(now), t = 0;
    for (; t < count; ++t) {
        if (t >= 2 && !warp_wait(&s.free[t & 1], ((t >> 1) - 1) & 1))
            break;
        if (lane < kCopyKeys)
            s.state[t & 1][key] = now.seen ? kTaken : kMissing;
        if (lane == 0)
            s.dirty[t & 1][warp] = now.dirty;
        __syncwarp();
        if (elected != 0u)
            mbar_arrive_expect_tx(&s.landed[t & 1], bytes);
        __syncwarp();
        const uint32_t to = smem + kKeys + uint32_t(t & 1) * kTileBytes + (key0 >> 3) * kGroupBytes;
        if (box >= 8) {
            for (int b = 0; b < boxes; ++b)
                copy_groups(to + b * (box >> 3) * kGroupBytes, &l.rows, __shfl_sync(kFull, row, b * box) >> 3,
                            &s.landed[t & 1], elected);
        } else {
            for (int g = 0; g < kCopyKeys; g += 4) {
                int at[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    at[i] = __shfl_sync(kFull, row, g + i);
#pragma unroll
                for (int i = 0; i < kChunks; ++i)
                    copy_four(to + (g >> 3) * kGroupBytes + i * 1024 + (g & 4) * 128, &l.rows, 64 * i, at,
                              &s.landed[t & 1], elected);
            }
        }
        now = next;
        row = resolve(now);
        if (box >= 8 && t + 1 < count)
            for (int b = 0; b < boxes; ++b)
                prefetch_groups(&l.rows, __shfl_sync(kFull, row, b * box) >> 3, elected);
        next = place_and_advance();
    }
    // nothing of this CTA's is on its way when it ends
    bool alive = t == count;
    for (int u = t >= 2 ? t - 2 : 0; u < t; ++u)
        alive = warp_wait(&s.landed[u & 1], (u >> 1) & 1) && alive;
    if (!alive)
        flag(p.a.b.err, DSV4_DEVERR_TIMEOUT);
}

// whether one of the copy warps found its keys of the tile in need of it
__device__ __forceinline__ bool is_dirty(const Shared &s, int slot)
{
    uint32_t any = 0u;
#pragma unroll
    for (int j = 0; j < kCopyWarps; ++j)
        any |= s.dirty[slot][j];
    return any != 0u;
}

__device__ __forceinline__ void clean_role(const AParams &p, Shared &s, uint32_t smem, int count)
{
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) - kRowWarp;
    for (int t = 0; t < count; ++t) {
        if (!warp_wait(&s.landed[t & 1], (t >> 1) & 1)) {
            flag(p.a.b.err, DSV4_DEVERR_TIMEOUT);
            return;
        }
        if (is_dirty(s, t & 1)) {
            constexpr int kOwn = kTileKeys / Kind<false>::row_warps;
#pragma unroll 2
            for (int i = 0; i < kOwn; ++i) {
                const int key = warp * kOwn + i;
                const uint32_t at = smem + kKeys + uint32_t(t & 1) * kTileBytes + piece_of(key, lane >> 3, lane & 7);
                const uint32_t bad =
                    bf16x8_not_finite(load_shared16(at)) | bf16x8_not_finite(load_shared16(at + 4 * 1024));
                if (!__any_sync(kFull, bad != 0u))
                    continue;
                store_shared16(at, make_uint4(0u, 0u, 0u, 0u));
                store_shared16(at + 4 * 1024, make_uint4(0u, 0u, 0u, 0u));
                if (lane == 0 && s.state[t & 1][key] == kTaken)
                    s.state[t & 1][key] = kNotFinite;
            }
            fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&s.full[t & 1]);
    }
}

// ---- The products, by one warp

// What they take their operands from.  Slots of the two tiles are template arguments, so that
// every descriptor is a constant away from these, in uniform registers.
struct Operands {
    Operand keys, query, values, probs;
    uint32_t tmem, scores_inst, elected;
};

// the first product of the tile in slot kSlot
template <int kSlot>
__device__ __forceinline__ void multiply_scores(const Operands &o)
{
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k)
            mma_bf16(o.tmem + kScoresAt + kSlot * kTileKeys, o.query + (i * kRows * 128 + 32 * k),
                     o.keys + (kSlot * kTileBytes + i * 1024 + 32 * k), o.scores_inst, i > 0 || k > 0,
                     o.elected);
}

// the second
template <int kSlot, int kProbSlot>
__device__ __forceinline__ void multiply_values(const Operands &o, uint32_t inst, bool first)
{
#pragma unroll
    for (int i = 0; i < kChunks / 2; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k)
            mma_bf16(o.tmem + i * kRows, o.values + (kSlot * kTileBytes + 2 * i * 1024 + 2 * kGroupBytes * k),
                     o.probs + (kProbSlot * kProbBytes + 32 * k), inst, !first || k > 0, o.elected);
}

// Tile t's first product may run as soon as its rows are there and the second product of tile t - 2
// has been issued, the second one as soon as its P is there: whichever is ready is issued.  (With
// a fixed order each waited for the other's operands.)
template <bool kFp8>
__device__ void multiply_role(const AParams &p, Shared &s, uint32_t smem, Cursor c)
{
    Operands o;
    o.keys = operand(smem + kKeys, 16, kGroupBytes);
    o.query = operand(smem + kQuery, 16, 1024);
    o.values = operand(smem + kKeys, 1024, kGroupBytes);
    o.probs = operand(smem + kProbs, 16, 1024);
    o.tmem = s.tmem;
    o.scores_inst = instruction_of(kRows, kTileKeys, false, false);
    o.elected = elect_one();
    const int count = c.left;
    int scores = 0, values = 0, segment = 0;  // the next tile of either product, and its segment
    bool first = true;                        // of its segment, the next tile of the first product
    uint32_t inst[2] = {0u, 0u};              // of the second products to come, by slot
    bool begins[2] = {false, false}, ends[2] = {false, false};
    const auto multiply_next_scores = [&](auto slot) {
        constexpr int kSlot = decltype(slot)::value;
        tmem_fence_after();
        multiply_scores<kSlot>(o);
        mma_commit(&s.scores[kSlot], o.elected);
        const bool last = c.ends_segment();
        if (last)
            mma_commit(&s.query_free, o.elected);
        inst[kSlot] = instruction_of(128, uint32_t((c.row1 - c.row0 + 15) & ~15), true, false);
        begins[kSlot] = first;
        ends[kSlot] = last;
        segment += first ? 1 : 0;
        first = last;
        c.advance(p);
        ++scores;
    };
    const auto multiply_next_values = [&](auto slot) {
        constexpr int kSlot = decltype(slot)::value;
        tmem_fence_after();
        multiply_values<kSlot, kFp8 ? 0 : kSlot>(o, inst[kSlot], begins[kSlot]);
        mma_commit(&s.free[kSlot], o.elected);
        if (ends[kSlot])
            mma_commit(&s.output, o.elected);
        ++values;
    };
    const auto ready = [&](uint64_t *bar, uint32_t parity) { return __all_sync(kFull, mbar_test(bar, parity)); };
    const auto rows_ready = [&](int t) {
        const int slot = t & 1;
        const uint32_t parity = (t >> 1) & 1;
        if constexpr (kFp8)
            return ready(&s.full[slot], parity);
        else
            return ready(&s.landed[slot], parity) && (!is_dirty(s, slot) || ready(&s.full[slot], parity));
    };
    long long since = clock64();
    while (values < count) {
        if (scores < count && scores - values < 2 && rows_ready(scores) && (!first || ready(&s.query, segment & 1))) {
            if (scores & 1)
                multiply_next_scores(std::integral_constant<int, 1>());
            else
                multiply_next_scores(std::integral_constant<int, 0>());
            since = clock64();
        }
        if (values < scores && ready(&s.probs[values & 1], (values >> 1) & 1)) {
            if (values & 1)
                multiply_next_values(std::integral_constant<int, 1>());
            else
                multiply_next_values(std::integral_constant<int, 0>());
            since = clock64();
        }
        if (__any_sync(kFull, clock64() - since > kWaitCycles)) {
            flag(p.a.b.err, DSV4_DEVERR_TIMEOUT);
            return;
        }
    }
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
        const auto load_scores = [&](float ref0, float ref1) {
            tmem_load16_rows16(tmem + kScoresAt + (t & 1) * kTileKeys + key0, v);
            tmem_wait_load();
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
                v[j] = __fmaf_rn(v[j], scale, -ref0);
                v[j + 1] = __fmaf_rn(v[j + 1], scale, -ref0);
                v[j + 2] = __fmaf_rn(v[j + 2], scale, -ref1);
                v[j + 3] = __fmaf_rn(v[j + 3], scale, -ref1);
            }
            // an infinite score is one of a row that is not finite, or of a sum outside fp32
            float least = v[0];
#pragma unroll
            for (int j = 1; j < 16; ++j)
                least = fminf(least, v[j]);
            if (least == -INFINITY) {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    v[j] = v[j] == -INFINITY ? __int_as_float(0x7FFFFFFF) : v[j];
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
        load_scores(m0, m1);
        // (rows past the unit's last move nothing)
        float over = -INFINITY;
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (((j & 2) ? valid_hi : valid_lo))
                over = fmaxf(over, v[j]);
        if (named_barrier_any(1, 256, failed || over > kSlack)) {
            if (!first)  // the second product of the tile before is done with O
                failed = !mbar_wait(&s.free[(t - 1) & 1], ((t - 1) >> 1) & 1) || failed;
            if (named_barrier_any(1, 256, failed)) {
                flag(a.b.err, DSV4_DEVERR_TIMEOUT);
                return;
            }
            tmem_fence_after();
            // move the references up to this tile's scores and rescale what was taken before
            load_scores(0.0f, 0.0f);
            float top0 = fmaxf(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[4], v[5])), fmaxf(fmaxf(v[8], v[9]), fmaxf(v[12], v[13])));
            float top1 = fmaxf(fmaxf(fmaxf(v[2], v[3]), fmaxf(v[6], v[7])), fmaxf(fmaxf(v[10], v[11]), fmaxf(v[14], v[15])));
#pragma unroll
            for (int d = 1; d <= 2; d <<= 1) {
                top0 = fmaxf(top0, __shfl_xor_sync(kFull, top0, d));
                top1 = fmaxf(top1, __shfl_xor_sync(kFull, top1, d));
            }
            if ((lane & 3) == 0) {
                s.half_rows[half][r] = top0;
                s.half_rows[half][r + 8] = top1;
            }
            named_barrier(1, 256);
            // (fmaxf takes the number of a NaN and a number)
            const float new0 = fmaxf(m0, fmaxf(s.half_rows[0][r], s.half_rows[1][r]));
            const float new1 = fmaxf(m1, fmaxf(s.half_rows[0][r + 8], s.half_rows[1][r + 8]));
            const float factor0 = exp2_approx(m0 - new0), factor1 = exp2_approx(m1 - new1);
            m0 = new0;
            m1 = new1;
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
            load_scores(m0, m1);
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
        if (Kind<kFp8>::prob_slots == 1 && t > 0 && !mbar_wait(&s.free[(t - 1) & 1], ((t - 1) >> 1) & 1)) {
            // (P of the tile before was not taken; the others of the CTA run out of time as well)
            flag(a.b.err, DSV4_DEVERR_TIMEOUT);
        }
        const uint32_t p_at = probs + (Kind<kFp8>::prob_slots == 1 ? 0u : (t & 1) * kProbBytes);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            store_shared4(p_at + swizzled(r, 4 * half + j), packed[2 * j]);
            store_shared4(p_at + swizzled(r + 8, 4 * half + j), packed[2 * j + 1]);
        }
        fence_proxy_async_smem();
        tmem_fence_before();
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&s.probs[t & 1]);
        if (last) {
            // the segment's result
#pragma unroll
            for (int d = 1; d <= 2; d <<= 1) {
                sum0 += __shfl_xor_sync(kFull, sum0, d);
                sum1 += __shfl_xor_sync(kFull, sum1, d);
            }
            if ((lane & 3) == 0) {
                s.half_rows[half][r] = sum0;
                s.half_rows[half][r + 8] = sum1;
                if (half == 0) {
                    s.m[r] = m0;
                    s.m[r + 8] = m1;
                }
            }
            failed = !mbar_wait(&s.output, segment & 1);
            ++segment;
            if (named_barrier_any(1, 256, failed)) {
                flag(a.b.err, DSV4_DEVERR_TIMEOUT);
                return;
            }
            tmem_fence_after();
            const int row0 = c.row0, rows = c.row1 - c.row0;
            const bool whole_range = from_tile == c.range.first() && c.tile + 1 == c.range.stop();
            const int64_t out_row = int64_t(c.request) * p.all_rows + row0;
            // the run's first segment or its last
            float *part = partial_at(w, blockIdx.x, t + 1 == uint32_t(c.tile + 1 - from_tile) ? 0 : 1);
            const Span ps = partial_span(w);
            if (threadIdx.x < kRows) {
                const int i = threadIdx.x;
                const float total = s.half_rows[0][i] + s.half_rows[1][i];
                if (whole_range) {
                    float lse = 0.0f;
                    if (i < rows)
                        s.factor[i] = finish(s.m[i], total, sink_of(a, row0 + i), w.unit, &lse);
                    if (i < rows && a.lse != nullptr)
                        st_f32_in(a.lse + out_row + i, lse, Span{a.lse, rows_of(a) * 4u}, a.b.err);
                } else {
                    st_f32_in(part + kRows * DSV4_HEAD_DIM + i, s.m[i], ps, a.b.err);
                    st_f32_in(part + kRows * DSV4_HEAD_DIM + kRows + i, total, ps, a.b.err);
                }
            }
            named_barrier(1, 256);
            const Span os{a.out, rows_of(a) * (DSV4_HEAD_DIM * 2u)};
            const int col0 = key0, mine = rows - col0 < 32 ? rows - col0 : 32;
            if (mine > 0) {
#pragma unroll 1
                for (int k = 0; k < 4; ++k) {
                    float o[32];
                    tmem_load16(tmem + k * kRows + col0, o);
                    tmem_load16(tmem + k * kRows + col0 + 16, o + 16);
                    tmem_wait_load();
                    const int dim = k * 128 + warp * 32 + lane;
                    if (whole_range) {
                        // neighbouring lanes swap, so that each stores two dims of one row
                        const int odd = lane & 1;
                        uint16_t *to = a.out + (out_row + col0 + odd) * DSV4_HEAD_DIM + (dim - odd);
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            // (a row without keys has factor 0 and may have anything in O)
                            const float f0 = s.factor[col0 + j], f1 = s.factor[col0 + j + 1];
                            const float o0 = f0 == 0.0f ? 0.0f : o[j] * f0;
                            const float o1 = f1 == 0.0f ? 0.0f : o[j + 1] * f1;
                            const float other = __shfl_xor_sync(kFull, odd ? o0 : o1, 1);
                            if (j + odd < mine)
                                st4_in(to + j * DSV4_HEAD_DIM, odd ? bf16x2_rn(other, o1) : bf16x2_rn(o0, other),
                                       os, a.b.err);
                        }
                    } else {
                        float *to = part + col0 * DSV4_HEAD_DIM + dim;
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (j < mine)
                                st_f32_in(to + j * DSV4_HEAD_DIM, o[j], ps, a.b.err);
                    }
                }
            }
            tmem_fence_before();
            named_barrier(1, 256);  // m, factor and the halves' rows are free for the next segment
        }
        first = last;
        __syncwarp();
        if (lane == 0)
            c.advance(p);
        __syncwarp();
    }
}

template <bool kFp8>
__global__ void __launch_bounds__(kThreads<kFp8>, 1) latent_attention_kernel(const __grid_constant__ LParams l)
{
    extern __shared__ __align__(1024) uint8_t smem_bytes[];
    Shared &s = *reinterpret_cast<Shared *>(smem_bytes + kShared<kFp8>);
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
                mbar_init(&s.landed[i], kCopyWarps);
                mbar_init(&s.full[i], Kind<kFp8>::row_warps);
                mbar_init(&s.free[i], 1);
                mbar_init(&s.scores[i], 1);
                mbar_init(&s.probs[i], kSoftmaxWarps);
            }
            mbar_init(&s.query, 1);
            mbar_init(&s.query_free, 1);
            mbar_init(&s.output, 1);
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
        else if (warp >= kMultiplyWarp<kFp8> + 4)
            copy_role(l, s, smem, c);
    } else if (c.left == 0) {
        // more CTAs than tiles
    } else if (warp < kSoftmaxWarps) {
        if constexpr (kFp8)
            registers_up<Kind<true>::softmax_regs>();
        softmax_role<kFp8>(l.w, s, smem, c);
    } else {
        if constexpr (kFp8)
            convert_role(p, s, smem, c);
        else
            clean_role(p, s, smem, c.left);
    }
    tmem_fence_before();
    __syncthreads();
    if (warp == kMultiplyWarp<kFp8>) {
        tmem_fence_after();
        tmem_free512(s.tmem);
    }
}

template <bool kFp8>
int launch(const AttentionArgs &a, void *workspace, cudaStream_t stream)
{
    static std::atomic<int> sm_count[64];
    int sms = 0;
    if (configure_runs(latent_attention_kernel<kFp8>, kSmemBytes<kFp8>, sm_count, &sms) != DSV4_OK)
        return DSV4_ERR_CUDA;
    LParams l;
    l.w = plan_runs<Tiles>(a, kFp8 ? kFp8OperandUnit : 1.0f, sms, workspace);
    // the largest boxes of rows that never cross a block's end
    l.box = kTileKeys;
    while (a.b.block_size % l.box != 0)
        l.box /= 2;
    if (l.box < 8)
        l.box = 1;
    const uint64_t rows = uint64_t(a.b.num_blocks) * uint32_t(a.b.block_size);
    int st = encode_rows(&l.q, a.q, uint64_t(a.b.batch) * uint32_t(l.w.p.all_rows), kRows);
    if (st == DSV4_OK && !kFp8)
        st = l.box >= 8 ? encode_groups(&l.rows, a.b.cache, rows / 8, uint32_t(l.box / 8))
                        : encode_single_rows(&l.rows, a.b.cache, rows);
    if (st != DSV4_OK)
        return st;
    st = launch_after(latent_attention_kernel<kFp8>, dim3(unsigned(l.w.runs)), dim3(kThreads<kFp8>), stream, l,
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
    return store_mode == DSV4_STORE_FP8 ? launch<true>(a, workspace, stream) : launch<false>(a, workspace, stream);
}

}  // namespace dsv4

DSV4_BOUNDS_FLAG_READER(bounds_flag_latent_attention)
