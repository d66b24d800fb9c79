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

#include "bounds.cuh"
#include "fp8_rows.cuh"
#include "key_tiles.cuh"
#include "launch_status.h"
#include "ops.h"
#include "run_join.cuh"
#include "tcgen05.cuh"

namespace dsv4 {
namespace {

constexpr int kTileKeys = kLatentTileKeys;
using Tiles = KeyTiles<kTileKeys, kLatentStartCost, true>;
using Cursor = Tiles::Cursor;

constexpr int kChunks = 8;  // a row in chunks of 64 dims
constexpr uint32_t kChunkBytes = kTileKeys * 128;
constexpr int kSoftmaxWarps = 8, kLoadWarp = kSoftmaxWarps, kLoadWarps = 16;
constexpr int kMultiplyWarp = kLoadWarp + kLoadWarps;
constexpr int kThreads = (kMultiplyWarp + 4) * 32;  // whole warpgroups: the last two warps idle
constexpr int kWarpKeys = kTileKeys / kLoadWarps;   // 4
// registers a thread: 72 at launch (896 * 72 = 64512), then
constexpr int kSoftmaxRegs = 88, kLoadRegs = 72, kMultiplyRegs = 40;
static_assert(128 * (2 * kSoftmaxRegs + 4 * kLoadRegs + kMultiplyRegs) <= kThreads * 72,
              "the shares exceed what the CTA was launched with");
static_assert(kRows == 64 && kTileKeys == 64 && kWarpKeys == 4, "the lanes are dealt for these");
constexpr float kSlack = 16.0f;

// Shared memory (from a 1024-byte boundary).
constexpr uint32_t kTileBytes = kChunks * kChunkBytes;
constexpr uint32_t kKeys = 0;                              // two tiles
constexpr uint32_t kQuery = kKeys + 2 * kTileBytes;        // 8 chunks of 64 rows
constexpr uint32_t kProbs = kQuery + kChunks * kRows * 128;  // two P: 64 rows of 64 keys
constexpr uint32_t kShared = kProbs + 2 * kRows * 128;

// Tensor memory: O^T in 4 blocks of 128 dims by 64 rows, then two S of 64 keys.
constexpr uint32_t kScoresAt = 4 * kRows;

struct Shared {
    uint64_t full[2], free[2], scores[2], probs[2];  // of the two tiles in flight
    uint64_t query, query_free, output;
    uint32_t tmem;
    int scratch[kDealWords];
    float m[kRows];
    alignas(16) float factor[kRows];
    float half_rows[2][kRows];  // maxima or sums over the keys of either half
    alignas(4) uint8_t state[2][kTileKeys];
};
constexpr size_t kSmemBytes = kShared + sizeof(Shared);
enum : uint8_t { kMissing = 0, kTaken = 1, kNotFinite = 2 };  // of a key
static_assert(kSmemBytes <= 227 * 1024, "too much shared memory");

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

// ---- Warps 8..23: cache rows and queries into operands

template <bool kFp8>
__device__ __forceinline__ Span cache_span(const PagedBatch &b)
{
    return Span{b.cache, uint64_t(b.num_blocks) * uint32_t(b.block_size) *
                             (kFp8 ? DSV4_FP8_SLOT_BYTES : DSV4_BF16_SLOT_BYTES)};
}

// Where key `kWarpKeys * warp + lane % kWarpKeys` of a tile is: its block (on its way when this
// returns) and the offset in it, UINT32_MAX for a key that no row of the unit may see.
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

// What a lane holds of its warp's keys of a tile.
//  FP8: of each row lanes 0..27 have 16 codes (and their block's exponent) and lanes 28..31
//  eight rope dims; the other 32 rope dims of all four rows are with lanes 0..15.
//  bf16: 16 bytes of either half of each row.
template <bool kFp8>
struct Raw;
template <>
struct Raw<true> {
    uint4 a[kWarpKeys], tail;
    uint32_t e[kWarpKeys];
};
template <>
struct Raw<false> {
    uint4 a[kWarpKeys], b[kWarpKeys];
};

// 16 bytes of an FP8 row, which is 16-byte aligned in caches with an even block size (wide)
__device__ __forceinline__ uint4 load_fp8_16(const AParams &p, const uint8_t *at, bool wide)
{
    const Span cs = cache_span<true>(p.a.b);
    if (wide)
        return ldg16_now_in(at, cs, p.a.b.err);
    const uint2 lo = ldg8_now_in(at, cs, p.a.b.err), hi = ldg8_now_in(at + 8, cs, p.a.b.err);
    return make_uint4(lo.x, lo.y, hi.x, hi.y);
}

// the warp's row i on its way (zeros for a key that is not there)
__device__ __forceinline__ void load_row(const AParams &p, const KeyPlace &k, int i, bool wide, Raw<true> &raw)
{
    const int lane = threadIdx.x & 31;
    const uint32_t block = __shfl_sync(kFull, k.block, i), off = __shfl_sync(kFull, k.off, i);
    raw.a[i] = make_uint4(0u, 0u, 0u, 0u);
    raw.e[i] = 0u;
    if (off == UINT32_MAX)
        return;
    const uint32_t bs = uint32_t(p.a.b.block_size);
    const uint8_t *page = p.a.b.cache + uint64_t(block) * bs * DSV4_FP8_SLOT_BYTES;
    raw.a[i] = load_fp8_16(p, page + uint64_t(off) * DSV4_FP8_DATA_BYTES + 16 * lane, wide);
    if (lane < 28)
        raw.e[i] = ldg_byte_now_in(page + uint64_t(bs) * DSV4_FP8_DATA_BYTES + uint64_t(off) * DSV4_FP8_SCALE_BYTES + (lane >> 2),
                                   cache_span<true>(p.a.b), p.a.b.err);
}

__device__ __forceinline__ void load_tail(const AParams &p, const KeyPlace &k, bool wide, Raw<true> &raw)
{
    const int lane = threadIdx.x & 31;
    const uint32_t block = __shfl_sync(kFull, k.block, (lane >> 2) & 3), off = __shfl_sync(kFull, k.off, (lane >> 2) & 3);
    raw.tail = make_uint4(0u, 0u, 0u, 0u);
    if (lane < 16 && off != UINT32_MAX) {
        const uint32_t bs = uint32_t(p.a.b.block_size);
        const uint8_t *page = p.a.b.cache + uint64_t(block) * bs * DSV4_FP8_SLOT_BYTES;
        raw.tail = load_fp8_16(p, page + uint64_t(off) * DSV4_FP8_DATA_BYTES + DSV4_NOPE_DIM + 64 + 16 * (lane & 3), wide);
    }
}

__device__ __forceinline__ void load_row(const AParams &p, const KeyPlace &k, int i, bool, Raw<false> &raw)
{
    const int lane = threadIdx.x & 31;
    const uint32_t block = __shfl_sync(kFull, k.block, i), off = __shfl_sync(kFull, k.off, i);
    raw.a[i] = raw.b[i] = make_uint4(0u, 0u, 0u, 0u);
    if (off == UINT32_MAX)
        return;
    const uint8_t *row = p.a.b.cache + (uint64_t(block) * uint32_t(p.a.b.block_size) + off) * DSV4_BF16_SLOT_BYTES + 16 * lane;
    raw.a[i] = ldg16_now_in(row, cache_span<false>(p.a.b), p.a.b.err);
    raw.b[i] = ldg16_now_in(row + 512, cache_span<false>(p.a.b), p.a.b.err);
}

__device__ __forceinline__ void load_tail(const AParams &, const KeyPlace &, bool, Raw<false> &) {}

// Row i of the warp's four into the operand at `tile` (key: its place there); true where it is not
// finite: it is then zeros.  kTail: the marks of the rows' other rope dims, by lane.
__device__ __forceinline__ bool store_row(const Raw<true> &raw, int i, uint32_t tile, int key, uint32_t tail_marks)
{
    const int lane = threadIdx.x & 31, chunk = lane >> 2, quarter = lane & 3;
    uint4 first, second;
    uint32_t bad;
    if (lane < 28) {
        const uint32_t e = raw.e[i];
        bad = e4m3x16_nan(raw.a[i]) | (e > kFp8OperandTop ? 1u : 0u);
        const uint32_t scale2 = fp8_operand_scale(e);
        const uint4 lo = e4m3x8_scaled(raw.a[i].x, raw.a[i].y, scale2);
        const uint4 hi = e4m3x8_scaled(raw.a[i].z, raw.a[i].w, scale2);
        // odd chunks store their pieces the other way round: no two of 8 lanes meet in a bank
        first = (chunk & 1) ? hi : lo;
        second = (chunk & 1) ? lo : hi;
    } else {
        bad = bf16x8_not_finite(raw.a[i]);
        first = second = fp8_rope_operand(raw.a[i]);
    }
    const bool not_finite = __any_sync(kFull, bad != 0u) || ((tail_marks >> (4 * i)) & 15u) != 0u;
    if (not_finite)
        first = second = make_uint4(0u, 0u, 0u, 0u);
    const uint32_t row = tile + chunk * kChunkBytes;
    const int piece = lane < 28 ? 2 * quarter + (chunk & 1) : quarter;
    store_shared16(row + swizzled(key, piece), first);
    if (lane < 28)
        store_shared16(row + swizzled(key, piece ^ 1), second);
    return not_finite;
}

__device__ __forceinline__ uint32_t tail_marks(const Raw<true> &raw)
{
    return __ballot_sync(kFull, bf16x8_not_finite(raw.tail) != 0u);
}

// the rope dims 32..63 of the warp's rows; `bad`: which of them are zeros instead
__device__ __forceinline__ void store_tail(const Raw<true> &raw, uint32_t tile, int key0, uint32_t bad)
{
    const int lane = threadIdx.x & 31;
    if (lane < 16)
        store_shared16(tile + 7 * kChunkBytes + swizzled(key0 + (lane >> 2), 4 + (lane & 3)),
                       ((bad >> (lane >> 2)) & 1u) ? make_uint4(0u, 0u, 0u, 0u) : fp8_rope_operand(raw.tail));
}

__device__ __forceinline__ bool store_row(const Raw<false> &raw, int i, uint32_t tile, int key, uint32_t)
{
    const int lane = threadIdx.x & 31;
    const bool not_finite =
        __any_sync(kFull, (bf16x8_not_finite(raw.a[i]) | bf16x8_not_finite(raw.b[i])) != 0u);
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    const uint32_t at = tile + (lane >> 3) * kChunkBytes + swizzled(key, lane & 7);
    store_shared16(at, not_finite ? zero : raw.a[i]);
    store_shared16(at + 4 * kChunkBytes, not_finite ? zero : raw.b[i]);
    return not_finite;
}

__device__ __forceinline__ uint32_t tail_marks(const Raw<false> &) { return 0u; }
__device__ __forceinline__ void store_tail(const Raw<false> &, uint32_t, int, uint32_t) {}

template <bool kFp8>
__device__ __forceinline__ void load_role(const AParams &p, Shared &s, uint8_t *smem, Cursor c)
{
    const int lane = threadIdx.x & 31, tid = threadIdx.x - kLoadWarp * 32;
    const int key0 = (tid >> 5) * kWarpKeys, key = key0 + (lane & (kWarpKeys - 1));
    const bool wide = ((reinterpret_cast<uintptr_t>(p.a.b.cache) | (8u * uint32_t(p.a.b.block_size))) & 15u) == 0u;
    const uint32_t base = smem_addr(smem);
    const int count = c.left;
    KeyPlace now = key_place(p, c, key);
    check_place(p, now);
    Raw<kFp8> raw;
#pragma unroll
    for (int i = 0; i < kWarpKeys; ++i)
        load_row(p, now, i, wide, raw);
    load_tail(p, now, wide, raw);
    const auto fill_query = [&](int request, int row0) {
        load_query(p, request, row0, smem + kQuery, kRows, tid, kLoadWarps * 32);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&s.query);
    };
    fill_query(c.request, c.row0);
    // the cursor runs a tile ahead of the rows and two ahead of what is stored
    bool next_begins = c.advance(p);
    int next_request = c.request, next_row0 = c.row0;
    KeyPlace next = key_place(p, c, key);
    bool begins = false;  // this tile begins another unit than the first
    int request = 0, row0 = 0, segment = 1;
    for (int t = 0; t < count; ++t) {
        bool after_begins = false;
        KeyPlace after{0u, UINT32_MAX};
        if (c.left > 0) {
            after_begins = c.advance(p);
            after = key_place(p, c, key);
        }
        bool alive = true;
        if (begins) {
            alive = __all_sync(kFull, mbar_wait(&s.query_free, (segment - 1) & 1));
            ++segment;
            if (alive)
                fill_query(request, row0);
        }
        if (alive && t >= 2)
            alive = __all_sync(kFull, mbar_wait(&s.free[t & 1], ((t >> 1) - 1) & 1));
        if (!alive) {
            flag(p.a.b.err, DSV4_DEVERR_TIMEOUT);
            break;
        }
        const uint32_t tile = base + kKeys + uint32_t(t & 1) * kTileBytes;
        const uint32_t marks = tail_marks(raw);
        const bool mine = now.off != UINT32_MAX;
        check_place(p, next);
        uint32_t bad = 0u;
#pragma unroll
        for (int i = 0; i < kWarpKeys; ++i) {
            bad |= store_row(raw, i, tile, key0 + i, marks) ? 1u << i : 0u;
            load_row(p, next, i, wide, raw);
        }
        store_tail(raw, tile, key0, bad);
        load_tail(p, next, wide, raw);
        if (lane < kWarpKeys)
            s.state[t & 1][key] = !mine ? kMissing : ((bad >> lane) & 1u) ? kNotFinite : kTaken;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&s.full[t & 1]);
        now = next;
        next = after;
        begins = next_begins;
        request = next_request;
        row0 = next_row0;
        next_begins = after_begins;
        next_request = c.request;
        next_row0 = c.row0;
    }
}

// ---- Warp 24: the products

__device__ void multiply_role(const AParams &p, Shared &s, uint32_t smem, Cursor c)
{
    const uint32_t elected = elect_one();
    const Operand keys = operand(smem + kKeys, 16, 1024), query = operand(smem + kQuery, 16, 1024);
    const Operand values = operand(smem + kKeys, kChunkBytes, 1024);
    const Operand probs = operand(smem + kProbs, 16, 1024);
    const uint32_t scores_inst = instruction_of(kRows, kTileKeys, false, false);
    // the second product of tile u
    const auto output = [&](uint32_t u, uint32_t inst, bool first, bool last) {
        if (!__all_sync(kFull, mbar_wait(&s.probs[u & 1], (u >> 1) & 1)))
            return false;
        tmem_fence_after();
        const uint32_t tile = (u & 1) * kTileBytes, p_at = (u & 1) * (kRows * 128);
#pragma unroll
        for (int i = 0; i < kChunks / 2; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                mma_bf16(s.tmem + i * kRows, values + (tile + 2 * i * kChunkBytes + 2048 * k),
                         probs + (p_at + 32 * k), inst, !first || k > 0, elected);
        mma_commit(&s.free[u & 1], elected);
        if (last)
            mma_commit(&s.output, elected);
        return true;
    };
    int segment = 0;
    bool first = true;  // of its segment
    uint32_t t = 0, before_inst = 0;
    bool before_first = false, before_last = false, alive = true;
    for (; c.left > 0; ++t) {
        if (first) {
            alive = __all_sync(kFull, mbar_wait(&s.query, segment & 1));
            ++segment;
        }
        alive = alive && __all_sync(kFull, mbar_wait(&s.full[t & 1], (t >> 1) & 1));
        if (!alive)
            break;
        tmem_fence_after();
        const uint32_t tile = (t & 1) * kTileBytes, d = s.tmem + kScoresAt + (t & 1) * kTileKeys;
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                mma_bf16(d, query + (i * kRows * 128 + 32 * k), keys + (tile + i * kChunkBytes + 32 * k),
                         scores_inst, i > 0 || k > 0, elected);
        const bool last = c.ends_segment();
        mma_commit(&s.scores[t & 1], elected);
        if (last)
            mma_commit(&s.query_free, elected);
        if (t > 0 && !output(t - 1, before_inst, before_first, before_last)) {
            alive = false;
            break;
        }
        before_inst = instruction_of(128, uint32_t((c.row1 - c.row0 + 15) & ~15), true, false);
        before_first = first;
        before_last = last;
        first = last;
        c.advance(p);
    }
    if (alive && t > 0)
        alive = output(t - 1, before_inst, before_first, before_last);
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
    // a row past the unit's last has zeros for a query, and its results go nowhere
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

__device__ void softmax_role(const WParams &w, Shared &s, uint8_t *smem, Cursor c)
{
    const AParams &p = w.p;
    const AttentionArgs &a = p.a;
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3, half = threadIdx.x >> 7;
    // rows r and r + 8; of each 8 keys of the half, the two from `pair` on
    const int r = 16 * warp + (lane >> 2), pair = 2 * (lane & 3), key0 = 32 * half;
    const uint32_t tmem = s.tmem + (uint32_t(warp * 32) << 16);
    const float scale = a.scale * (kLog2e * w.unit);
    const uint32_t probs = smem_addr(smem) + kProbs + 2 * pair;
    RowView lo{0, 0, 0u}, hi{0, 0, 0u};
    int whole_to = 0, whole_from = 0;  // keys that all of the warp's rows see
    float m0 = 0.0f, m1 = 0.0f, sum0 = 0.0f, sum1 = 0.0f;
    bool first = true;
    int segment = 0, from_tile = 0;
    for (uint32_t t = 0; c.left > 0; ++t) {
        if (first) {
            from_tile = c.tile;
            lo = view_of(p, c, r);
            hi = view_of(p, c, r + 8);
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
        float over = v[0];
#pragma unroll
        for (int j = 1; j < 16; ++j)
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
        const uint32_t p_at = probs + (t & 1) * (kRows * 128);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float a0 = exp2_approx(v[4 * j]), a1 = exp2_approx(v[4 * j + 1]);
            const float b0 = exp2_approx(v[4 * j + 2]), b1 = exp2_approx(v[4 * j + 3]);
            sum0 += a0 + a1;
            sum1 += b0 + b1;
            store_shared4(p_at + swizzled(r, 4 * half + j), bf16x2_rn(a0, a1));
            store_shared4(p_at + swizzled(r + 8, 4 * half + j), bf16x2_rn(b0, b1));
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
        c.advance(p);
    }
}

template <bool kFp8>
__global__ void __launch_bounds__(kThreads, 1) latent_attention_kernel(const __grid_constant__ WParams w)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    Shared &s = *reinterpret_cast<Shared *>(smem + kShared);
    const AParams &p = w.p;
    const int warp = threadIdx.x >> 5;
    wait_for_kernel_before();
    if ((smem_addr(smem) & 1023u) != 0u) {  // never: there is no static shared memory
        flag(p.a.b.err, DSV4_DEVERR_TIMEOUT);
        return;
    }
    if (warp == kMultiplyWarp) {
        tmem_alloc512(&s.tmem);
        if ((threadIdx.x & 31) == 0) {
            for (int i = 0; i < 2; ++i) {
                mbar_init(&s.full[i], kLoadWarps);
                mbar_init(&s.free[i], 1);
                mbar_init(&s.scores[i], 1);
                mbar_init(&s.probs[i], kSoftmaxWarps);
            }
            mbar_init(&s.query, kLoadWarps);
            mbar_init(&s.query_free, 1);
            mbar_init(&s.output, 1);
            mbar_init_fence();
        }
        tmem_fence_before();
    }
    Cursor c;
    Tiles::deal(p, blockIdx.x, gridDim.x, s.scratch, c);  // with barriers for the CTA
    tmem_fence_after();
    if (warp >= kMultiplyWarp) {
        registers_down<kMultiplyRegs>();
        if (warp == kMultiplyWarp)
            multiply_role(p, s, smem_addr(smem), c);
        else if (warp == kMultiplyWarp + 1)
            note_ends(w, c);
    } else if (c.left == 0) {
        // more CTAs than tiles
    } else if (warp < kSoftmaxWarps) {
        registers_up<kSoftmaxRegs>();
        softmax_role(w, s, smem, c);
    } else {
        load_role<kFp8>(p, s, smem, c);
    }
    tmem_fence_before();
    __syncthreads();
    if (warp == kMultiplyWarp) {
        tmem_fence_after();
        tmem_free512(s.tmem);
    }
}

}  // namespace

size_t latent_attention_workspace()
{
    return run_workspace();
}

int launch_latent_attention(int store_mode, const AttentionArgs &a, void *workspace, cudaStream_t stream)
{
    static std::atomic<int> sm_count[2][64];
    const bool fp8 = store_mode == DSV4_STORE_FP8;
    const auto kernel = fp8 ? latent_attention_kernel<true> : latent_attention_kernel<false>;
    int sms = 0;
    if (configure_runs(kernel, kSmemBytes, sm_count[fp8], &sms) != DSV4_OK)
        return DSV4_ERR_CUDA;
    return launch_runs<Tiles>(kernel, kThreads, kSmemBytes, sms, a, fp8 ? kFp8OperandUnit : 1.0f, workspace, stream);
}

}  // namespace dsv4

DSV4_BOUNDS_FLAG_READER(bounds_flag_latent_attention)
