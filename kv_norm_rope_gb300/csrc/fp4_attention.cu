// Attention over the 4-bit cache: out = softmax(scale * q k^T [sink]) k, where a
// request's latent rows are keys and values in one.
//
// Per (query row, key) it takes 2 * 512 multiplications for the score and as many
// for the value, and a key's 368 bytes are read once for all rows of its request:
// at 64 heads 356 operations a byte, which puts the matrix units and the memory
// near one another.  So the rows are multiplied with tcgen05 in bf16 (a 4-bit code
// times its scale is a bf16 exactly) and converted on the way:
//
//  * A CTA holds 64 query rows (the heads of one or more tokens of a request) and
//    walks its run of tiles of 128 keys (fp4_tiles.cuh).  Scores are computed
//    transposed, S^T[key, row] = K q^T, and so are the outputs, O^T[dim, row] =
//    K^T P^T: keys and dims take the 128 lanes of the tensor memory, so any number
//    of rows up to 64 costs in proportion (N = 16, 32, 48, 64), and O^T of 512
//    dims (4 x 64 columns) fits beside S^T.  Rows are held times 2^-80 (fp4.cuh).
//  * One converted tile serves both products: K-major as the left operand of the
//    first, read across (MN-major) as that of the second.  It is held in 4 pairs
//    of chunks of 64 dims, each filled, and freed by the second product, on its
//    own, so the next tile is converted under the products of this one.
//  * Warps 0..7 do the softmax: warp w has the keys of lanes 32 (w % 4).. and rows
//    32 (w / 4)..; a thread has one key and 32 rows.  Warps 8..23 convert, warp 24
//    issues the products, warp 25 notes the run's ends.  The teams of converting
//    warps share one code path, so that all loops fit the instruction cache together,
//    and warp 24's warpgroup gives registers to the softmax: a spill costs a trip to
//    L2, as shared memory leaves little of L1.
//  * The softmax needs no maximum per tile.  Each row has a reference m, the
//    largest score of the first tile it saw; p = 2^(x - m) is taken against that,
//    and only when some x exceeds m by more than kSlack is m moved and everything
//    rescaled (fp32 and bf16 have the same range, so a p of 2^kSlack loses
//    nothing).  Sums stay per thread, in fp32, until the segment ends.
//  * A run that covers all tiles of a request writes the output; else the
//    unnormalised O, m and the sum go to the workspace and a second kernel joins
//    them in the order of the runs, each of which has noted (warp 25) what it left.
//
// A key whose row is not finite may be masked for some rows of the tile, and 0 times
// an infinity is NaN in the second product.  So what is not finite of it enters the
// operands as a finite value and the key is marked: rows that see it get NaN as its score, whose P
// makes all of their dims NaN, and the others are left alone.
//
// P is rounded to bf16 as an operand (half a step, at most 2^-8 of the value, to
// either side); the sum that divides it is of the unrounded p.
//
// One request of 262147 keys, 128 heads: 115.5 to 119.4 us in several runs, 576 to 595
// TFLOP/s; 128 requests of 1024 to 8192 keys, 128 heads: 239 us, 607 TFLOP/s; 48 of up
// to 4096, 64 heads: 41 us (their results joined included).  By
// arithmetic, an instruction of either product reads 6 KB of shared memory for 32
// cycles of the matrix unit, so at 128 bytes a cycle shared memory bounds them at two
// thirds of the unit's rate, and the converted rows are written through it as well.
// Between the products stands the softmax: there is no room for a second tile of keys
// (128 KB) beside the queries' 64 KB.  On the second case, an earlier form took 289 us,
// and 220 in a copy without any of the conversion's work.  Tried and slower there:
// half of the keys staged in tensor memory so that the next tile's scores overlap the
// softmax (352 us), a warpgroup a pair (286), all warps on one pair at a time (270).

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include "fp4_tiles.cuh"
#include "launch_status.h"
#include "ops.h"
#include "run_join.cuh"

namespace dsv4 {
namespace {

constexpr int kGroups = 2;           // of 4 softmax warps
constexpr int kCols = kRows / kGroups;
constexpr int kConvertWarp = 4 * kGroups, kMultiplyWarp = kConvertWarp + 16;
constexpr int kThreads = (kMultiplyWarp + 4) * 32;  // whole warpgroups: the last two warps idle
// registers a thread: 72 at launch (896 * 72 = 64512), then
constexpr int kSoftmaxRegs = 88, kConvertRegs = 72, kMultiplyRegs = 40;
static_assert(128 * (kGroups * kSoftmaxRegs + 4 * kConvertRegs + kMultiplyRegs) <= kThreads * 72,
              "the shares exceed what the CTA was launched with");
constexpr float kSlack = 16.0f;

// Shared memory (from a 1024-byte boundary).
constexpr uint32_t kKeys = 0;                                  // 8 chunks of a converted tile
constexpr uint32_t kQuery = kKeys + kChunks * kChunkBytes;     // 8 chunks of 64 rows
constexpr uint32_t kProbs = kQuery + kChunks * kRows * 128;    // P^T: 128 keys of 64 rows
constexpr uint32_t kRing = kProbs + kTileKeys * 128;            // a slot of codes for each team
constexpr uint32_t kShared = kRing + 2 * kRingSlot;

struct Shared {
    uint64_t full[kChunks / 2], free[kChunks / 2];  // of a pair of chunks
    uint64_t scores, probs, query, query_free, output;
    uint32_t tmem;
    int scratch[kDealWords];
    alignas(16) float m[kRows];
    alignas(16) float factor[kRows];
    float warp_rows[4][kRows];  // maxima or sums of the four warps' keys
    int seen_to[kRows], seen_from[kRows];
    uint8_t key_state[kTileKeys];  // kMissing, kTaken or kNotFinite, by its exponents
    // bits of the keys whose rope dims are not finite: a word for each softmax warp,
    // which clears it
    uint32_t rope_marks[kGroups][4];
    Cursor place[4 * kGroups];  // of the softmax warps
};
constexpr size_t kSmemBytes = kShared + sizeof(Shared);
enum : uint8_t { kMissing = 0, kTaken = 1, kNotFinite = 2 };
static_assert(kSmemBytes <= 227 * 1024, "too much shared memory");

// monotone map of a float to an int, for integer maxima; NaN counts as -infinity
__device__ __forceinline__ int ordered(float x)
{
    const int b = __float_as_int(x == x ? x : -INFINITY);
    return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float unordered(int i)
{
    return __int_as_float(i ^ ((i >> 31) & 0x7fffffff));
}

// ---- Warps 8..23: cache rows and queries into operands

// a row's exponents; the two bytes without one become 1 where the row is not finite
// (found as they are loaded: among the conversion it cost 34 us more than 251)
__device__ __forceinline__ uint4 marked(uint4 scales)
{
    scales.w = (scales.w & 0xFFFFu) | (fp4_row_above(scales) ? 0x10000u : 0u);
    return scales;
}

__device__ __forceinline__ void mark_key(Shared &s, int key)
{
#pragma unroll
    for (int g = 0; g < kGroups; ++g)
        atomicOr(&s.rope_marks[g][key >> 5], 1u << (key & 31));
}

__device__ __forceinline__ void convert_role(const AParams &p, Shared &s, uint8_t *smem, Cursor c,
                                             const int team)
{
    const int tid = threadIdx.x - kConvertWarp * 32 - team * kTeam;
    const int key = tid >> 1, half = tid & 1, lane = tid & 31;
    const int count = c.left;
    const uint32_t base = smem_addr(smem), slot = base + kRing + team * kRingSlot;
    const uint32_t place = swizzled(key, 4 * half);
    KeyPlace now = key_place(p, c, true, key);
    Fp4Row row = row_at(p, now);
    copy_codes(p, slot, tid, row, team);
    uint4 scales = marked(load_raw(p, row.scale, row.data != nullptr));
    const auto fill_query = [&] {
        const int unit = ~now.unit, request = int(fastdiv(uint32_t(unit), p.tile_div));
        load_query(p, request, (unit - request * p.row_tiles) * kRows, smem + kQuery, kRows, tid + team * kTeam, 2 * kTeam);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&s.query);
    };
    fill_query();
    bool moved = c.advance(p);
    KeyPlace next = key_place(p, c, moved, key);
    int segment = 1;
    for (int t = 0; t < count; ++t) {
        const Fp4Row next_row = row_at(p, next);
        KeyPlace after = next;
        after.off = UINT32_MAX;
        if (c.left > 0) {
            moved = c.advance(p);
            after = key_place(p, c, moved, key);
        }
        const uint4 next_scales = load_raw(p, next_row.scale, next_row.data != nullptr);
        if (team == 1)
            prefetch64(p, row.data + kFp4Codes + 64 * half, row.data != nullptr);
        bool alive = true;
        if (now.unit < 0 && t > 0) {
            alive = __all_sync(kFull, mbar_wait(&s.query_free, (segment - 1) & 1));
            if (alive)
                fill_query();
            ++segment;
        }
        uint4 rope[4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int i = team + 2 * u;  // chunks 2i and 2i + 1
            const uint32_t to = base + kKeys + 2 * i * kChunkBytes;
            copy_wait();
            const uint4 a = load_shared16(slot + tid * 16), b = load_shared16(slot + 4096 + tid * 16);
            uint4 out[4];
            copy_codes(p, slot, tid, u == 0 ? row : next_row, u == 0 ? i + 2 : team);
            const uint32_t four = (i < 2 ? (i == 0 ? scales.x : scales.y) : i == 2 ? scales.z : scales.w) >>
                                  (8 * half);
            convert_group<true>(a, four, out);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                computed(out[k]);  // before the wait for its place
            if (t > 0 && alive)
                alive = __all_sync(kFull, mbar_wait(&s.free[i], (t - 1) & 1));
            if (!alive)
                break;
            if (i == 0 && half == 0)
                store_shared1(base + kShared + uint32_t(offsetof(Shared, key_state)) + key,
                              row.data == nullptr ? uint32_t(kMissing) : kTaken + (scales.w >> 16));
            store_half(to, place, out);
            if (i < 3) {
                convert_group<true>(b, four >> 16, out);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    out[k] = finite_bf16x8(mul_bf16x8(rope[k], kRopeToOperand));
            }
            store_half(to + kChunkBytes, place, out);
            if (i == 3) {
                // after the stores: its registers before them cost 15 us of 258
                uint32_t zero = 0u;  // or NaN, 0x7FFF, where a value is not finite
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    zero = zero_of_bf16x8(rope[k], zero);
                if ((zero & 0x7FFF7FFFu) != 0u)
                    mark_key(s, key);
            }
            if (i == 1) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    rope[k] = load_raw(p, row.data + kFp4Codes + 64 * half + 16 * k, row.data != nullptr);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&s.full[i]);
        }
        if (!alive) {
            flag(p.a.b.err, DSV4_DEVERR_TIMEOUT);
            break;
        }
        scales = marked(next_scales);
        row = next_row;
        now = next;
        next = after;
    }
    copy_wait();
}

// ---- Warp 24: the products

__device__ void multiply_role(const AParams &p, Shared &s, uint32_t smem, Cursor c)
{
    const uint32_t elected = elect_one();
    const uint32_t d_scores = s.tmem, d_output = s.tmem + kRows;
    const Operand keys = operand(smem + kKeys, 16, 1024), query = operand(smem + kQuery, 16, 1024);
    const Operand values = operand(smem + kKeys, kChunkBytes, 1024);
    const Operand probs = operand(smem + kProbs, kChunkBytes, 1024);
    uint32_t scores_inst = 0, output_inst = 0;
    int segment = 0;
    bool first = true;  // of its segment
    for (uint32_t t = 0; c.left > 0; ++t) {
        if (first) {
            const uint32_t n = uint32_t((c.row1 - c.row0 + 15) & ~15);
            scores_inst = instruction(n, false);
            output_inst = instruction(n, true);
            if (!__all_sync(kFull, mbar_wait(&s.query, segment & 1)))
                break;
            ++segment;
        }
        const bool last = c.ends_segment();
        bool alive = true;
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            if (i % 2 == 0) {
                alive = alive && __all_sync(kFull, mbar_wait(&s.full[i / 2], t & 1));
                if (!alive)
                    break;
                tmem_fence_after();
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                mma_bf16(d_scores, keys + (i * kChunkBytes + 32 * k), query + (i * kRows * 128 + 32 * k),
                         scores_inst, i > 0 || k > 0, elected);
        }
        if (!alive)
            break;
        mma_commit(&s.scores, elected);
        if (last)
            mma_commit(&s.query_free, elected);
        if (!__all_sync(kFull, mbar_wait(&s.probs, t & 1)))
            break;
        tmem_fence_after();
#pragma unroll
        for (int i = 0; i < kChunks / 2; ++i) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                mma_bf16(d_output + i * kRows, values + (2 * i * kChunkBytes + 2048 * k),
                         probs + 2048 * k, output_inst, !first || k > 0, elected);
            mma_commit(&s.free[i], elected);
        }
        if (last)
            mma_commit(&s.output, elected);
        first = last;
        c.advance(p);
    }
    if (c.left > 0)
        flag(p.a.b.err, DSV4_DEVERR_TIMEOUT);
}

// ---- Warps 0..7: softmax and results

// Move the references of a warpgroup's rows up to the scores x of this tile and
// rescale what was taken against the old ones.
__device__ __forceinline__ void move_references(Shared &s, const float *x, float *sum, uint32_t tmem,
                                                bool rescale_output)
{
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3, group = threadIdx.x >> 7;
    const int col0 = group * kCols;
    int mine = 0;
#pragma unroll
    for (int j = 0; j < kCols; ++j) {
        const int top = __reduce_max_sync(kFull, ordered(x[j]));
        if (lane == j)
            mine = top;
    }
    s.warp_rows[warp][col0 + lane] = unordered(mine);
    named_barrier(1 + group, 128);
    if (warp == 0) {
        const int j = col0 + lane;
        const float old = s.m[j];
        const float m = fmaxf(fmaxf(old, fmaxf(s.warp_rows[0][j], s.warp_rows[1][j])),
                              fmaxf(s.warp_rows[2][j], s.warp_rows[3][j]));
        s.m[j] = m;
        s.factor[j] = exp2_approx(old - m);
    }
    named_barrier(1 + group, 128);
#pragma unroll
    for (int j = 0; j < kCols; ++j)
        sum[j] *= s.factor[col0 + j];
    if (rescale_output) {
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
            const uint32_t at = tmem + kRows + (i >> 1) * kRows + col0 + (i & 1) * 16;
            float o[16];
            tmem_load16(at, o);
            tmem_wait_load();
#pragma unroll
            for (int j = 0; j < 16; ++j)
                o[j] *= s.factor[col0 + (i & 1) * 16 + j];
            tmem_store16(at, o);
        }
        tmem_wait_store();
    }
}

// sums of 32 values over the 32 lanes of a warp: lane j returns that of v[j]
__device__ __forceinline__ float transposed_sum(float *v, int lane)
{
#pragma unroll
    for (int half = 16; half >= 1; half >>= 1) {
        const bool upper = (lane & half) != 0;
#pragma unroll
        for (int j = 0; j < half; ++j) {
            const float keep = upper ? v[j + half] : v[j];
            const float give = upper ? v[j] : v[j + half];
            v[j] = keep + __shfl_xor_sync(kFull, give, half);
        }
    }
    return v[0];
}

__device__ void softmax_role(const WParams &w, Shared &s, uint8_t *smem, const Cursor &begin)
{
    const AParams &p = w.p;
    const AttentionArgs &a = p.a;
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3, group = threadIdx.x >> 7;
    const int key = warp * 32 + lane, col0 = group * kCols;
    // the warp's place lives in shared memory: what the softmax holds fills its registers
    Cursor &c = s.place[threadIdx.x >> 5];
    if (lane == 0)
        c = begin;
    __syncwarp();
    const uint32_t tmem = s.tmem + (uint32_t(warp * 32) << 16);
    const float scale = a.scale * (kLog2e * kOperandUnit);
    const uint32_t probs = smem_addr(smem) + kProbs, row = swizzled(key, group * (kCols / 8));
    float sum[kCols];
    bool first = true;
    int segment = 0, from_tile = 0;
    for (uint32_t t = 0; c.left > 0; ++t) {
        const int row0 = c.row0, rows = c.row1 - c.row0;
        if (first) {
            from_tile = c.tile;
            if (warp == 0) {
                const int r = col0 + lane;
                const int to = r < rows ? c.n - a.q_len + 1 + int(fastdiv(uint32_t(row0 + r), p.head_div)) : 0;
                s.seen_to[r] = to;
                s.seen_from[r] = a.window > 0 ? to - a.window : INT32_MIN;
                s.m[r] = kUnset;
            }
            named_barrier(1 + group, 128);
#pragma unroll
            for (int j = 0; j < kCols; ++j)
                sum[j] = 0.0f;
        }
        const bool last = c.ends_segment();
        bool failed = !mbar_wait(&s.scores, t & 1);
        tmem_fence_after();
        const int i = c.tile * kTileKeys + key;
        // every row of the group sees every key of the tile: the first row sees the
        // fewest at the end, the last one the fewest at the start
        const bool whole = rows >= col0 + kCols && (c.tile + 1) * kTileKeys <= s.seen_to[col0] &&
                           c.tile * kTileKeys >= s.seen_from[col0 + kCols - 1];
        const int state = s.key_state[key];
        const uint32_t marks = s.rope_marks[group][warp];
        const bool ok = state == kTaken && ((marks >> lane) & 1u) == 0u;
        if (marks != 0u) {
            __syncwarp();
            if (lane == 0)
                s.rope_marks[group][warp] = 0u;
        }
        float v[kCols];
        // v = the scores less `reference` (a row each; null: none), -infinity where unseen
        const auto load_scores = [&](const float *reference) {
            __syncwarp();
            tmem_load16(tmem + col0, v);
            tmem_load16(tmem + col0 + 16, v + 16);
            tmem_wait_load();
#pragma unroll
            for (int j = 0; j < kCols; j += 4) {
                const float4 m = reference != nullptr
                                     ? *reinterpret_cast<const float4 *>(reference + col0 + j)
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
                v[j] = __fmaf_rn(v[j], scale, -m.x);
                v[j + 1] = __fmaf_rn(v[j + 1], scale, -m.y);
                v[j + 2] = __fmaf_rn(v[j + 2], scale, -m.z);
                v[j + 3] = __fmaf_rn(v[j + 3], scale, -m.w);
            }
            if (!ok) {
                const float stand_in = state == kMissing ? -INFINITY : __int_as_float(0x7FFFFFFF);
#pragma unroll
                for (int j = 0; j < kCols; ++j)
                    v[j] = stand_in;
            }
            if (!whole) {
#pragma unroll
                for (int j = 0; j < kCols; ++j)
                    if (i >= s.seen_to[col0 + j] || i < s.seen_from[col0 + j])
                        v[j] = -INFINITY;
            }
        };
        load_scores(s.m);
        float over = v[0];
#pragma unroll
        for (int j = 1; j < kCols; ++j)
            over = fmaxf(over, v[j]);
        if (named_barrier_any(1 + group, 128, failed || over > kSlack)) {
            if (named_barrier_any(1 + group, 128, failed)) {
                flag(a.b.err, DSV4_DEVERR_TIMEOUT);
                return;
            }
            load_scores(nullptr);
            move_references(s, v, sum, tmem, !first);
            load_scores(s.m);
        }
#pragma unroll
        for (int k = 0; k < kCols / 8; ++k) {
            uint32_t packed[4];
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const float p0 = exp2_approx(v[8 * k + j]), p1 = exp2_approx(v[8 * k + j + 1]);
                sum[8 * k + j] += p0;
                sum[8 * k + j + 1] += p1;
                packed[j / 2] = bf16x2_rn(p0, p1);
            }
            store_shared16(probs + (row ^ (k << 4)), make_uint4(packed[0], packed[1], packed[2], packed[3]));
        }
        fence_proxy_async_smem();
        tmem_fence_before();
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&s.probs);
        if (last) {
            // the segment's result
            const float key_sum = transposed_sum(sum, lane);
            s.warp_rows[warp][col0 + lane] = key_sum;
            failed = !mbar_wait(&s.output, segment & 1);
            ++segment;
            if (named_barrier_any(1 + group, 128, failed)) {
                flag(a.b.err, DSV4_DEVERR_TIMEOUT);
                return;
            }
            tmem_fence_after();
            const bool whole_range = from_tile == c.range.first() && c.tile + 1 == c.range.stop();
            const int r = col0 + lane;
            const float total = (s.warp_rows[0][r] + s.warp_rows[1][r]) +
                                (s.warp_rows[2][r] + s.warp_rows[3][r]);
            const int64_t out_row = int64_t(c.request) * p.all_rows + row0;
            // the run's first segment or its last
            float *part = partial_at(w, blockIdx.x, t + 1 == uint32_t(c.tile + 1 - from_tile) ? 0 : 1);
            const Span ps = partial_span(w);
            if (warp == 0) {
                if (whole_range) {
                    float lse = 0.0f;
                    if (r < rows)
                        s.factor[r] = finish(s.m[r], total, sink_of(a, row0 + r), w.unit, &lse);
                    if (r < rows && a.lse != nullptr)
                        st_f32_in(a.lse + out_row + r, lse, Span{a.lse, rows_of(a) * 4u}, a.b.err);
                } else {
                    st_f32_in(part + kRows * DSV4_HEAD_DIM + r, s.m[r], ps, a.b.err);
                    st_f32_in(part + kRows * DSV4_HEAD_DIM + kRows + r, total, ps, a.b.err);
                }
            }
            named_barrier(1 + group, 128);
            const Span os{a.out, rows_of(a) * (DSV4_HEAD_DIM * 2u)};
            const int mine = rows - col0 < kCols ? rows - col0 : kCols;
            if (mine > 0) {
#pragma unroll 1
                for (int k = 0; k < 4; ++k) {
                    float o[kCols];
                    tmem_load16(tmem + kRows + k * kRows + col0, o);
                    tmem_load16(tmem + kRows + k * kRows + col0 + 16, o + 16);
                    tmem_wait_load();
                    const int dim = k * 128 + key;
                    if (whole_range) {
                        // neighbouring lanes swap, so that each stores two dims of one row
                        const int odd = lane & 1;
                        uint16_t *to = a.out + (out_row + col0 + odd) * DSV4_HEAD_DIM + (dim - odd);
#pragma unroll
                        for (int j = 0; j < kCols; j += 2) {
                            const float o0 = o[j] * s.factor[col0 + j];
                            const float o1 = o[j + 1] * s.factor[col0 + j + 1];
                            const float other = __shfl_xor_sync(kFull, odd ? o0 : o1, 1);
                            if (j + odd < mine)
                                st4_in(to + j * DSV4_HEAD_DIM, odd ? bf16x2_rn(other, o1) : bf16x2_rn(o0, other),
                                       os, a.b.err);
                        }
                    } else {
                        float *to = part + col0 * DSV4_HEAD_DIM + dim;
#pragma unroll
                        for (int j = 0; j < kCols; ++j)
                            if (j < mine)
                                st_f32_in(to + j * DSV4_HEAD_DIM, o[j], ps, a.b.err);
                    }
                }
            }
            tmem_fence_before();
            named_barrier(1 + group, 128);  // m, sum and factor are free for the next segment
        }
        first = last;
        __syncwarp();
        if (lane == 0)
            c.advance(p);
        __syncwarp();
    }
}

__global__ void __launch_bounds__(kThreads, 1) fp4_attention_kernel(const __grid_constant__ WParams w)
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
            for (int i = 0; i < kChunks / 2; ++i) {
                mbar_init(&s.full[i], 8);
                mbar_init(&s.free[i], 1);
            }
            mbar_init(&s.scores, 1);
            mbar_init(&s.probs, kConvertWarp);
            mbar_init(&s.query, 16);
            mbar_init(&s.query_free, 1);
            mbar_init(&s.output, 1);
            mbar_init_fence();
        }
        tmem_fence_before();
    }
    if (threadIdx.x < 4 * kGroups)
        s.rope_marks[threadIdx.x >> 2][threadIdx.x & 3] = 0u;
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
    } else if (warp < kConvertWarp) {
        registers_up<kSoftmaxRegs>();
        softmax_role(w, s, smem, c);
    } else {
        convert_role(p, s, smem, c, (warp - kConvertWarp) / 8);
    }
    tmem_fence_before();
    __syncthreads();
    if (warp == kMultiplyWarp) {
        tmem_fence_after();
        tmem_free512(s.tmem);
    }
}

}  // namespace

size_t fp4_attention_workspace()
{
    return run_workspace();
}

int launch_fp4_attention(const AttentionArgs &a, void *workspace, cudaStream_t stream)
{
    static std::atomic<int> sm_count[64];
    int sms = 0;
    if (configure_runs(fp4_attention_kernel, kSmemBytes, sm_count, &sms) != DSV4_OK)
        return DSV4_ERR_CUDA;
    const WParams w = plan_runs<Tiles>(a, kOperandUnit, sms, workspace);
    const int st = launch_after(fp4_attention_kernel, dim3(unsigned(w.runs)), dim3(kThreads), stream, w, kSmemBytes);
    return st != DSV4_OK ? st : launch_join<Tiles>(w, stream);
}

}  // namespace dsv4

DSV4_BOUNDS_FLAG_READER(bounds_flag_fp4_attention)
