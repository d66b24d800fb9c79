// The attention each key of the 4-bit cache gets: weights[key] += the sum over query
// rows of exp(scale * q . k - lse).
//
// The first product of the attention (fp4_attention.cu) with another end: S^T[key,
// row] = K q^T on the tensor cores, keys in the lanes, so a thread holds one key and
// its sum over rows needs no exchange.  2 * 512 multiplications a (row, key), no
// second product, and nothing for the matrix unit to wait for but converted rows:
//
//  * 128 query rows a pass (N = 128).  More rows take more passes over the same run
//    of keys, whose bytes then come from L2.
//  * Converted keys go to tensor memory, the left operand, a thread a key: 256 of its
//    512 columns are a tile's 512 dims, in four pairs of chunks, each filled by its
//    own warpgroup as soon as the product of the tile before has read it.  (Through
//    shared memory, as the attention has to, their 128 KB a tile contended with the
//    product's own reads: 89 us against 85 below, and 61 with those stores left out.)
//  * S^T has two places in the other 256 columns, so the sums of a tile run under the
//    product of the next.
//  * Each key's sum is finished by one thread of one CTA in a fixed order of rows
//    and added by it: no atomics, the same bits every time.
//
// 3 requests of up to 131072 keys, 2 x 128 rows: 85 us, 805 TFLOP/s; 48 of up to 4096,
// 64 rows: 25 us.  What bounds it is the conversion: the schedulers issue in 67% of the
// cycles (23 instructions for the 8 codes of a word), the matrix unit is busy in 37%.
// All converting warps run one code path: a copy of the loop for each pair did not fit
// the instruction cache with the rest and took 150 us.

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "fp4_tiles.cuh"
#include "launch_status.h"
#include "ops.h"

namespace dsv4 {
namespace {

constexpr int kRows = 128;  // query rows of a pass
constexpr int kGroups = 2;  // of 4 summing warps, each with half of the rows
constexpr int kCols = kRows / kGroups;
constexpr int kConvertWarp = 4 * kGroups, kMultiplyWarp = kConvertWarp + 16;
constexpr int kThreads = (kMultiplyWarp + 1) * 32;
constexpr float kLog2e = 1.4426950408889634f;
// Places for the words of which keys are there.  A tile's is written behind the wait for the
// product of the tile before, t - 1, which began after every summing warp had given back the
// scores of tile t - 3, and so after all of them had read the words of tile t - 4.
constexpr int kOkTiles = 4;

// Shared memory (from a 1024-byte boundary): 8 chunks of 128 rows, then what is on
// its way, a tile: 64 bytes a key for pairs 0..2, 32 of codes and 128 of rope for pair 3.
constexpr uint32_t kQuery = 0;
constexpr uint32_t kRing = kQuery + kChunks * kRows * 128;
constexpr uint32_t kRope = kRing + 4 * kTileKeys * 64;
constexpr uint32_t kShared = kRope + kTileKeys * 128;

// Tensor memory, 512 columns: S^T of two tiles, then the keys.
constexpr uint32_t kKeysAt = 2 * kRows;

struct Shared {
    uint64_t staged[4], staged_free[4], scores[2], scores_free[2], query, query_free;
    uint32_t tmem;
    int scratch[kDealWords];
    alignas(16) float lse[kRows];
    int seen_to[kRows], seen_from[kRows];
    float part[kTileKeys];
    uint32_t key_ok[kOkTiles][4];  // a bit a key
};
constexpr size_t kSmemBytes = kShared + sizeof(Shared);
static_assert(kSmemBytes <= 227 * 1024, "too much shared memory");

struct WParams {
    AParams p;   // one unit a request: all of its rows
    int passes;  // of 128 rows
};

// The order in which a CTA works: its run of tiles request by request, each
// request's part once a pass.
struct Sweep {
    Cursor c;
    int length, k, pass;
    bool live, new_pass;

    __device__ __forceinline__ void begin()
    {
        live = c.left > 0;
        const int rest = c.range.stop() - c.tile;
        length = c.left < rest ? c.left : rest;
        k = pass = 0;
        new_pass = true;
    }

    // the place as a cursor, for key_place
    __device__ __forceinline__ Cursor at() const
    {
        Cursor x = c;
        x.tile = c.tile + k;
        x.left = live ? 1 : 0;
        return x;
    }

    __device__ __forceinline__ void advance(const WParams &w)
    {
        new_pass = false;
        if (++k < length)
            return;
        k = 0;
        new_pass = true;
        if (++pass < w.passes)
            return;
        c.tile += length - 1;
        c.left -= length - 1;
        c.advance(w.p);
        begin();
    }
};

__device__ __forceinline__ int pass_rows(const WParams &w, int pass)
{
    const int rest = w.p.all_rows - pass * kRows;
    return rest < kRows ? rest : kRows;
}

// ---- Warps 8..23: cache rows and queries into operands

// `pieces` (<= kPlaces) 16-byte pieces of the warp's 32 keys into shared memory, kPlaces
// places a key side by side, from byte `at` of each row on: neighbouring lanes copy
// neighbouring pieces.  A key's pieces are permuted by `turn` of it, so that 8 lanes
// reading one piece each of their own keys meet different banks.
template <int kPlaces>
__device__ __forceinline__ uint32_t turn(int key)
{
    return uint32_t(kPlaces == 8 ? key : key >> 1) & (kPlaces - 1);
}

template <int kPlaces>
__device__ __forceinline__ void copy_pieces(const AParams &p, uint32_t to, int lane, const uint8_t *row,
                                            int at, int pieces)
{
    const int piece = lane % kPlaces;
#pragma unroll
    for (int k = 0; k < kPlaces; ++k) {
        const int key = lane / kPlaces + 32 / kPlaces * k;
        const uint64_t from = __shfl_sync(kFull, reinterpret_cast<uint64_t>(row), key);
        if (piece < pieces)
            copy16(p, to + key * (16 * kPlaces) + ((piece ^ turn<kPlaces>(key)) << 4),
                   reinterpret_cast<const uint8_t *>(from) + at + 16 * piece, from != 0u);
    }
}

template <int kPlaces>
__device__ __forceinline__ uint4 piece_of(uint32_t at, int lane, int piece)
{
    return load_shared16(at + lane * (16 * kPlaces) + ((piece ^ turn<kPlaces>(lane)) << 4));
}

// A warpgroup converts one pair of chunks, a thread a key: 128 dims, pair 3's the codes
// of chunk 6 and the rope dims.  The next tile's bytes are copied as soon as this
// one's are read.  The pair is no template argument: the warps' loops have to fit the
// instruction cache together.
__device__ __forceinline__ void convert_role(const WParams &w, Shared &s, uint8_t *smem, Sweep sw,
                                             const int pair)
{
    const AParams &p = w.p;
    const int tid = threadIdx.x - kConvertWarp * 32, lane = tid & 31, warp = (tid >> 5) & 3;
    const int key = warp * 32 + lane;
    const uint32_t ring = smem_addr(smem) + kRing + pair * (kTileKeys * 64) + warp * 2048;
    const uint32_t rope = smem_addr(smem) + kRope + warp * 4096;
    const uint32_t staged = s.tmem + (uint32_t(warp * 32) << 16) + kKeysAt + pair * 64;
    const auto copy = [&](const Fp4Row &row) {
        copy_pieces<4>(p, ring, lane, row.data, 64 * pair, pair < 3 ? 4 : 2);
        if (pair == 3)
            copy_pieces<8>(p, rope, lane, row.data, kFp4Codes, 8);
    };
    const auto load_scales = [&](const Fp4Row &row) {
        return row.data != nullptr ? ldg4_now_in(row.scale + 4 * pair, cache_span(p.a.b), p.a.b.err) : 0u;
    };
    KeyPlace now = key_place(p, sw.at(), true, key);
    int now_pass = 0;
    Fp4Row row = row_at(p, now);
    copy(row);
    uint32_t scales = load_scales(row);
    bool there = row.data != nullptr;
    sw.advance(w);
    KeyPlace next = key_place(p, sw.at(), sw.new_pass, key);
    bool next_live = sw.live;
    int next_pass = sw.pass;
    uint32_t passes = 0;
    for (uint32_t t = 0;; ++t) {
        row = row_at(p, next);
        const uint32_t next_scales = load_scales(row);
        KeyPlace after = next;
        after.off = UINT32_MAX;
        bool after_live = false;
        int after_pass = 0;
        if (next_live) {
            sw.advance(w);
            after = key_place(p, sw.at(), sw.new_pass, key);
            after_live = sw.live;
            after_pass = sw.pass;
        }
        bool alive = true;
        if (now.unit < 0) {
            if (passes > 0)
                alive = __all_sync(kFull, mbar_wait(&s.query_free, (passes - 1) & 1));
            if (alive) {
                load_query(p, ~now.unit, now_pass * kRows, smem + kQuery, kRows, tid, 512);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&s.query);
            }
            ++passes;
        }
        copy_wait();
        __syncwarp();  // the copies are the warp's together
        if (t > 0 && alive)
            alive = __all_sync(kFull, mbar_wait(&s.staged_free[pair], (t - 1) & 1));
        if (!alive) {
            flag(p.a.b.err, DSV4_DEVERR_TIMEOUT);
            break;
        }
        tmem_fence_after();
        __syncwarp();
        if (pair == 0) {
            const uint32_t bits = __ballot_sync(kFull, there);
            if (lane == 0)
                s.key_ok[t % kOkTiles][warp] = bits;
        }
#pragma unroll 1
        for (int g = 0; g < 4; ++g) {
            uint4 out[4];
            if (pair < 3 || g < 2) {
                convert_group<false>(piece_of<4>(ring, lane, g), scales >> (8 * g), out);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    out[k] = mul_bf16x8(piece_of<8>(rope, lane, 4 * (g - 2) + k), kRopeToOperand);
            }
            __syncwarp();
            tmem_store16(staged + 16 * g, out);
        }
        tmem_wait_store();
        tmem_fence_before();
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&s.staged[pair]);
        if (!next_live)
            break;
        copy(row);
        scales = next_scales;
        there = row.data != nullptr;
        now = next;
        now_pass = next_pass;
        next = after;
        next_live = after_live;
        next_pass = after_pass;
    }
    copy_wait();
}

// ---- Warp 24: the products

__device__ __forceinline__ void multiply_role(const WParams &w, Shared &s, uint32_t smem, Sweep sw)
{
    const uint32_t elected = elect_one();
    const Operand query = operand(smem + kQuery, 16, 1024);
    uint32_t inst = 0, passes = 0;
    for (uint32_t t = 0; sw.live; ++t) {
        bool alive = true;
        if (sw.new_pass) {
            inst = instruction(uint32_t((pass_rows(w, sw.pass) + 15) & ~15), false);
            alive = __all_sync(kFull, mbar_wait(&s.query, passes & 1));
            ++passes;
        }
        const bool last = sw.k + 1 == sw.length;
        if (t >= 2)
            alive = alive && __all_sync(kFull, mbar_wait(&s.scores_free[t & 1], (t / 2 - 1) & 1));
        const uint32_t d = s.tmem + (t & 1) * kRows;
#pragma unroll
        for (int i = 0; i < kChunks / 2; ++i) {
            alive = alive && __all_sync(kFull, mbar_wait(&s.staged[i], t & 1));
            if (!alive)
                break;
            tmem_fence_after();
#pragma unroll
            for (int k = 0; k < 8; ++k)
                mma_bf16_staged(d, s.tmem + kKeysAt + i * 64 + k * 8,
                                query + ((2 * i + (k >> 2)) * kRows * 128 + 32 * (k & 3)), inst,
                                i > 0 || k > 0, elected);
            mma_commit(&s.staged_free[i], elected);
        }
        if (!alive) {
            flag(w.p.a.b.err, DSV4_DEVERR_TIMEOUT);
            break;
        }
        mma_commit(&s.scores[t & 1], elected);
        if (last)
            mma_commit(&s.query_free, elected);
        sw.advance(w);
    }
}

// ---- Warps 0..7: the sums

__device__ __forceinline__ void sum_role(const WParams &w, Shared &s, Sweep sw)
{
    const AParams &p = w.p;
    const AttentionArgs &a = p.a;
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3, group = threadIdx.x >> 7;
    const int key = warp * 32 + lane, col0 = group * kCols, tid = threadIdx.x;
    const uint32_t tmem = s.tmem + (uint32_t(warp * 32) << 16);
    const float scale = a.scale * (kLog2e * kOperandUnit);
    const Span ws{a.weights, (uint64_t(a.b.batch - 1) * a.weights_stride + a.weights_width) * 4u};
    bool some_out = false;  // some row of the pass is left out
    for (uint32_t t = 0; sw.live; ++t) {
        const int rows = pass_rows(w, sw.pass), n = sw.c.n;
        if (sw.new_pass) {
            named_barrier(1, 256);  // the rows before are done with
            bool out = false;
            if (tid < kRows) {
                const int r = sw.pass * kRows + tid;
                float lse = INFINITY;  // no row: its exponentials are 0
                int to = 0;
                if (tid < rows) {
                    lse = kLog2e * ldg_f32_in(a.lse + int64_t(sw.c.request) * p.all_rows + r,
                                              Span{a.lse, rows_of(a) * 4u}, a.b.err);
                    to = n - a.q_len + 1 + int(fastdiv(uint32_t(r), p.head_div));
                    // a row without a sum adds nothing, and sees no key: one that is
                    // not finite would make NaN of its exponential
                    out = lse == -INFINITY;
                    if (out)
                        to = 0;
                }
                s.lse[tid] = lse;
                s.seen_to[tid] = to;
                s.seen_from[tid] = a.window > 0 ? to - a.window : INT32_MIN;
            }
            some_out = named_barrier_any(1, 256, out);
        }
        const int tile = sw.c.tile + sw.k, i = tile * kTileKeys + key;
        const bool mine = group == 0 && i >= sw.c.range.lo && i < sw.c.range.hi;
        if (mine && i >= a.weights_width)
            flag(a.b.err, DSV4_DEVERR_SLOT_RANGE);
        const bool add = mine && i < a.weights_width;
        float *to = a.weights + int64_t(sw.c.request) * a.weights_stride + i;
        const float before = add ? ld_f32_now_in(to, ws, a.b.err) : 0.0f;
        const bool failed = !mbar_wait(&s.scores[t & 1], (t / 2) & 1);
        if (named_barrier_any(1, 256, failed)) {
            flag(a.b.err, DSV4_DEVERR_TIMEOUT);
            return;
        }
        tmem_fence_after();
        // every row of the group sees every key of the tile
        const bool whole = !some_out && rows >= col0 + kCols && (tile + 1) * kTileKeys <= s.seen_to[col0] &&
                           tile * kTileKeys >= s.seen_from[col0 + kCols - 1];
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j0 = 0; j0 < kCols; j0 += 32) {
            if (col0 + j0 >= rows)
                break;
            float v[32];
            tmem_load16(tmem + (t & 1) * kRows + col0 + j0, v);
            tmem_load16(tmem + (t & 1) * kRows + col0 + j0 + 16, v + 16);
            tmem_wait_load();
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
                const float4 l = *reinterpret_cast<const float4 *>(&s.lse[col0 + j0 + j]);
                v[j] = exp2_approx(__fmaf_rn(v[j], scale, -l.x));
                v[j + 1] = exp2_approx(__fmaf_rn(v[j + 1], scale, -l.y));
                v[j + 2] = exp2_approx(__fmaf_rn(v[j + 2], scale, -l.z));
                v[j + 3] = exp2_approx(__fmaf_rn(v[j + 3], scale, -l.w));
            }
            if (!whole) {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (i >= s.seen_to[col0 + j0 + j] || i < s.seen_from[col0 + j0 + j])
                        v[j] = 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 32; ++j)
                sum[j & 3] += v[j];
        }
        tmem_fence_before();
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&s.scores_free[t & 1]);
        const float total = (sum[0] + sum[1]) + (sum[2] + sum[3]);
        if (group == 1)
            s.part[key] = total;
        named_barrier(1, 256);
        if (add && ((s.key_ok[t % kOkTiles][warp] >> lane) & 1u) != 0u)
            st_f32_in(to, before + (total + s.part[key]), ws, a.b.err);
        sw.advance(w);
    }
}

__global__ void __launch_bounds__(kThreads, 1) fp4_weights_kernel(const __grid_constant__ WParams w)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    Shared &s = *reinterpret_cast<Shared *>(smem + kShared);
    const int warp = threadIdx.x >> 5;
    Sweep sw;
    wait_for_kernel_before();
    Tiles::deal(w.p, blockIdx.x, gridDim.x, s.scratch, sw.c);
    if (sw.c.left == 0)
        return;
    if ((smem_addr(smem) & 1023u) != 0u) {  // never: there is no static shared memory
        flag(w.p.a.b.err, DSV4_DEVERR_TIMEOUT);
        return;
    }
    sw.begin();
    if (warp == kMultiplyWarp) {
        tmem_alloc512(&s.tmem);
        if ((threadIdx.x & 31) == 0) {
            for (int i = 0; i < 4; ++i) {
                mbar_init(&s.staged[i], 4);
                mbar_init(&s.staged_free[i], 1);
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(&s.scores[i], 1);
                mbar_init(&s.scores_free[i], 4 * kGroups);
            }
            mbar_init(&s.query, 16);
            mbar_init(&s.query_free, 1);
            mbar_init_fence();
        }
        tmem_fence_before();
    }
    __syncthreads();
    tmem_fence_after();
    if (warp < kConvertWarp) {
        sum_role(w, s, sw);
    } else if (warp < kMultiplyWarp) {
        convert_role(w, s, smem, sw, (warp - kConvertWarp) / 4);
    } else if (warp == kMultiplyWarp) {
        multiply_role(w, s, smem_addr(smem), sw);
    }
    tmem_fence_before();
    __syncthreads();
    if (warp == kMultiplyWarp) {
        tmem_fence_after();
        tmem_free512(s.tmem);
    }
}

int configure(int *sms)
{
    static std::atomic<int> sm_count[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return DSV4_ERR_CUDA;
    const bool cached = dev >= 0 && dev < 64;
    *sms = cached ? sm_count[dev].load(std::memory_order_relaxed) : 0;
    if (*sms > 0)
        return DSV4_OK;
    if (cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || *sms < 1 ||
        cudaFuncSetAttribute(fp4_weights_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             int(kSmemBytes)) != cudaSuccess)
        return DSV4_ERR_CUDA;
    if (cached)
        sm_count[dev].store(*sms, std::memory_order_relaxed);
    return DSV4_OK;
}

}  // namespace

int launch_fp4_weights(const AttentionArgs &a, cudaStream_t stream)
{
    int sms = 0;
    if (configure(&sms) != DSV4_OK)
        return DSV4_ERR_CUDA;
    WParams w;
    w.p = tile_params(a, a.q_len * a.heads);
    w.passes = (w.p.all_rows + kRows - 1) / kRows;
    const int64_t most = (int64_t(a.b.width) * a.b.block_size + kTileKeys - 1) / kTileKeys * w.p.units;
    return launch_after(fp4_weights_kernel, dim3(unsigned(most < sms ? most : sms)), dim3(kThreads),
                        stream, w, kSmemBytes);
}

}  // namespace dsv4

DSV4_BOUNDS_FLAG_READER(bounds_flag_fp4_weights)
