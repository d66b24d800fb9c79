// The attention each key of the 4-bit cache gets: weights[key] += the sum over query
// rows of exp(scale * q . k - lse).
//
// The first product of the attention (fp4_attention.cu) with another end: S^T[key,
// row] = K q^T on the tensor cores, keys in the lanes, so a thread holds one key and
// its sum over rows needs no exchange.  2 * 512 multiplications a (row, key), no
// second product, and nothing for the matrix unit to wait for but converted rows:
//
//  * 128 query rows a pass (N = 128: the rows' operand then costs the matrix unit no
//    more shared-memory reads than it has time for).  More rows take more passes
//    over the same run of keys, whose bytes then come from L2.
//  * The tile passes through two slots of two chunks, one for each converting team,
//    so a chunk is converted while the one before is multiplied; S^T has two
//    places, so the sums of a tile run under the product of the next.
//  * Each key's sum is finished by one thread of one CTA in a fixed order of rows
//    and added by it: no atomics, the same bits every time.

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
constexpr int kThreads = (kMultiplyWarp + 4) * 32;  // whole warpgroups: three warps idle
// registers a thread: 72 at launch, then (the converting warps spill below this, and
// spills go to L2: shared memory leaves little of L1)
constexpr int kSumRegs = 72 /* as launched */, kConvertRegs = 80, kMultiplyRegs = 40;
static_assert(128 * (kGroups * kSumRegs + 4 * kConvertRegs + kMultiplyRegs) <= kThreads * 72,
              "the shares exceed what the CTA was launched with");
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kOkTiles = 4;

// Shared memory (from a 1024-byte boundary).
constexpr uint32_t kSlotBytes = 2 * kChunkBytes;                // a pair of chunks
constexpr uint32_t kQuery = 2 * kSlotBytes;                     // 8 chunks of 128 rows
constexpr uint32_t kRing = kQuery + kChunks * kRows * 128;      // codes on their way
constexpr uint32_t kShared = kRing + 2 * kRingSlot;

struct Shared {
    uint64_t full[2], free[2], scores[2], scores_free[2], query, query_free;
    uint32_t tmem;
    int scratch[18];
    alignas(16) float lse[kRows];
    int seen_to[kRows], seen_from[kRows];
    float part[kTileKeys];
    uint8_t key_ok[kOkTiles][kTileKeys];
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

template <int team>
__device__ __forceinline__ void convert_role(const WParams &w, Shared &s, uint8_t *smem, Sweep sw)
{
    const AParams &p = w.p;
    const int tid = threadIdx.x - kConvertWarp * 32 - team * kTeam;
    const int key = tid >> 1, half = tid & 1, lane = tid & 31;
    const uint32_t base = smem_addr(smem), slot = base + kRing + team * kRingSlot;
    const uint32_t place = swizzled(key, 4 * half), to = base + team * kSlotBytes;
    KeyPlace now = key_place(p, sw.at(), true, key);
    int now_pass = 0;
    Fp4Row row = row_at(p, now);
    copy_codes<team>(p, slot, tid, row);
    uint4 scales = load_raw(p, row.scale, row.data != nullptr);
    sw.advance(w);
    KeyPlace next = key_place(p, sw.at(), sw.new_pass, key);
    bool next_live = sw.live;
    int next_pass = sw.pass;
    uint32_t passes = 0;
    for (uint32_t t = 0;; ++t) {
        const Fp4Row next_row = row_at(p, next);
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
        const uint4 next_scales = load_raw(p, next_row.scale, next_row.data != nullptr);
        if constexpr (team == 1)
            prefetch64(p, row.data + kFp4Codes + 64 * half, row.data != nullptr);
        bool alive = true;
        if (now.unit < 0) {
            if (passes > 0)
                alive = __all_sync(kFull, mbar_wait(&s.query_free, (passes - 1) & 1));
            if (alive) {
                load_query(p, ~now.unit, now_pass * kRows, smem + kQuery, kRows, tid + team * kTeam,
                           2 * kTeam);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&s.query);
            }
            ++passes;
        }
        uint4 rope[4];
        const auto pair = [&](auto ci) {
            constexpr int i = decltype(ci)::value;  // chunks 2i and 2i + 1, this slot's use 2t + i / 2
            const uint32_t use = 2 * t + i / 2;
            copy_wait();
            const uint4 a = load_shared16(slot + tid * 16);
            uint4 b = a, out[4];
            if constexpr (i < 3)
                b = load_shared16(slot + 4096 + tid * 16);
            if constexpr (i < 2)
                copy_codes<i + 2>(p, slot, tid, row);
            else
                copy_codes<i - 2>(p, slot, tid, next_row);
            convert_codes<2 * i>(scales, a, half, out);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                computed(out[k]);  // before the wait for its place
            if (use > 0 && alive)
                alive = __all_sync(kFull, mbar_wait(&s.free[team], (use - 1) & 1));
            if (!alive)
                return;
            if (i == 0 && half == 0)
                s.key_ok[t % kOkTiles][key] = row.data != nullptr ? 1 : 0;
            store_half(to, place, out);
            if constexpr (i < 3) {
                convert_codes<2 * i + 1>(scales, b, half, out);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    out[k] = mul_bf16x8(rope[k], kRopeToOperand);
            }
            store_half(to + kChunkBytes, place, out);
            if constexpr (i == 1) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    rope[k] = load_raw(p, row.data + kFp4Codes + 64 * half + 16 * k, row.data != nullptr);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&s.full[team]);
        };
        pair(std::integral_constant<int, team>{});
        pair(std::integral_constant<int, team + 2>{});
        if (!alive) {
            flag(p.a.b.err, DSV4_DEVERR_TIMEOUT);
            break;
        }
        if (!next_live)
            break;
        scales = next_scales;
        row = next_row;
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
    const Operand keys = operand(smem, 16, 1024), query = operand(smem + kQuery, 16, 1024);
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
            alive = alive && __all_sync(kFull, mbar_wait(&s.full[i & 1], (2 * t + i / 2) & 1));
            if (!alive)
                break;
            tmem_fence_after();
#pragma unroll
            for (int k = 0; k < 8; ++k)
                mma_bf16(d, keys + ((i & 1) * kSlotBytes + (k >> 2) * kChunkBytes + 32 * (k & 3)),
                         query + ((2 * i + (k >> 2)) * kRows * 128 + 32 * (k & 3)), inst, i > 0 || k > 0,
                         elected);
            mma_commit(&s.free[i & 1], elected);
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
    const Fp4AttentionArgs &a = p.a;
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3, group = threadIdx.x >> 7;
    const int key = warp * 32 + lane, col0 = group * kCols, tid = threadIdx.x;
    const uint32_t tmem = s.tmem + (uint32_t(warp * 32) << 16);
    const float scale = a.scale * (kLog2e * kOperandUnit);
    const Span ws{a.weights, (uint64_t(a.b.batch - 1) * a.weights_stride + a.weights_width) * 4u};
    for (uint32_t t = 0; sw.live; ++t) {
        const int rows = pass_rows(w, sw.pass), n = sw.c.n;
        if (sw.new_pass) {
            named_barrier(1, 256);  // the rows before are done with
            if (tid < kRows) {
                const int r = sw.pass * kRows + tid;
                float lse = INFINITY;  // no row: its exponentials are 0
                int to = 0;
                if (tid < rows) {
                    lse = kLog2e * ldg_f32_in(a.lse + int64_t(sw.c.request) * p.all_rows + r,
                                              Span{a.lse, rows_of(a) * 4u}, a.b.err);
                    if (lse == -INFINITY)
                        lse = INFINITY;  // a row that saw nothing adds nothing
                    to = n - a.q_len + 1 + int(fastdiv(uint32_t(r), p.head_div));
                }
                s.lse[tid] = lse;
                s.seen_to[tid] = to;
                s.seen_from[tid] = a.window > 0 ? to - a.window : INT32_MIN;
            }
            named_barrier(1, 256);
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
        const bool whole = rows >= col0 + kCols && (tile + 1) * kTileKeys <= s.seen_to[col0] &&
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
        if (add && s.key_ok[t % kOkTiles][key] != 0)
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
    deal(w.p, blockIdx.x, gridDim.x, s.scratch, sw.c);
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
            for (int i = 0; i < 2; ++i) {
                mbar_init(&s.full[i], 8);
                mbar_init(&s.free[i], 1);
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
        registers_up<kConvertRegs>();
        if (warp < kConvertWarp + 8)
            convert_role<0>(w, s, smem, sw);
        else
            convert_role<1>(w, s, smem, sw);
    } else {
        registers_down<kMultiplyRegs>();
        if (warp == kMultiplyWarp)
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

int launch_fp4_weights(const Fp4AttentionArgs &a, cudaStream_t stream)
{
    int sms = 0;
    if (configure(&sms) != DSV4_OK)
        return DSV4_ERR_CUDA;
    WParams w;
    w.p = tile_params(a, a.q_len * a.heads);
    w.passes = (w.p.all_rows + kRows - 1) / kRows;
    const int64_t most = (int64_t(a.b.width) * a.b.block_size + kTileKeys - 1) / kTileKeys * w.p.units;
    return launch_kernel(fp4_weights_kernel, dim3(unsigned(most < sms ? most : sms)), dim3(kThreads),
                         kSmemBytes, stream, w);
}

}  // namespace dsv4

DSV4_BOUNDS_FLAG_READER(bounds_flag_fp4_weights)
