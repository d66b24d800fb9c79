// What the attention over the 4-bit cache and the attention weights share: their tiles of
// keys, and how a tile of cache rows becomes a bf16 matrix operand.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "bounds.cuh"
#include "fp4.cuh"
#include "key_tiles.cuh"
#include "ops.h"
#include "tcgen05.cuh"

namespace dsv4 {
namespace {

constexpr int kTileKeys = 128;
constexpr int kChunks = 8;                    // a row in chunks of 64 dims: 7 of codes, 1 of rope
constexpr uint32_t kChunkBytes = kTileKeys * 128;

__device__ __forceinline__ Span cache_span(const PagedBatch &b)
{
    return Span{b.cache, uint64_t(b.num_blocks) * uint32_t(b.block_size) * kFp4Slot};
}

// Positions that beginning a unit takes: 0, 1, 2, 3, 4, 6 of them:
// attention over 48 requests of 64 to 4096 keys 47.9, 47.3, 41.0, 40.3, 40.1, 43.3 us;
// 24 of 1 to 6000 in windows of 2048 with three tokens 68, 47, 43, 46, 47, 51; 128 of
// 1024 to 8192 258, 252, 240, 245, 246, 248; the weights over the first gain
// nothing (24.2 without and 23.4 with it on one resident input, 24.9 and 25.3 on changing ones).
using Tiles = KeyTiles<kTileKeys, kFp4StartCost, false>;
using Range = Tiles::Range;
using Cursor = Tiles::Cursor;

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

}  // namespace
}  // namespace dsv4
