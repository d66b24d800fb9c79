// Rotation of rows by a table of cosines and sines: (a, b) -> (a cos - b sin, b cos + a sin) for
// the pairs of a row's rotated dims, or with -sin, which is the gradient and, by a table of magnitude 1,
// the inverse; in fp32 with one rounding to the row's type.  In place only the rotated dims are touched; out of place
// the others are copied.
//
// Bound by memory.  A thread has one column (a vector of 16 bytes; two of them in the half
// layout, one from either half of the rotated dims) of one or two rows at once.  Two rows of one
// token share the table's values, which come from L1 and L2.  Where a size, a stride or an address is
// not a multiple of 16 bytes, a column is one pair or one copied element.
//
// 16383 tokens of 32 heads of 128 fp16, 64 dims of them turned in halves out of place, take 51.5 us
// (80% of a copy's rate).  What counts is how many loads an SM holds: with ten CTAs of 128 threads
// (48 registers) 51.5 us, of 256 threads five 53 and as many as 60 registers let 56; four rows
// at once 61, one 74.5; two rows of different tokens, each with its table's row, 58.

#include <cuda_runtime.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "bounds.cuh"
#include "convert.cuh"
#include "fastdiv.h"
#include "launch_status.h"
#include "ops.h"

namespace dsv4 {
namespace {

constexpr int kRowThreads = 128;

struct RowParams {
    RopeRowsArgs a;
    int32_t columns;   // of a row: first those that turn, then those that are copied
    int32_t turned;
    int32_t lanes;     // columns that a CTA has at once
    uint32_t slots;    // rows that it has at once
    uint64_t lane_div, head_div;
    int64_t rows;
    uint64_t x_bytes, out_bytes;  // from the first element to behind the last
};

// elements of a vector as fp32, and back
template <int kType>
__device__ __forceinline__ void unpack(uint4 v, float *f)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (kType == DSV4_TYPE_FP32) {
            f[i] = __uint_as_float(w[i]);
        } else if constexpr (kType == DSV4_TYPE_BF16) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        } else {
            f[2 * i] = __half2float(__ushort_as_half(uint16_t(w[i])));
            f[2 * i + 1] = __half2float(__ushort_as_half(uint16_t(w[i] >> 16)));
        }
    }
}

template <int kType>
__device__ __forceinline__ uint32_t half_bits(float f)
{
    return kType == DSV4_TYPE_BF16 ? bf16x2_rn(f, 0.0f) & 0xffffu : uint32_t(__half_as_ushort(__float2half_rn(f)));
}

template <int kType>
__device__ __forceinline__ uint4 pack(const float *f)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (kType == DSV4_TYPE_FP32)
            w[i] = __float_as_uint(f[i]);
        else if constexpr (kType == DSV4_TYPE_BF16)
            w[i] = bf16x2_rn(f[2 * i], f[2 * i + 1]);
        else
            w[i] = half_bits<kType>(f[2 * i]) | half_bits<kType>(f[2 * i + 1]) << 16;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// a vector, or one element in its first bits
template <int kType, bool kVector>
__device__ __forceinline__ uint4 load_some(const uint8_t *p, Span s, int32_t *err)
{
    if constexpr (kVector)
        return ld16_in(p, s, err);
    else if constexpr (kType == DSV4_TYPE_FP32)
        return make_uint4(ld4_in(p, s, err), 0u, 0u, 0u);
    else
        return make_uint4(ld2_in(p, s, err), 0u, 0u, 0u);
}

template <int kType, bool kVector>
__device__ __forceinline__ void store_some(uint8_t *p, uint4 v, Span s, int32_t *err)
{
    if constexpr (kVector)
        st16_in(p, v, s, err);
    else if constexpr (kType == DSV4_TYPE_FP32)
        st4_in(p, v.x, s, err);
    else
        st2_in(p, v.x, s, err);
}

// kCount (1, 2, 4 or 8) fp32 of the table, aligned to as many up to four
template <int kCount>
__device__ __forceinline__ void load_table(const float *p, Span s, int32_t *err, float *f)
{
    if constexpr (kCount >= 4) {
#pragma unroll
        for (int i = 0; i < kCount; i += 4) {
            const float4 v = ldg_f4_in(p + i, s, err);
            f[i] = v.x;
            f[i + 1] = v.y;
            f[i + 2] = v.z;
            f[i + 3] = v.w;
        }
    } else if constexpr (kCount == 2) {
        const uint2 v = ldg8_in(p, s, err);
        f[0] = __uint_as_float(v.x);
        f[1] = __uint_as_float(v.y);
    } else {
        f[0] = ldg_f32_in(p, s, err);
    }
}

template <int kType, bool kVector, bool kHalf, int kRowsAtOnce, bool kOneToken>
__global__ void __launch_bounds__(kRowThreads, 10) rope_rows_kernel(const __grid_constant__ RowParams p)
{
    constexpr int kSize = kType == DSV4_TYPE_FP32 ? 4 : 2;
    constexpr int kElems = kVector ? 16 / kSize : 1;
    constexpr bool kTwo = kHalf || !kVector;                // a column that turns is two vectors
    constexpr int kPairs = kHalf || !kVector ? kElems : kElems / 2;  // of such a column
    const RopeRowsArgs &a = p.a;
    wait_for_kernel_before();
    const uint32_t slot = fastdiv(threadIdx.x, p.lane_div);
    if (slot >= p.slots)
        return;
    const int half = a.rope_dim / 2;
    const Span xs{a.x, p.x_bytes}, os{a.out, p.out_bytes};
    const Span ts{a.cos_sin, uint64_t(a.max_position) * uint32_t(a.rope_dim) * 4u};
    // a thread's rows: one after the other if they are one token's, else with the CTA's others between
    const int64_t row0 = int64_t(blockIdx.x) * (p.slots * kRowsAtOnce) + slot * (kOneToken ? kRowsAtOnce : 1);
    const uint32_t step = kOneToken ? 1u : p.slots;
    for (int column = threadIdx.x - slot * p.lanes; column < p.columns; column += p.lanes) {
        const bool turns = column < p.turned;
        // the column's first elements, and the pair that they begin with
        int at, pair = 0;
        if (turns) {
            pair = column * kPairs;
            at = a.offset + (kTwo && !kHalf ? 2 * column : column * kElems);
        } else {
            at = (column - p.turned) * kElems;
            at += at >= a.offset ? a.rope_dim : 0;
        }
        const int other = kHalf ? half : 1;
        int64_t x_at[kRowsAtOnce], out_at[kRowsAtOnce], position[kRowsAtOnce];
        bool live[kRowsAtOnce];
        uint4 first[kRowsAtOnce], second[kRowsAtOnce];
#pragma unroll
        for (int u = 0; u < kRowsAtOnce; ++u) {
            const int64_t row = row0 + int64_t(u) * step;
            live[u] = row < p.rows;
            if (!live[u])
                continue;
            const uint32_t token = fastdiv(uint32_t(row), p.head_div), head = uint32_t(row) - token * uint32_t(a.heads);
            if (!kOneToken || u == 0)
                position[u] = ldg_i64_in(a.positions + token, Span{a.positions, uint64_t(a.tokens) * 8u}, a.err);
            else
                position[u] = position[0];
            x_at[u] = (token * a.x_token_stride + head * a.x_head_stride + at) * kSize;
            out_at[u] = (token * a.out_token_stride + head * a.out_head_stride + at) * kSize;
            first[u] = load_some<kType, kVector>(a.x + x_at[u], xs, a.err);
            if (kTwo && turns)
                second[u] = load_some<kType, kVector>(a.x + x_at[u] + other * kSize, xs, a.err);
        }
        float c[kPairs], s[kPairs];
#pragma unroll
        for (int u = 0; u < kRowsAtOnce; ++u) {
            if (!live[u])
                continue;
            if (position[u] < 0 || position[u] >= a.max_position) {
                if (column == 0 && a.err != nullptr)
                    atomicOr(a.err, DSV4_DEVERR_POS_RANGE);
                continue;
            }
            if (turns) {
                if (!kOneToken || u == 0) {
                    const float *angles = a.cos_sin + position[u] * a.rope_dim + pair;
                    load_table<kPairs>(angles, ts, a.err, c);
                    load_table<kPairs>(angles + half, ts, a.err, s);
                }
                float f[2 * 8], g[8];
                unpack<kType>(first[u], f);
                if constexpr (kTwo)
                    unpack<kType>(second[u], g);
#pragma unroll
                for (int k = 0; k < kPairs; ++k) {
                    const float sine = a.inverse ? -s[k] : s[k];
                    float &even = kTwo ? f[k] : f[2 * k], &odd = kTwo ? g[k] : f[2 * k + 1];
                    const float turned = __fmaf_rn(even, c[k], -__fmul_rn(odd, sine));
                    odd = __fmaf_rn(odd, c[k], __fmul_rn(even, sine));
                    even = turned;
                }
                first[u] = pack<kType>(f);
                if constexpr (kTwo)
                    second[u] = pack<kType>(g);
            }
            store_some<kType, kVector>(a.out + out_at[u], first[u], os, a.err);
            if (kTwo && turns)
                store_some<kType, kVector>(a.out + out_at[u] + other * kSize, second[u], os, a.err);
        }
    }
}

template <int kType, bool kVector, bool kHalf, int kRowsAtOnce, bool kOneToken>
int launch_rows(const RowParams &p, cudaStream_t stream)
{
    const int64_t per = int64_t(p.slots) * kRowsAtOnce;
    return launch_after(rope_rows_kernel<kType, kVector, kHalf, kRowsAtOnce, kOneToken>,
                        dim3(unsigned((p.rows + per - 1) / per)), dim3(kRowThreads), stream, p);
}

template <int kType, bool kVector, bool kHalf>
int launch_kind(const RowParams &p, cudaStream_t stream)
{
    // Two rows at once where that still gives each SM eight CTAs, else one: 800 tokens of 32 heads of
    // 128 dims in halves take 3.6 us by one and 3.7 by two, 1600 of them 5.9 and 5.7; 600 of 64 dims in
    // pairs 1.85 and 1.86, 4000 of them 6.3 and 5.4.
    if constexpr (kVector) {
        if (p.rows / (int64_t(p.slots) * 2) >= 8 * p.a.sms)
            return p.a.heads % 2 == 0 ? launch_rows<kType, true, kHalf, 2, true>(p, stream)
                                      : launch_rows<kType, true, kHalf, 2, false>(p, stream);
    }
    return launch_rows<kType, kVector, kHalf, 1, false>(p, stream);
}

template <int kType>
int launch_type(const RowParams &p, bool vector, cudaStream_t stream)
{
    const bool half = p.a.layout == DSV4_ROPE_HALF;
    if (vector)
        return half ? launch_kind<kType, true, true>(p, stream) : launch_kind<kType, true, false>(p, stream);
    return half ? launch_kind<kType, false, true>(p, stream) : launch_kind<kType, false, false>(p, stream);
}

}  // namespace

int launch_rope_rows(const RopeRowsArgs &a, cudaStream_t stream)
{
    RowParams p;
    p.a = a;
    const bool in_place = a.x == a.out, half = a.layout == DSV4_ROPE_HALF;
    const int size = a.type == DSV4_TYPE_FP32 ? 4 : 2, elems = 16 / size;
    const auto whole = [&](int64_t n) { return n % elems == 0; };
    const bool vector = ((reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.out)) & 15u) == 0u &&
                        whole(a.x_token_stride) && whole(a.x_head_stride) && whole(a.out_token_stride) &&
                        whole(a.out_head_stride) && whole(a.offset) && whole(half ? a.rope_dim / 2 : a.rope_dim) &&
                        (in_place || whole(a.width));
    const int unit = vector ? elems : 1;
    p.turned = vector ? (half ? a.rope_dim / 2 : a.rope_dim) / unit : a.rope_dim / 2;
    p.columns = p.turned + (in_place ? 0 : (a.width - a.rope_dim) / unit);
    p.lanes = p.columns < kRowThreads ? p.columns : kRowThreads;
    p.slots = uint32_t(kRowThreads / p.lanes);
    p.lane_div = fastdiv_magic(uint32_t(p.lanes));
    p.head_div = fastdiv_magic(uint32_t(a.heads));
    p.rows = a.tokens * a.heads;
    p.x_bytes = uint64_t((a.tokens - 1) * a.x_token_stride + (a.heads - 1) * a.x_head_stride + a.width) * size;
    p.out_bytes = uint64_t((a.tokens - 1) * a.out_token_stride + (a.heads - 1) * a.out_head_stride + a.width) * size;
    switch (a.type) {
    case DSV4_TYPE_BF16: return launch_type<DSV4_TYPE_BF16>(p, vector, stream);
    case DSV4_TYPE_FP16: return launch_type<DSV4_TYPE_FP16>(p, vector, stream);
    default: return launch_type<DSV4_TYPE_FP32>(p, vector, stream);
    }
}

}  // namespace dsv4

DSV4_BOUNDS_FLAG_READER(bounds_flag_rope_rows)
