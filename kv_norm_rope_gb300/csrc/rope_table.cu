// The table of cosines and sines that the inserts and the rotation take: row p, pair i holds
// magnitude * cos(p f_i) and magnitude * sin(p f_i).
//
// The angle is held in turns: g_i is f_i / 2 pi modulo 1 as a 64-bit fraction, and p g_i modulo 1
// is the low half of an integer product, exact but for p times g_i's half unit (2^-33 turns for
// the farthest p).  A turn is cut into kTurnPoints arcs; with a the nearest point and b the rest
// (|b| <= pi / kTurnPoints),
//   cos(a + b) = cos a + (cos a (cos b - 1) - sin a sin b),   sin(a + b) alike,
// where sin b and cos b - 1 are the first terms of their series (the first left out is below
// 2^-40), and cos a and sin a are pairs of floats.  What is rounded before the last addition is
// below 2^-5 of the result's largest, so entries are within 0.6 steps of 1.
//
// Bound by its stores (8 bytes a pair): 1048576 rows of 64 columns take 40.8 us (98% of a copy's rate),
// 52 with positions given in any order.  With one copy of the points instead of eight their loads met in
// banks (46 us).  CTAs an SM, each with its part of the rows: 2 take 40 and 72 us, 3 41 and 58, 6 40 and
// 49 but more where the table is small (100000 rows: 6.6 by 4, 7.1 by 6).

#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "bounds.cuh"
#include "fastdiv.h"
#include "launch_status.h"
#include "ops.h"

namespace dsv4 {
namespace {

constexpr int kPointBits = 7;
constexpr int kPoints = 1 << kPointBits;
constexpr int kTableThreads = 256;
constexpr int kCtasPerSm = 4;

struct TableParams {
    float4 points[kPoints];           // magnitude * (cos high, cos low, sin high, sin low)
    uint64_t turns[kMaxRopeDim / 2];  // g_i
    float *out;
    const int64_t *positions;         // or null: first, first + 1, ...
    int64_t first, count;
    int32_t pairs;                    // of a row
    uint64_t group_div;               // fastdiv_magic of a row's groups of kPairs pairs
    int32_t *err;
};
static_assert(sizeof(TableParams) <= 4000, "kernel parameters");

template <int kPairs>
__global__ void __launch_bounds__(kTableThreads) rope_table_kernel(const __grid_constant__ TableParams p)
{
    // eight copies, each in its own banks: no two lanes that load at once meet in one
    __shared__ float4 points[kPoints * 8];
    for (int i = threadIdx.x; i < kPoints * 8; i += kTableThreads)
        points[i] = p.points[i >> 3];
    __syncthreads();
    wait_for_kernel_before();
    const uint32_t groups = uint32_t(p.pairs) / kPairs, rows = kTableThreads / groups;
    // the thread has the same pairs of every row it takes
    const uint32_t local = fastdiv(threadIdx.x, p.group_div), first = (threadIdx.x - local * groups) * kPairs;
    if (local >= rows)
        return;
    uint64_t turns[kPairs];
#pragma unroll
    for (int k = 0; k < kPairs; ++k)
        turns[k] = p.turns[first + k];
    const Span os{p.out, uint64_t(p.count) * uint32_t(p.pairs) * 8u};
    const int64_t step = int64_t(gridDim.x) * rows;
    const auto position = [&](int64_t row) {
        if (p.positions == nullptr)
            return p.first + row;
        if (row >= p.count)
            return int64_t(0);
        const uint2 v = ldg8_now_in(p.positions + row, Span{p.positions, uint64_t(p.count) * 8u}, p.err);
        return int64_t(uint64_t(v.y) << 32 | v.x);
    };
    int64_t next = position(int64_t(blockIdx.x) * rows + local);
    for (int64_t row = int64_t(blockIdx.x) * rows + local; row < p.count; row += step) {
        const int64_t at = next;
        next = position(row + step);  // on its way meanwhile
        if ((uint64_t(at) >> 32) != 0u) {
            if (p.err != nullptr)
                atomicOr(p.err, DSV4_DEVERR_POS_RANGE);
            continue;
        }
        float c[kPairs], s[kPairs];
#pragma unroll
        for (int k = 0; k < kPairs; ++k) {
            const uint64_t angle = uint64_t(at) * turns[k];
            // the nearest point, and what is left in 2^-39 turns
            const uint32_t point = (uint32_t(angle >> 32) + (1u << (31 - kPointBits))) >> (32 - kPointBits);
            const int32_t rest = int32_t(uint32_t(angle >> (32 - kPointBits)));
            const float b = float(rest) * (6.283185307179586f * 0x1p-39f), b2 = b * b;
            const float sin_b = __fmaf_rn(b * b2, __fmaf_rn(b2, 1.0f / 120.0f, -1.0f / 6.0f), b);
            const float cos_b1 = b2 * __fmaf_rn(b2, 1.0f / 24.0f, -0.5f);
            const float4 a = points[(point & (kPoints - 1)) * 8 + (threadIdx.x & 7)];
            c[k] = a.x + __fmaf_rn(-a.z, sin_b, __fmaf_rn(a.x, cos_b1, a.y));
            s[k] = a.z + __fmaf_rn(a.x, sin_b, __fmaf_rn(a.z, cos_b1, a.w));
        }
        float *to = p.out + row * (2 * p.pairs) + first;
        if constexpr (kPairs == 4) {
            st_f4_in(to, make_float4(c[0], c[1], c[2], c[3]), os, p.err);
            st_f4_in(to + p.pairs, make_float4(s[0], s[1], s[2], s[3]), os, p.err);
        } else {
            st_f32_in(to, c[0], os, p.err);
            st_f32_in(to + p.pairs, s[0], os, p.err);
        }
    }
}

// f / 2 pi modulo 1 as a 64-bit fraction, to the nearest; f finite, 0 <= f < 2^16
uint64_t turns_of(double f)
{
    // 1 / 2 pi = 0.28BE60DB 9391054A 7F09D5F4 7D4D3770 36D8... in base 16
    constexpr uint64_t kHigh = 0x28BE60DB9391054Aull, kLow = 0x7F09D5F47D4D3770ull;
    int e = 0;
    const double fraction = std::frexp(f, &e);  // f = fraction * 2^e, fraction in [1/2, 1)
    if (fraction == 0.0)
        return 0;
    const uint64_t m = uint64_t(std::ldexp(fraction, 53));  // f = m * 2^(e - 53)
    // m / 2 pi in units of 2^-128
    typedef unsigned __int128 Wide;
    const Wide low = Wide(m) * kLow, high = Wide(m) * kHigh + uint64_t(low >> 64);
    const uint64_t words[3] = {uint64_t(low), uint64_t(high), uint64_t(high >> 64)};  // 2^-128, 2^-64, 1
    // times 2^(e - 53): the fraction's 64 bits begin 53 - e bits above those of 2^-64
    const int up = 53 - e;  // 37 .. 53 + 1022 and more for tiny f
    if (up >= 128)
        return 0;
    const auto word = [&](int i) { return i < 3 ? words[i] : uint64_t(0); };
    const int at = 1 + up / 64, bit = up % 64;
    const uint64_t below = bit == 0 ? word(at - 1) >> 63 : (word(at) >> (bit - 1)) & 1u;
    return (bit == 0 ? word(at) : (word(at) >> bit) | (word(at + 1) << (64 - bit))) + below;
}

// cos and sin of the points in 64 bits, by the host's library
struct Points {
    double cos[kPoints], sin[kPoints];
    Points()
    {
        for (int i = 0; i < kPoints; ++i) {
            // from the first eighth of the turn, where both are exact at the ends
            const int eighth = i / (kPoints / 8), in = i % (kPoints / 8);
            const double a = 6.283185307179586476925 / kPoints * ((eighth & 1) ? kPoints / 8 - in : in);
            double c = std::cos(a), s = std::sin(a);
            if (((eighth + 1) & 2) != 0) {  // beyond pi/4 of the quarter's nearer axis
                const double t = c;
                c = s;
                s = t;
            }
            cos[i] = eighth >= 2 && eighth < 6 ? -c : c;
            sin[i] = eighth >= 4 ? -s : s;
        }
    }
};

}  // namespace

int launch_rope_table(const RopeTableArgs &a, cudaStream_t stream)
{
    static const Points points;
    TableParams p;
    for (int i = 0; i < kPoints; ++i) {
        const double c = points.cos[i] * a.magnitude, s = points.sin[i] * a.magnitude;
        const float ch = float(c), sh = float(s);
        p.points[i] = make_float4(ch, float(c - ch), sh, float(s - sh));
    }
    p.pairs = a.rope_dim / 2;
    for (int i = 0; i < p.pairs; ++i)
        p.turns[i] = turns_of(a.frequencies[i]);
    p.out = a.out;
    p.positions = a.positions;
    p.first = a.first;
    p.count = a.count;
    p.err = a.err;
    const bool four = p.pairs % 4 == 0 && (reinterpret_cast<uintptr_t>(a.out) & 15u) == 0u;
    const int groups = four ? p.pairs / 4 : p.pairs;
    p.group_div = fastdiv_magic(uint32_t(groups));
    const int64_t rows = kTableThreads / groups, most = int64_t(a.sms) * kCtasPerSm;
    const int64_t ctas = (a.count + rows - 1) / rows;
    return launch_after(four ? rope_table_kernel<4> : rope_table_kernel<1>, dim3(unsigned(ctas < most ? ctas : most)),
                        dim3(kTableThreads), stream, p);
}

}  // namespace dsv4

DSV4_BOUNDS_FLAG_READER(bounds_flag_rope_table)
