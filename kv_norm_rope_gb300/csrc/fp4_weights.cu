// The attention that each key of the 4-bit cache gets.

#include <cuda_runtime.h>
#include <stdint.h>

#include "fp4.cuh"
#include "launch_status.h"
#include "ops.h"

namespace dsv4 {
namespace {

constexpr unsigned kFull = 0xffffffffu;

struct AParams {
    Fp4AttentionArgs a;
    uint64_t block_div;
};

__device__ __forceinline__ Span cache_span(const Fp4Batch &b)
{
    return Span{b.cache, uint64_t(b.num_blocks) * uint32_t(b.block_size) * kFp4Slot};
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

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1)
        v += __shfl_xor_sync(kFull, v, m);
    return v;
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

// dims [8l, 8l+8) and [256+8l, 256+8l+8) of key i of request r as fp32; false for a bad block
__device__ __forceinline__ bool load_key(const AParams &p, int lane, int r, int i, float *x)
{
    const Fp4Batch &b = p.a.b;
    const uint32_t at = fastdiv(uint32_t(i), p.block_div);
    const int32_t *entry = b.table + r * b.table_stride + at;
    const uint32_t blk = ldg4_in(entry, Span{b.table, (uint64_t(b.batch - 1) * b.table_stride + b.width) * 4u}, b.err);
    if (int64_t(blk) >= b.num_blocks) {
        flag(b.err, DSV4_DEVERR_SLOT_RANGE);
        return false;
    }
    const Fp4Row row = fp4_row(b.cache, blk, uint32_t(i) - at * uint32_t(b.block_size), uint32_t(b.block_size));
    const Span cs = cache_span(b);
    const uint32_t e0 = ldg_byte_in(row.scale + (lane >> 2), cs, b.err);
    widen8(fp4x8_to_bf16(ldg4_in(row.data + 4 * lane, cs, b.err), fp4_scale_bf16x2(e0)), x);
    if (lane < 24) {
        const uint32_t e1 = ldg_byte_in(row.scale + 8 + (lane >> 2), cs, b.err);
        widen8(fp4x8_to_bf16(ldg4_in(row.data + 128 + 4 * lane, cs, b.err), fp4_scale_bf16x2(e1)), x + 8);
    } else {
        widen8(ldg16_in(row.data + kFp4Codes + 16 * (lane - 24), cs, b.err), x + 8);
    }
    return true;
}

__device__ __forceinline__ float dot16(const float *x, const float *y)
{
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        s = __fmaf_rn(x[i], y[i], s);
    return warp_sum(s);
}

// one warp per key, the rows in order
__global__ void __launch_bounds__(128) fp4_weights_kernel(const AParams p)
{
    const Fp4AttentionArgs &a = p.a;
    const int lane = threadIdx.x & 31;
    const int r = blockIdx.y;
    const int n = length_of(a.b, r);
    if (n > a.weights_width)
        flag(a.b.err, DSV4_DEVERR_SLOT_RANGE);
    const int most = n < a.weights_width ? n : a.weights_width;
    const Span qs{a.q, rows_of(a) * 1024u}, ls{a.lse, rows_of(a) * 4u};
    const Span ws{a.weights, (uint64_t(a.b.batch - 1) * a.weights_stride + a.weights_width) * 4u};
    for (int i = int(blockIdx.x) * 4 + (threadIdx.x >> 5); i < most; i += int(gridDim.x) * 4) {
        float x[16];
        if (!load_key(p, lane, r, i, x))
            continue;
        float sum = 0.0f;
        for (int j = 0; j < a.q_len; ++j) {
            const int to = n - a.q_len + 1 + j;
            if (i >= to || (a.window > 0 && i < to - a.window))
                continue;
            for (int h = 0; h < a.heads; ++h) {
                const int64_t row = (int64_t(r) * a.q_len + j) * a.heads + h;
                float q[16];
                widen8(ldg16_in(a.q + row * 512 + 8 * lane, qs, a.b.err), q);
                widen8(ldg16_in(a.q + row * 512 + 256 + 8 * lane, qs, a.b.err), q + 8);
                const float lse = ldg_f32_in(a.lse + row, ls, a.b.err);
                const float s = dot16(q, x) * a.scale;
                sum += lse == -INFINITY ? 0.0f : expf(s - lse);
            }
        }
        float *w = a.weights + r * a.weights_stride + i;
        if (lane == 0)
            st_f32_in(w, ld_f32_in(w, ws, a.b.err) + sum, ws, a.b.err);
    }
}

}  // namespace

int launch_fp4_weights(const Fp4AttentionArgs &a, cudaStream_t stream)
{
    AParams p{a, fastdiv_magic(uint32_t(a.b.block_size))};
    return launch_kernel(fp4_weights_kernel, dim3(1024, unsigned(a.b.batch)), dim3(128), 0, stream, p);
}

}  // namespace dsv4

DSV4_BOUNDS_FLAG_READER(bounds_flag_fp4_weights)
