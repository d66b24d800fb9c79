// C-ABI entry points of the rotary positions: the frequencies (host arithmetic), the table
// and the rotation of rows.

#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <utility>

#include "dsv4kv.h"
#include "hostcheck.h"
#include "ops.h"

namespace {

using dsv4::aligned;

constexpr int kMaxDevices = 64;
std::atomic<int> g_sms[kMaxDevices];

int sm_count(int32_t *sms)
{
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return DSV4_ERR_CUDA;
    const bool cached = dev >= 0 && dev < kMaxDevices;
    n = cached ? g_sms[dev].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1)
            return DSV4_ERR_CUDA;
        if (cached)
            g_sms[dev].store(n, std::memory_order_relaxed);
    }
    *sms = n;
    return DSV4_OK;
}

bool bad_rope_dim(int32_t rope_dim)
{
    return rope_dim < 2 || rope_dim > dsv4::kMaxRopeDim || rope_dim % 2 != 0;
}

// elements from the first of the rows to behind the last; strides to 2^31, tokens and heads below 2^31:
// at most 2^63
uint64_t extent(int64_t tokens, int64_t heads, int64_t width, int64_t token_stride, int64_t head_stride)
{
    return uint64_t(tokens - 1) * uint64_t(token_stride) + uint64_t(heads - 1) * uint64_t(head_stride) + width;
}

// strides that keep the rows of an output apart, whichever of tokens and heads lies inside
bool rows_apart(int64_t tokens, int64_t heads, int64_t width, int64_t token_stride, int64_t head_stride)
{
    const bool heads_inside = (heads == 1 || head_stride >= width) &&
                              (tokens == 1 || token_stride >= (heads - 1) * head_stride + width);
    const bool tokens_inside = (tokens == 1 || token_stride >= width) &&
                               (heads == 1 || head_stride >= (tokens - 1) * token_stride + width);
    return heads_inside || tokens_inside;
}

// For rows that lie apart: whether some of them, moved by `by` > 0 bytes, meet others or themselves.
// Strides and width in bytes.
bool moved_rows_meet(uint64_t by, int64_t tokens, int64_t heads, int64_t width, int64_t token_stride,
                     int64_t head_stride)
{
    int64_t outer = tokens, inner = heads, outer_stride = token_stride, inner_stride = head_stride;
    const bool heads_inside = (heads == 1 || head_stride >= width) &&
                              (tokens == 1 || token_stride >= (heads - 1) * head_stride + width);
    if (!heads_inside) {
        std::swap(outer, inner);
        std::swap(outer_stride, inner_stride);
    }
    // a multiple of each stride, less by `by`, that is below the width
    const auto meets = [&](int64_t rest) {  // of the inner stride
        rest = rest < 0 ? -rest : rest;
        const int64_t j = inner == 1 ? 0 : std::min(rest / inner_stride, inner - 1);
        return rest - j * inner_stride < width || (j + 1 < inner && (j + 1) * inner_stride - rest < width);
    };
    if (by > uint64_t(INT64_MAX))
        return false;
    const int64_t i = outer == 1 ? 0 : std::min(int64_t(by) / outer_stride, outer - 1);
    return meets(int64_t(by) - i * outer_stride) ||
           (i + 1 < outer && meets(int64_t(by) - (i + 1) * outer_stride));
}

}  // namespace

extern "C" {

int dsv4_rope_frequencies(int scaling, int32_t rope_dim, double theta, double factor,
                          double original_positions, double turns_fast, double turns_slow, double *frequencies)
{
    if (bad_rope_dim(rope_dim))
        return DSV4_ERR_SHAPE;
    if (scaling < DSV4_ROPE_PLAIN || scaling > DSV4_ROPE_YARN || !std::isfinite(theta) || !(theta > 1.0) ||
        theta > 1e12)
        return DSV4_ERR_VALUE;
    if (scaling != DSV4_ROPE_PLAIN && (!(factor >= 1.0) || !(factor <= 1e6)))
        return DSV4_ERR_VALUE;
    if (scaling == DSV4_ROPE_YARN &&
        (!(original_positions > 0.0) || !std::isfinite(original_positions) || !(turns_slow > 0.0) ||
         !(turns_fast > turns_slow) || !std::isfinite(turns_fast)))
        return DSV4_ERR_VALUE;
    if (!frequencies)
        return DSV4_ERR_NULL;
    const int pairs = rope_dim / 2;
    if (scaling == DSV4_ROPE_NTK && rope_dim > 2)
        theta *= std::pow(factor, double(rope_dim) / (rope_dim - 2));
    double low = 0.0, high = 0.0;
    if (scaling == DSV4_ROPE_YARN) {
        // the pair that makes so many turns over the original positions
        const auto pair_of = [&](double turns) {
            return pairs * std::log(original_positions / (6.283185307179586476925 * turns)) / std::log(theta);
        };
        low = std::max(0.0, std::floor(pair_of(turns_fast)));
        // (it may lie past the last pair: ended there, the ramp of 65536 positions and theta 10^4 would
        // leave pair 31 of 32 with 0.30 of its frequency)
        high = std::min(double(rope_dim - 1), std::ceil(pair_of(turns_slow)));
        high = std::max(high, low + 0.001);
    }
    for (int i = 0; i < pairs; ++i) {
        const double f = std::pow(theta, -2.0 * i / rope_dim);
        double slow = 0.0;  // how much of the frequency is divided by the factor
        if (scaling == DSV4_ROPE_LINEAR)
            slow = 1.0;
        else if (scaling == DSV4_ROPE_YARN)
            slow = std::min(1.0, std::max(0.0, (i - low) / (high - low)));
        frequencies[i] = slow == 0.0 ? f : slow == 1.0 ? f / factor : f * (1.0 - slow) + f / factor * slow;
    }
    return DSV4_OK;
}

int dsv4_rope_table(const double *frequencies, int32_t rope_dim, double magnitude, const int64_t *positions,
                    int64_t first, int64_t num_positions, float *cos_sin, int32_t *device_error, void *stream)
{
    constexpr int64_t kPositions = int64_t(1) << 32;
    if (bad_rope_dim(rope_dim) || num_positions < 0 || num_positions > kPositions)
        return DSV4_ERR_SHAPE;
    if (!positions && (first < 0 || first > kPositions - num_positions))
        return DSV4_ERR_SHAPE;
    if (!std::isfinite(magnitude) || std::fabs(magnitude) > 65536.0 ||
        (magnitude != 0.0 && std::fabs(magnitude) < 1.0 / 65536.0))
        return DSV4_ERR_VALUE;
    if (!frequencies)
        return DSV4_ERR_NULL;
    for (int i = 0; i < rope_dim / 2; ++i)
        if (!(frequencies[i] >= 0.0) || !(frequencies[i] < 65536.0))
            return DSV4_ERR_VALUE;
    if (num_positions == 0)
        return DSV4_OK;
    if (!cos_sin)
        return DSV4_ERR_NULL;
    if (!aligned(cos_sin, 4) || !aligned(positions, 8) || !aligned(device_error, 4))
        return DSV4_ERR_ALIGN;
    dsv4::RopeTableArgs a = {};
    a.frequencies = frequencies;
    a.rope_dim = rope_dim;
    a.magnitude = magnitude;
    a.positions = positions;
    a.first = first;
    a.count = num_positions;
    a.out = cos_sin;
    a.err = device_error;
    if (sm_count(&a.sms) != DSV4_OK)
        return DSV4_ERR_CUDA;
    return dsv4::launch_rope_table(a, static_cast<cudaStream_t>(stream));
}

int dsv4_rope_rows(int type, const void *x, int64_t x_token_stride, int64_t x_head_stride, void *out,
                   int64_t out_token_stride, int64_t out_head_stride, int64_t num_tokens, int32_t num_heads,
                   int32_t width, int32_t offset, int32_t rope_dim, int layout, int inverse,
                   const int64_t *positions, const float *cos_sin, int64_t max_position, int32_t *device_error,
                   void *stream)
{
    constexpr int64_t kMost = INT64_MAX / 65536;
    if (bad_rope_dim(rope_dim) || width < 1 || width > 65536 || offset < 0 || offset > width - rope_dim ||
        num_tokens < 0 || num_heads < 1 || max_position < 1 || max_position > kMost)
        return DSV4_ERR_SHAPE;
    if (num_tokens > INT32_MAX / num_heads)  // rows are counted in 32 bits
        return DSV4_ERR_SHAPE;
    for (const int64_t s : {x_token_stride, x_head_stride, out_token_stride, out_head_stride})
        if (s < 0 || s > (int64_t(1) << 31))
            return DSV4_ERR_SHAPE;
    if (type < DSV4_TYPE_BF16 || type > DSV4_TYPE_FP32 || (layout != DSV4_ROPE_PAIRS && layout != DSV4_ROPE_HALF) ||
        (inverse != 0 && inverse != 1))
        return DSV4_ERR_VALUE;
    if (num_tokens == 0)
        return DSV4_OK;
    // bytes are counted in 64 bits
    const int64_t size = type == DSV4_TYPE_FP32 ? 4 : 2;
    if (extent(num_tokens, num_heads, width, x_token_stride, x_head_stride) > INT64_MAX / size ||
        extent(num_tokens, num_heads, width, out_token_stride, out_head_stride) > INT64_MAX / size)
        return DSV4_ERR_SHAPE;
    if (!rows_apart(num_tokens, num_heads, width, out_token_stride, out_head_stride))
        return DSV4_ERR_SHAPE;
    if (x == out && (x_token_stride != out_token_stride || x_head_stride != out_head_stride))
        return DSV4_ERR_SHAPE;
    if (!x || !out || !positions || !cos_sin)
        return DSV4_ERR_NULL;
    if (!aligned(x, size) || !aligned(out, size) || !aligned(positions, 8) || !aligned(cos_sin, 16) ||
        !aligned(device_error, 4))
        return DSV4_ERR_ALIGN;
    const uint64_t x_at = reinterpret_cast<uintptr_t>(x), out_at = reinterpret_cast<uintptr_t>(out);
    if (x != out && (num_tokens == 1 || x_token_stride == out_token_stride) &&
        (num_heads == 1 || x_head_stride == out_head_stride) &&
        moved_rows_meet(x_at < out_at ? out_at - x_at : x_at - out_at, num_tokens, num_heads, width * size,
                        out_token_stride * size, out_head_stride * size))
        return DSV4_ERR_SHAPE;
    dsv4::RopeRowsArgs a = {};
    a.x = static_cast<const uint8_t *>(x);
    a.out = static_cast<uint8_t *>(out);
    a.type = type;
    a.tokens = num_tokens;
    a.heads = num_heads;
    a.width = width;
    a.x_token_stride = x_token_stride;
    a.x_head_stride = x_head_stride;
    a.out_token_stride = out_token_stride;
    a.out_head_stride = out_head_stride;
    a.offset = offset;
    a.rope_dim = rope_dim;
    a.layout = layout;
    a.inverse = inverse != 0;
    a.positions = positions;
    a.cos_sin = cos_sin;
    a.max_position = max_position;
    a.err = device_error;
    if (sm_count(&a.sms) != DSV4_OK)
        return DSV4_ERR_CUDA;
    return dsv4::launch_rope_rows(a, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
