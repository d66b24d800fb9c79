// Argument checks shared by the C-ABI files (api.cpp, fp4_api.cpp, latent_api.cpp).
#pragma once

#include <stdint.h>

#include "dsv4kv.h"

namespace dsv4 {

inline bool aligned(const void *p, uintptr_t a)
{
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

// Caches hold at most 2^32 slots (more than any one GPU can hold at 132 bytes
// per slot), so the kernels divide 32-bit slot numbers by the block size.
constexpr int64_t kMaxSlots = int64_t(1) << 32;

inline bool too_many_slots(int64_t num_blocks, int32_t block_size)
{
    return num_blocks > kMaxSlots / block_size;
}

// keys of a request that a table can name: key indices, less a window and a
// number of tokens, then stay in 32 bits
constexpr int64_t kMaxKeys = int64_t(1) << 30;

// sizes of what every operator over requests takes; pointers come after the
// early return for an empty batch
inline int check_sizes(int64_t num_blocks, int32_t block_size, int64_t table_stride,
                       int32_t table_width, int32_t batch)
{
    if (num_blocks < 1 || block_size < 1 || table_width < 1 || batch < 0 ||
        table_stride < table_width)
        return DSV4_ERR_SHAPE;
    if (too_many_slots(num_blocks, block_size) || num_blocks > INT32_MAX ||
        int64_t(table_width) * block_size > kMaxKeys || table_stride > INT64_MAX / 4096 / 65536 ||
        batch > 65535)
        return DSV4_ERR_SHAPE;
    return DSV4_OK;
}

inline int check_attention(int32_t q_len, int32_t num_heads, int32_t batch, float scale, int32_t window,
                           int64_t most_keys, int tile_keys, int start_cost)
{
    if (q_len < 1 || q_len > (1 << 24) || num_heads < 1 || window < 0)
        return DSV4_ERR_SHAPE;
    if (int64_t(q_len) * num_heads > INT32_MAX ||
        int64_t(q_len) * num_heads * batch > INT64_MAX / 4096 ||
        (batch > 0 && int64_t(q_len) * num_heads > INT32_MAX / batch))
        return DSV4_ERR_SHAPE;
    // The line of tiles of 64 rows and tile_keys keys with what is added to it is counted in 32
    // bits, up to a multiple of the CTAs (fewer than 1024).
    if (((int64_t(q_len) * num_heads + 63) / 64) * batch >
        (INT32_MAX - 1024) / ((most_keys + tile_keys - 1) / tile_keys + start_cost))
        return DSV4_ERR_SHAPE;
    if (!(scale > 0.0f && scale <= 4294967296.0f))  // it is multiplied by 2^82 in fp32
        return DSV4_ERR_VALUE;
    return DSV4_OK;
}

}  // namespace dsv4
