// Argument checks shared by the C-ABI files (api.cpp, fp4_api.cpp).
#pragma once

#include <stdint.h>

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

}  // namespace dsv4
