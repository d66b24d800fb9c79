// Copies of rows of 512 bf16 from global to shared memory by the tensor-copy unit
// (cp.async.bulk.tensor), in the 128-byte swizzle that the matrix unit reads (tcgen05.cuh), and
// the maps that describe the rows to it.
//
// A copy's first dim is a multiple of 64, so it starts on a 16-byte boundary.  Rows past the last
// read as zeros.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "bulkcopy.cuh"
#include "dsv4kv.h"

namespace dsv4 {
namespace {

// Rows [row, row + the map's box) as 8 chunks of 64 dims one after the other, counted on *bar.  The
// lane with elected != 0 issues it; every lane of the warp calls it with the same values.
// (Issued by lanes of their own, copies took about 80 cycles each.)
__device__ __forceinline__ void copy_rows(uint32_t to, const CUtensorMap *map, int row, uint64_t *bar, uint32_t elected)
{
    asm volatile("{\n\t.reg .pred e;\n\tsetp.ne.u32 e, %4, 0;\n\t"
                 "@e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%5, %2, %5}], [%3];\n\t}" ::"r"(to),
                 "l"(map), "r"(row), "r"(smem_addr(bar)), "r"(elected), "r"(0)
                 : "memory");
}

// The driver's encoder, found once (it is not linked: the library needs the driver at run time
// only); null without a driver.
typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiled tensor_map_encoder()
{
    static std::atomic<void *> found{nullptr};
    void *f = found.load(std::memory_order_relaxed);
    if (f == nullptr) {
        cudaDriverEntryPointQueryResult result;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &result) !=
                cudaSuccess ||
            result != cudaDriverEntryPointSuccess)
            return nullptr;
        found.store(f, std::memory_order_relaxed);
    }
    return reinterpret_cast<EncodeTiled>(f);
}

// `rows` rows at `base` (16-byte aligned), in boxes of `box` of them: (dim in chunk, row, chunk)
inline int encode_rows(CUtensorMap *map, const void *base, uint64_t rows, uint32_t box)
{
    const EncodeTiled encode = tensor_map_encoder();
    constexpr cuuint64_t row_bytes = DSV4_HEAD_DIM * 2;
    const cuuint64_t sizes[3] = {64, rows, 8}, strides[2] = {row_bytes, 128};
    const cuuint32_t boxes[3] = {64, box, 8}, steps[3] = {1, 1, 1};
    return encode != nullptr &&
                   encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), sizes, strides, boxes,
                          steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? DSV4_OK
               : DSV4_ERR_CUDA;
}

}  // namespace
}  // namespace dsv4
