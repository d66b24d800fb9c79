// Copies of rows of bf16 from global to shared memory by the tensor-copy unit (cp.async.bulk.tensor), in the 128-byte swizzle that the matrix unit reads (tcgen05.cuh),
// and the maps that describe the rows to it.
//
// A row is 512 bf16.  A copy's first dim is a multiple of 64, so it starts on a 16-byte
// boundary.  Rows past the last read as zeros.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "bulkcopy.cuh"
#include "dsv4kv.h"

namespace dsv4 {
namespace {

// All copies are issued by the lane with elected != 0 and counted on *bar; every lane calls them
// with the same values.

// rows [row, row + the map's box), all 512 dims, as 8 chunks one after the other (encode_rows)
__device__ __forceinline__ void copy_rows3(uint32_t to, const CUtensorMap *map, int row, uint64_t *bar, uint32_t elected)
{
    asm volatile(
        "{\n\t.reg .pred e;\n\tsetp.ne.u32 e, %4, 0;\n\t"
        "@e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%5, %2, %5}], [%3];\n\t}" ::
            "r"(to),
        "l"(map), "r"(row), "r"(smem_addr(bar)), "r"(elected), "r"(0)
        : "memory");
}

// chunks `chunk` and the next of groups of 8 rows from `group` on, each as 2 chunks of its 8 rows
// (encode_groups)
__device__ __forceinline__ void copy_groups(uint32_t to, const CUtensorMap *map, int chunk, int group, uint64_t *bar,
                                            uint32_t elected)
{
    asm volatile(
        "{\n\t.reg .pred e;\n\tsetp.ne.u32 e, %5, 0;\n\t"
        "@e cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%6, %6, %2, %3}], [%4];\n\t}" ::"r"(to),
        "l"(map), "r"(chunk), "r"(group), "r"(smem_addr(bar)), "r"(elected), "r"(0)
        : "memory");
}

// dims [dim, dim + 64) of four rows anywhere (encode_single_rows)
__device__ __forceinline__ void copy_four(uint32_t to, const CUtensorMap *map, int dim, const int *rows, uint64_t *bar,
                                          uint32_t elected)
{
    asm volatile(
        "{\n\t.reg .pred e;\n\tsetp.ne.u32 e, %8, 0;\n\t"
        "@e cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];\n\t}" ::"r"(to),
        "l"(map), "r"(dim), "r"(rows[0]), "r"(rows[1]), "r"(rows[2]), "r"(rows[3]), "r"(smem_addr(bar)), "r"(elected)
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

inline int encode_map(CUtensorMap *map, const void *base, int rank, const cuuint64_t *sizes, const cuuint64_t *strides,
                      const cuuint32_t *box)
{
    const EncodeTiled encode = tensor_map_encoder();
    const cuuint32_t steps[4] = {1, 1, 1, 1};
    return encode != nullptr &&
                   encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, cuuint32_t(rank), const_cast<void *>(base), sizes,
                          strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? DSV4_OK
               : DSV4_ERR_CUDA;
}

constexpr cuuint64_t kRowBytes = DSV4_HEAD_DIM * 2;

// `rows` rows at `base` (16-byte aligned), in boxes of `box` rows: (dim in chunk, row, chunk)
inline int encode_rows(CUtensorMap *map, const void *base, uint64_t rows, uint32_t box)
{
    const cuuint64_t sizes[3] = {64, rows, 8}, strides[2] = {kRowBytes, 128};
    const cuuint32_t boxes[3] = {64, box, 8};
    return encode_map(map, base, 3, sizes, strides, boxes);
}

// `groups` groups of 8 rows, in boxes of 2 chunks of `box` groups: (dim in chunk, row in group,
// chunk, group)
inline int encode_groups(CUtensorMap *map, const void *base, uint64_t groups, uint32_t box)
{
    const cuuint64_t sizes[4] = {64, 8, 8, groups}, strides[3] = {kRowBytes, 128, 8 * kRowBytes};
    const cuuint32_t boxes[4] = {64, 8, 2, box};
    return encode_map(map, base, 4, sizes, strides, boxes);
}

// `rows` rows, to be gathered: (dim, row)
inline int encode_single_rows(CUtensorMap *map, const void *base, uint64_t rows)
{
    const cuuint64_t sizes[2] = {DSV4_HEAD_DIM, rows}, strides[1] = {kRowBytes};
    const cuuint32_t boxes[2] = {64, 1};
    return encode_map(map, base, 2, sizes, strides, boxes);
}

}  // namespace
}  // namespace dsv4
