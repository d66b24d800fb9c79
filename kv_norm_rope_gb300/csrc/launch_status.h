// Kernel launches that report their own status.
//
// A <<< >>> launch returns nothing, and cudaGetLastError() after it returns,
// and clears, the last error of any earlier runtime call on the thread: an
// unrelated error the caller left pending would be reported as this launch's
// failure and lost to the caller.  cudaLaunchKernel returns the status of the
// launch itself (plus errors that already broke the context, which any call
// returns).  Every kernel of the library takes one parameter struct.
#pragma once

#include <cuda_runtime.h>

#include "dsv4kv.h"

namespace dsv4 {

template <typename P>
inline int launch_kernel(void (*kernel)(P), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                         const P &p)
{
    void *args[] = {const_cast<P *>(&p)};
    return cudaLaunchKernel(reinterpret_cast<const void *>(kernel), grid, block, args, smem,
                            stream) == cudaSuccess
               ? DSV4_OK
               : DSV4_ERR_CUDA;
}

// the same in clusters of `cluster` CTAs
template <typename P>
inline int launch_cluster(void (*kernel)(P), dim3 grid, dim3 block, unsigned cluster,
                          cudaStream_t stream, const P &p)
{
    void *args[] = {const_cast<P *>(&p)};
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t config = {};
    config.gridDim = grid;
    config.blockDim = block;
    config.stream = stream;
    config.attrs = &attr;
    config.numAttrs = 1;
    return cudaLaunchKernelExC(&config, reinterpret_cast<const void *>(kernel), args) == cudaSuccess
               ? DSV4_OK
               : DSV4_ERR_CUDA;
}

// A launch that may begin while the kernel before it on the stream still runs, once
// every CTA of that one has ended or called let_kernel_after_begin().  Every thread
// of it that reads what that kernel writes, and at least one thread of every CTA,
// calls wait_for_kernel_before() first.
template <typename P>
inline int launch_after(void (*kernel)(P), dim3 grid, dim3 block, cudaStream_t stream, const P &p,
                        size_t smem = 0)
{
    void *args[] = {const_cast<P *>(&p)};
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t config = {};
    config.gridDim = grid;
    config.blockDim = block;
    config.dynamicSmemBytes = smem;
    config.stream = stream;
    config.attrs = &attr;
    config.numAttrs = 1;
    return cudaLaunchKernelExC(&config, reinterpret_cast<const void *>(kernel), args) == cudaSuccess
               ? DSV4_OK
               : DSV4_ERR_CUDA;
}

#ifdef __CUDACC__
__device__ __forceinline__ void let_kernel_after_begin()
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// until the kernel before it has ended and its writes are visible
__device__ __forceinline__ void wait_for_kernel_before()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
#endif

}  // namespace dsv4
