// Launch helpers of the few-token kernels (internal).
#pragma once

#include "ep_internal.h"

namespace ep {

// Allows `kernel` up to smem bytes of dynamic shared memory on the current device.
template <class Kernel>
inline int raise_smem(Kernel kernel, size_t smem, PerDevice &set)
{
    const int dev = current_device();
    if ((int)smem > set.get(dev)) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) {
            cudaGetLastError();
            return EP_ERR_CUDA;
        }
        set.put(dev, (int)smem);
    }
    return EP_OK;
}

// Launches a kernel that calls grid_dependency_wait() before it touches
// anything that earlier work of the stream may write or read: it may be
// scheduled while that work drains.
template <class... Params, class... Args>
inline int launch_dependent(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                            const Args &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) {
        cudaGetLastError();
        return EP_ERR_CUDA;
    }
    return EP_OK;
}

}  // namespace ep
