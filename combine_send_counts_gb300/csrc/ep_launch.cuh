// Launch helpers of the few-token kernels (internal).
#pragma once

#include "ep_internal.h"

namespace ep {

// Allows `kernel` up to smem bytes of dynamic shared memory on the current
// device.  smem is the same in every call for one kernel, so that concurrent
// first calls cannot lower it.
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

// How many of a block's `blocks` row blocks a warp takes at a time, up to four
// (`most`): each x it loads serves them all, but an item that has fewer still
// takes the time of all, which counts where the codes' arithmetic is what takes
// time (4-bit weights; a stage of it is about 270 instructions, and a unit's x
// 40: one row with 50021x7168 took 48 us in the largest equal items, 45 so).
// bf16: the largest equal items (128 tokens of 128 experts 4096x1536: 814 us;
// with three, two, one of up's blocks at a time 818, 829, 868, with one of down's
// 980.  One token of 6 experts 2048x1024 would be 20.2 us with one of up's,
// instead of 21.3).  The 270 instructions are those of groups of 128 and one
// plane of x, but the choices hold for the others: with 1, 13 and 128 tokens and
// groups of 32, 64 and 128, no other number of blocks in up or in down (three
// planes) took 1.5% less, and most took 2 to 20% more.
inline int blocks_at_once(int64_t blocks, int most, bool w4)
{
    int best = (int)ceil_div(blocks, ceil_div(blocks, most));
    if (w4) {
        int64_t least = INT64_MAX;
        for (int n = most; n >= 1; --n) {
            const int64_t cost = ceil_div(blocks, n) * (270 * n + 40);
            if (cost < least) {
                least = cost;
                best = n;
            }
        }
    }
    return best;
}

}  // namespace ep
