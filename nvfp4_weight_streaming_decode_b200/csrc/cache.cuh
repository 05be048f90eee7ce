// cache.cuh -- device-side view of a paged cache (nvfp4_cache): where a lane's
// slot lies, which lane a row belongs to, and small pieces that the cache,
// rotary and attention kernels share.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "nvfp4decode.h"

namespace nvfp4 {

// Rows of a call and their lanes: lane b has rows [lo, hi) of row_start,
// clamped so that whatever the device memory holds stays inside the call.
__device__ __forceinline__ void lane_rows(const int32_t* row_start, int b, int rows, int& lo, int& hi)
{
    if (row_start) {
        lo = min(max(__ldg(row_start + b), 0), rows);
        hi = min(max(__ldg(row_start + b + 1), lo), rows);
    } else {
        lo = min(b, rows);
        hi = min(b + 1, rows);
    }
}

// Wait for the kernels before this one in its stream (a programmatic
// dependent launch starts early), after letting the next one start.
__device__ __forceinline__ void pdl_begin()
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// One arrival on a GPU-scope counter: publishes the caller's writes (the CTA
// barrier before it orders the other threads') and sees those of every
// earlier arrival.
__device__ __forceinline__ unsigned count_in(unsigned* counter)
{
    unsigned old;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(old) : "l"(counter) : "memory");
    return old;
}

// Host: a launch as a programmatic dependent of the work before it.
template <class... Args>
inline cudaError_t launch_pdl(void (*kernel)(Args...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                              Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace nvfp4
