// Host-side launch helper shared by the kernels' files.
#pragma once

#include <cuda_runtime.h>

#include <utility>

namespace pa {
namespace {

// Tokens that a row of the block tables has room for, at most INT32_MAX: the product itself may be larger.
__device__ __forceinline__ int table_tokens(int max_blocks_per_seq, int block_size)
{
    return (int)min((long long)max_blocks_per_seq * block_size, 0x7fffffffll);
}

// Launches a kernel with programmatic dependent launch: its CTAs may be scheduled
// while the previous kernel in the stream drains; they wait (griddepcontrol.wait)
// before touching that kernel's results.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                       Args&&... args)
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
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

}  // namespace
}  // namespace pa
