// What the kernels of the paged cache's own operations share.
#pragma once

#include <cuda_runtime_api.h>

#include <cstdint>

#include "fa_paged.h"

namespace fa {
namespace {

// Small integers through L2: the kernels are programmatic dependents (see
// fa_paged_sched.cuh), and fork rewrites tables in place.
__device__ __forceinline__ int ldi(const int32_t* p) { return __ldcg(p); }

__device__ __forceinline__ void bad_page(uint32_t* status, uint32_t site) {
    atomicCAS(status + PAGE_WORD, 0u, STATUS_PAGE | (site << 8) | ((blockIdx.x & 0xFFFFu) << 16));
}

// Launch as a programmatic dependent of the work before it on the stream.
template <typename K, typename P>
inline cudaError_t launch_dependent(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream, const P& p) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace
}  // namespace fa
