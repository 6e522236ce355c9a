// launch.h -- a kernel launched as a programmatic dependent of the work before it on the stream: its CTAs may be
// scheduled while that work drains, and the kernel waits for it (wait_prior_grid) before it touches memory.
#pragma once

#include "qsa_internal.h"

namespace qsa {

template <typename... Params, typename... Args>
qsa_status launch_dependent(const char *what, void (*kern)(Params...), int grid, int threads, size_t smem, cudaStream_t s,
                            Args... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return check_cuda(cudaLaunchKernelEx(&cfg, kern, static_cast<Params>(args)...), what);
}

}  // namespace qsa
