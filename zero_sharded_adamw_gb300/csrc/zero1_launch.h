// zero1_launch.h -- a kernel launch whose status is its own: what
// cudaGetLastError returns after <<<>>> may be an earlier call's error (an
// allocation that did not fit, say), and the launch would be taken for failed.
#pragma once

#include <cuda_runtime.h>

namespace zero1 {

// early: the kernel may begin while the one before it on the stream still
// runs, and waits for its end (griddepcontrol.wait) before it reads anything.
template <bool EARLY, typename... Params, typename... Args>
cudaError_t launch_as(void (*kernel)(Params...), dim3 grid, uint32_t threads, size_t smem, cudaStream_t stream,
                      const Args &... args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = EARLY ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename... Params, typename... Args>
cudaError_t launch(void (*kernel)(Params...), dim3 grid, uint32_t threads, size_t smem, cudaStream_t stream,
                   const Args &... args)
{
    return launch_as<false>(kernel, grid, threads, smem, stream, args...);
}

template <typename... Params, typename... Args>
cudaError_t launch_early(void (*kernel)(Params...), dim3 grid, uint32_t threads, size_t smem, cudaStream_t stream,
                         const Args &... args)
{
    return launch_as<true>(kernel, grid, threads, smem, stream, args...);
}

}  // namespace zero1
