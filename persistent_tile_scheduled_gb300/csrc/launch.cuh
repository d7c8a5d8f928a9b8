// One launch with the attributes that the small kernels use.
#pragma once
#include <cuda_runtime.h>

namespace pts {

// cluster: CTAs along x of a cluster; overlap: the launch may start while the
// kernel before it finishes (it waits for it before it reads memory).
template <class... P, class... A>
cudaError_t launch_kernel(void (*kernel)(P...), dim3 grid, int block, size_t smem, int cluster, cudaStream_t stream, bool overlap, A... args)
{
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(block), 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    int n = 0;
    if (overlap) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = static_cast<unsigned>(cluster);
        attr[n].val.clusterDim.y = 1;
        attr[n].val.clusterDim.z = 1;
        ++n;
    }
    cfg.numAttrs = static_cast<unsigned>(n);
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace pts
