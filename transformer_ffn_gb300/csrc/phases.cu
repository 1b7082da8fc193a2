// phases.cu -- cluster launch of the phase kernel (clusters of two CTAs, grid
// capped at the CTA pairs the GPU keeps resident).
#include <cuda_runtime.h>

#include "phases.cuh"
#include "train.h"

namespace tffn {

static int phase_config(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr, int* resident)
{
    static int pairs = 0;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.blockDim = dim3(phases::NUM_THREADS);
    cfg.dynamicSmemBytes = phases::SMEM_BYTES;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(2);
    if (pairs == 0) {
        if (cudaFuncSetAttribute(phases::phase_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 phases::SMEM_BYTES) != cudaSuccess)
            return -1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, phases::phase_kernel, &cfg) != cudaSuccess || n < 1)
            return -1;
        pairs = n;
    }
    *resident = pairs;
    return 0;
}

int phase_pairs()
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    int resident = 0;
    return phase_config(cfg, attr, &resident) == 0 ? resident : -1;
}

int launch_phases(const phases::Params& p, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    int resident = 0;
    if (phase_config(cfg, attr, &resident) != 0)
        return -1;
    cfg.stream = s;
    cfg.gridDim = dim3(2 * static_cast<unsigned>(p.total < resident ? p.total : resident));
    if (cudaLaunchKernelEx(&cfg, phases::phase_kernel, p) != cudaSuccess)
        return -1;
    return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace tffn
