// dependent.cuh -- launches that begin while the kernel before them on the stream still ends (programmatic dependent
// launch). A kernel that is launched so calls begin_dependent() before it touches memory, and reads what kernels before it
// wrote with loads that the compiler keeps behind that call (volatile; __ldg it may move).
//
// Back to back, a launch of a few microseconds' work otherwise leaves the GPU idle for about 2 us.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace qn {

// Waits until the kernels before this one are done, then lets the next one be set up.
__device__ __forceinline__ void begin_dependent() {
    grid_dependency_wait();
    grid_dependents_launch();
}

__device__ __forceinline__ uint32_t ld_nc_u16(const uint16_t *p) {
    uint16_t v;
    asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ uint32_t ld_nc_u8(const uint8_t *p) {
    uint16_t v;
    asm volatile("ld.global.nc.u8 %0, [%1];" : "=h"(v) : "l"(p));
    return v;
}

// One launch of `grid` CTAs without dynamic shared memory.
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kern)(P...), unsigned grid, int threads, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
    if (e == cudaSuccess) count_launch();
    return e;
}

}  // namespace qn
