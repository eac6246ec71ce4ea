// selftest_sm100.cuh -- a bounded wait that runs out, for every translation
// unit that has a device status word of its own.
#pragma once

#include "ptx_sm100.cuh"

namespace ajvp {

// One warp waits on a barrier that nothing ever arrives on, with no copies in
// flight, gives up after bound_ns, sets this unit's status word and returns.
static __global__ void selftest_wait_kernel(unsigned long long bound_ns, bool idle) {
    __shared__ __align__(8) uint64_t bar;
    __shared__ int abort_flag;
    const uint32_t b = smem_u32(&bar);
    if (threadIdx.x == 0) {
        mbar_init(b, 1);
        abort_flag = 0;
        fence_barrier_init();
    }
    __syncwarp();
    volatile int *const flag = reinterpret_cast<volatile int *>(&abort_flag);
    bool ok = idle ? mbar_wait_idle(b, 0, flag, bound_ns) : mbar_wait(b, 0, flag, bound_ns);
    ok = __all_sync(0xffffffffu, ok);
    (void)ok;
}

static inline cudaError_t selftest_wait(uint64_t bound_ns, bool idle, cudaStream_t stream) {
    selftest_wait_kernel<<<1, 32, 0, stream>>>((unsigned long long)bound_ns, idle);
    return cudaGetLastError();
}

}  // namespace ajvp
