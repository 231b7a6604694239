// Kernels and switches for tests of the bounded waits: they make the rare
// event that a wait must survive, and nothing faults, traps or hangs.
#include <atomic>

#include "zs_device.cuh"
#include "zs_launch.h"

static std::atomic<int> g_give_up{-1};       // zs_test_give_up

int zsl_test_give_up() { return g_give_up.load(std::memory_order_relaxed); }

extern "C" zs_status zs_test_give_up(int32_t at) {
    if (at < -1) return zs_fail(ZS_EINVAL, "zs_test_give_up: %d", at);
    g_give_up.store(at, std::memory_order_relaxed);
    zs_clear_error();
    return ZS_OK;
}

namespace zsk {

// Lets its dependents begin at once, works on for delay_ns, and then copies:
// a dependent that reads dst, or begins to count its time, before this kernel
// has completed is found out.
__global__ void late_copy_kernel(uint4 *dst, const uint4 *src, int64_t n, uint64_t delay_ns) {
    pdl_trigger();
    if (threadIdx.x == 0) {
        const uint64_t t0 = global_ns();
        for (int i = 0; i < (1 << 30) && global_ns() - t0 < delay_ns; ++i) __nanosleep(1000);
    }
    __syncthreads();
    for (int64_t i = threadIdx.x; i < n; i += blockDim.x) dst[i] = src[i];
}

}  // namespace zsk

extern "C" zs_status zs_test_late_copy(void *dst, const void *src, int64_t bytes, int64_t delay_ns, void *stream) {
    const char *fn = "zs_test_late_copy";
    if (!dst || !src || bytes < 0 || bytes % 16 || reinterpret_cast<uintptr_t>(dst) % 16 || reinterpret_cast<uintptr_t>(src) % 16)
        return zs_fail(ZS_EINVAL, "%s: NULL or not 16-byte aligned, or %lld bytes", fn, (long long)bytes);
    if (delay_ns <= 0 || delay_ns > 2000000000ll)
        return zs_fail(ZS_EINVAL, "%s: delay_ns %lld not in (0, 2e9]", fn, (long long)delay_ns);
    zsk::late_copy_kernel<<<1, 256, 0, (cudaStream_t)stream>>>(static_cast<uint4 *>(dst), static_cast<const uint4 *>(src),
                                                              bytes / 16, (uint64_t)delay_ns);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return zs_fail(ZS_ECUDA, "%s: %s (%s)", fn, cudaGetErrorName(e), cudaGetErrorString(e));
    zs_clear_error();
    return ZS_OK;
}
