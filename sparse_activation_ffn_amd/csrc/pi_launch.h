// pi_launch.h -- host helpers shared by the translation units of libpi.so: the
// error message of a call, argument checks, and kernel launches with the timing
// hooks of pi_kernel_timer_start / _stop.  Defined in pi_api.hip.
#pragma once
#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>

#include <cstdint>
#include <vector>

#include "pi.h"

namespace pi {

// stores the message pi_last_error() returns (thread-local) and returns s
pi_status fail(pi_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));

#define CHECK(cond, status, ...)                              \
    do {                                                      \
        if (!(cond)) return ::pi::fail(status, __VA_ARGS__);  \
    } while (0)

#define TRY(expr)                         \
    do {                                  \
        pi_status _s = (expr);            \
        if (_s != PI_OK) return _s;       \
    } while (0)

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct Timer {
    bool armed = false;
    int max = 0, used = 0;
    std::vector<hipEvent_t> ev;   // 2 per launch
};
Timer& kernel_timer(int kid);     // this host thread's timer of kernel kid

template <typename K, typename... Args>
pi_status launch(int kid, K kernel, dim3 grid, dim3 block, size_t shmem, hipStream_t s,
                 Args... args) {
    Timer& t = kernel_timer(kid);
    if (t.armed && t.used < t.max) {
        hipExtLaunchKernelGGL(kernel, grid, block, (uint32_t)shmem, s, t.ev[2 * t.used],
                              t.ev[2 * t.used + 1], 0, args...);
        ++t.used;
    } else {
        hipLaunchKernelGGL(kernel, grid, block, shmem, s, args...);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return fail(PI_ERR_HIP, "%s launch: %s", pi_kernel_name(kid), hipGetErrorString(e));
    return PI_OK;
}

// kernels with more than 64 KiB of dynamic LDS must opt in
template <typename K>
pi_status allow_lds(K kernel, size_t bytes) {
    if (bytes <= 65536) return PI_OK;
    hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                       hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != hipSuccess) return fail(PI_ERR_HIP, "LDS attribute: %s", hipGetErrorString(e));
    return PI_OK;
}

}  // namespace pi
