// Launch helpers shared by the library's HIP sources.
#pragma once

#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>

#include "lora_internal.hpp"

namespace lora {

// Event pair attached to this thread's next kernel launch (lora_set_launch_events).
extern thread_local hipEvent_t t_ev_start, t_ev_stop;

template <typename Kernel, typename... A>
void launch_args(Kernel kernel, dim3 grid, int threads, size_t lds, hipStream_t s, const A &...a)
{
    const dim3 block(threads);
    if (t_ev_start || t_ev_stop) {
        hipEvent_t e0 = t_ev_start, e1 = t_ev_stop;
        t_ev_start = t_ev_stop = nullptr;
        hipExtLaunchKernelGGL(kernel, grid, block, lds, s, e0, e1, 0, a...);
    } else {
        hipLaunchKernelGGL(kernel, grid, block, lds, s, a...);
    }
}

inline int launch_status(const char *what)
{
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(LORA_E_HIP, "%s: launch failed: %s", what, hipGetErrorString(e));
    return LORA_OK;
}

}  // namespace lora
