// Host-side helpers shared by the translation units that implement C entry
// points: the view of a context that they need, errors, the device guard.
#pragma once

#include <cuda_runtime.h>

#include "pi.h"

namespace pi {

struct DeviceGuard {
    int prev = -1;
    explicit DeviceGuard(int dev)
    {
        if (cudaGetDevice(&prev) != cudaSuccess) prev = -1;
        if (prev != dev) cudaSetDevice(dev);
    }
    ~DeviceGuard()
    {
        int cur = -1;
        if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev) cudaSetDevice(prev);
    }
};

// What a call of the block operators needs of its context.
struct CtxView {
    int device;
    cudaStream_t stream;
    int sms;         // streaming multiprocessors
    int smem_optin;  // dynamic shared memory limit per CTA
    int *status;     // device words: first device error, abort flag
    int *abort_flag;
    unsigned long long wait_ns;
};

CtxView ctx_view(pi_ctx *c);
pi_status ctx_fail(pi_ctx *c, pi_status code, const char *fmt, ...);

} // namespace pi
