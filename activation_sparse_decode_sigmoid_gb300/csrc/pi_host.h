// Host-side helpers shared by the translation units that implement C entry
// points: the view of a context that they need, errors, the device guard.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <initializer_list>

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

// Raises a kernel's limit of dynamic shared memory on the current device to all
// that its static arrays leave, once per device (`ready`: the kernel's own,
// devices by bit).  The limit belongs to the function on a device, not to a
// launch: set to one call's size, it made launches of another thread's context
// fail (881 of 5000 norms of 4096 columns beside norms of 64).
inline cudaError_t raise_limit(const void *kern, std::atomic<uint64_t> &ready)
{
    int dev = 0, most = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && (ready.load(std::memory_order_relaxed) >> dev & 1))) return e;
    cudaFuncAttributes a;
    e = cudaFuncGetAttributes(&a, kern);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most - (int)a.sharedSizeBytes);
    if (e == cudaSuccess && dev < 64) ready.fetch_or(1ull << dev);
    return e;
}

CtxView ctx_view(pi_ctx *c);
pi_status ctx_fail(pi_ctx *c, pi_status code, const char *fmt, ...);

// Refuses buffers of elements of `elem` bytes that start between two elements:
// a kernel's access there would fault.
inline pi_status check_elements(pi_ctx *c, int elem, std::initializer_list<const void *> buffers)
{
    for (const void *p : buffers)
        if ((uintptr_t)p % elem)
            return ctx_fail(c, PI_ERR_ARG, "address %p is not a multiple of the element's %d bytes", p, elem);
    return PI_OK;
}

} // namespace pi
