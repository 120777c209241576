// device_guard.h -- makes a device current for one library call and restores
// the caller's current device when the call returns.
#pragma once

#include <cuda_runtime.h>

namespace ckv {

struct DeviceGuard {
    int prev = -1;
    cudaError_t enter(int dev)
    {
        cudaError_t e = cudaGetDevice(&prev);
        if (e != cudaSuccess) { prev = -1; return e; }
        return prev == dev ? cudaSuccess : cudaSetDevice(dev);
    }
    ~DeviceGuard()
    {
        int cur = -1;
        if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev) cudaSetDevice(prev);
    }
};

}  // namespace ckv
