// sv_host.h -- host-side helpers shared by the entry points: the current
// device for the length of a call, and a handle's workspace.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "spec_verify.h"

namespace sv {

struct DeviceGuard {
    int prev = -1;
    bool ok = false, changed = false;
    explicit DeviceGuard(int dev)
    {
        if (cudaGetDevice(&prev) != cudaSuccess) return;
        changed = prev != dev;
        ok = !changed || cudaSetDevice(dev) == cudaSuccess;
    }
    ~DeviceGuard()
    {
        if (changed) cudaSetDevice(prev);
    }
};

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// device memory from the allocator of spec_verify_set_allocator, or cudaMalloc
// when none is set; it goes back the way it came (NULL functions: cudaFree)
struct Workspace {
    void* base;
    spec_alloc_fn alloc_fn;
    spec_release_fn release_fn;
    void* ctx;
};

// `bytes` of zeroed memory on `device` (which must be current), aligned to 256
// bytes; the zeros have arrived when it returns.  SPEC_ERR_OOM, SPEC_ERR_INVALID_ARG (a misaligned block of the
// caller's allocator) or SPEC_ERR_CUDA leave nothing allocated.
spec_status workspace_take(Workspace* w, int device, size_t bytes);

// returns it (synchronises the device, which must be current)
spec_status workspace_give(Workspace* w, int device);

}  // namespace sv
