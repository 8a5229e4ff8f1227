// Argument checks shared by the C ABI entry points (host side; nothing is
// launched by any of them).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "cssd_internal.h"

namespace cssd {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Device of the stream (or the current device for the default stream).
inline int stream_device(cudaStream_t s, int* dev) {
    if (s == nullptr) return cudaGetDevice(dev) == cudaSuccess ? CSSD_OK : CSSD_ERR_CUDA;
    return stream_device_of(s, dev) == cudaSuccess ? CSSD_OK : CSSD_ERR_CUDA;
}

// The pointer must be device (or managed) memory usable on `dev`.
inline int check_device_ptr(const void* p, int dev) {
    cudaPointerAttributes at;
    if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
        cudaGetLastError();  // clear the sticky-free error this query may set
        return CSSD_ERR_DEVICE;
    }
    if (at.type == cudaMemoryTypeManaged) return CSSD_OK;
    if (at.type != cudaMemoryTypeDevice || at.device != dev) return CSSD_ERR_DEVICE;
    return CSSD_OK;
}

template <typename... Ts>
int check_all_device(int dev, Ts... ptrs) {
    const void* arr[] = {ptrs...};
    for (const void* p : arr) {
        if (!p) continue;
        const int s = check_device_ptr(p, dev);
        if (s != CSSD_OK) return s;
    }
    return CSSD_OK;
}

}  // namespace cssd
