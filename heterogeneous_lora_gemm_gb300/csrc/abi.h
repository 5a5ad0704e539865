// What the C entry points of the caches and of the rotation share (cache.cu, rotary.cu): errors, the
// device of a handle, checks of row operands.
#pragma once
#include <cuda_runtime.h>

#include <cstdarg>
#include <cstdio>

#include "../../include/mlora.h"
#include "internal.h"

namespace mlora {

inline mlora_status fail(mlora_status s, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    set_last_error(buf);
    return s;
}

inline mlora_status cuda_fail(cudaError_t e, const char* what) {
    cudaGetLastError();   // reported here: not the next launch's error
    return fail(MLORA_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

// Makes a handle's device current for the scope of one call and restores the caller's.
struct DeviceGuard {
    int prev = -1;
    bool moved = false;
    cudaError_t err = cudaSuccess;
    explicit DeviceGuard(int dev) {
        err = cudaGetDevice(&prev);
        if (err == cudaSuccess && prev != dev) {
            err = cudaSetDevice(dev);
            moved = err == cudaSuccess;
        }
    }
    ~DeviceGuard() {
        if (moved) cudaSetDevice(prev);
    }
};

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

inline mlora_status check_rows(const char* name, const void* p, int64_t row, int64_t head, mlora_dtype dtype) {
    const int64_t unit = dtype == MLORA_BF16 ? 8 : 4;   // elements per 16 bytes
    if (!p) return fail(MLORA_ERR_INVALID_ARG, "%s is NULL", name);
    if (!aligned16(p) || row % unit || head % unit || row < 0 || head < 0)
        return fail(MLORA_ERR_INVALID_ARG, "%s: 16-byte alignment (strides %lld, %lld elements)", name, (long long)row,
                    (long long)head);
    return MLORA_OK;
}

}  // namespace mlora
