// internal.h -- entry points shared between the library's own translation units.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "mlora.h"

// mlora_apply with the long-segment H workspace in caller-provided device memory of
// `ws_bytes` bytes; never allocates.  MLORA_ERR_UNSUPPORTED if the batch needs more.
mlora_status mlora_apply_with_workspace(mlora_pool *pool, const mlora_segments *segs,
                                        const void *X, int64_t ldx, void *Y, int64_t ldy,
                                        void *stream, float *ws, size_t ws_bytes);

// Look up (and so reserve, under lazy module loading) the no-allocation entry point's
// scratch array on device `dev`, which must be current; cached per device.
mlora_status mlora_noalloc_reserve(int dev);

// Device the pool was created on (-1 for NULL).
int mlora_pool_device(const mlora_pool *pool);

// What the row kernels need of a pool.
struct mlora_pool_view {
    int device;
    int32_t n_slots;
    const int32_t *slot_rank;    // device
    unsigned int *status;        // device
};
bool mlora_pool_get_view(const mlora_pool *pool, mlora_pool_view *view);   // false for NULL

// Kernel attributes on device `dev`, which must be current; once per device.
mlora_status mlora_prepare_device(int dev);

// Sizes, strides and pointers of a quantised matrix.
mlora_status mlora_mx_check_matrix(const mlora_mx_matrix *Q);

// Makes `dev` current for the guard's life, restoring the caller's device.
struct mlora_device_guard {
    int prev = -1;
    bool ok = true;
    explicit mlora_device_guard(int dev)
    {
        if (cudaGetDevice(&prev) != cudaSuccess) {
            ok = false;
            return;
        }
        if (prev != dev && cudaSetDevice(dev) != cudaSuccess) ok = false;
    }
    ~mlora_device_guard()
    {
        int cur = -1;
        if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev) cudaSetDevice(prev);
    }
};
