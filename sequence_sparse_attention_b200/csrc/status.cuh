// status.cuh -- host-side error helpers of the C ABI's translation units.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/spava.h"

namespace spava {

// Workspace status bit of the cache calls (bit 0 is a wait that gave up): a
// length or a page outside its table or pool.
constexpr int kStatusBadBatch = 2;

// CUDA error code of this thread's last SPAVA_ERR_CUDA (spava_last_cuda_error).
inline thread_local int32_t g_last_cuda_error = 0;

// Also takes the error from the runtime, which would give it to the next launched().
inline spava_status cuda_fail(cudaError_t e) {
    cudaGetLastError();
    g_last_cuda_error = static_cast<int32_t>(e);
    return SPAVA_ERR_CUDA;
}

inline spava_status cuda_ok(cudaError_t e) { return e == cudaSuccess ? SPAVA_OK : cuda_fail(e); }

inline spava_status check_ptr(const void *p, bool required = true) {
    if (!p) return required ? SPAVA_ERR_INVALID_ARG : SPAVA_OK;
    return (reinterpret_cast<uintptr_t>(p) & 15) ? SPAVA_ERR_MISALIGNED : SPAVA_OK;
}

inline spava_status launched() { return cuda_ok(cudaGetLastError()); }

}  // namespace spava

#define SPAVA_CUDA(...)                                    \
    do {                                                   \
        cudaError_t e_ = (__VA_ARGS__);                           \
        if (e_ != cudaSuccess) return ::spava::cuda_fail(e_);       \
    } while (0)

#define SPAVA_TRY(...)                                     \
    do {                                                   \
        spava_status s_ = (__VA_ARGS__);                          \
        if (s_ != SPAVA_OK) return s_;                     \
    } while (0)
