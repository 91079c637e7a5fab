// Host helpers of the C-ABI layer shared by its translation units (defined
// with the entry points of the verify attention).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/swa.h"

namespace swa {

constexpr int kMaxDevices = 64;
constexpr int kMaxBlockLen = 512;  // MAX_NUM_BATCHED_TOKENS: rows of a block

// Sets the thread's last-error message and returns `st`.
swa_status api_fail(swa_status st, const char *fmt, ...);
swa_status api_cuda_fail(cudaError_t e, const char *what);
// Clears the message: the call succeeded.
swa_status api_ok();
// The current device's ordinal and its fault word's device address.
swa_status api_device(int *dev, uint32_t **fault);
int api_device_sms(int dev);
// Host checks of a paged cache description against dims.
swa_status api_check_paged(const swa_paged *paged, const swa_dims *dims);

inline bool aligned_to(const void *p, uintptr_t n) {
    return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

}  // namespace swa
