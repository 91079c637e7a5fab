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

// The checks of an attention call's dims and window.
swa_status api_check_dims(const swa_dims *dims, int32_t window);
// The device's workspace of at least `need` bytes (see swa_verify_attn).
swa_status api_workspace(int dev, size_t need, cudaStream_t stream, void **out);
// Bytes of split partials a plain contiguous call of these dims takes, and that
// call with the partials in `parts`.
size_t api_plan_bytes(const swa_dims *dims, int32_t window, int dev);
swa_status api_verify_rows(const void *q, const void *k, const void *v, const int32_t *seq_lens,
                           const int32_t *q_pos, int32_t window, float scale, void *out, float *lse,
                           const swa_dims *dims, void *parts, swa_stream_t stream);

// The merge of split partials (P.splits > 1); nan_lse: rows of NaN get that lse too.
struct AttnParams;
cudaError_t api_merge(const AttnParams &P, int head_dim, bool nan_lse, cudaStream_t s);
// swa_debug_options in effect: the kernel override, the bounded waits' limit in
// SM cycles, the withheld fill.
int api_forced_kernel();
long long api_wait_limit();
int api_withhold_fill();

inline bool aligned_to(const void *p, uintptr_t n) {
    return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

}  // namespace swa
