// Internal interface between the 8-bit cache's entry points and its tensor-core
// kernel.
#pragma once

#include "swa_tc_host.h"

namespace swa {

struct Q8TcLaunch {
    TcParams T;
    const int8_t *k_exp, *v_exp;
    const void *k, *v;
    int head_dim, n, grid;  // padded rows per item, persistent CTAs
    long long cache_rows;   // rows of each of the K and V tensors
};

// Encodes the tensor maps and launches; on failure writes a message.
cudaError_t q8_tc_launch(const Q8TcLaunch &L, cudaStream_t stream, char *err, size_t errlen);

}  // namespace swa
