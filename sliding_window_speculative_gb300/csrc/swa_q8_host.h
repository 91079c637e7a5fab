// Internal interface between the 8-bit cache's entry points and its tensor-core
// kernel.
#pragma once

#include "swa_tc_host.h"

namespace swa {

// Keys that an item of that kernel takes at most: small weights may be off by 2^-21 of
// the item's largest each (see swa_q8_tc.cuh), by 2^-8 of it together if all are off the
// same way.  Shorter items cost time: 152 windows of 8000 keys, 8 rows, 4 heads of 128
// to a KV head, 82 us in one item each, 97 in two.
constexpr int kQ8ItemKeys = 8192;

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
