// Log probabilities of given tokens, entropies and the likeliest tokens.
#pragma once

#include "swa_common.cuh"

namespace swa {

constexpr int kLogpThreads = 256;
constexpr int kLogpMaxTop = 32;

struct LogpParams {
    const uint16_t *logits;
    const int32_t *keep, *tokens;
    const float *temperature;
    float *logprobs, *entropy, *top_logprobs;
    int32_t *ranks, *top_tokens;
    int q_len, V, top;
};

// A logit as the order takes it: NaN is -inf, -0 is 0.
__device__ __forceinline__ float logp_value(uint16_t b) {
    const float x = __uint_as_float((uint32_t)b << 16);
    return x == x ? x + 0.f : -__int_as_float(0x7f800000);
}

// Rising with the value, and with a falling column.
__device__ __forceinline__ unsigned long long logp_key(float x, int col) {
    const uint32_t u = __float_as_uint(x);
    return ((unsigned long long)(u & 0x80000000u ? ~u : u | 0x80000000u) << 32) | (uint32_t)~col;
}

// One row per CTA.
__global__ void __launch_bounds__(kLogpThreads) swa_logprobs_kernel(const LogpParams A) {
    const float INF = __int_as_float(0x7f800000);
    __shared__ float red[3][kLogpThreads];
    __shared__ unsigned long long best[kLogpThreads];
    __shared__ int col_sm, count[kLogpThreads];
    grid_dep_wait();
    grid_dep_trigger();
    const long long row = blockIdx.x;
    const int t = threadIdx.x;
    const uint16_t *x = A.logits + row * A.V;
    float T = A.temperature ? A.temperature[row / A.q_len] : 1.f;
    T = T > 0.f ? fminf(T, 3.0e38f) : 1.f;
    // the given token's column
    const int tok = A.tokens[row];
    if (t == 0) col_sm = A.keep || tok < 0 || tok >= A.V ? 0x7fffffff : tok;
    __syncthreads();
    if (A.keep && tok >= 0)
        for (int j = t; j < A.V; j += kLogpThreads)
            if (A.keep[j] == tok) atomicMin(&col_sm, j);
    __syncthreads();
    const int col = col_sm < A.V ? col_sm : -1;
    const float xt = col >= 0 ? logp_value(x[col]) : 0.f;
    float m = -INF;
    int before = 0;
    for (int j = t; j < A.V; j += kLogpThreads) {
        const float v = logp_value(x[j]);
        m = fmaxf(m, v);
        before += col >= 0 && (v > xt || (v == xt && j < col));
    }
    red[0][t] = m;
    count[t] = before;
    __syncthreads();
    for (int n = kLogpThreads / 2; n > 0; n >>= 1) {
        if (t < n) {
            red[0][t] = fmaxf(red[0][t], red[0][t + n]);
            count[t] += count[t + n];
        }
        __syncthreads();
    }
    m = red[0][0];
    float s = 0.f, u = 0.f;
    for (int j = t; j < A.V; j += kLogpThreads) {
        const float v = logp_value(x[j]);
        const float y = v == m ? 0.f : (v - m) / T;  // (both may be infinite)
        const float e = expf(y);
        s += e;
        if (e > 0.f) u += e * y;
    }
    red[1][t] = s;
    red[2][t] = u;
    __syncthreads();
    for (int n = kLogpThreads / 2; n > 0; n >>= 1) {
        if (t < n) {
            red[1][t] += red[1][t + n];
            red[2][t] += red[2][t + n];
        }
        __syncthreads();
    }
    s = red[1][0];
    u = red[2][0];
    const float ls = logf(s);
    const bool none = m == -INF;
    auto logprob = [&](float v) {
        return none ? -INF : (v == m ? 0.f : (v - m) / T) - ls;
    };
    if (t == 0) {
        A.logprobs[row] = col >= 0 ? logprob(xt) : -INF;
        if (A.ranks) A.ranks[row] = col >= 0 ? count[0] + 1 : 0;
        if (A.entropy) A.entropy[row] = none ? 0.f : ls - u / s;
    }
    unsigned long long last = ~0ull;
    for (int k = 0; k < A.top; ++k) {
        unsigned long long b = 0;
        for (int j = t; j < A.V; j += kLogpThreads) {
            const unsigned long long key = logp_key(logp_value(x[j]), j);
            if (key < last && key > b) b = key;
        }
        __syncthreads();
        best[t] = b;
        __syncthreads();
        for (int n = kLogpThreads / 2; n > 0; n >>= 1) {
            if (t < n && best[t + n] > best[t]) best[t] = best[t + n];
            __syncthreads();
        }
        last = best[0];
        if (t == 0) {
            const int j = (int)~(uint32_t)last;
            A.top_tokens[row * A.top + k] = A.keep ? A.keep[j] : j;
            A.top_logprobs[row * A.top + k] = logprob(logp_value(x[j]));
        }
    }
}

}  // namespace swa
