// The 8-bit KV cache: rows quantised to e4m3 as they are written, and read back.
//
// A row x of D elements becomes x8_d = e4m3(x_d 2^-e) and the exponent e, the
// smallest with max |x_d| <= 448 2^e.  The scale is a power of two, so that
// scaling is exact either way: a row's only rounding is the one to e4m3's four
// significant bits (2^-4 of the value at most, as for any other scale: the
// format is a floating one, its range is what a finer scale would change), and
// x8_d 2^e is a bf16 number, which the attention and swa_q8_read take as is.
#pragma once

#include <cuda_fp16.h>

#include "swa_simt.cuh"

namespace swa {

constexpr int kQ8Threads = 256;
constexpr int kQ8MinExp = -50, kQ8MaxExp = 50;

// Two floats -> two e4m3 bytes (first in the low byte), nearest even, at most
// 448 in size; NaN -> NaN.
__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two e4m3 bytes -> two fp16 (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t v) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
    return r;
}

// 2^e for e in [-126, 127]
__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }

struct Q8AppendParams {
    const __nv_bfloat16 *src[2];  // k_new, v_new
    long long row[2];             // elements from one token to the next
    uint8_t *dst[2];
    int8_t *exp[2];
    AttnParams cache;  // seq_lens, q_pos, q_len, Hkv, L, the block table
    long long rows;    // batch * q_len * Hkv
};

// One row per D / 8 lanes, 8 elements each.
template <int D>
__global__ void __launch_bounds__(kQ8Threads) swa_q8_append_kernel(const Q8AppendParams A) {
    constexpr int LPR = D / 8, RPW = 32 / LPR;  // lanes per row, rows per warp
    grid_dep_wait();
    grid_dep_trigger();
    const AttnParams &P = A.cache;
    const int l = threadIdx.x % LPR, sub = (threadIdx.x % 32) / LPR;
    const long long warp = (long long)blockIdx.x * (kQ8Threads / 32) + threadIdx.x / 32;
    const long long step = (long long)gridDim.x * (kQ8Threads / 32) * RPW;
    // (the trip count is the warp's: lanes past the last row take part in the
    // shuffles with zeros)
    for (long long r0 = warp * RPW; r0 < 2 * A.rows; r0 += step) {
        const long long r = r0 + sub;
        const bool there = r < 2 * A.rows;
        const int kv = r >= A.rows;
        const long long rr = there ? r - (kv ? A.rows : 0) : 0;
        const long long tok = rr / P.Hkv;
        const int h = (int)(rr - tok * P.Hkv);
        const int b = (int)(tok / P.q_len), i = (int)(tok - (long long)b * P.q_len);
        uint4 w = make_uint4(0, 0, 0, 0);
        if (there)
            w = __ldg(reinterpret_cast<const uint4 *>(A.src[kv] + tok * A.row[kv] +
                                                      (long long)h * D + l * 8));
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
        float x[8], a = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[2 * e] = bf16lo(u[e]);
            x[2 * e + 1] = bf16hi(u[e]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (!(fabsf(x[e]) < __int_as_float(0x7f800000))) x[e] = __int_as_float(0x7fffffff);
            a = fmaxf(a, fabsf(x[e]));  // (a NaN is ignored)
        }
#pragma unroll
        for (int off = LPR / 2; off >= 1; off >>= 1)
            a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
        // a = 1.f 2^k: 448 = 1.75 2^8 holds it at e = k - 8 up to 1.75, else k - 7
        const uint32_t ab = __float_as_uint(a);
        int e = (int)(ab >> 23) - 127 - 8 + ((ab & 0x7fffffu) > 0x600000u ? 1 : 0);
        e = e < kQ8MinExp ? kQ8MinExp : (e > kQ8MaxExp ? kQ8MaxExp : e);
        const float sc = pow2f(-e);
        uint32_t y[2];
#pragma unroll
        for (int p = 0; p < 2; ++p)
            y[p] = (uint32_t)e4m3x2(x[4 * p] * sc, x[4 * p + 1] * sc) |
                   ((uint32_t)e4m3x2(x[4 * p + 2] * sc, x[4 * p + 3] * sc) << 16);
        const long long pos = (long long)P.q_pos[b] + i;
        long long end = P.seq_lens[b];
        if constexpr (kDebugChecks)
            if (there && l == 0 && (end < 0 || end > P.L)) debug_oob(P.fault);
        if (end > P.L) end = P.L;
        if (!there || pos < 0 || pos >= end) continue;
        bool bad = false;
        const long long row = cache_row(P, b, h, (int)pos, &bad);
        if (bad) continue;
        *reinterpret_cast<uint2 *>(A.dst[kv] + row * D + l * 8) = make_uint2(y[0], y[1]);
        if (l == 0) A.exp[kv][row] = (int8_t)e;
    }
}

struct Q8ReadParams {
    const uint8_t *src[2];
    const int8_t *exp[2];
    __nv_bfloat16 *dst[2];  // [B, Hkv, n, D]
    AttnParams cache;       // seq_lens, Hkv, L, the block table
    const int32_t *start;   // first position of each sequence; NULL: that of its window
    int32_t *shifted;       // (start NULL) [2][B]: lengths and q_pos counted from there
    int n;
    long long rows;         // batch * Hkv * n
};

// First position of a sequence's windows, in [0, L].
__device__ __forceinline__ int q8_window_start(const AttnParams &P, int b) {
    const long long lo = (long long)P.q_pos[b] - P.window + 1;
    return (int)(lo < 0 ? 0 : (lo > P.L ? P.L : lo));
}

// One row per D / 16 lanes, 16 elements each.
template <int D>
__global__ void __launch_bounds__(kQ8Threads) swa_q8_read_kernel(const Q8ReadParams A) {
    constexpr int LPR = D / 16;
    grid_dep_wait();
    grid_dep_trigger();
    const AttnParams &P = A.cache;
    const int l = threadIdx.x % LPR;
    const long long step = (long long)gridDim.x * (kQ8Threads / LPR);
    if (A.start == nullptr) {
        for (long long b = (long long)blockIdx.x * kQ8Threads + threadIdx.x; b < P.B;
             b += (long long)gridDim.x * kQ8Threads) {
            const int lo = q8_window_start(P, (int)b);
            const long long len = min((long long)P.seq_lens[b], (long long)P.L) - lo;
            A.shifted[b] = (int)(len < 0 ? 0 : (len > A.n ? A.n : len));
            A.shifted[P.B + b] = (int)max((long long)P.q_pos[b] - lo, -(1LL << 31));
        }
    }
    for (long long r = (long long)blockIdx.x * (kQ8Threads / LPR) + threadIdx.x / LPR;
         r < 2 * A.rows; r += step) {
        const int kv = r >= A.rows;
        const long long rr = r - (kv ? A.rows : 0);
        const long long unit = rr / A.n;
        const int i = (int)(rr - unit * A.n);
        const int b = (int)(unit / P.Hkv), h = (int)(unit - (long long)b * P.Hkv);
        const long long pos = (A.start ? (long long)A.start[b] : q8_window_start(P, b)) + i;
        long long end = P.seq_lens[b];
        if constexpr (kDebugChecks)
            if (l == 0 && (end < 0 || end > P.L)) debug_oob(P.fault);
        if (end > P.L) end = P.L;
        uint32_t o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (pos >= 0 && pos < end) {
            const long long row = cache_row(P, b, h, (int)pos);
            const uint4 w = *reinterpret_cast<const uint4 *>(A.src[kv] + row * D + l * 16);
            int e = A.exp[kv][row];
            const float sc = pow2f(e < -126 ? -126 : e);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int p = 0; p < 8; ++p) {
                const uint32_t f = e4m3x2_to_f16x2((uint16_t)(u[p >> 1] >> (16 * (p & 1))));
                const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&f));
                o[p] = pack_bf16x2(x.x * sc, x.y * sc);
            }
        }
        uint4 *d = reinterpret_cast<uint4 *>(A.dst[kv] + rr * D + l * 16);
        d[0] = make_uint4(o[0], o[1], o[2], o[3]);
        d[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

}  // namespace swa
