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

__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// (2^e, 2^e) in bf16 for e in [-126, 127]
__device__ __forceinline__ uint32_t bf16x2_of_pow2(int e) {
    return (uint32_t)(e + 127) * 0x00800080u;
}

struct Q8AppendParams {
    const __nv_bfloat16 *src[2];  // k_new, v_new
    long long row[2];             // elements from one token to the next
    uint8_t *dst[2];
    int8_t *exp[2];
    AttnParams cache;  // seq_lens, q_pos, q_len, Hkv, L, the block table
    int step_tok, step_h;  // tokens and heads from one of a thread's rows to the next
    uint32_t page_inv;
};

// What bounds both kernels is the one read and one write of the rows.  A CTA takes
// U rows per group of lanes from one sequence (and one of K and V), all loads in
// flight at once; the grid is (chunks of rows, sequences).
// Measured: 512 sequences of 64 tokens and 2 heads of 256 written into pages of 16 and
// read back (202 MB) 34.2 us, 5.9 TB/s; 59 with one row at a time and divisions.

// The cache row of position pos of head h, as cache_row, the page found without a
// division: page_inv = (2^32 - 1) / page_size gives the quotient or one less.
__device__ __forceinline__ long long q8_cache_row(const AttnParams &P, uint32_t page_inv, int b,
                                                  int h, uint32_t pos, bool *bad) {
    if (P.block_table == nullptr) return ((long long)b * P.Hkv + h) * P.L + pos;
    const uint32_t ps = (uint32_t)P.page_size;
    uint32_t blk = __umulhi(pos, page_inv), in = pos - blk * ps;
    if (in >= ps) {
        ++blk;
        in -= ps;
    }
    const int page =
        checked_page(P, __ldg(P.block_table + (long long)b * P.max_blocks + blk), bad);
    return ((long long)page * P.Hkv + h) * ps + in;
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t max_u16x2_half(uint32_t v) { return max(v & 0xffffu, v >> 16); }
// The largest 16-bit half over the LPR lanes of a row.  All lanes of the warp call
// it where LPR is 32; otherwise those of whole rows.
template <int LPR>
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
    v = max_u16x2_half(v);
    if constexpr (LPR == 32) return __reduce_max_sync(0xffffffffu, v);
    const uint32_t mask = (LPR == 16 ? 0xffffu : 0xffu) << ((threadIdx.x & 31) / LPR * LPR);
#pragma unroll
    for (int off = LPR / 2; off >= 1; off >>= 1) v = max(v, __shfl_xor_sync(mask, v, off));
    return v;
}

// One row per D / 8 lanes, 8 elements each.
template <int D, int U>
__global__ void __launch_bounds__(kQ8Threads) swa_q8_append_kernel(const Q8AppendParams A) {
    constexpr int LPR = D / 8, GROUPS = kQ8Threads / LPR;
    grid_dep_wait();
    grid_dep_trigger();
    const AttnParams &P = A.cache;
    const int l = threadIdx.x % LPR;
    const int n = P.q_len * P.Hkv;  // rows of a sequence: token, then head
    // (K's and V's rows of a token are neighbours in a fused projection)
    const int kv = (int)(blockIdx.x & 1);
    const int r0 = (int)(blockIdx.x >> 1) * (GROUPS * U) + threadIdx.x / LPR;
    const int b = (int)blockIdx.y;
    uint4 w[U];
    long long to[U];  // cache rows, -1: none
    int tok[U], h[U];
    tok[0] = r0 / P.Hkv;
    h[0] = r0 - tok[0] * P.Hkv;
    const __nv_bfloat16 *src = A.src[kv] + (long long)b * P.q_len * A.row[kv] + l * 8;
#pragma unroll
    for (int j = 0; j < U; ++j) {
        if (j > 0) {
            tok[j] = tok[j - 1] + A.step_tok;
            h[j] = h[j - 1] + A.step_h;
            if (h[j] >= P.Hkv) {
                h[j] -= P.Hkv;
                ++tok[j];
            }
        }
        w[j] = make_uint4(0, 0, 0, 0);
        if (r0 + GROUPS * j < n)
            w[j] = __ldcs(reinterpret_cast<const uint4 *>(src + tok[j] * A.row[kv] + h[j] * D));
    }
    const long long q_pos = P.q_pos[b];
    long long end = P.seq_lens[b];
    if constexpr (kDebugChecks)
        if (threadIdx.x == 0 && (end < 0 || end > P.L)) debug_oob(P.fault);
    if (end > P.L) end = P.L;
#pragma unroll
    for (int j = 0; j < U; ++j) {
        to[j] = -1;
        const long long pos = q_pos + tok[j];
        if (r0 + GROUPS * j < n && pos >= 0 && pos < end) {
            bool bad = false;
            const long long row = q8_cache_row(P, A.page_inv, b, h[j], (uint32_t)pos, &bad);
            if (!bad) to[j] = row;
        }
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
        uint32_t u[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
        // the largest magnitude: a bf16's bits without the sign rise with it
        uint32_t a = row_max<LPR>(max_u16x2(max_u16x2(u[0] & 0x7fff7fffu, u[1] & 0x7fff7fffu),
                                            max_u16x2(u[2] & 0x7fff7fffu, u[3] & 0x7fff7fffu)));
        if (a >= 0x7f80u) {
            // infinities or NaN: NaN all, the largest of the others
            uint32_t fin = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t v = (u[e >> 1] >> (16 * (e & 1))) & 0x7fffu;
                if (v >= 0x7f80u) u[e >> 1] |= 0x7fffu << (16 * (e & 1));
                else fin = max(fin, v);
            }
            a = row_max<LPR>(fin);
        }
        // a = 1.f 2^k: 448 = 1.75 2^8 holds it at e = k - 8 up to 1.75, else k - 7
        int e = (int)(a >> 7) - 127 - 8 + ((a & 0x7fu) > 0x60u ? 1 : 0);
        e = e < kQ8MinExp ? kQ8MinExp : (e > kQ8MaxExp ? kQ8MaxExp : e);
        // (the product is exact, or below any e4m3 number)
        const uint32_t sc = bf16x2_of_pow2(-e);
        uint32_t y[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const uint32_t z = bf16x2_mul(u[p], sc);
            y[p] = e4m3x2(bf16lo(z), bf16hi(z));
        }
        if (to[j] < 0) continue;
        *reinterpret_cast<uint2 *>(A.dst[kv] + to[j] * D + l * 8) =
            make_uint2(y[0] | (y[1] << 16), y[2] | (y[3] << 16));
        if (l == 0) A.exp[kv][to[j]] = (int8_t)e;
    }
}

struct Q8ReadParams {
    const uint8_t *src[2];
    const int8_t *exp[2];
    __nv_bfloat16 *dst[2];  // [B, Hkv, n, D]
    AttnParams cache;       // seq_lens, Hkv, L, the block table
    const int32_t *start;   // first position of each sequence; NULL: that of its window
    int32_t *shifted;       // (start NULL) [2][B]: lengths and q_pos counted from there
    int n;                  // positions per sequence
    uint32_t page_inv;
};

// First position of a sequence's windows, in [0, L].
__device__ __forceinline__ int q8_window_start(const AttnParams &P, int b) {
    const long long lo = (long long)P.q_pos[b] - P.window + 1;
    return (int)(lo < 0 ? 0 : (lo > P.L ? P.L : lo));
}

// One row per D / 8 lanes, 8 elements each.
template <int D, int U>
__global__ void __launch_bounds__(kQ8Threads) swa_q8_read_kernel(const Q8ReadParams A) {
    constexpr int LPR = D / 8, GROUPS = kQ8Threads / LPR;
    grid_dep_wait();
    grid_dep_trigger();
    const AttnParams &P = A.cache;
    const int l = threadIdx.x % LPR;
    const int b = (int)blockIdx.y;
    if (A.start == nullptr && blockIdx.x == 0 && blockIdx.z == 0 && threadIdx.x == 0) {
        const int lo = q8_window_start(P, b);
        const long long len = min((long long)P.seq_lens[b], (long long)P.L) - lo;
        A.shifted[b] = (int)(len < 0 ? 0 : (len > A.n ? A.n : len));
        A.shifted[P.B + b] = (int)max((long long)P.q_pos[b] - lo, -(1LL << 31));
    }
    const int i0 = (int)blockIdx.x * (GROUPS * U) + threadIdx.x / LPR;
    for (int z = (int)blockIdx.z; z < 2 * P.Hkv; z += (int)gridDim.z) {
        const int kv = z & 1, h = z >> 1;
        const long long unit = (long long)b * P.Hkv + h;
        const long long first = A.start ? (long long)A.start[b] : q8_window_start(P, b);
        long long end = P.seq_lens[b];
        if constexpr (kDebugChecks)
            if (threadIdx.x == 0 && (end < 0 || end > P.L)) debug_oob(P.fault);
        if (end > P.L) end = P.L;
        __nv_bfloat16 *dst = A.dst[kv] + unit * A.n * D + l * 8;
        uint2 w[U];
        int e[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int i = i0 + GROUPS * j;
            const long long pos = first + i;
            w[j] = make_uint2(0, 0);
            e[j] = 0;
            if (i < A.n && pos >= 0 && pos < end) {
                const long long row = q8_cache_row(P, A.page_inv, b, h, (uint32_t)pos, nullptr);
                w[j] = __ldcs(reinterpret_cast<const uint2 *>(A.src[kv] + row * D + l * 8));
                e[j] = A.exp[kv][row];
            }
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int i = i0 + GROUPS * j;
            if (i >= A.n) break;
            const uint32_t sc = bf16x2_of_pow2(e[j] < -126 ? -126 : e[j]);
            const uint32_t u[2] = {w[j].x, w[j].y};
            uint32_t o[4];
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const uint32_t f = e4m3x2_to_f16x2((uint16_t)(u[p >> 1] >> (16 * (p & 1))));
                const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&f));
                o[p] = bf16x2_mul(pack_bf16x2(x.x, x.y), sc);  // (bf16 times a power of two)
            }
            *reinterpret_cast<uint4 *>(dst + (long long)i * D) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

}  // namespace swa
